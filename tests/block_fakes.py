"""Plain CPU stand-ins for the library's calls, for tests of the torch modules
around them.  They take a matrix as a kernel does, by its storage and row
stride, and refuse what the binding refuses."""
import torch

import fp32_emulated_gemm_split_gb300 as emu
import layer_ref as ref
from fp32_emulated_gemm_split_gb300.layers import version_of


def _matrix(X, rows=None, cols=None):
    """X as emu_layers.h's functions take it: rows of unit stride that do not overlap."""
    if X.dtype != torch.float32:
        raise TypeError("must be float32")
    if X.dim() != 2 or (rows is not None and X.size(0) != rows) or (cols is not None and X.size(1) != cols):
        raise ValueError(f"wrong shape {tuple(X.shape)}")
    if X.stride(1) != 1 and X.size(1) > 1:
        raise ValueError("needs unit stride along its rows")
    if X.size(0) > 1 and X.stride(0) < X.size(1):
        raise ValueError("rows overlap")
    return X.detach().double()


def _read(X, trans):
    """op(X) as emu_sgemm reads it (as_strided raises where that leaves the storage)."""
    S, t, ld = emu._stored(X, trans)
    S = torch.as_strided(S.detach(), S.shape, (ld, 1)).double()
    return S.t() if t else S


def emu_sgemm(A, B, C=None, *, transA=False, transB=False, alpha=1.0, beta=0.0, mode="bf16x9", stream=None):
    Y = alpha * (_read(A, transA) @ _read(B, transB))
    if C is None:
        return Y.float()
    return C.copy_(Y + beta * C if beta else Y)


def emu_split_b(B, transB=False, mode="bf16x9", stream=None):
    return _read(B, transB).clone()


def emu_sgemm_bsplit(A, Bp, C=None, *, transA=False, alpha=1.0, beta=0.0, mode="bf16x9", stream=None):
    return emu_sgemm(A, Bp.float(), C, transA=transA, alpha=alpha, beta=beta)


class Packed:
    """What a pack function returns: the values of its time, and the tensors with their versions."""

    def __init__(self, *tensors):
        self.tensors = [t.detach() for t in tensors]
        self.values = [_matrix(t).clone() for t in tensors]
        self.versions = [version_of(t) for t in self.tensors]

    def checked(self):
        if self.versions != [version_of(t) for t in self.tensors]:
            raise ValueError("changed in place: pack again")
        return self.values


def emu_gated_pack(Wg, Wu, *, stream=None):
    return Packed(Wg, Wu)


def emu_gated(X, w, act="silu", save=False, out=None, *, stream=None):
    Wg, Wu = w.checked()
    X = _matrix(X, cols=Wg.size(1))
    G, U = X @ Wg.t(), X @ Wu.t()
    H = ref.act(act, G)[0] * U
    return tuple(t.float() for t in (H, G, U)) if save else H.float()


def emu_gated_bwd(dH, X, w, G, U, act="silu", need_dx=True, need_dw=True, *, stream=None):
    Wg, Wu = w.checked()
    X = _matrix(X, cols=Wg.size(1))
    d = [_matrix(t, X.size(0), Wg.size(0)) for t in (dH, G, U)]
    a, da = ref.act(act, d[1])
    dG, dU = d[0] * d[2] * da, d[0] * a
    return ((dG @ Wg + dU @ Wu).float() if need_dx else None,
            *((t.float() if need_dw else None) for t in (dG.t() @ X, dU.t() @ X)))


def emu_lora_pack(W, bias=None, *, stream=None):
    return Packed(W)


def emu_lora(X, w, A, B, index, scale=None, out=None, *, stream=None):
    W, = w.checked()
    _matrix(X, cols=W.size(1))
    return ref.lora(X.detach(), W, None, A.detach(), B.detach(), index, scale)[0].float()


def _head(x, w, cos, sin, positions, eps, interleaved):
    return ref.qk(x, w, cos, sin, positions, eps, interleaved)[0].to(x.dtype)


def emu_qk_norm_rope(q, k, wq, wk, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False, out=None, *,
                     stream=None):
    how = cos, sin, positions, eps, interleaved
    return _head(q.detach(), wq, *how).detach(), _head(k.detach(), wk, *how).detach()


def emu_qk_norm_rope_bwd(dq_out, dk_out, q, k, wq, wk, cos=None, sin=None, positions=None, eps=1e-6,
                         interleaved=False, *, stream=None):
    how = cos, sin, positions, eps, interleaved
    (dq, dwq), _ = ref.qk_bwd(dq_out, q.detach(), wq.detach(), *how)
    (dk, dwk), _ = ref.qk_bwd(dk_out, k.detach(), wk.detach(), *how)
    return dq.to(q.dtype), dk.to(k.dtype), dwq.float(), dwk.float()


def put_in(monkeypatch):
    """block.py and linear.py on these."""
    from fp32_emulated_gemm_split_gb300 import block, linear
    for name in ("emu_gated", "emu_gated_bwd", "emu_gated_pack", "emu_lora", "emu_lora_pack", "emu_qk_norm_rope",
                 "emu_qk_norm_rope_bwd"):
        monkeypatch.setattr(block, name, globals()[name])
    for name in ("emu_sgemm", "emu_sgemm_bsplit", "emu_split_b"):
        monkeypatch.setattr(linear, name, globals()[name])
