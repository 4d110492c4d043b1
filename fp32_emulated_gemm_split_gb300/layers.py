"""Python binding of include/emu_layers.h: the gated feed-forward, the
low-rank adapters of many requests beside a projection, and the norm and
rotation of query and key heads, each as the C entry point of its name.

The functions check shapes, types and devices, allocate the outputs, and
enqueue the library's kernels on the current CUDA stream (or ``stream``, a
``torch.cuda.Stream``).  All tensors of a call are on the current device.
Outputs are allocated where they are not given.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _check, _i64, _int, _f32, _vp, _stored, emu_split_b, lib

ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4}
DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

_ready = None


class _Heads(ctypes.Structure):
    _fields_ = [("data", _vp), ("heads", _i64), ("token_stride", _i64), ("head_stride", _i64)]


def _L():
    """The library with this header's entry points declared."""
    global _ready
    if _ready is None:
        L = lib()
        L.emu_gated_rows.argtypes, L.emu_gated_rows.restype = [_i64], _i64
        L.emu_gated_pack.argtypes = [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
        L.emu_gated.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                                _vp, _i64, _vp, _vp, _i64, _vp]
        L.emu_gated_bwd.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp,
                                    _i64, _vp, _i64, _vp, _i64, _vp]
        L.emu_lora.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i64,
                               _vp, _vp, _vp, _vp, _vp, _i64, _vp]
        qk = [_int, _i64, _i64, _i64, _int, _f32]
        tables = [_vp, _vp, _vp, _vp, _i64, _vp]
        L.emu_qk_norm_rope.argtypes = qk + [_Heads] * 2 + tables + [_Heads] * 2 + [_vp]
        L.emu_qk_norm_rope_bwd.argtypes = qk + [_Heads] * 4 + tables + [_Heads] * 2 + [_vp] * 3
        for f in (L.emu_gated_pack, L.emu_gated, L.emu_gated_bwd, L.emu_lora, L.emu_qk_norm_rope,
                  L.emu_qk_norm_rope_bwd):
            f.restype = _int
        _ready = L
    return _ready


def _on(stream):
    """Outputs and work of a call belong to `stream` (None: the current one)."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _handle():
    return torch.cuda.current_stream().cuda_stream


def _here(*tensors):
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and (not t.is_cuda or t.device.index != dev):
            raise ValueError(f"expected tensors on the current CUDA device (cuda:{dev}), got {t.device}")


def _rows(X, name, rows=None, cols=None):
    """Row stride of a 2-D float32 matrix with unit stride along its rows."""
    if X.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {X.dtype}")
    if X.dim() != 2 or (rows is not None and X.size(0) != rows) or (cols is not None and X.size(1) != cols):
        raise ValueError(f"{name} must be {'M' if rows is None else rows} x {'K' if cols is None else cols}, "
                         f"got {tuple(X.shape)}")
    if X.size(1) > 1 and X.stride(1) != 1:
        raise ValueError(f"{name} needs unit stride along its rows")
    ld = X.stride(0) if X.size(0) > 1 else X.size(1)
    if ld < X.size(1):
        raise ValueError(f"{name}'s rows overlap")
    return max(ld, 1)


def _vector(x, name, n):
    if x is None:
        return None
    if x.dtype != torch.float32 or x.dim() != 1 or x.numel() != n or (n > 1 and x.stride(0) != 1):
        raise ValueError(f"{name} must be {n} contiguous float32 values")
    return x.data_ptr()


def _act(act):
    if act not in ACT:
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACT)}")
    return ACT[act]


# ----------------------------------------------------- gated feed-forward --

class GatedWeights:
    """The gate and up weights of a gated feed-forward with their packed
    pieces (``emu_gated_pack``).  The pieces hold the values that the weights
    had then: pack again after changing them."""

    __slots__ = ("Wg", "Wu", "pieces", "F", "K", "ldg", "ldu", "ldp", "rows")

    def __init__(self, Wg, Wu, pieces, ldg, ldu, rows):
        self.Wg, self.Wu, self.pieces = Wg, Wu, pieces
        self.F, self.K = Wg.shape
        self.ldg, self.ldu, self.ldp, self.rows = ldg, ldu, pieces.size(2), rows


def emu_gated_pack(Wg, Wu, stream=None) -> GatedWeights:
    """The weights Wg and Wu (F x K each) ready for ``emu_gated``."""
    Wg, Wu = Wg.detach(), Wu.detach()
    ldg = _rows(Wg, "Wg")
    F, K = Wg.shape
    ldu = _rows(Wu, "Wu", F, K)
    _here(Wg, Wu)
    rows = _L().emu_gated_rows(F)
    with _on(stream):
        P = torch.empty((3, 2 * rows, max((K + 63) // 64 * 64, 64)), dtype=torch.int16, device=Wg.device)
        _check(_L().emu_gated_pack(F, K, Wg.data_ptr(), ldg, Wu.data_ptr(), ldu, P.data_ptr(), P.size(2),
                                   _handle()), "emu_gated_pack")
    return GatedWeights(Wg, Wu, P, ldg, ldu, rows)


def emu_gated(X, w: GatedWeights, act="silu", save=False, out=None, stream=None):
    """H = act(X Wg^T) * (X Wu^T), or (H, G, U) with save=True: the two
    products as well, for ``emu_gated_bwd``."""
    a = _act(act)
    ldx = _rows(X, "X", cols=w.K)
    M = X.size(0)
    _here(X, w.Wg, out)
    with _on(stream):
        H = torch.empty((M, w.F), dtype=torch.float32, device=X.device) if out is None else out
        ldh = _rows(H, "out", M, w.F)
        G = U = None
        ldg = 0
        if save:
            # rows of whole 16-byte groups, so that they can be stored and read as such
            ldg = max((w.F + 3) // 4 * 4, 4)
            GU = torch.empty((2, M, ldg), dtype=torch.float32, device=X.device)
            G, U = GU[0, :, :w.F], GU[1, :, :w.F]
        _check(_L().emu_gated(a, M, w.F, w.K, X.data_ptr(), ldx, w.Wg.data_ptr(), w.ldg, w.Wu.data_ptr(),
                              w.ldu, w.pieces.data_ptr(), w.ldp, H.data_ptr(), ldh,
                              G.data_ptr() if save else None, U.data_ptr() if save else None, ldg,
                              _handle()), "emu_gated")
    return (H, G, U) if save else H


def emu_gated_bwd(dH, X, w: GatedWeights, G, U, act="silu", need_dx=True, need_dw=True, stream=None):
    """(dX, dWg, dWu) from the gradient dH of H and what ``emu_gated`` saved;
    None in the place of a gradient that is not needed."""
    a = _act(act)
    M, F, K = X.size(0), w.F, w.K
    ldx, lddh = _rows(X, "X", cols=K), _rows(dH, "dH", M, F)
    ldg = _rows(G, "G", M, F)
    if _rows(U, "U", M, F) != ldg:
        raise ValueError("G and U need the same row stride")
    _here(dH, X, G, U, w.Wg)
    with _on(stream):
        dX = torch.empty((M, K), dtype=torch.float32, device=X.device) if need_dx else None
        dW = torch.empty((2 * w.rows, K), dtype=torch.float32, device=X.device) if need_dw else None
        _check(_L().emu_gated_bwd(a, M, F, K, dH.data_ptr(), lddh, X.data_ptr(), ldx,
                                  w.pieces.data_ptr(), w.ldp, G.data_ptr(), U.data_ptr(), ldg,
                                  dX.data_ptr() if need_dx else None, max(K, 1),
                                  dW.data_ptr() if need_dw else None, max(K, 1), _handle()),
               "emu_gated_bwd")
    return dX, dW[:F] if need_dw else None, dW[w.rows:w.rows + F] if need_dw else None


# ------------------------------------------------------ low-rank adapters --

class LoraWeights:
    """The weight (N x K) and bias of a shared projection with the weight's
    pieces (``emu_lora_pack``); pack again after changing the weight."""

    __slots__ = ("W", "bias", "pieces", "N", "K", "ldw", "ldp")

    def __init__(self, W, bias, pieces, ldw):
        self.W, self.bias, self.pieces, self.ldw = W, bias, pieces, ldw
        self.N, self.K = W.shape
        self.ldp = pieces.size(2)


def emu_lora_pack(W, bias=None, stream=None) -> LoraWeights:
    """The projection's weight W (N x K) and bias ready for ``emu_lora``."""
    W = W.detach()
    bias = None if bias is None else bias.detach()
    ldw = _rows(W, "W")
    _vector(bias, "bias", W.size(0))
    _here(W, bias)
    with _on(stream):
        P = emu_split_b(W, transB=True)
    return LoraWeights(W, bias, P, ldw)


def emu_lora(X, w: LoraWeights, A, B, index, scale=None, out=None, stream=None):
    """Y = X W^T + bias + scale_i (X A_i^T) B_i^T with i = index[row] (-1: no
    adapter); A is adapters x R x K, B adapters x N x R, scale `adapters`
    values, index int32."""
    ldx = _rows(X, "X", cols=w.K)
    M = X.size(0)
    if A.dtype != torch.float32 or B.dtype != torch.float32:
        raise TypeError("A and B must be float32")
    if A.dim() != 3 or B.dim() != 3 or A.size(2) != w.K or B.size(1) != w.N or A.size(0) != B.size(0) \
            or A.size(1) != B.size(2):
        raise ValueError(f"A must be adapters x R x {w.K} and B adapters x {w.N} x R, "
                         f"got {tuple(A.shape)} and {tuple(B.shape)}")
    if not A.is_contiguous() or not B.is_contiguous():
        raise ValueError("A and B must be contiguous")
    n, R = A.size(0), A.size(1)
    if index.dtype != torch.int32 or index.dim() != 1 or index.numel() != M or (M > 1 and index.stride(0) != 1):
        raise ValueError(f"index must be {M} contiguous int32 values")
    sp = _vector(scale, "scale", n)
    _here(X, w.W, A, B, index, scale, out)
    with _on(stream):
        Y = torch.empty((M, w.N), dtype=torch.float32, device=X.device) if out is None else out
        ldy = _rows(Y, "out", M, w.N)
        _check(_L().emu_lora(M, w.N, w.K, X.data_ptr(), ldx, w.W.data_ptr(), w.ldw, w.pieces.data_ptr(),
                             w.ldp, None if w.bias is None else w.bias.data_ptr(), R, n, A.data_ptr(),
                             B.data_ptr(), sp, index.data_ptr(), Y.data_ptr(), ldy, _handle()), "emu_lora")
    return Y


# --------------------------------- norm and rotation of queries and keys --

def _heads(x, name, like=None):
    if x.dim() != 3 or (like is not None and x.shape != like.shape):
        raise ValueError(f"{name} must be tokens x heads x D"
                         + (f" = {tuple(like.shape)}" if like is not None else "") + f", got {tuple(x.shape)}")
    if x.size(2) > 1 and x.stride(2) != 1:
        raise ValueError(f"{name} needs unit stride along the values of a head")
    return _Heads(x.data_ptr(), x.size(1), x.stride(0), x.stride(1))


def _qk_args(q, k, wq, wk, cos, sin, positions, rest):
    if q.dtype not in DTYPE:
        raise TypeError(f"q and k must be float32, bfloat16 or float16, got {q.dtype}")
    for t in (k, *rest):
        if t.dtype != q.dtype:
            raise TypeError(f"expected tensors of one type, got {q.dtype} and {t.dtype}")
    hq, hk = _heads(q, "q"), _heads(k, "k")
    T, _, D = q.shape
    if k.size(0) != T or k.size(2) != D:
        raise ValueError(f"q and k differ in tokens or head size: {tuple(q.shape)}, {tuple(k.shape)}")
    if cos is None:
        if sin is not None:
            raise ValueError("cos and sin go together")
        rot, rows, tables = 0, 0, (None, None, 0, None)
    else:
        if cos.dtype != torch.float32 or sin.dtype != torch.float32:
            raise TypeError("cos and sin must be float32")
        if cos.dim() != 2 or cos.shape != sin.shape or not cos.is_contiguous() or not sin.is_contiguous():
            raise ValueError("cos and sin must be contiguous matrices of one shape, positions x rot/2")
        rows, rot = cos.size(0), 2 * cos.size(1)
        if positions is None or positions.dtype != torch.int32 or positions.dim() != 1 \
                or positions.numel() != T or (T > 1 and positions.stride(0) != 1):
            raise ValueError(f"positions must be {T} contiguous int32 values")
        tables = (cos.data_ptr(), sin.data_ptr(), rows, positions.data_ptr())
    _here(q, k, wq, wk, cos, sin, positions, *rest)
    return T, D, rot, hq, hk, (_vector(wq, "wq", D), _vector(wk, "wk", D)) + tables


def emu_qk_norm_rope(q, k, wq, wk, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False, out=None,
                     stream=None):
    """Norm of each head of q and k (tokens x heads x D, any token and head
    strides) times wq / wk (None: ones), and the rotation of its first
    2 * cos.size(1) values by the tables' row positions[token]; returns
    (q', k').  out=(q, k) writes in place."""
    T, D, rot, hq, hk, tables = _qk_args(q, k, wq, wk, cos, sin, positions, out or ())
    with _on(stream):
        qo, ko = out if out is not None else (torch.empty(q.shape, dtype=q.dtype, device=q.device),
                                              torch.empty(k.shape, dtype=k.dtype, device=k.device))
        _check(_L().emu_qk_norm_rope(DTYPE[q.dtype], T, D, rot, int(interleaved), eps, hq, hk, *tables,
                                     _heads(qo, "out[0]", q), _heads(ko, "out[1]", k), _handle()),
               "emu_qk_norm_rope")
    return qo, ko


def emu_qk_norm_rope_bwd(dq_out, dk_out, q, k, wq, wk, cos=None, sin=None, positions=None, eps=1e-6,
                         interleaved=False, stream=None):
    """(dq, dk, dwq, dwk) from the gradients of ``emu_qk_norm_rope``'s outputs
    and its inputs; dwq / dwk are None where wq / wk are."""
    T, D, rot, hq, hk, tables = _qk_args(q, k, wq, wk, cos, sin, positions, (dq_out, dk_out))
    with _on(stream):
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        dk = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        dw = torch.empty((2, D), dtype=torch.float32, device=q.device)
        _check(_L().emu_qk_norm_rope_bwd(
            DTYPE[q.dtype], T, D, rot, int(interleaved), eps, _heads(dq_out, "dq_out", q),
            _heads(dk_out, "dk_out", k), hq, hk, *tables, _heads(dq, "dq"), _heads(dk, "dk"),
            dw[0].data_ptr() if wq is not None else None, dw[1].data_ptr() if wk is not None else None,
            _handle()), "emu_qk_norm_rope_bwd")
    return dq, dk, dw[0] if wq is not None else None, dw[1] if wk is not None else None
