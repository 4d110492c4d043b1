"""Python binding of include/emu_layers.h: the gated feed-forward, the
low-rank adapters of many requests beside a projection, and the norm and
rotation of query and key heads, each as the C entry point of its name.

The functions check shapes, types and devices, allocate the outputs, and
enqueue the library's kernels on the current CUDA stream (or ``stream``, a
``torch.cuda.Stream``).  All tensors of a call are on the current device.
Outputs are allocated where they are not given.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _check, _i64, _int, _f32, _vp, _stored, emu_split_b, lib

ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4}
DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_F32 = torch.float32

_ready = None


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
        qk = [_int, _i64, _i64, _i64, _int, _f32, ctypes.c_char_p, _vp, _vp, _vp, _vp, _i64, _vp]
        L.emu_qk_norm_rope.argtypes = qk + [_vp]
        L.emu_qk_norm_rope_bwd.argtypes = qk + [_vp, _vp, _vp]
        for f in (L.emu_gated_pack, L.emu_gated, L.emu_gated_bwd, L.emu_lora, L.emu_qk_norm_rope,
                  L.emu_qk_norm_rope_bwd):
            f.restype = _int
        _ready = L
    return _ready


# A call for a few tokens takes the GPU 10 to 30 us, so the wrappers count:
# each tensor's shape and strides are read once and compared as tuples, and the
# stream's handle comes without making a Stream object.

def _on_stream(fn):
    """Gives fn a ``stream``: its outputs and work belong to it (None: to the
    current one)."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kwargs):
        if stream is None:
            return fn(*args, **kwargs)
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return call


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _handle(dev):
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _device(X, *tensors):
    """The index of the current device, which holds every tensor of the call."""
    dev = torch.cuda.current_device()
    for t in (X, *tensors):
        if t is not None and t.get_device() != dev:
            raise ValueError(f"expected tensors on the current CUDA device (cuda:{dev}), got {t.device}")
    return dev


def _rows(X, name, rows=None, cols=None):
    """Row stride of a 2-D float32 matrix with unit stride along its rows."""
    if X.dtype is not _F32:
        raise TypeError(f"{name} must be float32, got {X.dtype}")
    shape = X.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (cols is not None and shape[1] != cols):
        raise ValueError(f"{name} must be {'M' if rows is None else rows} x {'K' if cols is None else cols}, "
                         f"got {tuple(shape)}")
    ld, unit = X.stride()
    r, c = shape
    if unit != 1 and c > 1:
        raise ValueError(f"{name} needs unit stride along its rows")
    if r <= 1:
        return c if c > 0 else 1
    if ld < c:
        raise ValueError(f"{name}'s rows overlap")
    return ld if ld > 0 else 1


def _vector(x, name, n):
    if x is None:
        return None
    if x.dtype is not _F32 or x.shape != (n,) or (n > 1 and x.stride(0) != 1):
        raise ValueError(f"{name} must be {n} contiguous float32 values")
    return x.data_ptr()


def _indices(x, name, n):
    if x is None or x.dtype is not torch.int32 or x.shape != (n,) or (n > 1 and x.stride(0) != 1):
        raise ValueError(f"{name} must be {n} contiguous int32 values")
    return x.data_ptr()


def _act(act):
    a = ACT.get(act)
    if a is None:
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACT)}")
    return a


# ----------------------------------------------------- gated feed-forward --

class GatedWeights:
    """The gate and up weights of a gated feed-forward with their packed
    pieces (``emu_gated_pack``).  The kernels read one or the other, so a
    weight changed in place since then is refused: pack again."""

    __slots__ = ("Wg", "Wu", "pieces", "F", "K", "rows", "_weights", "_pieces", "_versions")

    def __init__(self, Wg, Wu, pieces, ldg, ldu, rows):
        self.Wg, self.Wu, self.pieces, self.rows = Wg, Wu, pieces, rows
        self.F, self.K = Wg.shape
        self._versions = Wg._version, Wu._version
        # the entry points' arguments (the tensors above keep the memory)
        self._weights = (Wg.data_ptr(), ldg, Wu.data_ptr(), ldu)
        self._pieces = (pieces.data_ptr(), pieces.size(2))

    def check(self):
        if (self.Wg._version, self.Wu._version) != self._versions:
            raise ValueError("a weight was changed in place since emu_gated_pack: pack again")


@_on_stream
def emu_gated_pack(Wg, Wu) -> GatedWeights:
    """The weights Wg and Wu (F x K each) ready for ``emu_gated``."""
    Wg, Wu = Wg.detach(), Wu.detach()
    ldg = _rows(Wg, "Wg")
    F, K = Wg.shape
    ldu = _rows(Wu, "Wu", F, K)
    dev = _device(Wg, Wu)
    rows = _L().emu_gated_rows(F)
    P = torch.empty((3, 2 * rows, max((K + 63) // 64 * 64, 64)), dtype=torch.int16, device=Wg.device)
    _check(_L().emu_gated_pack(F, K, Wg.data_ptr(), ldg, Wu.data_ptr(), ldu, P.data_ptr(), P.size(2),
                               _handle(dev)), "emu_gated_pack")
    return GatedWeights(Wg, Wu, P, ldg, ldu, rows)


@_on_stream
def emu_gated(X, w: GatedWeights, act="silu", save=False, out=None):
    """H = act(X Wg^T) * (X Wu^T), or (H, G, U) with save=True: the two
    products as well, for ``emu_gated_bwd``."""
    a = _act(act)
    w.check()
    F, K = w.F, w.K
    ldx = _rows(X, "X", None, K)
    M = X.shape[0]
    dev = _device(X, w.Wg, out)
    if out is None:
        H, ldh = torch.empty((M, F), dtype=_F32, device=X.device), F if F > 0 else 1
    else:
        H, ldh = out, _rows(out, "out", M, F)
    G = U = pG = pU = None
    ldg = 0
    if save:
        # rows of whole 16-byte groups, so that they can be stored and read as such
        ldg = max((F + 3) // 4 * 4, 4)
        G = torch.empty((M, ldg), dtype=_F32, device=X.device)
        U = torch.empty((M, ldg), dtype=_F32, device=X.device)
        if ldg != F:
            G, U = G[:, :F], U[:, :F]
        pG, pU = G.data_ptr(), U.data_ptr()
    _check(_L().emu_gated(a, M, F, K, X.data_ptr(), ldx, *w._weights, *w._pieces, H.data_ptr(), ldh,
                          pG, pU, ldg, _handle(dev)), "emu_gated")
    return (H, G, U) if save else H


@_on_stream
def emu_gated_bwd(dH, X, w: GatedWeights, G, U, act="silu", need_dx=True, need_dw=True):
    """(dX, dWg, dWu) from the gradient dH of H and what ``emu_gated`` saved;
    None in the place of a gradient that is not needed."""
    a = _act(act)
    w.check()
    M, F, K = X.size(0), w.F, w.K
    ldx, lddh = _rows(X, "X", cols=K), _rows(dH, "dH", M, F)
    ldg = _rows(G, "G", M, F)
    if _rows(U, "U", M, F) != ldg:
        raise ValueError("G and U need the same row stride")
    dev = _device(dH, X, G, U, w.Wg)
    dX = torch.empty((M, K), dtype=_F32, device=X.device) if need_dx else None
    dW = torch.empty((2 * w.rows, K), dtype=_F32, device=X.device) if need_dw else None
    _check(_L().emu_gated_bwd(a, M, F, K, dH.data_ptr(), lddh, X.data_ptr(), ldx, *w._pieces,
                              G.data_ptr(), U.data_ptr(), ldg,
                              dX.data_ptr() if need_dx else None, max(K, 1),
                              dW.data_ptr() if need_dw else None, max(K, 1), _handle(dev)),
           "emu_gated_bwd")
    return dX, dW[:F] if need_dw else None, dW[w.rows:w.rows + F] if need_dw else None


# ------------------------------------------------------ low-rank adapters --

class LoraWeights:
    """The weight (N x K) and bias of a shared projection with the weight's
    pieces (``emu_lora_pack``).  The kernels read one or the other, so a weight
    changed in place since then is refused: pack again."""

    __slots__ = ("W", "bias", "pieces", "N", "K", "_weight", "_version")

    def __init__(self, W, bias, pieces, ldw):
        self.W, self.bias, self.pieces = W, bias, pieces
        self.N, self.K = W.shape
        self._version = W._version
        # the entry point's arguments (the tensors above keep the memory)
        self._weight = (W.data_ptr(), ldw, pieces.data_ptr(), pieces.size(2),
                        None if bias is None else bias.data_ptr())


@_on_stream
def emu_lora_pack(W, bias=None) -> LoraWeights:
    """The projection's weight W (N x K) and bias ready for ``emu_lora``."""
    W = W.detach()
    bias = None if bias is None else bias.detach()
    ldw = _rows(W, "W")
    _vector(bias, "bias", W.size(0))
    _device(W, bias)
    P = emu_split_b(W, transB=True)
    return LoraWeights(W, bias, P, ldw)


@_on_stream
def emu_lora(X, w: LoraWeights, A, B, index, scale=None, out=None):
    """Y = X W^T + bias + scale_i (X A_i^T) B_i^T with i = index[row] (-1: no
    adapter); A is adapters x R x K, B adapters x N x R, scale `adapters`
    values, index int32."""
    if w.W._version != w._version:
        raise ValueError("the weight was changed in place since emu_lora_pack: pack again")
    N, K = w.N, w.K
    ldx = _rows(X, "X", None, K)
    M = X.shape[0]
    if A.dtype is not _F32 or B.dtype is not _F32:
        raise TypeError("A and B must be float32")
    shape = A.shape
    if len(shape) != 3 or shape[2] != K or B.shape != (shape[0], N, shape[1]):
        raise ValueError(f"A must be adapters x R x {K} and B adapters x {N} x R, "
                         f"got {tuple(A.shape)} and {tuple(B.shape)}")
    if not A.is_contiguous() or not B.is_contiguous():
        raise ValueError("A and B must be contiguous")
    n, R = shape[0], shape[1]
    ip = _indices(index, "index", M)
    sp = _vector(scale, "scale", n)
    dev = _device(X, w.W, A, B, index, scale, out)
    if out is None:
        Y, ldy = torch.empty((M, N), dtype=_F32, device=X.device), N if N > 0 else 1
    else:
        Y, ldy = out, _rows(out, "out", M, N)
    _check(_L().emu_lora(M, N, K, X.data_ptr(), ldx, *w._weight, R, n, A.data_ptr(), B.data_ptr(), sp, ip,
                         Y.data_ptr(), ldy, _handle(dev)), "emu_lora")
    return Y


# --------------------------------- norm and rotation of queries and keys --

_4_heads, _6_heads = struct.Struct("4q4q4q4q"), struct.Struct("4q4q4q4q4q4q")      # emu_heads_t each


def _heads(x, name, shape, dtype):
    """The emu_heads_t of a tokens x heads x D tensor of the given shape."""
    if x.dtype is not dtype:
        raise TypeError(f"expected tensors of one type, got {dtype} and {x.dtype} for {name}")
    if x.shape != shape:
        raise ValueError(f"{name} must be tokens x heads x D = {tuple(shape)}, got {tuple(x.shape)}")
    st, sh, unit = x.stride()
    if unit != 1 and shape[2] > 1:
        raise ValueError(f"{name} needs unit stride along the values of a head")
    return x.data_ptr(), shape[1], st, sh


def _qk_args(q, k, wq, wk, cos, sin, positions):
    """Checks of both directions: (dtype, T, D, rot), q and k as emu_heads_t,
    and the weights' and tables' arguments."""
    kind = q.dtype
    dt = DTYPE.get(kind)
    if dt is None:
        raise TypeError(f"q and k must be float32, bfloat16 or float16, got {kind}")
    qs, ks = q.shape, k.shape
    if len(qs) != 3 or len(ks) != 3 or ks[0] != qs[0] or ks[2] != qs[2]:
        raise ValueError(f"q and k must be tokens x heads x D with the same tokens and D, got {tuple(qs)}, {tuple(ks)}")
    T, _, D = qs
    hq, hk = _heads(q, "q", qs, kind), _heads(k, "k", ks, kind)
    pq, pk = _vector(wq, "wq", D), _vector(wk, "wk", D)
    if cos is None:
        if sin is not None:
            raise ValueError("cos and sin go together")
        return (dt, T, D, 0), hq, hk, (pq, pk, None, None, 0, None)
    shape = cos.shape
    if cos.dtype is not _F32 or sin.dtype is not _F32:
        raise TypeError("cos and sin must be float32")
    if len(shape) != 2 or sin.shape != shape or not cos.is_contiguous() or not sin.is_contiguous():
        raise ValueError("cos and sin must be contiguous matrices of one shape, positions x rot/2")
    return (dt, T, D, 2 * shape[1]), hq, hk, (pq, pk, cos.data_ptr(), sin.data_ptr(), shape[0],
                                              _indices(positions, "positions", T))


@_on_stream
def emu_qk_norm_rope(q, k, wq, wk, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False, out=None):
    """Norm of each head of q and k (tokens x heads x D, any token and head
    strides) times wq / wk (None: ones), and the rotation of its first
    2 * cos.size(1) values by the tables' row positions[token]; returns
    (q', k').  out=(q, k) writes in place."""
    size, hq, hk, tables = _qk_args(q, k, wq, wk, cos, sin, positions)
    D = size[2]
    if out is None:
        dev = _device(q, k, wq, wk, cos, sin, positions)
        kind, on = q.dtype, q.device
        qo, ko = torch.empty(q.shape, dtype=kind, device=on), torch.empty(k.shape, dtype=kind, device=on)
        ho, hp = (qo.data_ptr(), hq[1], hq[1] * D, D), (ko.data_ptr(), hk[1], hk[1] * D, D)
    else:
        qo, ko = out
        dev = _device(q, k, wq, wk, cos, sin, positions, qo, ko)
        ho, hp = _heads(qo, "out[0]", q.shape, q.dtype), _heads(ko, "out[1]", k.shape, q.dtype)
    heads = _4_heads.pack(*hq, *hk, *ho, *hp)
    _check(_L().emu_qk_norm_rope(*size, 1 if interleaved else 0, eps, heads, *tables, _handle(dev)),
           "emu_qk_norm_rope")
    return qo, ko


@_on_stream
def emu_qk_norm_rope_bwd(dq_out, dk_out, q, k, wq, wk, cos=None, sin=None, positions=None, eps=1e-6,
                         interleaved=False):
    """(dq, dk, dwq, dwk) from the gradients of ``emu_qk_norm_rope``'s outputs
    and its inputs; dwq / dwk are None where wq / wk are."""
    size, hq, hk, tables = _qk_args(q, k, wq, wk, cos, sin, positions)
    dev = _device(q, k, wq, wk, cos, sin, positions, dq_out, dk_out)
    D, kind, on = size[2], q.dtype, q.device
    hdq, hdk = _heads(dq_out, "dq_out", q.shape, kind), _heads(dk_out, "dk_out", k.shape, kind)
    dq, dk = torch.empty(q.shape, dtype=kind, device=on), torch.empty(k.shape, dtype=kind, device=on)
    dwq = torch.empty(D, dtype=_F32, device=on) if wq is not None else None
    dwk = torch.empty(D, dtype=_F32, device=on) if wk is not None else None
    heads = _6_heads.pack(*hq, *hk, dq.data_ptr(), hq[1], hq[1] * D, D, dk.data_ptr(), hk[1], hk[1] * D, D,
                          *hdq, *hdk)
    _check(_L().emu_qk_norm_rope_bwd(*size, 1 if interleaved else 0, eps, heads, *tables,
                                     None if dwq is None else dwq.data_ptr(),
                                     None if dwk is None else dwk.data_ptr(), _handle(dev)),
           "emu_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk
