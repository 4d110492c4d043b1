"""Python binding of include/emu_layers.h: the gated feed-forward, the
low-rank adapters of many requests beside a projection, and the norm and
rotation of query and key heads, each as the C entry point of its name.

The functions check shapes, types, strides and devices, allocate the outputs
that are not given, and enqueue the library's kernels on the current CUDA stream
(or ``stream``, a ``torch.cuda.Stream``).  All tensors of a call are on the
current device; an output that is given may not overlap an input (q and k in
place excepted).  Autograd does not see the calls: block.py has the modules with
gradients.  csrc/layers_bind.cpp does the work in C++.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import _build, _check, _i64, _int, _f32, _vp, emu_split_b, lib

ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4}

_ready = None
_bound = None


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


def _C():
    """csrc/layers_bind.cpp, bound to the library."""
    global _bound
    if _bound is None:
        L = _L()
        if not os.path.exists(_build.BIND_PATH):
            raise RuntimeError(f"the binding of emu_layers.h is not built ({_build.BIND_PATH} is missing); run "
                               "`python -c 'import __graft_entry__ as g; g.build()'` first")
        spec = importlib.util.spec_from_file_location("emu_layers_bind", _build.BIND_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(_check, *(ctypes.cast(f, _vp).value for f in (
            L.emu_gated_rows, L.emu_gated_pack, L.emu_gated, L.emu_gated_bwd, L.emu_lora, L.emu_qk_norm_rope,
            L.emu_qk_norm_rope_bwd)))
        _bound = module
    return _bound


def _on(stream, fn, *args):
    """fn's call whose outputs and work belong to ``stream``."""
    with torch.cuda.stream(stream):
        return fn(*args)


def _act(act):
    a = ACT.get(act)
    if a is None:
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACT)}")
    return a


def version_of(t):
    """The version that in-place changes of t raise; -1 for an inference
    tensor, which has none."""
    return -1 if t.is_inference() else t._version


def _kept(t):
    """A weight as a pack keeps it: itself, or a copy where its changes could not be seen."""
    t = t.detach()
    return t.clone() if t.is_inference() else t


# ----------------------------------------------------- gated feed-forward --

class GatedWeights:
    """The gate and up weights of a gated feed-forward with their packed
    pieces (``emu_gated_pack``).  The kernels read one or the other, so a
    weight changed in place since then is refused: pack again.  A write that
    leaves the tensor's version as it was (through ``.data``) cannot be seen,
    and few rows would read the new values where many read the old: pack again
    after it, or pack a copy.  Of inference tensors, which have no version, a
    copy is kept."""

    __slots__ = ("Wg", "Wu", "pieces", "F", "K", "rows", "_args")

    def __init__(self, Wg, Wu, pieces):
        self.Wg, self.Wu, self.pieces, self.rows = Wg, Wu, pieces, pieces.size(1) // 2
        self.F, self.K = Wg.shape
        self._args = Wg, Wu, pieces, version_of(Wg), version_of(Wu)


def emu_gated_pack(Wg, Wu, *, stream=None) -> GatedWeights:
    """The weights Wg and Wu (F x K each) ready for ``emu_gated``."""
    if stream is not None:
        return _on(stream, emu_gated_pack, Wg, Wu)
    Wg, Wu = _kept(Wg), _kept(Wu)
    return GatedWeights(Wg, Wu, _C().gated_pack(Wg, Wu))


def emu_gated(X, w: GatedWeights, act="silu", save=False, out=None, *, stream=None):
    """H = act(X Wg^T) * (X Wu^T), or (H, G, U) with save=True: the two
    products as well, for ``emu_gated_bwd``."""
    if stream is not None:
        return _on(stream, emu_gated, X, w, act, save, out)
    return _C().gated(_act(act), X, w._args, save, out)


def emu_gated_bwd(dH, X, w: GatedWeights, G, U, act="silu", need_dx=True, need_dw=True, *, stream=None):
    """(dX, dWg, dWu) from the gradient dH of H and what ``emu_gated`` saved;
    None in the place of a gradient that is not needed."""
    if stream is not None:
        return _on(stream, emu_gated_bwd, dH, X, w, G, U, act, need_dx, need_dw)
    return _C().gated_bwd(_act(act), dH, X, w._args, G, U, need_dx, need_dw)


# ------------------------------------------------------ low-rank adapters --

class LoraWeights:
    """The weight (N x K) and bias of a shared projection with the weight's
    pieces (``emu_lora_pack``).  The kernels read one or the other, so a weight
    changed in place since then is refused: pack again (after a write through
    ``.data`` as well, which cannot be seen).  Of an inference tensor, which has
    no version, a copy is kept."""

    __slots__ = ("W", "bias", "pieces", "N", "K", "_args")

    def __init__(self, W, bias, pieces):
        self.W, self.bias, self.pieces = W, bias, pieces
        self.N, self.K = W.shape
        self._args = W, bias, pieces, version_of(W)


def emu_lora_pack(W, bias=None, *, stream=None) -> LoraWeights:
    """The projection's weight W (N x K) and bias ready for ``emu_lora``."""
    if stream is not None:
        return _on(stream, emu_lora_pack, W, bias)
    W = _kept(W)
    bias = None if bias is None else bias.detach()
    _C().lora_weights(W, bias)
    return LoraWeights(W, bias, emu_split_b(W, transB=True))


def emu_lora(X, w: LoraWeights, A, B, index, scale=None, out=None, *, stream=None):
    """Y = X W^T + bias + scale_i (X A_i^T) B_i^T with i = index[row] (-1: no
    adapter); A is adapters x R x K, B adapters x N x R, scale `adapters`
    values, index int32."""
    if stream is not None:
        return _on(stream, emu_lora, X, w, A, B, index, scale, out)
    return _C().lora(X, w._args, A, B, index, scale, out)


# --------------------------------- norm and rotation of queries and keys --

def emu_qk_norm_rope(q, k, wq, wk, cos=None, sin=None, positions=None, eps=1e-6, interleaved=False, out=None,
                     *, stream=None):
    """Norm of each head of q and k (tokens x heads x D, any token and head
    strides) times wq / wk (None: ones), and the rotation of its first
    2 * cos.size(1) values by the tables' row positions[token]; returns
    (q', k').  out=(q, k) writes in place."""
    if stream is not None:
        return _on(stream, emu_qk_norm_rope, q, k, wq, wk, cos, sin, positions, eps, interleaved, out)
    qo, ko = out if out is not None else (None, None)
    return _C().qk_norm_rope(q, k, wq, wk, cos, sin, positions, eps, interleaved, qo, ko)


def emu_qk_norm_rope_bwd(dq_out, dk_out, q, k, wq, wk, cos=None, sin=None, positions=None, eps=1e-6,
                         interleaved=False, *, stream=None):
    """(dq, dk, dwq, dwk) from the gradients of ``emu_qk_norm_rope``'s outputs
    and its inputs; dwq / dwk are None where wq / wk are."""
    if stream is not None:
        return _on(stream, emu_qk_norm_rope_bwd, dq_out, dk_out, q, k, wq, wk, cos, sin, positions, eps, interleaved)
    return _C().qk_norm_rope_bwd(q, k, wq, wk, cos, sin, positions, eps, interleaved, dq_out, dk_out)
