"""Python binding of include/emu_layers.h: the gated feed-forward, the
low-rank adapters of many requests beside a projection, the norm and rotation
of query and key heads, and the pages of keys and values kept in 8 bits with the
attention over them, each as the C entry point of its name.

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
from typing import NamedTuple

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
        L.emu_kv_tables.argtypes = [_i64, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp,
                                    _vp, _vp]
        L.emu_kv_store.argtypes = [_int, _i64, ctypes.c_char_p, ctypes.c_char_p, _vp, ctypes.c_char_p, _vp]
        L.emu_kv_attention.argtypes = [_int, _i64, ctypes.c_char_p, ctypes.c_char_p, ctypes.c_char_p, _i64, _vp, _i64,
                                       _vp, _vp, _f32, _i64, _i64, _vp]
        for f in (L.emu_gated_pack, L.emu_gated, L.emu_gated_bwd, L.emu_lora, L.emu_qk_norm_rope,
                  L.emu_qk_norm_rope_bwd, L.emu_kv_tables, L.emu_kv_store, L.emu_kv_attention):
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
            L.emu_qk_norm_rope_bwd, L.emu_kv_tables, L.emu_kv_store, L.emu_kv_attention)))
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


# ----------------------------------------- keys and values kept in 8 bits --

class KvCache(NamedTuple):
    """Pages of keys and values: e4m3 codes (pages x heads x page x D, contiguous)
    and a scale for each page and head (pages x heads, float32); a value is code
    times scale.  The functions below also take a plain tuple of the four."""

    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


class KvPlan(NamedTuple):
    """A step's places (``emu_kv_tables``), int32: sequence b's rows are starts[b]
    to starts[b + 1] - 1 and it holds lengths[b] tokens with them; each row's slot
    (-1 behind the last sequence) and position; how many free pages are given away."""

    starts: torch.Tensor
    lengths: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    taken: torch.Tensor


def emu_kv_cache(pages, heads, D, page=64, device="cuda") -> KvCache:
    """An empty cache of pages * page tokens: 2 * D + 8 / page bytes for each token
    and key head.  page: 16, 32, 64, 128 or 256; D: a multiple of 16, up to 256."""
    codes = [torch.zeros(pages, heads, page, D, device=device, dtype=torch.float8_e4m3fn) for _ in range(2)]
    return KvCache(*codes, *(torch.zeros(pages, heads, device=device) for _ in range(2)))


def emu_kv_tables(kept, new, table, free, pages, page, tokens, taken=None, *, stream=None) -> KvPlan:
    """The places of a step in which sequence b, of kept[b] tokens, gets new[b]
    more, in a cache of `pages` pages of `page` tokens.  The pages that the sequences
    lack are written into `table` (sequences x pages, int32, in place), from
    free[taken] on; `taken` (one int32 on the GPU, None for 0) is what the plan of
    the step before gave.  `tokens`: the step's rows, new.sum() or more."""
    if stream is not None:
        return _on(stream, emu_kv_tables, kept, new, table, free, pages, page, tokens, taken)
    return KvPlan(*_C().kv_tables(kept, new, table, free, pages, page, tokens, taken))


def emu_kv_store(k, v, cache: KvCache, slots, *, stream=None) -> None:
    """Keys and values (tokens x heads x D, any token and head strides; float32,
    bfloat16 or float16) into their slots of the cache (-1: none), a page's
    slots one after another.  A page's scale is a power of two that grows as it
    has to; a run that writes a page's first row begins it anew."""
    if stream is not None:
        return _on(stream, emu_kv_store, k, v, cache, slots)
    _C().kv_store(k, v, cache, slots)


def emu_kv_attention(q, cache: KvCache, table, starts, lengths, scale=None, window=0, max_new=None, out=None, *,
                     stream=None):
    """Causal attention of the rows of q (tokens x heads x D, any token and head
    strides), sequence b's from starts[b] to starts[b + 1], the last of its
    lengths[b] tokens, over the cache.  scale: D ** -0.5 by default; window: how
    many tokens a row sees at most, itself among them (0: all); max_new: rows
    of a sequence at most, None where the caller does not know. It chooses kernels,
    not what is computed (always two launches): without it a batch of next tokens
    goes through those for prompts (96 sequences of 600,000 tokens: 630 us for 196).
    A row that sees nothing is zero, as are the rows before the first
    and behind the last sequence.  out may be q."""
    if stream is not None:
        return _on(stream, emu_kv_attention, q, cache, table, starts, lengths, scale, window, max_new, out)
    if scale is None:
        scale = q.size(-1) ** -0.5
    return _C().kv_attention(q, cache, table, starts, lengths, scale, window, max_new or 0, out)
