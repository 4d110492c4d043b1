"""A transformer block on the emulated FP32 GEMM: the operators of layers.py
as torch modules, and a small decoder block that runs them together.

  EmuGatedLinear   act(x Wg^T) * (x Wu^T), forward and backward
  qk_norm_rope     norm and rotation of query and key heads, forward and
                   backward
  EmuDecoderBlock  norm, one projection to queries, keys and values (with each
                   token's low-rank adapter where adapters are given), norm and
                   rotation of the heads, attention (for serving over the pages
                   of a KvCache, many sequences at once), output projection;
                   norm, gated feed-forward, down projection

The operators have first derivatives; a derivative of a gradient (a loss made of
forces) raises.

``python -m fp32_emulated_gemm_split_gb300.block`` runs the block on a prompt,
then token by token on the same sequence, and prints how far the two are apart;
then on three sequences at once whose keys and values are kept in 8 bits, and
prints how far that is from keeping them in FP32.
"""
from __future__ import annotations

import math
from typing import NamedTuple

import torch

from .layers import (KvCache, KvPlan, emu_gated, emu_gated_bwd, emu_gated_pack, emu_kv_attention, emu_kv_cache, emu_kv_store,
                     emu_kv_tables, emu_lora, emu_lora_pack, emu_qk_norm_rope, emu_qk_norm_rope_bwd, version_of)
from .linear import EmuLinear, as_rows, readable, underivable


class _GatedFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, up, act):
        x2 = as_rows(x, x.shape[-1])
        w = emu_gated_pack(gate, up)
        h, g, u = emu_gated(x2, w, act=act, save=True)
        ctx.save_for_backward(x, x2, g, u)
        ctx.w, ctx.act, ctx.weights = w, act, (gate, up)
        return h.view(*x.shape[:-1], gate.shape[0])

    @staticmethod
    def backward(ctx, dh):
        x, x2, g, u = ctx.saved_tensors
        dh2 = as_rows(dh, dh.shape[-1])
        need_w = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        dx, dg, du = emu_gated_bwd(dh2, x2, ctx.w, g, u, act=ctx.act, need_dx=ctx.needs_input_grad[0],
                                   need_dw=need_w)
        if dx is not None:
            dx = dx.view(x.shape)
        return (*underivable("EmuGatedLinear", (dx, dg, du), dh, x, *ctx.weights), None)


class EmuGatedLinear(torch.nn.Module):
    """act(x Wg^T) * (x Wu^T) with FP32 parameters ``gate`` and ``up``
    (hidden x in).  A call that needs no gradients uses the weights as
    ``pack()`` laid them out, if it was called; otherwise each call lays them
    out itself.

    ``pack()`` keeps the weights' values of its time: a copy (4 bytes a value,
    for few rows) and the pieces (6 bytes).  A call after the parameters were
    changed in place, replaced, or given other data is refused: call ``pack()``
    again (``train()`` drops what it made; a copy of the module has none).  What
    is written in place through ``parameter.data`` leaves no trace that could
    be looked at: it takes effect with the next ``pack()``."""

    def __init__(self, in_features, hidden_features, activation="silu", device=None):
        super().__init__()
        std = in_features ** -0.5
        shape = (hidden_features, in_features)
        self.gate = torch.nn.Parameter(torch.randn(shape, device=device) * std)
        self.up = torch.nn.Parameter(torch.randn(shape, device=device) * std)
        self.activation = activation
        self._packed = self._packed_of = None

    def _weights(self):
        """What tells today's parameters from others."""
        return [(w.data_ptr(), version_of(w), w.shape, w.stride(), w.device) for w in (self.gate, self.up)]

    def pack(self):
        gate, up = self.gate.detach(), self.up.detach()
        self._packed = emu_gated_pack(*(w.clone(memory_format=torch.contiguous_format) for w in (gate, up)))
        # gate and up are held, so that no other tensor gets their addresses
        self._packed_of = self._weights(), gate, up
        return self

    def __getstate__(self):
        return {**self.__dict__, "_packed": None, "_packed_of": None}

    def train(self, mode=True):
        if mode:
            self._packed = self._packed_of = None
        return super().train(mode)

    def forward(self, x):
        if x.dtype != torch.float32:
            raise TypeError("EmuGatedLinear computes FP32 in and out")
        if torch.is_grad_enabled() and (x.requires_grad or self.gate.requires_grad or self.up.requires_grad):
            return _GatedFn.apply(readable(x), self.gate, self.up, self.activation)
        w = self._packed
        if w is None:
            w = emu_gated_pack(self.gate, self.up)
        elif self._packed_of[0] != self._weights():
            raise ValueError("the weights were changed since pack(): call it again")
        x2 = as_rows(x, x.shape[-1])
        return emu_gated(x2, w, act=self.activation).view(*x.shape[:-1], self.gate.shape[0])


class _QkFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin, positions, eps, interleaved):
        ctx.save_for_backward(q, k, wq, wk, cos, sin, positions)
        ctx.how = dict(eps=eps, interleaved=interleaved)
        return emu_qk_norm_rope(q, k, wq, wk, cos, sin, positions, **ctx.how)

    @staticmethod
    def backward(ctx, dq, dk):
        unit = [d if d.stride(-1) == 1 else d.contiguous() for d in (dq, dk)]
        saved = ctx.saved_tensors
        grads = emu_qk_norm_rope_bwd(*unit, *saved, **ctx.how)
        return (*underivable("qk_norm_rope", grads, dq, dk, *saved[:4]), None, None, None, None, None)


def qk_norm_rope(q, k, wq, wk, cos, sin, positions, eps=1e-6, interleaved=False):
    """``emu_qk_norm_rope`` with gradients for q, k, wq and wk."""
    return _QkFn.apply(q, k, wq, wk, cos, sin, positions, eps, interleaved)


def rotary_tables(positions, rot, base=10000.0, device=None):
    """cos and sin (positions x rot/2) of the usual geometric frequencies."""
    at = torch.arange(positions, device=device, dtype=torch.float64)[:, None]
    f = base ** (-torch.arange(rot // 2, device=device, dtype=torch.float64) * 2 / rot)
    return (at * f).cos().float(), (at * f).sin().float()


class KvStep(NamedTuple):
    """What a step of many sequences attends to: a block's cache, the sequences'
    pages (``table``) and the step's places (``emu_kv_tables``); max_new as in
    ``emu_kv_attention``: 1 for a step of next tokens, which is three times as slow
    without.  The blocks of a model have a cache each and share the rest."""

    cache: KvCache
    table: torch.Tensor
    plan: KvPlan
    max_new: int | None = None


class EmuDecoderBlock(torch.nn.Module):
    """One decoder block, FP32.  ``forward(x, start)`` takes tokens x width and
    the position of the first token, attends to the keys and values kept from
    earlier calls, which have to stand before it, when ``keep`` is true (to its
    own tokens otherwise), and adds the adapters' part to the first projection
    where ``adapters`` = (A, B, scale) and ``index`` are given.  That part is for
    serving: it has no backward pass, and where a gradient would have to go
    through it the call raises.

    With ``kv`` (a KvStep) the rows of x are the new tokens of many sequences, in the
    plan's order: their keys and values are rounded into the cache's pages, and each
    attends to its own sequence's.  For serving, too; ``start`` and ``keep`` do not
    go with it.  Rows behind the last sequence come out of a block as any others do
    that attend to nothing."""

    def __init__(self, width, heads, kv_heads, hidden, max_positions=4096, eps=1e-6, device="cuda"):
        super().__init__()
        self.heads, self.kv_heads, self.dim, self.eps = heads, kv_heads, width // heads, eps
        ones = lambda n: torch.nn.Parameter(torch.ones(n, device=device))  # noqa: E731
        self.norm1, self.norm2 = ones(width), ones(width)
        self.wq, self.wk = ones(self.dim), ones(self.dim)
        self.qkv = EmuLinear(width, (heads + 2 * kv_heads) * self.dim, bias=False, device=device)
        self.out = EmuLinear(heads * self.dim, width, bias=False, device=device)
        self.gated = EmuGatedLinear(width, hidden, device=device)
        self.down = EmuLinear(hidden, width, bias=False, device=device)
        cos, sin = rotary_tables(max_positions, self.dim, device=device)
        self.register_buffer("cos", cos)
        self.register_buffer("sin", sin)
        self.kept = None

    def _norm(self, x, w):
        return x * (x.square().mean(-1, keepdim=True) + self.eps).rsqrt() * w

    def _attention(self, q, k, v):
        """Plain causal attention; the queries are the last of the keys' tokens."""
        group = self.heads // self.kv_heads
        k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
        s = torch.einsum("qhd,khd->hqk", q, k) / math.sqrt(self.dim)
        before = k.size(0) - q.size(0)
        seen = torch.arange(k.size(0), device=q.device) <= before + torch.arange(q.size(0), device=q.device)[:, None]
        s = s.masked_fill(~seen, float("-inf"))
        return torch.einsum("hqk,khd->qhd", s.softmax(-1), v).reshape(q.size(0), -1)

    def _serves(self, what, *tensors):
        """Raises where a gradient would have to go through what has no backward pass."""
        if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
            raise RuntimeError(f"{what} no backward pass: call the block under torch.no_grad(), or train without them")

    def forward(self, x, start=0, adapters=None, index=None, keep=False, kv=None):
        T, D = x.size(0), self.dim
        if kv is not None:
            if start != 0 or keep:
                raise ValueError("start and keep are one sequence's: with kv the plan has the positions, the cache the tokens")
            if kv.plan.positions.size(0) != T:
                raise ValueError(f"the plan has places for {kv.plan.positions.size(0)} rows, x has {T}")
        elif start < 0 or start + T > self.cos.size(0):
            raise ValueError(f"positions {start} to {start + T - 1} are not all in the tables' {self.cos.size(0)}")
        if keep and start > 0 and (self.kept is None or self.kept[0].size(0) > start):
            held = "none" if self.kept is None else f"{self.kept[0].size(0)} tokens"
            raise ValueError(f"start is {start}: the tokens before it have to be kept, and no others ({held} kept)")
        n = self._norm(x, self.norm1)
        if adapters is None:
            qkv = self.qkv(n)
        else:
            A, B, scale = adapters
            self._serves("the adapters have", n, self.qkv.weight, A, B, scale)
            qkv = emu_lora(n, emu_lora_pack(self.qkv.weight), A, B, index, scale)
        q, k, v = qkv.view(T, -1, D).split((self.heads, self.kv_heads, self.kv_heads), 1)
        if kv is not None:
            self._serves("keys and values in 8 bits have", qkv, self.wq, self.wk)
            q, k = emu_qk_norm_rope(q, k, self.wq, self.wk, self.cos, self.sin, kv.plan.positions, self.eps)
            emu_kv_store(k, v, kv.cache, kv.plan.slots)
            y = emu_kv_attention(q, kv.cache, kv.table, kv.plan.starts, kv.plan.lengths, max_new=kv.max_new)
            x = x + self.out(y.view(T, -1))
            return x + self.down(self.gated(self._norm(x, self.norm2)))
        positions = torch.arange(start, start + T, device=x.device, dtype=torch.int32)
        q, k = qk_norm_rope(q, k, self.wq, self.wk, self.cos, self.sin, positions, self.eps)
        if keep:
            if start > 0:
                k, v = torch.cat((self.kept[0], k)), torch.cat((self.kept[1], v))
            self.kept = k, v
        x = x + self.out(self._attention(q, k, v))
        return x + self.down(self.gated(self._norm(x, self.norm2)))


def main():
    torch.manual_seed(0)
    width, T, new = 512, 100, 8
    block = EmuDecoderBlock(width, 8, 2, 1408).eval()
    A = torch.randn(3, 8, width, device="cuda") / width ** 0.5
    B = torch.randn(3, block.qkv.out_features, 8, device="cuda") / 8 ** 0.5
    adapters = (A, B, torch.tensor([0.5, 1.0, 2.0], device="cuda"))
    x = torch.randn(T + new, width, device="cuda")
    index = torch.full((T + new,), 1, device="cuda", dtype=torch.int32)
    with torch.no_grad():
        whole = block(x, adapters=adapters, index=index)
        block.gated.pack()
        parts = [block(x[:T], adapters=adapters, index=index[:T], keep=True)]
        for t in range(T, T + new):
            parts.append(block(x[t:t + 1], start=t, adapters=adapters, index=index[t:t + 1], keep=True))
    off = (torch.cat(parts) - whole).norm() / whole.norm()
    print(f"prompt of {T} and {new} single tokens against one pass: {float(off):.2e} apart")

    # three sequences at once, each the first tokens of x, over pages of 8-bit keys and values
    page, pages = 16, 32
    cache = emu_kv_cache(pages, block.kv_heads, block.dim, page=page)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, free = torch.full((3, 8), -1, dtype=torch.int32, device="cuda"), torch.arange(pages, device="cuda", dtype=torch.int32)
    kept, taken, prompts = ints(0, 0, 0), None, (T, 1, 37)
    with torch.no_grad():
        for step in range(new + 1):
            rows = prompts if step == 0 else (1, 1, 1)
            plan = emu_kv_tables(kept, ints(*rows), table, free, pages, page, sum(rows), taken)
            first = prompts if step else (0, 0, 0)
            x_new = torch.cat([x[f + max(step - 1, 0):f + max(step - 1, 0) + n] for f, n in zip(first, rows)])
            y = block(x_new, kv=KvStep(cache, table, plan, max(rows)))
            kept, taken = plan.lengths, plan.taken
        want = torch.stack([block(x[:n + new])[-1] for n in prompts])
    off = (y - want).norm() / want.norm()
    print(f"three sequences over 8-bit keys and values, against FP32: {float(off):.2e} apart")


if __name__ == "__main__":
    main()
