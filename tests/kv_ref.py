"""Plain implementations of the operators on keys and values kept in 8 bits:
tables and store exactly, the attention in float64 with a bound of what the
kernels may be off, counted in roundings.
"""
import math

import torch

from layer_ref import HALF_ULP, LEAST

F8 = torch.float8_e4m3fn


def tables(kept, new, table, free, page, tokens, taken=0):
    """(table, starts, lengths, slots, positions, taken) as lists, token by token."""
    table, at = [list(r) for r in table], taken
    starts, slots, positions = [0], [], []
    for b, (k, n) in enumerate(zip(kept, new)):
        for j in range(-(-k // page), -(-(k + n) // page)):
            table[b][j] = free[at]
            at += 1
        for p in range(k, k + n):
            slots.append(table[b][p // page] * page + p % page)
            positions.append(p)
        starts.append(len(slots))
    behind = tokens - len(slots)
    return table, starts, [k + n for k, n in zip(kept, new)], slots + [-1] * behind, positions + [0] * behind, at


def e4m3(x):
    """float64 values rounded to e4m3's (|x| <= 448), ties to even."""
    step = torch.exp2((torch.frexp(x)[1] - 1).clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def page_scale(top):
    """The least power of two s >= 2^-126 with top <= 448 s, by trying."""
    e = -126
    while top > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def store(x, codes, scales, slots, page):
    """x (T x heads x D) into copies of codes and scales (float64), run by run."""
    x, codes, scales, slots = x.double().cpu(), codes.double().cpu(), scales.double().cpu(), slots.tolist()
    t = 0
    while t < len(slots):
        if slots[t] < 0 or slots[t] >= codes.size(0) * page:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == slots[t] + n and slots[t + n] % page:
            n += 1
        p, r0 = slots[t] // page, slots[t] % page
        for h in range(x.size(1)):
            run = x[t:t + n, h]
            finite = run[torch.isfinite(run)].abs()
            s = page_scale(float(finite.max()) if finite.numel() else 0.0)
            if r0:
                old = float(scales[p, h])
                s = max(s, old)
                if s > old:
                    others = torch.ones(page, dtype=torch.bool)
                    others[r0:r0 + n] = False
                    codes[p, h, others] = e4m3(codes[p, h, others] * (old / s))
            scales[p, h] = s
            codes[p, h, r0:r0 + n] = torch.where(torch.isfinite(run), e4m3(torch.where(torch.isfinite(run), run, 0.0) / s),
                                                 math.nan)
        t += n
    return codes, scales


def attention(q, k, v, k_scale, v_scale, table, starts, lengths, scale, window=0):
    """(out, bound), float64.  A row's sums leave out what it does not see, NaN
    among it.  What a score may be off, with A = scale s_k sum |q| |K| and u = 2^-24:
    the products' sums (two pieces, D / 16 steps each, a step good to 4 u of A),
    the pieces themselves (2 u; 2^-38 of the row's largest value where that is
    more), 6 roundings of factors; its weight in addition the difference to
    the maximum (2 u of it, twice) and two approximate powers of two (4 u each, and
    as many again where parts are joined); 16-bit rows: the weight's own rounding,
    2^-11.  Sums over tokens: a step of 16 is good to 4 u of the weights' sum of |v|.
    """
    u = 2.0 ** -24
    T, Hq, D = q.shape
    Hk, P = k.size(1), k.size(2)
    G = Hq // Hk
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b, L in enumerate(lengths):
        first, n = starts[b], starts[b + 1] - starts[b]
        if n == 0 or L == 0:
            continue
        pages = table[b, : -(-L // P)].long()

        def dense(codes, scales):
            x = codes[pages].double() * scales[pages].double()[..., None, None]
            return x.transpose(1, 2).reshape(-1, Hk, D)[:L].repeat_interleave(G, 1)
        K, V = dense(k, k_scale), dense(v, v_scale)
        x = q[first:first + n].double()
        at = torch.arange(L - n, L, device=q.device)[:, None]
        token = torch.arange(L, device=q.device)
        seen = (token <= at) & ((token > at - window) if window else torch.ones_like(token, dtype=torch.bool))
        seen = seen[:, None]                                     # n x 1 x L
        some = seen.any(-1, keepdim=True)
        s = torch.einsum("nhd,lhd->nhl", x, K) * scale
        A = torch.einsum("nhd,lhd->nhl", x.abs(), K.abs()) * abs(scale)
        A = A + 2.0 ** -14 * x.abs().amax(-1, keepdim=True) * K.abs().sum(-1).t() * abs(scale)
        s, A = torch.where(seen, s, -math.inf), torch.where(seen, A, 0.0)
        top = torch.where(some, s.amax(-1, keepdim=True), 0.0)
        p = torch.where(seen, torch.exp(s - top), 0.0)
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(some, total, 1.0)
        off = A * (2 * 4 * (D / 16 + 1) + 2 + 6) * u + torch.where(seen, top - s, 0.0) * 4 * u + 16 * u
        off = off + A.amax(-1, keepdim=True) * 6 * u
        if q.dtype != torch.float32:
            off = off + 2.0 ** -11
        clean = torch.nan_to_num(V, nan=0.0)
        y = torch.einsum("nhl,lhd->nhd", p, clean)
        hurt = torch.einsum("nhl,lhd->nhd", seen.double().expand(p.shape), torch.isnan(V).double()) > 0
        size = torch.einsum("nhl,lhd->nhd", p * off, clean.abs()) + (p * off).sum(-1, keepdim=True) * y.abs()
        size = 1.01 * size + (L / 16 + 80) * 4 * u * torch.einsum("nhl,lhd->nhd", p, clean.abs())
        size = size + HALF_ULP.get(q.dtype, 0.0) * (y.abs() + size) + LEAST.get(q.dtype, 0.0) + 1e-37
        out[first:first + n] = torch.where(some, torch.where(hurt, math.nan, y), 0.0)
        bound[first:first + n] = torch.where(some, size, 0.0)
    return out, bound


def within(got, want, bound):
    """Whether got is NaN exactly where want is, infinite where want is past the
    type's largest value, and within the bound elsewhere."""
    info = torch.finfo(got.dtype)
    got = got.double()
    bad = torch.isnan(want)
    if not torch.equal(torch.isnan(got), bad):
        return False
    past = want.abs() - bound > info.max * (1 + info.eps)
    if not torch.equal(got[past], torch.sign(want[past]) * math.inf):
        return False
    # (next to the largest value either is right)
    near = (want.abs() + bound >= info.max) & torch.isinf(got)
    return bool(((got - want).abs() <= bound)[~bad & ~past & ~near].all())
