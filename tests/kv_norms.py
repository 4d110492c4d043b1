"""What a bound for each element cannot see of the attention over 8-bit keys and
values: relative errors of whole sequences, where roundings that are independent
average out and a lost piece, or a sum that drifts, does not."""
import math

import torch

# FP32 rows.  A weight is two FP16 pieces (2^-23 of itself) times two approximate powers of two, its score off by a few 2^-23 of
# its size: some 1e-6 in all, with either sign, so less in a sum of many.  One piece of the queries or of the weights: 1e-4.
TWO_PIECES = 5e-6


def relative(got, want):
    """The Frobenius norm of the difference over want's."""
    return float((got.double() - want).norm() / want.norm())


def halves(x, pieces):
    """x (float64) as the sum of so many FP16 values, scaled so that a row's largest lies in 2^14..2^15."""
    up = torch.exp2(15 - torch.frexp(x.abs().amax(-1, keepdim=True).clamp(min=1e-300))[1].double())
    left, sum = x * up, torch.zeros_like(x)
    for _ in range(pieces):
        h = left.half().double()
        sum, left = sum + h, left - h
    return sum / up


def in_pieces(q, K, V, of_q, of_p):
    """Attention of one token (heads x D) over all of K and V (tokens x heads x D) in float64, the queries and the weights held in
    so many FP16 pieces."""
    s = torch.einsum("hd,lhd->hl", halves(q.double(), of_q), K) * q.size(-1) ** -0.5
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return torch.einsum("hl,lhd->hd", halves(p, of_p), V) / p.sum(-1, keepdim=True)


def one_sign(type, n, B, L, D, Hk, P=64, seed=0, device="cuda"):
    """B sequences of L tokens, the last n of them rows, over the same pages; scores of ordinary size, values all positive."""
    g = torch.Generator(device=device).manual_seed(seed)
    pages = -(-L // P)

    def codes(size, more):
        x = torch.randn(pages, Hk, P, D, generator=g, device=device) * size + more
        return x.clamp(-448, 448).to(torch.float8_e4m3fn)
    cache = (codes(100, 0), codes(40, 200), torch.full((pages, Hk), 2.0 ** -7, device=device),
             torch.exp2(torch.randint(-8, -5, (pages, Hk), generator=g, device=device).float()))
    table = torch.randperm(pages, generator=g, device=device).to(torch.int32).expand(B, -1).contiguous()
    q = torch.randn(B * n, Hk, D, generator=g, device=device).to(type)
    return q, cache, table, [n * b for b in range(B + 1)], [L] * B


def rows_exactly(made, rows):
    """The outputs of some rows (all of the sequences have as many) in float64, without a window."""
    q, (k, v, ks, vs), table, starts, lengths = made
    Hk, P, D, n = k.size(1), k.size(2), k.size(3), starts[1]
    out = []
    for row in rows:
        b, L = row // n, lengths[row // n] - n + row % n + 1
        pages = table[b, : -(-L // P)].long()
        K, V = ((c[pages].double() * s[pages].double()[..., None, None]).transpose(1, 2).reshape(-1, Hk, D)[:L]
                .repeat_interleave(q.size(1) // Hk, 1) for c, s in ((k, ks), (v, vs)))
        s = torch.einsum("hd,lhd->hl", q[row].double(), K) * D ** -0.5
        out.append(torch.einsum("hl,lhd->hd", s.softmax(-1), V))
    return torch.stack(out)


def far_below(top, scale, gap, n, zero_first, Hq=4, Hk=2, D=64, P=16, pages=10, device="cuda"):
    """One sequence whose page of zero values (scale 2^-126, as the store leaves it) has the largest scores, and whose other
    pages, of the value scale `scale`, have scores lower by `gap` (an e4m3 value) and a bit: q = 1, scale 1 / D."""
    g = torch.Generator(device=device).manual_seed(n)
    L = pages * P - 3
    k = -gap + torch.randn(pages, Hk, P, D, generator=g, device=device) * gap / 64
    v = torch.randn(pages, Hk, P, D, generator=g, device=device) * 90
    at = 0 if zero_first else 4
    k[at], v[at] = top, 0.0
    vs = torch.full((pages, Hk), scale, device=device)
    vs[at] = 2.0 ** -126
    table = torch.arange(pages, dtype=torch.int32, device=device)[None]
    q = torch.ones(n, Hq, D, device=device)
    f8 = torch.float8_e4m3fn
    return q, (k.clamp(-448, 448).to(f8), v.clamp(-448, 448).to(f8), torch.ones(pages, Hk, device=device), vs), table, [0, n], [L]


def flushed(made):
    """How far outputs may be off where weights below 2^-125 of the row's largest are left out: 2^-125 of all |v|."""
    v, vs = made[1][1], made[1][3]
    return 2.0 ** -125 * float((torch.nan_to_num(v.double()).abs() * vs.double()[..., None, None]).sum((0, 2)).max())
