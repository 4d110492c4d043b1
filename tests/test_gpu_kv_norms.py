"""Attention over keys and values kept in 8 bits, on the GPU: what the elementwise
bounds of test_gpu_kv_attention.py cannot see (kv_norms.py), and values whose sizes
lie far apart."""
import gc
import math

import pytest

import kv_norms as norms
import kv_ref as ref
from gpu_util import emu_module
from test_gpu_kv_attention import TYPES, _check, _error, _ints, _make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()                                     # tensors that graphs and tracebacks still hold


def _type(type):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[type]


def _attend(emu, made, **how):
    q, cache, table, starts, lengths = made
    return emu.emu_kv_attention(q, cache, table, _ints(starts), _ints(lengths), **how)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("n", [1, 40, 140])
@pytest.mark.parametrize("zero_first", [True, False])
def test_zero_values_with_the_largest_scores(emu, type, n, zero_first):
    """Pages of zero values have the least scale there is; other pages' values are finite beside them,
    and count where their weights do (those below 2^-126 of the row's largest may be left out)."""
    import torch
    for scale in (1.0, 2.0 ** 3, 2.0 ** 9, 2.0 ** 20, 2.0 ** 40, 2.0 ** 100):
        for gap in (60, 80, 88, 120, 208):
            made = norms.far_below(0.0, scale, gap, n, zero_first)
            made = (made[0].to(_type(type)), *made[1:])
            out = _attend(emu, made, scale=1 / 64, max_new=n)
            want, bound = ref.attention(*made[:1], *made[1], *made[2:], 1 / 64)
            assert not torch.isnan(out).any(), (scale, gap)
            assert ref.within(out, want, bound + (norms.flushed(made) if gap > 83 else 0.0)), (scale, gap)
    assert _error(emu) == 0


@pytest.mark.parametrize("kept,new,Hq,Hk,D", [([20011], [1], 8, 2, 128), ([9000, 10], [3, 4], 4, 1, 64), ([3000, 700], [300, 129], 4, 2, 128),
                                              ([40000, 300], [40, 50], 4, 1, 128), ([900], [700], 3, 3, 96), ([1500], [40], 16, 1, 256)])
def test_both_pieces_of_fp32(emu, kept, new, Hq, Hk, D):
    import torch
    made = _make(kept, new, Hq, Hk, D, 32, "f32")
    want = ref.attention(*made[:1], *made[1], *made[2:], D ** -0.5)[0]
    for most in (max(new), 1):                       # (kernels for many rows, and for few)
        out = _attend(emu, made, max_new=most)
        for b in range(len(kept)):
            rows = slice(made[3][b], made[3][b + 1])
            assert norms.relative(out[rows], want[rows]) <= norms.TWO_PIECES


# Sums of one sign, segments that one CTA goes through alone.  The products' accumulators round toward zero, half a step (2^-24) of
# the sum on the average: what an FP32 sum may lose is bounded by its parts of 64 such additions (32 steps, 2^-25 each on the average as
# it grows), 2e-6 with the rest; in 16 bits by half a step of the type's 11 bits.
@pytest.mark.parametrize("n,B,most", [(128, 40, 128), (4, 120, 4)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L", [1000, 8000, 40000])
def test_long_sums_of_one_sign(emu, n, B, most, D, L):
    import torch
    made = norms.one_sign(torch.float32, n, B, L, D, 4)
    out = _attend(emu, made, max_new=most)
    rows = [0, n * (B // 2) + n // 2, n * B - 1]
    assert norms.relative(out[rows], norms.rows_exactly(made, rows)) <= 3e-6
    assert _error(emu) == 0


@pytest.mark.parametrize("n,B,L", [(128, 40, 200000), (300, 20, 200000), (4, 120, 400000)])
def test_long_sums_in_16_bits(emu, n, B, L):
    """The mean error stays below a quarter of FP16's half step: roundings of weights and outputs average out, what sums
    lose does not."""
    import torch
    made = norms.one_sign(torch.float16, n, B, L, 64, 4)
    out = _attend(emu, made, max_new=n)
    rows = [n * b + (n // 12 * b) % n for b in range(0, B, max(1, B // 12))]
    want = norms.rows_exactly(made, rows)
    assert abs(float((out[rows].double() / want - 1).mean())) <= 2.0 ** -14
    assert _error(emu) == 0


@pytest.mark.parametrize("type,most", [("bf16", 2.0 ** -8), ("f16", 2.0 ** -11)])
@pytest.mark.parametrize("D", [48, 64, 128, 192, 256])
@pytest.mark.parametrize("n,B", [(2, 160), (12, 120)])
def test_sums_in_parts_of_few_rows(emu, type, most, D, n, B):
    """Next tokens and drafts whose warps have hundreds of steps each."""
    import torch
    made = norms.one_sign(_type(type), n, B, 70000, D, 4)
    out = _attend(emu, made, max_new=n)
    rows = [0, n * (B // 3) + n - 1, n * B - 1]
    assert norms.relative(out[rows], norms.rows_exactly(made, rows)) <= most
    assert torch.isfinite(out).all() and _error(emu) == 0


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("D", [16, 48, 96, 128])
@pytest.mark.parametrize("n,window", [(100, 0), (300, 0), (300, 12000), (129, 5000)])
def test_sums_in_parts(emu, type, D, n, window):
    """Segments whose outputs are added up in several parts, with a NaN that some rows see."""
    import torch
    q, cache, table, starts, lengths = _make([20000, 5], [n, n], 2, 2, D, 32, type, seed=D)
    v = cache[1].float()
    at = lengths[0] - n // 2
    v[int(table[0, at // 32]), 1, at % 32, 3] = math.nan
    _check(emu, (q, (cache[0], v.to(ref.F8), *cache[2:]), table, starts, lengths), window=window)


@pytest.mark.parametrize("type,own,large", [("f32", norms.TWO_PIECES, 2.0 ** -38), ("bf16", 2.0 ** -8, 2.0 ** -32), ("f16", 2.0 ** -11, 2.0 ** -32)])
@pytest.mark.parametrize("gap", [0, 7, 11, 14, 18])
@pytest.mark.parametrize("n", [1, 140])
def test_weights_beside_a_large_one(emu, type, own, large, gap, n):
    """Rows whose first token has nearly all the weight, and zero values: the others count as the header says, to a share of
    themselves or of that one (times a value of the size 100 2^-7, independent in 700 tokens)."""
    import torch
    q, cache, table, starts, lengths = _make([700], [n], 4, 2, 64, 32, type, size=(-7, -7))
    k, v = cache[0].float(), cache[1].float()
    page = int(table[0, 0])
    # its score: the queries' first value times its code, 2^-7 and 1/8; no other code there
    k[..., 0] = 0.0
    k[page, :, 0, 0] = min(448.0, gap * 32.0)
    q[..., 0] = gap * 1024.0 / max(float(k[page, 0, 0, 0].to(ref.F8)), 1.0)
    v[page, :, 0] = 0.0
    made = (q, (k.to(ref.F8), v.to(ref.F8), *cache[2:]), table, starts, lengths)
    want = ref.attention(q, *made[1], table, starts, lengths, 0.125)[0]
    out = _attend(emu, made, scale=0.125, max_new=n)
    size = 2.0 ** -7 * 100 * math.sqrt(840 * want.numel())
    least = 2.0 ** -25 * math.sqrt(want.numel()) if type == "f16" else 0.0   # of FP16 outputs
    assert float((out.double() - want).norm()) <= own * float(want.norm()) + large * size + least
    assert _error(emu) == 0


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("n", [1, 40, 140])
def test_infinite_queries_and_codes_of_one_sign(emu, type, n):
    """All scores are the same infinity, of which no softmax is a number, and rows that see nothing are zero still."""
    import torch
    q, cache, table, starts, lengths = _make([100], [n], 4, 2, 64, 32, type)
    for sign in (1.0, -1.0):
        k = cache[0].float()
        k[..., 5] = sign * k[..., 5].abs().clamp(min=1.0)
        for value in (math.inf, -math.inf):
            x = q.clone()
            x[0, 1, 5] = value
            made = (x, (k.to(ref.F8), *cache[1:]), table, starts, lengths)
            out = _attend(emu, made, max_new=n)
            others = torch.ones(x.shape[:2], dtype=torch.bool, device="cuda")
            others[0, 1] = False
            x = torch.where(others[..., None], x, 0.0)
            want, bound = ref.attention(x, *made[1], table, starts, lengths, 0.125)
            assert torch.isnan(out[0, 1]).all(), (sign, value)
            assert ref.within(out[others], want[others], bound[others])
            assert not _attend(emu, (*made[:4], [0]), max_new=n).any()
    assert _error(emu) == 0


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("n", [1, 100])
def test_rows_before_the_first_sequence(emu, type, n):
    """Rows that no sequence has are zero, before the first one as behind the last."""
    import torch
    q, cache, table, starts, lengths = _make([50, 9], [n, n], 4, 2, 64, 16, type, behind=7)
    starts = [s + 4 for s in starts]
    out = torch.full_like(q, 7.0)
    _attend(emu, (q, cache, table, starts, lengths), max_new=n, out=out)
    want, bound = ref.attention(q, *cache, table, starts, lengths, 0.125)
    assert ref.within(out, want, bound) and not out[:4].any() and not out[2 * n + 4:].any()
    assert _error(emu) == 0


@pytest.mark.parametrize("type", TYPES)
def test_same_bits_of_all_types(emu, type):
    import torch
    made = _make([5000, 100, 3000, 0], [1, 4, 1, 300], 8, 2, 128, 16, type)
    for most in (4, None):                           # (kernels for few rows, and for many)
        first = _attend(emu, made, max_new=most)
        for _ in range(10):
            assert torch.equal(_attend(emu, made, max_new=most), first)
