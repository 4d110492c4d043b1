"""Attention over keys and values kept in 8 bits, on the GPU, against its
definition in 64 bits (kv_ref.py has the bound)."""
import gc
import math

import pytest

import kv_ref as ref
from gpu_util import emu_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()                                     # tensors that graphs and tracebacks still hold


def _make(kept, new, Hq, Hk, D, P, type, seed=0, behind=0, spare=2, size=(-9, -4)):
    """q, cache, table, starts, lengths (the last two as lists): pages in random
    order, codes behind a sequence's last token NaN."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    lengths = [k + n for k, n in zip(kept, new)]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    need = [-(-L // P) for L in lengths]
    pages, width = sum(need) + spare, max(need + [0]) + 1
    order = torch.randperm(pages, generator=g, device="cuda").tolist()
    table = torch.full((len(kept), width), -1, dtype=torch.int32)
    codes = [(torch.randn(pages, Hk, P, D, generator=g, device="cuda") * 100).clamp(-448, 448) for _ in range(2)]
    for b, n in enumerate(need):
        for j in range(n):
            table[b, j] = order.pop()
        if lengths[b] % P:
            for c in codes:
                c[table[b, n - 1], :, lengths[b] % P:] = math.nan
    for i in order:
        for c in codes:
            c[i] = math.nan
    scales = [torch.exp2(torch.randint(size[0], size[1] + 1, (pages, Hk), generator=g, device="cuda").float())
              for _ in range(2)]
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[type]
    q = torch.randn(starts[-1] + behind, Hq, D, generator=g, device="cuda").to(dtype)
    cache = (codes[0].to(ref.F8), codes[1].to(ref.F8), scales[0], scales[1])
    return q, cache, table.cuda(), starts, lengths


def _error(emu):
    """The device's error word, which is cleared."""
    code = emu.emu_get_last_device_error()
    emu.emu_clear_device_error()
    return code


def _ints(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _check(emu, made, window=0, scale=None, **how):
    q, cache, table, starts, lengths = made
    out = emu.emu_kv_attention(q, cache, table, _ints(starts), _ints(lengths), scale=scale, window=window, **how)
    want, bound = ref.attention(q, *cache, table, starts, lengths, q.size(-1) ** -0.5 if scale is None else scale,
                                window)
    assert ref.within(out, want, bound)
    assert _error(emu) == 0
    return out


TYPES = ["f32", "bf16", "f16"]


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("Hq,Hk,D,P", [(4, 4, 64, 16), (8, 2, 128, 16), (6, 2, 80, 32), (16, 1, 256, 64), (7, 1, 16, 128),
                                       (5, 5, 96, 16), (40, 2, 32, 256), (3, 3, 192, 64), (4, 1, 144, 32)])
def test_next_tokens(emu, type, Hq, Hk, D, P):
    kept = [0, 1, 14, 15, 16, 17, 62, 63, 64, 65, 127, 200, 777]
    _check(emu, _make(kept, [1] * len(kept), Hq, Hk, D, P, type, seed=D), max_new=1)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("Hq,Hk,D,P", [(8, 2, 64, 16), (12, 4, 128, 64), (2, 1, 256, 32), (20, 4, 80, 16)])
@pytest.mark.parametrize("window", [0, 1, 40])
def test_ragged(emu, type, Hq, Hk, D, P, window):
    kept = [0, 5, 100, 0, 33, 300, 64]
    new = [7, 0, 3, 70, 1, 37, 130]
    _check(emu, _make(kept, new, Hq, Hk, D, P, type, seed=window, behind=5), window=window)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("Hq,Hk,D,P,n", [(4, 1, 128, 64, 300), (8, 8, 64, 16, 517), (3, 1, 96, 32, 129), (16, 2, 256, 16, 65)])
@pytest.mark.parametrize("kept", [0, 1, 400])
def test_prompts(emu, type, Hq, Hk, D, P, n, kept):
    _check(emu, _make([kept, 3], [n, 2], Hq, Hk, D, P, type, seed=n))


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("Hq,Hk,D,P,most", [(16, 2, 128, 32, 7), (24, 3, 64, 16, 4), (10, 2, 80, 64, 9), (17, 1, 32, 16, 2),
                                            (16, 1, 256, 32, 3), (40, 1, 112, 128, 1)])
def test_drafts(emu, type, Hq, Hk, D, P, most):
    """A few rows of many heads: 17 to 63 of a sequence and key head."""
    kept = [0, 3, 40, 127, 128, 300, 2000]
    new = [1 + i % most for i in range(len(kept))]
    _check(emu, _make(kept, new, Hq, Hk, D, P, type, seed=most, behind=2), max_new=most)
    _check(emu, _make(kept, new, Hq, Hk, D, P, type, seed=most), max_new=most, window=35)


@pytest.mark.parametrize("type", TYPES)
def test_long_and_many(emu, type):
    _check(emu, _make([20011], [1], 8, 2, 128, 16, type))
    _check(emu, _make([9000, 10], [3, 4], 4, 1, 64, 128, type))
    _check(emu, _make([(37 * i) % 211 for i in range(700)], [1 + (i % 7 == 0) for i in range(700)], 4, 2, 64, 16, type))


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("D", list(range(16, 257, 16)))
def test_many_steps(emu, type, D):
    """Long enough that every stage of every ring is filled and read, and pages are looked up ahead."""
    import torch
    for P, G, window in ((16, 3, 0), (64, 9, 700)):
        q, cache, table, starts, lengths = _make([2500 + 33 * i for i in range(30)], [1 + i % 2 for i in range(30)], 8 * G, 8,
                                                 D, P, type, seed=D)
        for most in (2, None):                       # (kernels for few rows, and for many)
            out = emu.emu_kv_attention(q, cache, table, _ints(starts), _ints(lengths), window=window, max_new=most)
            for b in (0, 13, 29):                    # (the reference of all would take long)
                rows = slice(starts[b], starts[b + 1])
                want, bound = ref.attention(q[rows], *cache, table[b:b + 1], [0, starts[b + 1] - starts[b]], [lengths[b]],
                                            D ** -0.5, window)
                assert ref.within(out[rows], want, bound)
            assert torch.isfinite(out).all() and _error(emu) == 0


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("window", [0, 300])
def test_many_tiles(emu, type, D, window):
    """Prompts of more tiles than the GPU has SMs, of different lengths: every CTA has parts of several."""
    new = [700, 1, 0, 333, 1025, 64]
    made = _make([0, 600, 50, 1000, 129, 3], new, 10, 2, D, 32, type, seed=D, behind=3)
    _check(emu, made, window=window)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("n", [1, 200])
def test_zeros(emu, type, n):
    """Keys and values of zero, as the store leaves them (scale 2^-126), alone and beside others."""
    import torch
    q, cache, table, starts, lengths = _make([100, 100], [n, n], 4, 2, 64, 32, type)
    for pages in (table[0], table[0, 1:3]):
        k, v, ks, vs = (x.clone() for x in cache)
        at = pages[pages >= 0].long()
        for codes, scale in ((k, ks), (v, vs)):
            codes.view(torch.uint8)[at] = 0
            scale[at] = 2.0 ** -126
        out = _check(emu, (q, (k, v, ks, vs), table, starts, lengths), max_new=n)
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("scale", [0.0, -0.3, 40.0])
def test_scale(emu, type, scale):
    for kept, new in (([70, 9], [1, 1]), ([70, 9], [40, 150])):
        _check(emu, _make(kept, new, 4, 2, 64, 32, type), scale=scale, max_new=max(new))


@pytest.mark.parametrize("D", [64, 256])
def test_max_new_is_a_hint(emu, D):
    """Too small a max_new changes kernels only."""
    made = _make([300, 40], [30, 3], 6, 2, D, 16, "f32")
    for most in (1, 2, 30, 1000):
        _check(emu, made, max_new=most)


def test_rows_that_see_nothing(emu):
    """Length 0, fewer tokens than rows, rows behind the last sequence, no sequence."""
    import torch
    q, cache, table, starts, lengths = _make([0, 20], [2, 6], 4, 2, 64, 16, "f32", behind=3)
    lengths = [0, 4]
    out = _check(emu, (q, cache, table, starts, lengths))
    assert not out[:4].any() and not out[8:].any() and out[4:8].any()
    none = emu.emu_kv_attention(q, cache, table[:0], _ints([0]), _ints([]))
    assert none.shape == q.shape and not none.any()
    assert emu.emu_kv_attention(q[:0], cache, table[:0], _ints([0]), _ints([])).shape == (0, 4, 64)
    torch.cuda.synchronize()


@pytest.mark.parametrize("type", TYPES)
def test_nan_where_nothing_looks(emu, type):
    """NaN in a key or value reaches the rows that see it and no others."""
    import torch
    made = _make([30, 50], [5, 150], 6, 2, 64, 32, type)
    q, cache, table, starts, lengths = made
    k, v = cache[0].float(), cache[1].float()
    for codes, at in ((k, (0, 33)), (v, (0, 32)), (v, (1, 130)), (k, (1, 60)), (v, (1, 199))):
        page, row = int(table[at[0], at[1] // 32]), at[1] % 32
        codes[page, 1, row, 3] = math.nan
    made = (q, (k.to(ref.F8), v.to(ref.F8), *cache[2:]), table, starts, lengths)
    for window in (0, 20):
        out = _check(emu, made, window=window)
        assert torch.isnan(out).any() and not torch.isnan(out[:, :3]).any()


@pytest.mark.parametrize("type", TYPES)
def test_scales_far_apart(emu, type):
    """Pages whose scales differ by many powers of two: values of a small one
    count fully where their weights do."""
    import torch
    q, cache, table, starts, lengths = _make([150], [3], 4, 2, 64, 16, type, size=(-7, -5))
    vs = cache[3].clone()
    vs[table[0, 2].long()] = 2.0 ** 40
    vs[table[0, 5].long()] = 2.0 ** -100
    k = cache[0].float()
    k[table[0, 2].long()] = -448 * torch.sign(q.float().mean((0, 1)))
    _check(emu, (q, (k.to(ref.F8), cache[1], cache[2], vs), table, starts, lengths))
    # queries from the smallest to the largest
    for e in (-100, -30, 30, 60):
        if type == "f16" and abs(e) > 14:
            continue
        big = (q.float() * 2.0 ** e).to(q.dtype)
        ks = torch.full_like(cache[2], 2.0 ** (-e - 7))
        _check(emu, (big, (cache[0], cache[1], ks, cache[3]), table, starts, lengths))


def test_strides_and_in_place(emu):
    import torch
    q, cache, table, starts, lengths = _make([40, 9], [3, 20], 4, 2, 64, 16, "bf16")
    want = _check(emu, (q, cache, table, starts, lengths))
    for odd in (0, 1):
        wide = torch.zeros(23, 4 * 70 + odd, device="cuda", dtype=q.dtype)
        view = wide[:, :280].view(23, 4, 70)[..., 2 - odd:66 - odd]
        view.copy_(q)
        out = torch.full_like(wide, 7.0)
        here = out[:, :280].view(23, 4, 70)[..., 2 - odd:66 - odd]
        got = emu.emu_kv_attention(view, cache, table, _ints(starts), _ints(lengths), out=here)
        assert got.data_ptr() == here.data_ptr() and torch.equal(here, want)
        here.fill_(7.0)
        assert (out == 7.0).all()
        emu.emu_kv_attention(view, cache, table, _ints(starts), _ints(lengths), out=view)
        assert torch.equal(view, want)
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(emu.emu_kv_attention(turned, cache, table, _ints(starts), _ints(lengths)), want)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_strides_and_in_place_of_prompts(emu, type, D):
    import torch
    q, cache, table, starts, lengths = _make([40, 700], [150, 33], 6, 2, D, 32, type, behind=2)
    want = _check(emu, (q, cache, table, starts, lengths))
    for odd in (0, 1):
        wide = torch.zeros(185, 6 * (D + 16) + odd, device="cuda", dtype=q.dtype)
        view = wide[:, odd:odd + 6 * (D + 16)].view(185, 6, D + 16)[..., :D]
        view.copy_(q)
        out = torch.full_like(wide, 7.0)
        here = out[:, odd:odd + 6 * (D + 16)].view(185, 6, D + 16)[..., :D]
        emu.emu_kv_attention(view, cache, table, _ints(starts), _ints(lengths), out=here)
        assert torch.equal(here, want)
        here.fill_(7.0)
        assert (out == 7.0).all()
        emu.emu_kv_attention(view, cache, table, _ints(starts), _ints(lengths), out=view)
        assert torch.equal(view, want)


def test_same_bits_again(emu):
    import torch
    made = _make([5000, 100, 3000], [1, 4, 1], 8, 2, 128, 16, "f32")
    q, cache, table, starts, lengths = made
    args = (q, cache, table, _ints(starts), _ints(lengths))
    for most in (4, None):                           # (both kernels)
        first = emu.emu_kv_attention(*args, max_new=most)
        for _ in range(20):
            assert torch.equal(emu.emu_kv_attention(*args, max_new=most), first)


def test_bad_values_on_the_device(emu):
    """Page numbers, lengths and starts out of range: an error word, NaN where
    they count, the other sequences as they are."""
    import torch
    q, cache, table, starts, lengths = _make([70, 70, 70], [2, 2, 2], 4, 2, 64, 16, "f32")
    want = emu.emu_kv_attention(q, cache, table, _ints(starts), _ints(lengths))
    for page in (-1, cache[0].size(0), 1 << 30):
        bad = table.clone()
        bad[1, 1] = page
        out = emu.emu_kv_attention(q, cache, bad, _ints(starts), _ints(lengths))
        assert _error(emu) == -1
        assert torch.isnan(out[2:4]).all() and torch.equal(out[:2], want[:2]) and torch.equal(out[4:], want[4:])
    for length in (-1, table.size(1) * 16 + 1, 1 << 30):
        out = emu.emu_kv_attention(q, cache, table, _ints(starts), _ints([lengths[0], length, lengths[2]]))
        assert _error(emu) == -1
        assert torch.isnan(out[2:4]).all() and torch.equal(out[:2], want[:2]) and torch.equal(out[4:], want[4:])
    for wrong in ([0, 2, 1, 6], [0, 2, 9, 6], [0, -2, 2, 6]):
        emu.emu_kv_attention(q, cache, table, _ints(wrong), _ints(lengths))
        assert _error(emu) == -1
    assert torch.equal(emu.emu_kv_attention(q, cache, table, _ints(starts), _ints(lengths)), want)
    assert _error(emu) == 0


def test_stream_and_graph(emu):
    """Another stream; a captured call replayed with other lengths and values, while a
    larger call runs in between."""
    import torch
    made = _make([300, 40], [2, 1], 8, 2, 128, 16, "bf16")
    q, cache, table, starts, lengths = made
    want = _check(emu, made)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = emu.emu_kv_attention(q, cache, table, _ints(starts), _ints(lengths), stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    s, n = _ints(starts), _ints(lengths)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = emu.emu_kv_attention(q, cache, table, s, n)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    _check(emu, _make([30000], [1], 16, 2, 256, 16, "f32"))
    n.copy_(_ints([290, 33]))
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    other, bound = ref.attention(q, *cache, table, starts, [290, 33], 128 ** -0.5)
    assert ref.within(out, other, bound)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("most,window", [(100, 0), (30, 0), (30, 70)])
def test_many_short_segments(emu, type, most, window):
    """Hundreds of sequences of a tile or two, most of one unit: a CTA goes through many
    segments, of which many have no second tile."""
    kept = [(37 * b) % 90 if b % 9 else (211 * b) % 700 for b in range(400)]
    new = [1 + (53 * b) % most for b in range(400)]
    _check(emu, _make(kept, new, 8, 2, 64, 16, type), window=window, max_new=100)


@pytest.mark.parametrize("type", TYPES)
def test_one_segment_over_all(emu, type):
    """A few tiles with hundreds of units, and one with fewer than CTAs."""
    _check(emu, _make([40000, 300], [40, 50], 4, 1, 128, 64, type))


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("n", [1, 200])
def test_queries_that_are_not_finite(emu, type, n):
    """They change their own rows only."""
    import torch
    q, cache, table, starts, lengths = _make([300, 40], [n, n], 4, 2, 64, 16, type)
    want, bound = ref.attention(q, *cache, table, starts, lengths, 0.125, 0)
    at = {(0, 1): math.nan, (n, 0): math.inf, (2 * n - 1, 3): -math.inf}
    others = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    for (row, head), value in at.items():
        q[row, head, 5] = value
        others[row, head] = False
    out = emu.emu_kv_attention(q, cache, table, _ints(starts), _ints(lengths), scale=0.125, max_new=n)
    assert torch.isnan(out[0, 1]).all()
    assert ref.within(out[others], want[others], bound[others])
    assert _error(emu) == 0


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("n", [2, 150])
def test_expanded_queries(emu, type, n):
    """One head's queries for all heads, one token's for all tokens."""
    import torch
    q, cache, table, starts, lengths = _make([70, 20], [n, n], 4, 2, 128, 32, type)
    for wide in (q[:, :1].expand(-1, 4, -1), q[:1].expand(2 * n, -1, -1)):
        got = emu.emu_kv_attention(wide, cache, table, _ints(starts), _ints(lengths))
        assert torch.equal(got, emu.emu_kv_attention(wide.contiguous(), cache, table, _ints(starts), _ints(lengths)))
