"""Norm and rotation of query and key heads on the GPU, forward and backward,
against the definition in 64 bits."""
import gc

import pytest

import layer_ref as ref
from gpu_util import emu_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()                                     # tensors that graphs and tracebacks still hold


def _make(T, Hq, Hk, D, rot, dtype, seed, rows=400):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    qkv = (r(T, (Hq + 2 * Hk) * D) * 2).to(getattr(torch, dtype))
    q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    wq, wk = 1 + 0.3 * r(D), 1 + 0.3 * r(D)
    ang = r(rows, rot // 2) * 3
    cos, sin = (ang.cos(), ang.sin()) if rot else (None, None)
    pos = torch.randint(0, rows, (T,), generator=g, device="cuda", dtype=torch.int32) if rot else None
    return q, k, wq, wk, cos, sin, pos


# head sizes: whole 16-byte chunks, powers of two or not; halves that are not; odd; the smallest and largest
CASES = [(1, 1, 1, 64, 64), (3, 4, 2, 128, 128), (5, 8, 1, 96, 96), (7, 3, 3, 80, 40), (2, 6, 2, 256, 64),
         (4, 2, 1, 512, 512), (9, 5, 4, 66, 66), (6, 3, 2, 33, 16), (3, 2, 1, 1, 0), (4, 2, 2, 2, 2), (5, 1, 1, 511, 510),
         (300, 12, 4, 64, 32), (1200, 8, 2, 128, 128), (33, 40, 7, 192, 128), (17, 0, 3, 64, 64), (8, 3, 0, 64, 0)]


@pytest.mark.parametrize("T,Hq,Hk,D,rot", CASES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("pairs", [False, True])
def test_forward_and_backward(emu, T, Hq, Hk, D, rot, dtype, pairs):
    import torch
    q, k, wq, wk, cos, sin, pos = _make(T, Hq, Hk, D, rot, dtype, seed=T + D)
    eps = 1e-5
    got = emu.emu_qk_norm_rope(q, k, wq, wk, cos, sin, pos, eps=eps, interleaved=pairs)
    for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
        assert y.dtype == x.dtype and y.shape == x.shape
        if x.numel():
            want, bound = ref.qk(x, w, cos, sin, pos, eps, pairs)
            assert ref.ratio(y, want, bound) <= 1.0
    dq, dk = torch.randn(q.shape, device="cuda").to(q.dtype), torch.randn(k.shape, device="cuda").to(q.dtype)
    gq, gk, gwq, gwk = emu.emu_qk_norm_rope_bwd(dq, dk, q, k, wq, wk, cos, sin, pos, eps=eps, interleaved=pairs)
    for d, x, w, g, gw in ((dq, q, wq, gq, gwq), (dk, k, wk, gk, gwk)):
        assert g.dtype == x.dtype and g.shape == x.shape and gw.dtype == torch.float32
        if x.numel():
            want, bound = ref.qk_bwd(d, x, w, cos, sin, pos, eps, pairs)
            assert ref.ratio(g, want[0], bound[0]) <= 1.0
            assert ref.ratio(gw, want[1], bound[1]) <= 1.0
        else:
            assert bool((gw == 0).all())
    assert emu.emu_get_last_device_error() == 0


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_in_place_without_weights_and_other_strides(emu, dtype):
    """heads x tokens storage, a sequence in every other row, in place."""
    import torch
    q, k, _, _, cos, sin, pos = _make(50, 6, 2, 64, 64, dtype, seed=4)
    want, bound = ref.qk(q, None, cos, sin, pos, 1e-6, False)
    wide = torch.full((6, 100, 72), float("nan"), device="cuda", dtype=q.dtype)
    qs = wide[:, ::2, :64].transpose(0, 1)
    qs.copy_(q)
    k0 = k.clone()
    out = emu.emu_qk_norm_rope(qs, k0, None, None, cos, sin, pos, out=(qs, k0))
    assert out[0] is qs and out[1] is k0
    assert ref.ratio(qs, want, bound) <= 1.0
    assert bool(torch.isnan(wide[:, 1::2]).all()) and bool(torch.isnan(wide[:, :, 64:]).all())
    want, bound = ref.qk(k, None, cos, sin, pos, 1e-6, False)
    assert ref.ratio(k0, want, bound) <= 1.0
    d = torch.randn(q.shape, device="cuda").to(q.dtype)
    got = emu.emu_qk_norm_rope_bwd(d, torch.zeros_like(k), q, k, None, None, cos, sin, pos)
    assert got[2] is None and got[3] is None and bool((got[1] == 0).all())


def test_off_the_16_byte_grid(emu):
    import torch
    q, k, wq, wk, cos, sin, pos = _make(40, 4, 2, 64, 64, "bfloat16", seed=12)
    buf = torch.zeros(40 * 4 * 64 + 1, device="cuda", dtype=q.dtype)
    odd = buf[1:].view(40, 4, 64)
    odd.copy_(q)
    a = emu.emu_qk_norm_rope(q, k, wq, wk, cos, sin, pos)
    b = emu.emu_qk_norm_rope(odd, k, wq, wk, cos, sin, pos)
    want, bound = ref.qk(q, wq, cos, sin, pos, 1e-6, False)
    assert ref.ratio(a[0], want, bound) <= 1.0 and ref.ratio(b[0], want, bound) <= 1.0


def test_gradients_against_differences(emu):
    """Central differences of sum(dy y) in 64 bits; their error is of the
    order of h^2 = 1e-8, the kernel's 1e-6 of the sums of sizes."""
    import torch
    q, k, wq, wk, cos, sin, pos = _make(20, 4, 2, 64, 32, "float32", seed=31)
    dq, dk = torch.randn(q.shape, device="cuda"), torch.randn(k.shape, device="cuda")
    got = emu.emu_qk_norm_rope_bwd(dq, dk, q, k, wq, wk, cos, sin, pos, interleaved=True)
    at = [t.double() for t in (q, k, wq, wk)]

    def loss(ts):
        y = ref.qk(ts[0], ts[2], cos, sin, pos, 1e-6, True)[0]
        z = ref.qk(ts[1], ts[3], cos, sin, pos, 1e-6, True)[0]
        return float((y * dq.double()).sum() + (z * dk.double()).sum())
    ref.HALF_ULP[torch.float64] = ref.LEAST[torch.float64] = 0.0
    h = 1e-4
    for i, g in enumerate(got):
        v = torch.randn(at[i].shape, dtype=torch.float64, device="cuda")
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * v, at[i] - h * v
        slope = (loss(up) - loss(down)) / (2 * h)
        assert abs(slope - float((g.double() * v).sum())) <= 1e-5 * float((g.double() * v).abs().sum())


def test_positions_out_of_the_table(emu):
    """NaN in that token's rotated values, the rest as it should be, and the
    device's error word set."""
    import torch
    for D, rot in ((64, 32), (33, 16)):
        q, k, wq, wk, cos, sin, pos = _make(12, 4, 2, D, rot, "float32", seed=2)
        good = emu.emu_qk_norm_rope(q, k, wq, wk, cos, sin, pos)
        emu.emu_clear_device_error()
        bad = pos.clone()
        bad[3], bad[8] = 400, -1
        y, z = emu.emu_qk_norm_rope(q, k, wq, wk, cos, sin, bad)
        assert emu.emu_get_last_device_error() == -1
        emu.emu_clear_device_error()
        for a, b in ((y, good[0]), (z, good[1])):
            assert bool(torch.isnan(a[[3, 8], :, :rot]).all())
            assert bool((a[[3, 8], :, rot:] == b[[3, 8], :, rot:]).all())
            keep = [i for i in range(12) if i not in (3, 8)]
            assert bool((a[keep] == b[keep]).all())


def test_zeros_and_non_finite_heads(emu):
    import torch
    q, k, wq, wk, cos, sin, pos = _make(6, 4, 2, 64, 64, "float32", seed=2)
    q, k = q.clone(), k.clone()
    good = emu.emu_qk_norm_rope(q, k, wq, wk, cos, sin, pos)[0]
    q[1, 2] = 0.0
    q[2, 0, 5] = float("nan")
    q[3, 1, 7] = float("inf")
    y = emu.emu_qk_norm_rope(q, k, wq, wk, cos, sin, pos)[0]
    assert bool((y[1, 2] == 0).all()) and bool(torch.isnan(y[2, 0]).all())
    assert not bool(torch.isfinite(y[3, 1, 7])) and not bool(torch.isnan(y[3, 0]).any())
    same = torch.ones(6, 4, dtype=torch.bool, device="cuda")
    same[1, 2] = same[2, 0] = same[3, 1] = False
    assert bool((y[same] == good[same]).all())


def test_empty_streams_graph_and_bits(emu):
    import torch
    q, k, wq, wk, cos, sin, pos = _make(700, 8, 2, 128, 128, "bfloat16", seed=7)
    none = emu.emu_qk_norm_rope(q[:0], k[:0], wq, wk, cos, sin, pos[:0])
    assert none[0].shape == (0, 8, 128)
    g0 = emu.emu_qk_norm_rope_bwd(q[:0], k[:0], q[:0], k[:0], wq, wk, cos, sin, pos[:0])
    assert bool((g0[2] == 0).all()) and bool((g0[3] == 0).all())
    dq, dk = torch.randn(q.shape, device="cuda").bfloat16(), torch.randn(k.shape, device="cuda").bfloat16()

    def both(**kw):
        return (*emu.emu_qk_norm_rope(q, k, wq, wk, cos, sin, pos, **kw),
                *emu.emu_qk_norm_rope_bwd(dq, dk, q, k, wq, wk, cos, sin, pos, **kw))
    first = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    again = both(stream=s)
    s.synchronize()
    assert all(bool((a == b).all()) for a, b in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    pos.copy_(pos.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert all(bool((a == b).all()) for a, b in zip(out, both()))


def test_refusals(emu):
    import torch
    q, k, wq, wk, cos, sin, pos = _make(6, 4, 2, 64, 64, "float32", seed=2)
    bad = [dict(wq=wq[:32]), dict(positions=pos[:5]), dict(positions=pos.long()), dict(cos=cos.t()),
           dict(k=k[:5]), dict(k=k[:, :, :32]), dict(q=q.cpu()), dict(sin=sin[:, :16]),
           dict(q=q.transpose(1, 2)), dict(eps=-1.0), dict(out=(q, q))]
    for change in bad:
        args = dict(q=q, k=k, wq=wq, wk=wk, cos=cos, sin=sin, positions=pos) | change
        with pytest.raises((ValueError, RuntimeError)):
            emu.emu_qk_norm_rope(**args)
    with pytest.raises(TypeError):
        emu.emu_qk_norm_rope(q.double(), k.double(), wq, wk, cos, sin, pos)
    with pytest.raises(TypeError):
        emu.emu_qk_norm_rope(q, k.half(), wq, wk, cos, sin, pos)
    wide = torch.randn(2, 1, 514, device="cuda")
    with pytest.raises(RuntimeError):
        emu.emu_qk_norm_rope(wide, wide, None, None)
