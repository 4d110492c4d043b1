"""The gated feed-forward on the GPU against its definition in 64 bits:
every element within the bound that the number of roundings gives
(layer_ref.py), over row counts from one up, odd widths, strides, each
activation; the gradients against the formula and against differences."""
import gc

import pytest

import layer_ref as ref
from gpu_util import emu_module

pytestmark = pytest.mark.gpu

# the products' 2-norm error: three BF16 pieces hold an FP32 value exactly, a
# partial sum of 64 products is rounded a few times at 2^-24 of its size and
# the partial sums add up in FP32: well below 1e-6 (a lost piece gives 1e-5)
REL = 1.5e-6


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()                                     # tensors that graphs and tracebacks still hold


def _make(M, K, F, seed, pad=0, offset=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def mat(r, c, std=1.0):
        whole = torch.randn(r, c + pad + offset, generator=g, device="cuda") * std
        whole[:, c + offset:] = float("nan")
        return whole[:, offset:c + offset]
    return mat(M, K), mat(F, K, K ** -0.5), mat(F, K, K ** -0.5), mat(M, F)


SHAPES = [(1, 64, 64), (1, 2048, 1024), (2, 200, 130), (3, 33, 1), (7, 1, 40), (16, 512, 96), (17, 520, 256),
          (31, 1000, 300), (64, 256, 129), (65, 96, 1000), (128, 128, 33), (129, 100, 257), (200, 72, 640),
          (256, 256, 256), (257, 65, 127), (777, 640, 520), (1500, 36, 28)]


@pytest.mark.parametrize("M,K,F", SHAPES)
@pytest.mark.parametrize("save", [False, True])
def test_forward(emu, M, K, F, save):
    import torch
    X, Wg, Wu, _ = _make(M, K, F, seed=M + 3 * K + 7 * F)
    w = emu.emu_gated_pack(Wg, Wu)
    got = emu.emu_gated(X, w, act="silu", save=save)
    want, bound = ref.gated("silu", X, Wg, Wu)
    got = got if save else (got,)
    for g, r, b in zip(got, want, bound):
        assert g.shape == r.shape and g.dtype == torch.float32
        assert ref.ratio(g, r, b) <= 1.0
        assert ref.rel(g, r) <= REL
    assert emu.emu_get_last_device_error() == 0


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
@pytest.mark.parametrize("M", [5, 300])
def test_activations(emu, act, M):
    X, Wg, Wu, _ = _make(M, 192, 200, seed=5)
    X = X * 4                                        # gates from -15 to 15
    H, G, U = emu.emu_gated(X, emu.emu_gated_pack(Wg, Wu), act=act, save=True)
    want, bound = ref.gated(act, X, Wg, Wu)
    for g, r, b in zip((H, G, U), want, bound):
        assert ref.ratio(g, r, b) <= 1.0


@pytest.mark.parametrize("M,K,F,pad,offset", [(5, 96, 70, 4, 0), (40, 96, 70, 3, 1), (300, 96, 72, 5, 0),
                                               (300, 100, 72, 4, 4), (130, 51, 35, 1, 2)])
def test_strides_and_alignment(emu, M, K, F, pad, offset):
    """Rows longer than the matrix (NaN between), rows off the 16-byte grid,
    an output inside a larger buffer that must stay as it was around it."""
    import torch
    X, Wg, Wu, dH = _make(M, K, F, seed=9, pad=pad, offset=offset)
    w = emu.emu_gated_pack(Wg, Wu)
    room = torch.full((M + 2, F + pad + offset), 7.0, device="cuda")
    out = room[1:M + 1, offset:F + offset]
    assert emu.emu_gated(X, w, out=out) is out
    want, bound = ref.gated("silu", X, Wg, Wu)
    assert ref.ratio(out, want[0], bound[0]) <= 1.0
    around = room.clone()
    around[1:M + 1, offset:F + offset] = 7.0
    assert bool((around == 7.0).all())
    _, G, U = emu.emu_gated(X, w, save=True)
    got = emu.emu_gated_bwd(dH, X, w, G, U)
    want, bound = ref.gated_bwd("silu", dH, X, Wg, Wu, G, U)
    for g, r, b in zip(got, want, bound):
        assert ref.ratio(g, r, b) <= 1.0


@pytest.mark.parametrize("M,K,F", [(1, 64, 64), (3, 33, 1), (17, 520, 256), (64, 1, 129), (257, 65, 127),
                                   (777, 320, 520), (2000, 36, 28)])
@pytest.mark.parametrize("act", ["silu", "relu"])
def test_backward(emu, M, K, F, act):
    X, Wg, Wu, dH = _make(M, K, F, seed=M + K + F)
    w = emu.emu_gated_pack(Wg, Wu)
    _, G, U = emu.emu_gated(X, w, act=act, save=True)
    got = emu.emu_gated_bwd(dH, X, w, G, U, act=act)
    want, bound = ref.gated_bwd(act, dH, X, Wg, Wu, G, U)
    for g, r, b in zip(got, want, bound):
        assert g.shape == r.shape
        assert ref.ratio(g, r, b) <= 1.0
        assert ref.rel(g, r) <= 2 * REL
    only_x = emu.emu_gated_bwd(dH, X, w, G, U, act=act, need_dw=False)
    only_w = emu.emu_gated_bwd(dH, X, w, G, U, act=act, need_dx=False)
    assert only_x[1] is None and only_x[2] is None and only_w[0] is None
    assert bool((only_x[0] == got[0]).all())
    assert bool((only_w[1] == got[1]).all()) and bool((only_w[2] == got[2]).all())


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "sigmoid"])
def test_backward_activations(emu, act):
    X, Wg, Wu, dH = _make(150, 96, 88, seed=3)
    X = X * 3
    w = emu.emu_gated_pack(Wg, Wu)
    _, G, U = emu.emu_gated(X, w, act=act, save=True)
    got = emu.emu_gated_bwd(dH, X, w, G, U, act=act)
    want, bound = ref.gated_bwd(act, dH, X, Wg, Wu, G, U)
    for g, r, b in zip(got, want, bound):
        assert ref.ratio(g, r, b) <= 1.0


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "sigmoid"])
def test_gradients_against_differences(emu, act):
    """Central differences of the loss sum(dH * H) in 64 bits along random
    directions: their own error is of the order h^2 = 1e-8, the kernels' 1e-6
    of the sums of sizes."""
    import torch
    X, Wg, Wu, dH = _make(96, 80, 72, seed=21)
    w = emu.emu_gated_pack(Wg, Wu)
    _, G, U = emu.emu_gated(X, w, act=act, save=True)
    grads = emu.emu_gated_bwd(dH, X, w, G, U, act=act)
    at = [t.double() for t in (X, Wg, Wu)]

    def loss(ts):
        return float((ref.act(act, ts[0] @ ts[1].t())[0] * (ts[0] @ ts[2].t()) * dH.double()).sum())
    h = 1e-4
    for i, g in enumerate(grads):
        v = torch.randn(at[i].shape, dtype=torch.float64, device="cuda")
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * v, at[i] - h * v
        slope = (loss(up) - loss(down)) / (2 * h)
        assert abs(slope - float((g.double() * v).sum())) <= 1e-5 * float((g.double() * v).abs().sum())


def test_empty(emu):
    import torch
    Wg, Wu = torch.randn(24, 16, device="cuda"), torch.randn(24, 16, device="cuda")
    w = emu.emu_gated_pack(Wg, Wu)
    X = torch.empty(0, 16, device="cuda")
    H, G, U = emu.emu_gated(X, w, save=True)
    assert H.shape == (0, 24)
    dX, dWg, dWu = emu.emu_gated_bwd(torch.empty(0, 24, device="cuda"), X, w, G, U)
    assert dX.shape == (0, 16) and bool((dWg == 0).all()) and bool((dWu == 0).all())
    w0 = emu.emu_gated_pack(torch.empty(24, 0, device="cuda"), torch.empty(24, 0, device="cuda"))
    assert bool((emu.emu_gated(torch.empty(3, 0, device="cuda"), w0) == 0).all())


def test_nan_and_infinity_stay_in_their_rows(emu):
    import torch
    for M in (6, 300):
        X, Wg, Wu, _ = _make(M, 64, 64, seed=2)
        clean = emu.emu_gated(X, emu.emu_gated_pack(Wg, Wu))
        X[1, 3], X[4, 5] = float("nan"), float("inf")
        H = emu.emu_gated(X, emu.emu_gated_pack(Wg, Wu))
        assert bool(torch.isnan(H[1]).all()) and not bool(torch.isfinite(H[4]).any())
        keep = [i for i in range(M) if i not in (1, 4)]
        assert bool((H[keep] == clean[keep]).all())


def test_same_bits_again_and_on_another_stream(emu):
    import torch
    for M in (9, 400):
        X, Wg, Wu, dH = _make(M, 320, 200, seed=4)
        w = emu.emu_gated_pack(Wg, Wu)
        H, G, U = emu.emu_gated(X, w, save=True)
        first = (H, *emu.emu_gated_bwd(dH, X, w, G, U))
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        H, G, U = emu.emu_gated(X, w, save=True, stream=s)
        again = (H, *emu.emu_gated_bwd(dH, X, w, G, U, stream=s))
        s.synchronize()
        assert all(bool((a == b).all()) for a, b in zip(first, again))


@pytest.mark.parametrize("M", [4, 200])
def test_graph_replay(emu, M):
    import torch
    X, Wg, Wu, dH = _make(M, 256, 192, seed=6)
    w = emu.emu_gated_pack(Wg, Wu)

    def step():
        H, G, U = emu.emu_gated(X, w, save=True)
        return (H, *emu.emu_gated_bwd(dH, X, w, G, U))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    other, _, _, _ = _make(M, 256, 192, seed=7)
    X.copy_(other)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, step()):
        assert bool((a == b).all())


def test_refusals(emu):
    import torch
    Wg, Wu = torch.randn(24, 16, device="cuda"), torch.randn(24, 16, device="cuda")
    X = torch.randn(5, 16, device="cuda")
    w = emu.emu_gated_pack(Wg, Wu)
    with pytest.raises(ValueError):
        emu.emu_gated_pack(Wg, Wu[:, :8])
    with pytest.raises(TypeError):
        emu.emu_gated_pack(Wg.bfloat16(), Wu.bfloat16())
    with pytest.raises(ValueError):
        emu.emu_gated(X, w, act="swish")
    with pytest.raises(ValueError):
        emu.emu_gated(X[:, :8], w)
    with pytest.raises(ValueError):
        emu.emu_gated(X.cpu(), w)
    with pytest.raises(TypeError):
        emu.emu_gated(X.half(), w)
    with pytest.raises(ValueError):
        emu.emu_gated(torch.randn(16, 5, device="cuda").t(), w)
    with pytest.raises(ValueError):
        emu.emu_gated(X, w, out=torch.empty(5, 23, device="cuda"))
    _, G, U = emu.emu_gated(X, w, save=True)
    with pytest.raises(ValueError):
        emu.emu_gated_bwd(torch.randn(4, 24, device="cuda"), X, w, G, U)
    with pytest.raises(ValueError):
        emu.emu_gated_bwd(torch.randn(5, 24, device="cuda"), X, w, G, U.contiguous().clone()[:, :23])
