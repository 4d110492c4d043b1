"""The adapters of many requests beside a shared projection, on the GPU,
against their definition in 64 bits."""
import gc

import pytest

import layer_ref as ref
from gpu_util import emu_module

pytestmark = pytest.mark.gpu

REL = 1.5e-6


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()                                     # tensors that graphs and tracebacks still hold


def _make(M, K, N, R, n, seed, order="random", bias=True, scale=True):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std
    X, W = r(M, K), r(N, K, std=K ** -0.5)
    A, B = r(n, R, K, std=K ** -0.5), r(n, N, R, std=max(R, 1) ** -0.5)
    if order == "random":
        index = torch.randint(-1, n, (M,), generator=g, device="cuda")
    elif order == "runs":
        index = (torch.arange(M, device="cuda") * (n + 1) // max(M, 1)) - 1
    elif order == "none":
        index = torch.full((M,), -1, device="cuda")
    else:
        index = torch.zeros(M, device="cuda")
    return (X, W, r(N) if bias else None, A, B, index.to(torch.int32),
            torch.rand(n, generator=g, device="cuda") + 0.5 if scale else None)


SHAPES = [(1, 64, 64, 8, 3), (1, 2048, 1000, 16, 5), (2, 100, 33, 4, 1), (5, 37, 130, 3, 9), (16, 512, 256, 16, 64),
          (31, 260, 257, 32, 4), (64, 128, 640, 64, 40), (131, 300, 96, 17, 12), (200, 1, 50, 1, 2),
          (256, 256, 256, 16, 8), (513, 72, 384, 40, 6), (1030, 96, 130, 8, 100), (2000, 64, 1, 5, 3)]


@pytest.mark.parametrize("M,K,N,R,n", SHAPES)
@pytest.mark.parametrize("order", ["random", "runs"])
def test_forward(emu, M, K, N, R, n, order):
    X, W, bias, A, B, index, scale = _make(M, K, N, R, n, seed=M + K + N, order=order)
    Y = emu.emu_lora(X, emu.emu_lora_pack(W, bias), A, B, index, scale)
    want, bound = ref.lora(X, W, bias, A, B, index, scale)
    assert ref.ratio(Y, want, bound) <= 1.0
    assert ref.rel(Y, want) <= REL
    assert emu.emu_get_last_device_error() == 0


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("order", ["none", "one"])
@pytest.mark.parametrize("bias,scale", [(False, False), (True, False), (False, True)])
def test_absent_parts(emu, M, order, bias, scale):
    X, W, b, A, B, index, s = _make(M, 96, 200, 8, 4, seed=M, order=order, bias=bias, scale=scale)
    Y = emu.emu_lora(X, emu.emu_lora_pack(W, b), A, B, index, s)
    want, bound = ref.lora(X, W, b, A, B, index, s)
    assert ref.ratio(Y, want, bound) <= 1.0


@pytest.mark.parametrize("R,n", [(0, 3), (4, 0)])
def test_no_adapters(emu, R, n):
    import torch
    X, W, b, A, B, _, _ = _make(20, 64, 72, R, max(n, 1), seed=1)
    index = torch.full((20,), -1, device="cuda", dtype=torch.int32)
    Y = emu.emu_lora(X, emu.emu_lora_pack(W, b), A[:n], B[:n], index)
    want, bound = ref.lora(X, W, b, A[:0], B[:0], index, None)
    assert ref.ratio(Y, want, bound) <= 1.0


@pytest.mark.parametrize("M,K,N", [(12, 99, 70), (300, 101, 135)])
def test_strides_and_alignment(emu, M, K, N):
    """Rows longer than the matrix with NaN between, off the 16-byte grid; an
    output inside a larger buffer."""
    import torch
    X, W, b, A, B, index, s = _make(M, K, N, 6, 5, seed=K)
    Xw = torch.full((M, K + 3), float("nan"), device="cuda")
    Xw[:, 1:K + 1] = X
    Ww = torch.full((N, K + 2), float("nan"), device="cuda")
    Ww[:, :K] = W
    room = torch.full((M + 2, N + 3), 7.0, device="cuda")
    out = room[1:M + 1, 2:N + 2]
    emu.emu_lora(Xw[:, 1:K + 1], emu.emu_lora_pack(Ww[:, :K], b), A, B, index, s, out=out)
    want, bound = ref.lora(X, W, b, A, B, index, s)
    assert ref.ratio(out, want, bound) <= 1.0
    around = room.clone()
    around[1:M + 1, 2:N + 2] = 7.0
    assert bool((around == 7.0).all())


def test_order_of_tokens_does_not_change_bits(emu):
    """A token's result does not depend on where in the batch it stands."""
    import torch
    for M in (24, 700):
        X, W, b, A, B, index, s = _make(M, 128, 96, 16, 7, seed=3)
        w = emu.emu_lora_pack(W, b)
        Y = emu.emu_lora(X, w, A, B, index, s)
        p = torch.randperm(M, device="cuda")
        assert bool((emu.emu_lora(X[p], w, A, B, index[p], s) == Y[p]).all())


def test_nan_stays_with_its_adapter_and_token(emu):
    import torch
    for M in (20, 300):
        X, W, b, A, B, index, s = _make(M, 64, 64, 8, 4, seed=8)
        index[:] = torch.arange(M, device="cuda", dtype=torch.int32) % 5 - 1
        w = emu.emu_lora_pack(W, b)
        clean = emu.emu_lora(X, w, A, B, index, s)
        A[2] = float("nan")
        X[0] = float("inf")
        Y = emu.emu_lora(X, w, A, B, index, s)
        hit = (index == 2) | (torch.arange(M, device="cuda") == 0)
        assert not bool(torch.isfinite(Y[hit]).any())
        assert bool((Y[~hit] == clean[~hit]).all())


def test_index_out_of_range_counts_as_none_and_is_recorded(emu):
    import torch
    for M in (10, 300):
        X, W, b, A, B, index, s = _make(M, 64, 48, 4, 3, seed=5)
        w = emu.emu_lora_pack(W, b)
        emu.emu_clear_device_error()
        bad = index.clone()
        bad[3], bad[7] = 3, -2
        good = index.clone()
        good[3] = good[7] = -1
        Y = emu.emu_lora(X, w, A, B, bad, s)
        assert emu.emu_get_last_device_error() == -1
        emu.emu_clear_device_error()
        assert bool((Y == emu.emu_lora(X, w, A, B, good, s)).all())
        assert emu.emu_get_last_device_error() == 0


def test_empty(emu):
    import torch
    X, W, b, A, B, index, s = _make(4, 16, 24, 4, 2, seed=1)
    w = emu.emu_lora_pack(W, b)
    assert emu.emu_lora(X[:0], w, A, B, index[:0], s).shape == (0, 24)
    w0 = emu.emu_lora_pack(torch.empty(24, 0, device="cuda"), b)
    Y = emu.emu_lora(X[:, :0], w0, A[:, :, :0].contiguous(), B, index, s)
    assert bool((Y == b).all())


@pytest.mark.parametrize("M", [6, 300])
def test_stream_and_graph(emu, M):
    import torch
    X, W, b, A, B, index, s = _make(M, 128, 160, 8, 5, seed=6)
    w = emu.emu_lora_pack(W, b)
    first = emu.emu_lora(X, w, A, B, index, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = emu.emu_lora(X, w, A, B, index, s, stream=side)
    side.synchronize()
    assert bool((first == other).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = emu.emu_lora(X, w, A, B, index, s)
    index.copy_(index.flip(0))
    X.mul_(1.5)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert bool((out == emu.emu_lora(X, w, A, B, index, s)).all())


def test_refusals(emu):
    import torch
    X, W, b, A, B, index, s = _make(5, 16, 24, 4, 2, seed=1)
    w = emu.emu_lora_pack(W, b)
    with pytest.raises(ValueError):
        emu.emu_lora_pack(W, b[:5])
    with pytest.raises(ValueError):
        emu.emu_lora(X, w, A[:, :, :8], B, index, s)
    with pytest.raises(ValueError):
        emu.emu_lora(X, w, A, B[:1], index, s)
    with pytest.raises(ValueError):
        emu.emu_lora(X, w, A, B, index.long(), s)
    with pytest.raises(ValueError):
        emu.emu_lora(X, w, A, B, index[:4], s)
    with pytest.raises(ValueError):
        emu.emu_lora(X, w, A, B, index, s[:1])
    with pytest.raises(TypeError):
        emu.emu_lora(X, w, A.half(), B.half(), index, s)
    with pytest.raises(ValueError):
        emu.emu_lora(X.cpu(), w, A, B, index, s)
    with pytest.raises(ValueError):
        emu.emu_lora(X, w, A.transpose(0, 1).contiguous().transpose(0, 1), B, index, s)
