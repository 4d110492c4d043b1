"""What of the adapters beside a projection depends on a token's place in the
batch: nothing of the adapter's term; of the projection the last rounding only
(whole tiles, the last rows of a ragged batch and tiles that share K add up in
other orders), so both orders stay within the error bound."""
import gc

import pytest

import layer_ref as ref
from gpu_util import emu_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()


# 542 = 2 x 256 + 30: the last 30 rows stream a weight of this size; 700: tiles that share K; 100: few rows
SHAPES = [(542, 1028, 8000), (700, 1000, 4000), (100, 520, 3000)]


def _make(M, K, N, R=8, n=5):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    index = torch.randint(-1, n, (M,), generator=g, device="cuda", dtype=torch.int32)
    order = torch.randperm(M, generator=g, device="cuda")
    return (r(M, K), r(N, K) * K ** -0.5, r(N), r(n, R, K) * K ** -0.5, r(n, N, R) * R ** -0.5, index,
            torch.rand(n, generator=g, device="cuda") + 0.5, order)


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_permuted_batches_are_within_the_bound(emu, M, K, N):
    X, W, b, A, B, index, s, p = _make(M, K, N)
    w = emu.emu_lora_pack(W, b)
    want, bound = ref.lora(X, W, b, A, B, index, s)
    assert ref.ratio(emu.emu_lora(X, w, A, B, index, s), want, bound) <= 1.0
    assert ref.ratio(emu.emu_lora(X[p], w, A, B, index[p], s), want[p], bound[p]) <= 1.0


@pytest.mark.parametrize("M,K,N", SHAPES)
def test_the_adapters_term_keeps_its_bits(emu, M, K, N):
    """With a weight of zeros the projection adds 0 to it."""
    import torch
    X, W, b, A, B, index, s, p = _make(M, K, N)
    w = emu.emu_lora_pack(torch.zeros_like(W), b)
    Y = emu.emu_lora(X, w, A, B, index, s)
    assert bool((emu.emu_lora(X[p], w, A, B, index[p], s) == Y[p]).all())
