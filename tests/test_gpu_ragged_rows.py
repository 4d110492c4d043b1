"""More than 256 rows whose last ones leave a 256-row tile mostly empty: with large
weights those rows stream the FP32 weights, the others use the pieces.  All rows
against 64 bits, and the two kinds of rows apart.
"""
import gc

import pytest

import layer_ref as ref
from gpu_util import emu_module

pytestmark = pytest.mark.gpu

REL = 1.5e-6             # as in test_gpu_gated.py


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()


# (rows, K, width of one weight): 1, 30, 64, 100 and 150 rows left
@pytest.mark.parametrize("M,K,F", [(257, 1100, 3600), (542, 1028, 4000), (320, 2052, 3400), (356, 2060, 6200),
                                   (662, 2500, 6300)])
def test_gated(emu, M, K, F):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + K + F)
    X = torch.randn(M, K, device="cuda", generator=g)
    Wg, Wu = (torch.randn(F, K, device="cuda", generator=g) * K ** -0.5 for _ in range(2))
    got = emu.emu_gated(X, emu.emu_gated_pack(Wg, Wu), act="silu", save=True)
    want, bound = ref.gated("silu", X, Wg, Wu)
    for o, r, b in zip(got, want, bound):
        for part in (slice(0, M - M % 256), slice(M - M % 256, M)):
            assert ref.ratio(o[part], r[part], b[part]) <= 1.0
            assert ref.rel(o[part], r[part]) <= REL
    assert emu.emu_get_last_device_error() == 0


@pytest.mark.parametrize("M,K,N", [(257, 1100, 7000), (320, 2052, 6804), (356, 2060, 12400), (406, 2500, 12500)])
def test_adapters(emu, M, K, N):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + K + N)
    X = torch.randn(M, K, device="cuda", generator=g)
    W = torch.randn(N, K, device="cuda", generator=g) * K ** -0.5
    A = torch.randn(5, 8, K, device="cuda", generator=g) * K ** -0.5
    B = torch.randn(5, N, 8, device="cuda", generator=g) * 8 ** -0.5
    bias = torch.randn(N, device="cuda", generator=g)
    index = torch.randint(-1, 5, (M,), device="cuda", generator=g).int()
    Y = emu.emu_lora(X, emu.emu_lora_pack(W, bias), A, B, index)
    want, bound = ref.lora(X, W, bias, A, B, index, None)
    for part in (slice(0, M - M % 256), slice(M - M % 256, M)):
        assert ref.ratio(Y[part], want[part], bound[part]) <= 1.0
        assert ref.rel(Y[part], want[part]) <= REL
    assert emu.emu_get_last_device_error() == 0
