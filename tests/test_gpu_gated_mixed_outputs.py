"""The gated forward pass with H in rows that are not 16-byte aligned and G and U in
rows that are: the outputs go through one staging buffer by different ways, and
each has to be there whole before the next one's values are.
"""
import gc

import pytest

import layer_ref as ref
from gpu_util import emu_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()


@pytest.mark.parametrize("M,K,F", [(295, 209, 4909), (512, 64, 8190), (2048, 129, 1023), (4096, 64, 2049)])
@pytest.mark.parametrize("act", ["relu", "silu"])
def test_every_output_is_whole(emu, M, K, F, act):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + K + F)
    X = torch.randn(M, K, device="cuda", generator=g)
    Wg, Wu = (torch.randn(F, K, device="cuda", generator=g) * K ** -0.5 for _ in range(2))
    w = emu.emu_gated_pack(Wg, Wu)
    want, bound = ref.gated(act, X, Wg, Wu)
    for _ in range(3):
        for got, r, b in zip(emu.emu_gated(X, w, act=act, save=True), want, bound):
            assert ref.ratio(got, r, b) <= 1.0


@pytest.mark.parametrize("aligned", [0, 1])
def test_output_of_other_alignment(emu, aligned):
    """H of aligned rows (out) has the same bits as H of unaligned ones."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(7)
    M, K, F = 1024, 96, 1501
    X = torch.randn(M, K, device="cuda", generator=g)
    w = emu.emu_gated_pack(*(torch.randn(F, K, device="cuda", generator=g) for _ in range(2)))
    H = emu.emu_gated(X, w)
    out = torch.empty(M, F + (3 if aligned else 2), device="cuda")[:, :F]
    got, G, U = emu.emu_gated(X, w, save=True, out=out)
    assert torch.equal(got, H)
    got2, G2, U2 = emu.emu_gated(X, w, save=True)
    assert torch.equal(got2, H) and torch.equal(G, G2) and torch.equal(U, U2)
