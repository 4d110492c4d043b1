"""Norm and rotation with eps = 0, forward and backward, against the definition
in 64 bits: heads that are not zero need no eps, however many of them there are
(a round of a warp's that they do not fill has idle lanes, whose zeros have no
norm)."""
import gc

import pytest

import layer_ref as ref
from gpu_util import emu_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()


# whole 16-byte chunks (64, 96, 128) and not (66, 33, 10); heads that fill rounds of 4, 2 or 32 and that do not
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(1, 3, 1, 64, 64), (6, 4, 4, 64, 32), (7, 3, 5, 96, 64), (5, 1, 3, 128, 128),
                                           (9, 5, 4, 66, 66), (6, 3, 2, 33, 16), (40, 7, 0, 10, 4), (3, 2, 1, 512, 0)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("pairs", [False, True])
def test_forward_and_backward(emu, T, Hq, Hk, D, rot, dtype, pairs):
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + D)
    kind = getattr(torch, dtype)

    def r(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    q, k, dq, dk = (r(T, h, D).to(kind) for h in (Hq, Hk, Hq, Hk))
    wq, wk = 1 + 0.3 * r(D), 1 + 0.3 * r(D)
    cos, sin, pos = None, None, None
    if rot:
        angle = r(50, rot // 2) * 3
        cos, sin = angle.cos(), angle.sin()
        pos = torch.randint(0, 50, (T,), generator=g, device="cuda", dtype=torch.int32)
    at = (cos, sin, pos)
    out = emu.emu_qk_norm_rope(q, k, wq, wk, *at, eps=0.0, interleaved=pairs)
    gq, gk, gwq, gwk = emu.emu_qk_norm_rope_bwd(dq, dk, q, k, wq, wk, *at, eps=0.0, interleaved=pairs)
    for x, w, y, d, gx, gw in ((q, wq, out[0], dq, gq, gwq), (k, wk, out[1], dk, gk, gwk)):
        if x.numel() == 0:
            assert bool((gw == 0).all())
            continue
        want, bound = ref.qk(x, w, *at, 0.0, pairs)
        assert ref.ratio(y, want, bound) <= 1.0
        (dx, dw), (bx, bw) = ref.qk_bwd(d, x, w, *at, 0.0, pairs)
        assert ref.ratio(gx, dx, bx) <= 1.0
        assert ref.ratio(gw, dw, bw) <= 1.0
    assert emu.emu_get_last_device_error() == 0


def test_a_position_out_of_the_table_and_idle_lanes(emu):
    """The gradients that have a NaN position in them are NaN; the side's other tokens' dx are as without it."""
    import torch
    torch.manual_seed(1)
    q, k, dq, dk = (torch.randn(6, h, 64, device="cuda") for h in (3, 1, 3, 1))
    w = torch.ones(64, device="cuda")
    angle = torch.randn(20, 16, device="cuda")
    pos = torch.arange(6, device="cuda", dtype=torch.int32)
    good = emu.emu_qk_norm_rope_bwd(dq, dk, q, k, w, w, angle.cos(), angle.sin(), pos, eps=0.0)
    bad = pos.clone()
    bad[2] = 20
    emu.emu_clear_device_error()
    got = emu.emu_qk_norm_rope_bwd(dq, dk, q, k, w, w, angle.cos(), angle.sin(), bad, eps=0.0)
    assert emu.emu_get_last_device_error() == -1
    emu.emu_clear_device_error()
    keep = [0, 1, 3, 4, 5]
    for a, b in zip(got[:2], good[:2]):
        assert bool((a[keep] == b[keep]).all()) and bool(torch.isnan(a[2]).all())
    for a, b in zip(got[2:], good[2:]):
        assert bool(torch.isnan(a[:32]).all()) and bool((a[32:] == b[32:]).all())
