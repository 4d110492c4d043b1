"""The torch modules on the GPU with what autograd and a serving program hand
them: expanded gradients and inputs, weights replaced after pack(), weights made
in inference mode, derivatives of gradients."""
import gc

import pytest

from gpu_util import emu_module

pytestmark = pytest.mark.gpu

TOL = 1e-5                  # of the norm: an FP32 product or two, and an activation


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()


def _near(got, want):
    assert float((got.double() - want).norm()) <= TOL * float(want.norm())


def _gated(x, gate, up):
    import torch
    return torch.nn.functional.silu(x @ gate.t()) * (x @ up.t())


@pytest.mark.parametrize("M", [5, 300])
def test_expanded_gradients_and_inputs(emu, M):
    import torch
    from fp32_emulated_gemm_split_gb300.block import EmuGatedLinear
    from fp32_emulated_gemm_split_gb300.linear import EmuLinear
    torch.manual_seed(0)
    gated, linear = EmuGatedLinear(64, 72, device="cuda"), EmuLinear(64, 72, device="cuda")
    v = torch.randn(72, device="cuda")
    for layer, plain in ((gated, lambda x, g, u: _gated(x, g, u)),
                         (linear, lambda x, w, b: torch.nn.functional.linear(x, w, b))):
        x = torch.randn(M, 64, device="cuda", requires_grad=True)
        params = list(layer.parameters())
        for loss in (lambda y: (y.sum(0) * v.to(y.dtype)).sum(), lambda y: y.mean(0).square().sum()):
            got = torch.autograd.grad(loss(layer(x)), [x, *params])
            at = [t.detach().double().requires_grad_() for t in (x, *params)]
            for a, b in zip(got, torch.autograd.grad(loss(plain(*at)), at)):
                _near(a, b)
        rows = torch.randn(64, device="cuda").expand(M, 64)
        with torch.no_grad():
            _near(layer(rows), plain(*(t.double() for t in (rows, *params))))


@pytest.mark.parametrize("M", [3, 300])
def test_weights_replaced_after_pack(emu, M):
    import torch
    from fp32_emulated_gemm_split_gb300.block import EmuGatedLinear
    torch.manual_seed(1)
    layer = EmuGatedLinear(64, 72, device="cuda").eval().pack()
    x = torch.randn(M, 64, device="cuda")
    with torch.no_grad():
        old = layer(x)
        layer.gate.data.mul_(2)                      # seen by none of the kernels before pack()
        assert torch.equal(layer(x), old)
        _near(layer.pack()(x), _gated(x.double(), layer.gate.double(), layer.up.double()))
        layer.gate.data = torch.randn(72, 64, device="cuda")
        with pytest.raises(ValueError, match="pack"):
            layer(x)
        _near(layer.pack()(x), _gated(x.double(), layer.gate.double(), layer.up.double()))


@pytest.mark.parametrize("M", [3, 300])
def test_inference_mode(emu, M):
    import torch
    from fp32_emulated_gemm_split_gb300.block import EmuDecoderBlock, EmuGatedLinear
    torch.manual_seed(2)
    with torch.inference_mode():
        layer, x = EmuGatedLinear(64, 72, device="cuda"), torch.randn(M, 64, device="cuda")
        want = _gated(x.double(), layer.gate.double(), layer.up.double())
        _near(layer(x), want)
        _near(layer.pack()(x), want)
        W = torch.randn(48, 64, device="cuda")
        w = emu.emu_lora_pack(W)
        index = torch.full((M,), -1, device="cuda", dtype=torch.int32)
        A, B = torch.randn(1, 4, 64, device="cuda"), torch.randn(1, 48, 4, device="cuda")
        _near(emu.emu_lora(x, w, A, B, index), x.double() @ W.double().t())
        block = EmuDecoderBlock(64, 4, 2, 72, max_positions=512).eval()
        _near(block(x[:, :64]), _decoder64(block, x.double()))
    index = torch.zeros(M, device="cuda", dtype=torch.int32)
    _near(emu.emu_lora(x, w, A, B, index), x.double() @ (W.double() + B[0].double() @ A[0].double()).t())


def _decoder64(block, x):
    """The block's definition in float64, its products by torch."""
    import copy
    import torch
    b = copy.deepcopy(block).double()
    T, D, H, Hk = x.size(0), b.dim, b.heads, b.kv_heads

    def norm(v, w):
        return v / (v.square().mean(-1, keepdim=True) + b.eps).sqrt() * w

    def turn(v):
        c, s = b.cos[:T, None], b.sin[:T, None]
        p, q = v[..., :D // 2], v[..., D // 2:]
        return torch.cat((p * c - q * s, p * s + q * c), -1)
    q, k, v = (norm(x, b.norm1) @ b.qkv.weight.t()).view(T, -1, D).split((H, Hk, Hk), 1)
    q, k = turn(norm(q, b.wq)), turn(norm(k, b.wk))
    x = x + b._attention(q, k, v) @ b.out.weight.t()
    return x + _gated(norm(x, b.norm2), b.gated.gate, b.gated.up) @ b.down.weight.t()


def test_second_derivatives_raise(emu):
    import torch
    from fp32_emulated_gemm_split_gb300.block import EmuGatedLinear, qk_norm_rope
    from fp32_emulated_gemm_split_gb300.linear import EmuLinear
    torch.manual_seed(3)
    k, w = torch.randn(7, 1, 64, device="cuda"), torch.rand(64, device="cuda")
    angle = torch.randn(7, 32, device="cuda")
    at = k, w, w, angle.cos(), angle.sin(), torch.arange(7, device="cuda", dtype=torch.int32)
    for f in (EmuGatedLinear(64, 72, device="cuda"), EmuLinear(64, 72, device="cuda"),
              lambda x: qk_norm_rope(x.view(7, 1, 64), *at)[0]):
        x = torch.randn(7, 64, device="cuda", requires_grad=True)
        e = f(x).sum()
        force, = torch.autograd.grad(e, x, create_graph=True)
        with pytest.raises(RuntimeError, match="no second derivative"):
            (e + force.square().sum()).backward()
        assert torch.equal(torch.autograd.grad(f(x).sum(), x)[0], force)
