"""The torch modules of block.py on the CPU: what they hand to the library and
what autograd makes of it.  The library's calls are stand-ins that refuse what
the binding refuses (block_fakes.py)."""
import pytest
import torch

import block_fakes


@pytest.fixture
def block(monkeypatch):
    block_fakes.put_in(monkeypatch)
    from fp32_emulated_gemm_split_gb300 import block
    torch.manual_seed(0)
    return block


def _gated64(x, gate, up):
    return torch.nn.functional.silu(x @ gate.t()) * (x @ up.t())


@pytest.mark.parametrize("loss", [
    lambda y: (y.sum(0) * torch.arange(6)).sum(), lambda y: (y.mean(0) ** 2).sum(), lambda y: y.sum(),
    lambda y: (y.sum(1) * torch.arange(5)).sum()])
def test_gated_takes_expanded_gradients(block, loss):
    layer = block.EmuGatedLinear(4, 6)
    x = torch.randn(5, 4, requires_grad=True)
    got = torch.autograd.grad(loss(layer(x)), [x, layer.gate, layer.up])
    at = [t.detach().double().requires_grad_() for t in (x, layer.gate, layer.up)]
    for a, b in zip(got, torch.autograd.grad(loss(_gated64(*at)), at)):
        assert torch.allclose(a.double(), b, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("x", [torch.randn(4).expand(5, 4), torch.randn(5, 1).expand(5, 4), torch.randn(4, 5).t(),
                               torch.randn(12).unfold(0, 4, 2)])
@pytest.mark.parametrize("grad", [False, True])
def test_gated_takes_inputs_of_any_strides(block, x, grad):
    layer = block.EmuGatedLinear(4, 6)
    with torch.set_grad_enabled(grad):
        y = layer(x)
    want = _gated64(x.double(), layer.gate.double(), layer.up.double())
    assert torch.allclose(y.double(), want, rtol=1e-5, atol=1e-6)
