"""EmuLinear's inputs and gradients with strides that the GEMM cannot read as
they are, on the CPU through stand-ins that read a matrix as the kernels do."""
import pytest
import torch

import block_fakes


@pytest.fixture
def linear(monkeypatch):
    block_fakes.put_in(monkeypatch)
    from fp32_emulated_gemm_split_gb300.linear import EmuLinear
    torch.manual_seed(0)
    return EmuLinear(5, 7)


def _same(linear, x, loss):
    """The layer's output and gradients against torch's own, in float64."""
    params = [linear.weight, linear.bias]
    y = linear(x)
    got = (y, *torch.autograd.grad(loss(y), [x, *params]))
    x64, *p64 = (t.detach().double().requires_grad_() for t in (x, *params))
    y64 = torch.nn.functional.linear(x64, *p64)
    for a, b in zip(got, (y64, *torch.autograd.grad(loss(y64), [x64, *p64]))):
        assert torch.allclose(a.double(), b, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("loss", [
    lambda y: (y.sum(0) * torch.arange(7)).sum(), lambda y: (y.mean(0) ** 2).sum(),
    lambda y: y.sum(), lambda y: (y.sum(1) * torch.arange(6)).sum(), lambda y: (y.t().contiguous() ** 2).sum()])
def test_expanded_gradients(linear, loss):
    _same(linear, torch.randn(6, 5, requires_grad=True), loss)


@pytest.mark.parametrize("x", [
    torch.randn(5).expand(6, 5), torch.randn(6, 1).expand(6, 5), torch.randn(5, 6).t(),
    torch.randn(20).unfold(0, 5, 3), torch.randn(6, 10)[:, ::2], torch.randn(6, 8)[:, 1:6]])
def test_inputs_of_any_strides(linear, x):
    _same(linear, x.detach().requires_grad_(), lambda y: (y ** 2).sum())


@pytest.mark.parametrize("energy", [lambda y: y.sum(), lambda y: y.square().sum()])
def test_a_second_derivative_is_refused(linear, energy):
    """A loss made of forces raises, where it would be trained on the energy alone."""
    x = torch.randn(6, 5, requires_grad=True)
    for wanted in (None, [x], [linear.weight]):
        e = energy(linear(x))
        force, = torch.autograd.grad(e, x, create_graph=True)
        with pytest.raises(RuntimeError, match="no second derivative"):
            (e + force.square().sum()).backward(inputs=wanted)
    assert torch.equal(torch.autograd.grad(energy(linear(x)), x)[0], force)


def test_the_bias_gradient_can_be_differentiated(linear):
    """It is a sum of the incoming gradient, by torch itself."""
    x = torch.randn(6, 5)
    g = torch.randn(6, 7, requires_grad=True)
    db, = torch.autograd.grad(linear(x), linear.bias, g, create_graph=True)
    assert torch.allclose(torch.autograd.grad(db.square().sum(), g)[0], (2 * db).expand(6, 7))


def test_a_weight_made_in_inference_mode(linear):
    """It has no version that would tell of a change: its pieces are made for each call."""
    from fp32_emulated_gemm_split_gb300.linear import EmuLinear
    with torch.inference_mode():
        layer, x = EmuLinear(5, 7), torch.randn(6, 5)
        for _ in range(2):
            want = torch.nn.functional.linear(x, layer.weight, layer.bias)
            assert torch.allclose(layer(x), want, atol=1e-6)
            layer.weight.mul_(2)
    with torch.no_grad():
        want = torch.nn.functional.linear(x, layer.weight, layer.bias)
        assert torch.allclose(layer(x), want, atol=1e-6)


@pytest.mark.parametrize("strided", [lambda: torch.randn(4, 6, 5).transpose(0, 1), lambda: torch.randn(5, 6).t(),
                                     lambda: torch.randn(5).expand(6, 5).detach()])
def test_a_copied_input_may_change_before_the_backward_pass(linear, monkeypatch, strided):
    from fp32_emulated_gemm_split_gb300 import block
    gated = block.EmuGatedLinear(5, 7)
    for layer in (linear, gated):
        x = strided()
        want = [torch.autograd.grad(layer(x.contiguous()).square().sum(), p)[0] for p in layer.parameters()]
        y = layer(x)
        x.copy_(torch.zeros(())) if x.stride(0) else x[0].zero_()
        for a, b in zip(torch.autograd.grad(y.square().sum(), list(layer.parameters())), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("strided", [lambda x: x.t().contiguous().t(), lambda x: x[:1].expand(6, 5),
                                     lambda x: torch.cat((x, x), 1)[:, :5], lambda x: x])
def test_a_second_derivative_is_refused_for_any_strides(linear, strided):
    x = torch.randn(6, 5, requires_grad=True)
    force, = torch.autograd.grad(linear(strided(x)).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        torch.autograd.grad(force.square().sum(), x)
