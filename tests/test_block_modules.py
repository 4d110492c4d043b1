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


def _assign(layer, new):
    layer.load_state_dict({"gate": new, "up": layer.up.detach().clone()}, assign=True)


def _set_data(layer, new):
    layer.gate.data = new


def _replace(layer, new):
    layer.gate = torch.nn.Parameter(new)


def _in_place(layer, new):
    with torch.no_grad():
        layer.gate.copy_(new)


def _load(layer, new):
    layer.load_state_dict({"gate": new, "up": layer.up.detach().clone()})


def _other_strides(layer, new):
    layer.gate.data = new.t().contiguous().t()


@pytest.mark.parametrize("change", [_assign, _set_data, _replace, _in_place, _load, _other_strides])
def test_weights_changed_since_pack_are_refused(block, change):
    layer = block.EmuGatedLinear(4, 6).eval().pack()
    x = torch.randn(3, 4)
    with torch.no_grad():
        old = layer(x)
        change(layer, torch.randn(6, 4))
        with pytest.raises(ValueError, match="pack"):
            layer(x)
        y = layer.pack()(x)
    assert not torch.allclose(y, old)
    assert torch.allclose(y.double(), _gated64(x.double(), layer.gate.double(), layer.up.double()), atol=1e-6)


def test_a_new_weight_at_the_old_address_is_refused(block):
    """The pack holds the storage that it was made of, so no later tensor can have its address."""
    layer = block.EmuGatedLinear(64, 64).eval().pack()
    was = layer.gate.data_ptr()
    for _ in range(8):
        layer.gate = torch.nn.Parameter(torch.randn(64, 64))
        assert layer.gate.data_ptr() != was
    with torch.no_grad(), pytest.raises(ValueError, match="pack"):
        layer(torch.randn(3, 64))


def test_packed_values_are_one_set(block, monkeypatch):
    """A write through .data bumps no version.  It reaches neither what the
    tiles read (the pieces) nor what few rows read (the weights): both are the
    pack's own, the values of its time."""
    layer = block.EmuGatedLinear(4, 6).eval().pack()
    x = torch.randn(3, 4)
    with torch.no_grad():
        old = layer(x)
        layer.gate.data.mul_(2)
        assert torch.equal(layer(x), old)
        mine = {t.data_ptr() for t in layer._packed.tensors}
        assert mine.isdisjoint({layer.gate.data_ptr(), layer.up.data_ptr()})
        assert not torch.allclose(layer.pack()(x), old)


def test_copies_of_a_packed_layer(block):
    import copy
    import pickle
    layer = block.EmuGatedLinear(4, 6).eval().pack()
    x = torch.randn(3, 4)
    with torch.no_grad():
        want = layer(x)
        for other in (copy.deepcopy(layer), pickle.loads(pickle.dumps(layer))):
            assert torch.equal(other(x), want) and other._packed is None
            other.gate.mul_(2)
            assert not torch.allclose(other(x), want)
        assert torch.equal(layer(x), want)


def _qk_inputs():
    q, k = torch.randn(5, 2, 8), torch.randn(5, 1, 8)
    cos, sin = torch.randn(5, 4), torch.randn(5, 4)
    return q, k, torch.rand(8), torch.rand(8), cos, sin, torch.arange(5, dtype=torch.int32)


def _gated_case(block):
    layer = block.EmuGatedLinear(4, 6)
    return layer, torch.randn(5, 4)


def _qk_case(block):
    q, *rest = _qk_inputs()
    return lambda x: block.qk_norm_rope(x, *rest)[0], q


@pytest.mark.parametrize("case", [_gated_case, _qk_case])
@pytest.mark.parametrize("energy", [lambda y: y.sum(), lambda y: y.square().sum()])
def test_a_second_derivative_is_refused(block, case, energy):
    """The backward passes run kernels that autograd does not see: a loss made
    of a gradient raises, where it would be trained on a part of itself (with a
    constant incoming gradient, too: the gradient depends on x and the weights)."""
    f, x = case(block)
    x.requires_grad_()
    for wanted in (None, x):
        e = energy(f(x))
        force, = torch.autograd.grad(e, x, create_graph=True)
        with pytest.raises(RuntimeError, match="no second derivative"):
            (e + force.square().sum()).backward(inputs=wanted)
    # one derivative is as before, asked for with a graph or not
    assert torch.equal(torch.autograd.grad(energy(f(x)), x)[0], force)
    energy(f(x)).backward(create_graph=True)
    assert torch.equal(x.grad, force)


def test_a_second_derivative_by_the_weights_is_refused(block):
    layer, x = _gated_case(block)
    x.requires_grad_()
    force, = torch.autograd.grad(layer(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivative"):
        torch.autograd.grad(force.square().sum(), [layer.gate])


def _decoder(block, **kw):
    b = block.EmuDecoderBlock(8, 2, 1, 12, max_positions=16, device="cpu", **kw)
    A, B = torch.randn(2, 3, 8), torch.randn(2, 16, 3)
    return b, torch.randn(5, 8), (A, B, torch.rand(2)), torch.tensor([0, 1, -1, 1, 0], dtype=torch.int32)


@pytest.mark.parametrize("who", ["all", "x", "norm1", "qkv.weight", "A", "B", "scale"])
def test_adapters_where_gradients_are_wanted_are_refused(block, who):
    """The adapters' product has no backward pass: a loss would flow past it
    through the residual only."""
    b, x, adapters, index = _decoder(block)
    if who != "all":
        b.requires_grad_(False)
        named = dict(b.named_parameters(), x=x, **dict(zip(("A", "B", "scale"), adapters)))
        named[who].requires_grad_()
    with pytest.raises(RuntimeError, match="adapters.*no_grad"):
        b(x, adapters=adapters, index=index)
    with torch.no_grad():
        b(x, adapters=adapters, index=index)


def test_adapters_beside_a_part_that_is_trained(block):
    """What comes behind the adapters can be trained: no gradient goes through them."""
    b, x, adapters, index = _decoder(block)
    b.requires_grad_(False)
    b.gated.requires_grad_()
    b(x, adapters=adapters, index=index).sum().backward()
    assert b.gated.gate.grad is not None


def test_tokens_from_a_later_position_on_see_no_later_token(block):
    """A call with a start that keeps nothing: causal among its own tokens."""
    b, x, _, _ = _decoder(block)
    with torch.no_grad():
        whole = b(x, start=7)
        for t in range(1, 5):
            assert torch.allclose(b(x[:t], start=7), whole[:t], atol=1e-6)


def test_start_has_to_follow_what_is_kept(block):
    b, x, _, _ = _decoder(block)
    with torch.no_grad():
        with pytest.raises(ValueError, match="kept"):
            b(x[3:], start=3, keep=True)
        whole = b(x)
        b(x[:3], keep=True)
        with pytest.raises(ValueError, match="kept"):
            b(x[3:], start=2, keep=True)
        assert torch.allclose(b(x[3:], start=3, keep=True), whole[3:], atol=1e-6)
        assert torch.equal(b(x, keep=True), whole)       # from the start again


@pytest.mark.parametrize("start", [-1, 12, 16])
def test_positions_past_the_tables_are_refused(block, start):
    b, x, _, _ = _decoder(block)
    with torch.no_grad(), pytest.raises(ValueError, match="positions"):
        b(x, start=start)


def test_gated_weights_made_in_inference_mode(block):
    """Such tensors have no version counter."""
    with torch.inference_mode():
        layer = block.EmuGatedLinear(4, 6).eval()
        x = torch.randn(3, 4)
        want = _gated64(x.double(), layer.gate.double(), layer.up.double())
        assert torch.allclose(layer(x).double(), want, atol=1e-6)
        assert torch.allclose(layer.pack()(x).double(), want, atol=1e-6)
        layer.gate = torch.nn.Parameter(torch.randn(6, 4), requires_grad=False)
        with pytest.raises(ValueError, match="pack"):
            layer(x)


def test_decoder_made_in_inference_mode(block):
    with torch.inference_mode():
        b, x, adapters, index = _decoder(block)
        whole = b.eval()(x, adapters=adapters, index=index)
        b.gated.pack()
        parts = [b(x[:3], adapters=adapters, index=index[:3], keep=True)]
        for t in (3, 4):
            parts.append(b(x[t:t + 1], start=t, adapters=adapters, index=index[t:t + 1], keep=True))
        assert torch.allclose(torch.cat(parts), whole, atol=1e-6)
