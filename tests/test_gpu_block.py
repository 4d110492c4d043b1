"""The block operators as torch modules and run together in a small decoder
block, against float64 PyTorch (autograd of plain operations)."""
import gc
import math

import pytest

from gpu_util import emu_module

pytestmark = pytest.mark.gpu

# a block is a dozen FP32 steps of 2^-24 relative error each, amplified by sums
# of a few hundred terms: 1e-5 of the result's norm leaves a factor of ten
TOL = 1e-5


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()                                     # tensors that graphs and tracebacks still hold


def _plain(block, x, start=0, adapters=None, index=None):
    """The block's definition in float64."""
    import torch
    p = {n: v.double() for n, v in block.state_dict().items()}
    for n in p:
        p[n].requires_grad_(not n.startswith(("cos", "sin")))
    H, Hk, D, T = block.heads, block.kv_heads, block.dim, x.size(0)

    def norm(v, w):
        return v / (v.square().mean(-1, keepdim=True) + block.eps).sqrt() * w

    def turn(v):
        c, s = p["cos"][start:start + T, None], p["sin"][start:start + T, None]
        a, b = v[..., :D // 2], v[..., D // 2:]
        return torch.cat((a * c - b * s, a * s + b * c), -1)
    n = norm(x, p["norm1"])
    y = n @ p["qkv.weight"].t()
    if adapters is not None:
        A, B, scale = (a.double() for a in adapters)
        y = y + torch.stack([scale[i] * (B[i] @ (A[i] @ n[t])) if i >= 0 else torch.zeros_like(y[t])
                             for t, i in enumerate(index.tolist())])
    q, k, v = y.view(T, -1, D).split((H, Hk, Hk), 1)
    q, k = turn(norm(q, p["wq"])), turn(norm(k, p["wk"]))
    k, v = k.repeat_interleave(H // Hk, 1), v.repeat_interleave(H // Hk, 1)
    s = torch.einsum("qhd,khd->hqk", q, k) / math.sqrt(D)
    s = s.masked_fill(torch.ones(T, T, device=x.device).triu(1).bool(), float("-inf"))
    x = x + torch.einsum("hqk,khd->qhd", s.softmax(-1), v).reshape(T, -1) @ p["out.weight"].t()
    n = norm(x, p["norm2"])
    h = torch.nn.functional.silu(n @ p["gated.gate"].t()) * (n @ p["gated.up"].t())
    return x + h @ p["down.weight"].t(), p


def _block(seed=0):
    import torch
    from fp32_emulated_gemm_split_gb300.block import EmuDecoderBlock
    torch.manual_seed(seed)
    block = EmuDecoderBlock(128, 4, 2, 328, max_positions=256)
    with torch.no_grad():
        for w in (block.norm1, block.norm2, block.wq, block.wk):
            w.add_(0.2 * torch.randn_like(w))
    return block


def test_training_step(emu):
    import torch
    block = _block()
    x = torch.randn(70, 128, device="cuda", requires_grad=True)
    d = torch.randn(70, 128, device="cuda")
    y = block(x)
    y.backward(d)
    x64 = x.detach().double().requires_grad_(True)
    want, p = _plain(block, x64)
    want.backward(d.double())
    y, want = y.detach(), want.detach()
    assert float((y.double() - want).norm() / want.norm()) <= TOL
    assert float((x.grad.double() - x64.grad).norm() / x64.grad.norm()) <= TOL
    for n, v in block.named_parameters():
        assert float((v.grad.double() - p[n].grad).norm() / p[n].grad.norm()) <= TOL, n


def test_serving_with_adapters(emu):
    """A prompt and then single tokens give what one pass over all gives, and
    both what float64 gives."""
    import torch
    block = _block(1).eval()
    T, new = 60, 5
    x = torch.randn(T + new, 128, device="cuda")
    A, B = torch.randn(3, 4, 128, device="cuda") / 11, torch.randn(3, 256, 4, device="cuda") / 2
    adapters = (A, B, torch.tensor([0.5, 1.0, 1.5], device="cuda"))
    index = torch.randint(-1, 3, (T + new,), device="cuda", dtype=torch.int32)
    with torch.no_grad():
        whole = block(x, adapters=adapters, index=index)
        block.gated.pack()
        parts = [block(x[:T], adapters=adapters, index=index[:T], keep=True)]
        for t in range(T, T + new):
            parts.append(block(x[t:t + 1], start=t, adapters=adapters, index=index[t:t + 1], keep=True))
        want, _ = _plain(block, x.double(), adapters=adapters, index=index)
    assert float((whole.double() - want).norm() / want.norm()) <= TOL
    assert float((torch.cat(parts).double() - want).norm() / want.norm()) <= TOL


def test_gated_module(emu):
    """Leading dimensions, parts without gradients, packed weights, and an
    in-place change between forward and backward."""
    import torch
    from fp32_emulated_gemm_split_gb300.block import EmuGatedLinear
    torch.manual_seed(3)
    layer = EmuGatedLinear(40, 72, activation="gelu", device="cuda")
    x = torch.randn(2, 9, 40, device="cuda")
    y = layer(x)
    assert y.shape == (2, 9, 72)
    y.sum().backward()
    assert x.grad is None and layer.gate.grad is not None
    with torch.no_grad():
        plain = layer(x)
        layer.eval().pack()
        assert bool((layer(x) == plain).all()) and bool((plain == y).all())
        layer.gate.mul_(2)
        with pytest.raises(ValueError):                  # until packed again
            layer(x)
        assert not bool((layer.pack()(x) == plain).all())
    layer.train()
    y = layer(x)
    with torch.no_grad():
        layer.up.add_(1)
    with pytest.raises(ValueError):
        y.sum().backward()
    with pytest.raises(TypeError):
        layer(x.half())


def test_example_runs(emu, capsys):
    from fp32_emulated_gemm_split_gb300 import block
    block.main()
    assert "apart" in capsys.readouterr().out


def test_changed_weights_are_refused(emu):
    import torch
    W = torch.randn(24, 16, device="cuda")
    X = torch.randn(5, 16, device="cuda")
    index = torch.zeros(5, dtype=torch.int32, device="cuda")
    A, B = torch.randn(1, 2, 16, device="cuda"), torch.randn(1, 24, 2, device="cuda")
    w, g = emu.emu_lora_pack(W), emu.emu_gated_pack(W, W.clone())
    emu.emu_lora(X, w, A, B, index)
    _, G, U = emu.emu_gated(X, g, save=True)
    W.add_(1)
    with pytest.raises(ValueError):
        emu.emu_lora(X, w, A, B, index)
    with pytest.raises(ValueError):
        emu.emu_gated(X, g)
    with pytest.raises(ValueError):
        emu.emu_gated_bwd(G, X, g, G, U)
