"""Tables, store and attention run together, in the decoder block: prompts and next
tokens of several sequences against float64, and a captured step replayed."""
import gc

import pytest

import kv_ref as ref
from gpu_util import emu_module
from test_gpu_block import TOL, _block

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()                                     # tensors that graphs and tracebacks still hold


def _ints(*v):
    import torch
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _plain(block, x, positions, attend):
    """The block's definition in float64 with an attention of its own; (y, k, v)."""
    import torch
    p = {n: t.double() for n, t in block.state_dict().items()}
    H, Hk, D, T = block.heads, block.kv_heads, block.dim, x.size(0)

    def norm(v, w):
        return v / (v.square().mean(-1, keepdim=True) + block.eps).sqrt() * w

    def turn(v):
        c, s = p["cos"][positions.long(), None], p["sin"][positions.long(), None]
        a, b = v[..., :D // 2], v[..., D // 2:]
        return torch.cat((a * c - b * s, a * s + b * c), -1)
    x = x.double()
    q, k, v = (norm(x, p["norm1"]) @ p["qkv.weight"].t()).view(T, -1, D).split((H, Hk, Hk), 1)
    q, k = turn(norm(q, p["wq"])), turn(norm(k, p["wk"]))
    x = x + attend(q).reshape(T, -1) @ p["out.weight"].t()
    n = norm(x, p["norm2"])
    h = torch.nn.functional.silu(n @ p["gated.gate"].t()) * (n @ p["gated.up"].t())
    return x + h @ p["down.weight"].t(), k, v


@pytest.mark.parametrize("page", [16, 64])
def test_sequences_over_pages(emu, page):
    import torch
    from fp32_emulated_gemm_split_gb300.block import KvStep
    block = _block(4).eval()
    pages = 40
    cache = emu.emu_kv_cache(pages, block.kv_heads, block.dim, page=page)
    table = torch.full((4, 160 // page), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, device="cuda").to(torch.int32)
    kept, taken = _ints(0, 0, 0, 0), None
    with torch.no_grad():
        # prompts (one sequence comes later), next tokens, drafts and a second part of a prompt; rows behind them
        for step, new in enumerate([(70, 0, 3, 17), (1, 90, 1, 1), (1, 1, 1, 1), (4, 1, 60, 3), (1, 1, 1, 1)]):
            rows = sum(new) + step
            x = torch.randn(rows, 128, device="cuda")
            plan = emu.emu_kv_tables(kept, _ints(*new), table, free, pages, page, rows, taken)
            y = block(x, kv=KvStep(cache, table, plan, max(new)))
            lengths = plan.lengths.tolist()

            def attend(q):
                return ref.attention(q, *cache, table, plan.starts.tolist(), lengths, block.dim ** -0.5)[0]
            want, k, v = _plain(block, x, plan.positions, attend)
            assert float((y.double() - want).norm() / want.norm()) <= TOL
            # what was stored is the keys and values, rounded: half a step of e4m3, or of its least values (2^-10 of the
            # scale); a page's first rows once more for each time that its scale has grown, so three halves for all
            live = plan.slots >= 0
            at = plan.slots[live].long()
            for t, codes, scales in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
                s = scales[at // page].double()[..., None]
                got = codes.double()[at // page, :, at % page] * s
                assert ((got - t[live]).abs() <= 3 * (2.0 ** -4 * t[live].abs() + 2.0 ** -10 * s)).all()
            kept, taken = plan.lengths, plan.taken
    assert emu.emu_get_last_device_error() == 0


def test_captured_step(emu):
    """A step of fixed size, captured once and replayed token after token, gives
    what single calls give."""
    import torch
    from fp32_emulated_gemm_split_gb300.block import KvStep
    block = _block(5).eval()
    page, pages = 16, 30
    g = torch.Generator(device="cuda").manual_seed(0)
    xs = [torch.randn(6, 128, generator=g, device="cuda") for _ in range(20)]

    def state():
        return (emu.emu_kv_cache(pages, block.kv_heads, block.dim, page=page), _ints(0, 0, 0, 0), _ints(0),
                torch.full((4, 6), -1, dtype=torch.int32, device="cuda"), torch.arange(pages, device="cuda", dtype=torch.int32))

    def step(x, new, cache, kept, taken, table, free):
        plan = emu.emu_kv_tables(kept, new, table, free, pages, page, x.size(0), taken)
        y = block(x, kv=KvStep(cache, table, plan, 2))
        kept.copy_(plan.lengths)
        taken.copy_(plan.taken)
        return y
    counts = [_ints(*((i + b) % 3 for b in range(4))) for i in range(20)]
    with torch.no_grad():
        block.gated.pack()
        single = state()
        want = [step(x, n, *single) for x, n in zip(xs, counts)]
        held, x, n = state(), torch.zeros(6, 128, device="cuda"), _ints(0, 0, 0, 0)
        step(x, n, *held)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = step(x, n, *held)
        for i in range(20):
            x.copy_(xs[i])
            n.copy_(counts[i])
            graph.replay()
            # (rows behind the last sequence are computed from their own values only)
            assert torch.equal(y, want[i]), i
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(single[0], held[0]))
    assert torch.equal(single[3], held[3]) and emu.emu_get_last_device_error() == 0


def test_example_runs(emu, capsys):
    from fp32_emulated_gemm_split_gb300 import block
    block.main()
    assert "8-bit" in capsys.readouterr().out


def test_other_device_and_mixed_devices_are_refused(emu):
    """Tensors that are not on the current GPU."""
    import torch
    c = emu.emu_kv_cache(4, 2, 32, page=16)
    k = torch.zeros(3, 2, 32, device="cuda")
    for bad in (dict(k=k.cpu()), dict(slots=torch.zeros(3, dtype=torch.int32)), dict(cache=tuple(t.cpu() for t in c))):
        with pytest.raises(ValueError, match="current CUDA device"):
            emu.emu_kv_store(**{**dict(k=k, v=k, cache=c, slots=_ints(0, 1, 2)), **bad})
    with pytest.raises(ValueError, match="current CUDA device"):
        emu.emu_kv_attention(k, c, torch.zeros(1, 2, dtype=torch.int32), _ints(0, 3), _ints(3))
    with pytest.raises(ValueError, match="current CUDA device"):
        emu.emu_kv_tables(_ints(0), _ints(1), torch.zeros(1, 2, dtype=torch.int32), _ints(0), 4, 16, 1)
