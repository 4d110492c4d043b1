"""What the decoder block refuses of a step over pages, on the CPU: before any kernel."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def block():
    from fp32_emulated_gemm_split_gb300.block import EmuDecoderBlock
    return EmuDecoderBlock(32, 4, 2, 48, max_positions=16, device="cpu").eval()


def _step(rows):
    import fp32_emulated_gemm_split_gb300 as emu
    from fp32_emulated_gemm_split_gb300.block import KvStep
    z = torch.zeros(rows, dtype=torch.int32)
    return KvStep(emu.emu_kv_cache(4, 2, 16, page=16, device="cpu"), torch.zeros(1, 2, dtype=torch.int32),
                  emu.KvPlan(torch.tensor([0, rows]), z[:1], z, z, z[:1]))


def test_start_and_keep_are_refused(block):
    for kw in (dict(start=1), dict(keep=True)):
        with pytest.raises(ValueError, match="the plan has the positions"):
            block(torch.zeros(3, 32), kv=_step(3), **kw)


def test_a_plan_of_another_size_is_refused(block):
    with pytest.raises(ValueError, match="places for 4 rows, x has 3"):
        block(torch.zeros(3, 32), kv=_step(4))


def test_gradients_are_refused(block, monkeypatch):
    from fp32_emulated_gemm_split_gb300 import block as module
    monkeypatch.setattr(block, "qkv", torch.nn.Linear(32, 64, bias=False))
    monkeypatch.setattr(module, "emu_kv_store", None)
    with pytest.raises(RuntimeError, match="no backward pass"):
        block(torch.zeros(3, 32), kv=_step(3))
