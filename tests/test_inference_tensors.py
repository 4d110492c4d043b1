"""Weights made under torch.inference_mode have no version counter: packing and
using them works all the same, on copies of the pack's own."""
import pytest
import torch


@pytest.fixture(scope="module")
def layers():
    from fp32_emulated_gemm_split_gb300 import layers
    layers._C()
    return layers


def _weights():
    with torch.inference_mode():
        return torch.zeros(6, 4), torch.zeros(6, 4)


def test_packs_keep_copies(layers, monkeypatch):
    class C:
        gated_pack = staticmethod(lambda Wg, Wu: torch.zeros(3, 64, 64, dtype=torch.int16))
        lora_weights = staticmethod(lambda W, bias: None)
    monkeypatch.setattr(layers, "_C", lambda: C)
    monkeypatch.setattr(layers, "emu_split_b", lambda W, transB: torch.zeros(3, 6, 8, dtype=torch.int16))
    for mode in (torch.inference_mode, torch.no_grad):
        with mode():
            Wg, Wu = _weights()
            g, w = layers.emu_gated_pack(Wg, Wu), layers.emu_lora_pack(Wg, Wu[:, 0].contiguous())
            assert {Wg.data_ptr(), Wu.data_ptr()}.isdisjoint({g.Wg.data_ptr(), g.Wu.data_ptr(), w.W.data_ptr()})
    # others are kept as they are
    Wg, Wu = torch.zeros(6, 4), torch.nn.Parameter(torch.zeros(6, 4))
    with torch.inference_mode():
        g = layers.emu_gated_pack(Wg, Wu)
    assert g.Wg.data_ptr() == Wg.data_ptr() and g.Wu.data_ptr() == Wu.data_ptr()
    assert g._args[3:] == (Wg._version, Wu._version)


@pytest.mark.parametrize("mode", [torch.inference_mode, torch.no_grad])
def test_the_binding_takes_them(layers, mode):
    """As far as a call gets before it needs a GPU: an argument is refused for what it is."""
    C = layers._C()
    Wg, Wu = _weights()
    with mode():
        X = torch.zeros(2, 5)
        with pytest.raises(ValueError, match="X must be M x 4"):
            C.gated(0, X, (Wg, Wu, torch.zeros(3, 64, 64, dtype=torch.int16), -1, -1), False, None)
        with pytest.raises(ValueError, match="X must be M x 4"):
            C.lora(X, (Wg, None, torch.zeros(3, 6, 64, dtype=torch.int16), -1), X, X, X, None, None)
        with pytest.raises(ValueError, match="pack again"):
            C.gated(0, X, (Wg, Wu, torch.zeros(3, 64, 64, dtype=torch.int16), 0, -1), False, None)
