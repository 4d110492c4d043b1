"""Outputs that are given: one whose elements share memory is refused before
anything is launched (no GPU needed)."""
import pytest
import torch


@pytest.fixture(scope="module")
def C():
    from fp32_emulated_gemm_split_gb300 import layers
    return layers._C()


Z = torch.zeros


@pytest.mark.parametrize("q, k", [
    (Z(1, 2, 8).expand(3, 2, 8), Z(3, 1, 8)), (Z(3, 1, 8).expand(3, 2, 8), Z(3, 1, 8)), (Z(3, 2, 8), Z(1, 1, 8).expand(3, 1, 8)),
])
def test_heads_that_share_memory(C, q, k):
    with pytest.raises(ValueError, match="share memory"):
        C.qk_norm_rope(Z(3, 2, 8), Z(3, 1, 8), None, None, None, None, None, 1e-6, False, q, k)


@pytest.mark.parametrize("q, k", [
    (Z(3, 4, 8)[:, ::2], Z(2, 6, 8).transpose(0, 1)[::2, :1]), (Z(3, 2, 8), Z(3, 1, 8)),
    (Z(3, 2, 8), Z(3, 1, 8)[:, :0].expand(3, 0, 8)),
])
def test_other_strides_pass(C, q, k):
    """(as far as the call gets without a GPU)"""
    with pytest.raises(Exception) as e:
        C.qk_norm_rope(Z(3, 2, 8), Z(3, k.size(1), 8), None, None, None, None, None, 1e-6, False, q, k)
    assert "share memory" not in str(e.value)
