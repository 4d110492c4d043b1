"""Operands whose rows overlap (expanded tensors, sliding windows): their row
stride is shorter than their rows, which no leading dimension can say.  The
binding refuses them on the host; no GPU is needed, the calls never launch."""
import pytest
import torch

import fp32_emulated_gemm_split_gb300 as emu


def _overlapping():
    v = torch.arange(8.0)
    return {
        "one row for all": v.expand(5, 8),
        "one column for all": v[:, None].expand(8, 5),
        "one value for all": torch.ones(1, 1).expand(6, 1),
        "windows": v.unfold(0, 4, 2),
        "windows along columns": v.unfold(0, 4, 2).t(),
    }


@pytest.mark.parametrize("name", _overlapping())
def test_overlapping_rows_are_refused(name):
    with pytest.raises(ValueError, match="overlap"):
        emu._stored(_overlapping()[name], False)


@pytest.mark.parametrize("X, trans, ld", [
    (torch.zeros(4, 6), False, 6), (torch.zeros(4, 9)[:, 2:8], False, 9), (torch.zeros(6, 4).t(), True, 4),
    (torch.zeros(1, 6).expand(1, 6), False, 6), (torch.zeros(9, 1), False, 1), (torch.zeros(9, 4)[:, :1], False, 4),
    (torch.zeros(0, 6), False, 6), (torch.zeros(6, 0), False, 1), (torch.zeros(1, 1), False, 1),
])
def test_other_strides_are_taken_as_they_are(X, trans, ld):
    """A kernel reads element (i, j) of what is stored at i * ld + j: inside the tensor's storage."""
    S, t, got = emu._stored(X, False)
    assert (t, got) == (trans, ld)
    assert torch.equal(torch.as_strided(S, S.shape, (got, 1)), S)


@pytest.mark.parametrize("C", [torch.zeros(8).expand(4, 8), torch.zeros(1, 1).expand(4, 1),
                               torch.zeros(14).unfold(0, 8, 2)])
def test_overlapping_outputs_are_refused(C):
    M, N = C.shape
    A, B = torch.zeros(M, 6), torch.zeros(6, N)
    for call in (lambda: emu.emu_sgemm(A, B, C), lambda: emu.emu_sgemm_noalloc(A, B, C),
                 lambda: emu.emu_sgemm_bsplit(A, torch.zeros(3, N, 8, dtype=torch.int16), C)):
        with pytest.raises(ValueError, match="overlap"):
            call()
