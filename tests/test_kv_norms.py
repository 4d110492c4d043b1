"""The relative errors that the GPU tests of the attention over 8-bit keys and
values hold FP32 rows to: passed with two FP16 pieces of queries and weights, failed
with one of either, at every length used (on the CPU, the arithmetic emulated)."""
import pytest

torch = pytest.importorskip("torch")

import kv_norms as norms  # noqa: E402


@pytest.mark.parametrize("L", [16, 777, 1000, 4000, 20011, 40000])
@pytest.mark.parametrize("D", [64, 128])
def test_a_lost_piece_is_seen(L, D):
    g, heads = torch.Generator().manual_seed(L + D), 16

    def values():
        codes = (torch.randn(L, heads, D, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).double()
        pages = torch.randint(-9, -3, (-(-L // 32), heads), generator=g)
        return codes * torch.exp2(pages.double()).repeat_interleave(32, 0)[:L, :, None]
    K, V = values(), values()
    q = torch.randn(heads, D, generator=g)
    want = norms.in_pieces(q, K, V, 8, 8)
    s = torch.einsum("hd,lhd->hl", q.double(), K) * D ** -0.5
    assert norms.relative(want, torch.einsum("hl,lhd->hd", s.softmax(-1), V)) <= 1e-9
    assert norms.relative(norms.in_pieces(q, K, V, 2, 2), want) <= norms.TWO_PIECES / 4
    for pieces in ((1, 2), (2, 1), (1, 1)):
        assert norms.relative(norms.in_pieces(q, K, V, *pieces), want) > 2 * norms.TWO_PIECES, pieces


def test_pieces():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(50, 300, generator=g).double() * torch.exp2(torch.randint(-30, 30, (50, 1), generator=g).double())
    top = x.abs().amax(-1, keepdim=True)
    for pieces, bits in ((1, 11), (2, 22)):
        off = (norms.halves(x, pieces) - x).abs()
        assert (off <= torch.maximum(x.abs() * 2.0 ** -bits, top * 2.0 ** -39)).all()
        assert (off > x.abs() * 2.0 ** -(bits + 3)).any()
