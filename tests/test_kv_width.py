"""emu_kv_attention refuses tables whose rows hold more tokens than its positions
reach, tiles' ends among them; without a GPU, before anything is launched."""
import pytest

torch = pytest.importorskip("torch")

from test_kv_abi import _attend, _cache, layers  # noqa: E402, F401


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_positions_of_a_row(layers, page):  # noqa: F811
    most = (2 ** 31 - 256) // page
    for width in (most + 1, (2 ** 31 - 1) // page + 1, 2 ** 31):
        assert _attend(layers._L(), cache=_cache(page=page), width=width) == -1
    if not torch.cuda.is_available():                # (would launch on addresses that are not there)
        assert _attend(layers._L(), cache=_cache(page=page), width=most) != -1
