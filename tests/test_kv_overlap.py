"""emu_kv_tables refuses outputs over its inputs or over one another: its blocks read
the inputs each for itself, so one that started late would see the outputs of
another.  Without a GPU; pointers are never dereferenced."""
import pytest

torch = pytest.importorskip("torch")

SIZES = dict(kept=4, new=4, free=9, taken=1, table=12, starts=5, lengths=4, slots=700, positions=700, out=1)
WRITTEN = ("table", "starts", "lengths", "slots", "positions", "out")


@pytest.fixture(scope="module")
def call():
    from fp32_emulated_gemm_split_gb300 import _build, layers
    _build.build()
    L = layers._L()

    def tables(B=4, T=700, width=3, **at):
        place, p = {}, 1 << 20
        for name, n in SIZES.items():                # one behind another, without a gap
            place[name] = p
            p += 4 * n
        place.update(at)
        p = place
        return L.emu_kv_tables(B, p["kept"], p["new"], 8, 16, p["free"], 9, p["taken"], p["table"], width, T, p["starts"],
                               p["lengths"], p["slots"], p["positions"], p["out"], None), place
    return tables


def test_neighbours_are_not_refused(call):
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are not there")
    assert call()[0] != -1


@pytest.mark.parametrize("written", WRITTEN)
@pytest.mark.parametrize("other", list(SIZES))
@pytest.mark.parametrize("end", ["first", "last"])
def test_overlaps_are_refused(call, written, other, end):
    """The written array's first element over the other's last, or its last over the other's first."""
    if written == other:
        return
    far = 1 << 24                                    # (away from all the others)
    to = far if end == "first" else far + 4 * (SIZES[other] - 1)
    at = {other: far, written: to if end == "last" else far - 4 * (SIZES[written] - 1)}
    assert call(**at)[0] == -1


def test_lengths_over_kept(call):
    assert call(lengths=call(T=0, B=-1)[1]["kept"])[0] == -1
    assert call(out=call(T=0, B=-1)[1]["taken"])[0] == -1
