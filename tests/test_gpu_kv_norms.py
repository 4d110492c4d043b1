"""Attention over keys and values kept in 8 bits, on the GPU: what the elementwise
bounds of test_gpu_kv_attention.py cannot see (kv_norms.py), and values whose sizes
lie far apart."""
import gc
import math

import pytest

import kv_norms as norms
import kv_ref as ref
from gpu_util import emu_module
from test_gpu_kv_attention import TYPES, _error, _ints, _make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()                                     # tensors that graphs and tracebacks still hold


def _type(type):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[type]


def _attend(emu, made, **how):
    q, cache, table, starts, lengths = made
    return emu.emu_kv_attention(q, cache, table, _ints(starts), _ints(lengths), **how)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("n", [1, 40, 140])
@pytest.mark.parametrize("zero_first", [True, False])
def test_zero_values_with_the_largest_scores(emu, type, n, zero_first):
    """Pages of zero values have the least scale there is; other pages' values are finite beside them,
    and count where their weights do (those below 2^-126 of the row's largest may be left out)."""
    import torch
    for scale in (1.0, 2.0 ** 3, 2.0 ** 9, 2.0 ** 20, 2.0 ** 40, 2.0 ** 100):
        for gap in (60, 80, 88, 120, 208):
            made = norms.far_below(0.0, scale, gap, n, zero_first)
            made = (made[0].to(_type(type)), *made[1:])
            out = _attend(emu, made, scale=1 / 64, max_new=n)
            want, bound = ref.attention(*made[:1], *made[1], *made[2:], 1 / 64)
            assert not torch.isnan(out).any(), (scale, gap)
            assert ref.within(out, want, bound + (norms.flushed(made) if gap > 83 else 0.0)), (scale, gap)
    assert _error(emu) == 0
