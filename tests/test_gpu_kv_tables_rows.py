"""emu_kv_tables where a step has fewer rows than its sequences' new tokens, on the
GPU, against token by token Python."""
import gc

import pytest

import kv_ref as ref
from gpu_util import emu_module
from test_gpu_kv_cache import _error, _ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()                                     # tensors that graphs and tracebacks still hold


def test_pages_of_rows_left_out_are_not_given(emu):
    """More rows than the step has: the pages of tokens that are left out stay free, the others' are as ever."""
    import torch

    def run(kept, new, tokens, taken=0):
        table = torch.full((len(kept), 20), -1, dtype=torch.int32, device="cuda")
        held = 0
        for b, n in enumerate(kept):
            for j in range(-(-n // 16)):
                table[b, j], held = 900 + held, held + 1
        plan = emu.emu_kv_tables(_ints(kept), _ints(new), table, _ints(list(range(800))), 1000, 16, tokens, _ints([taken]))
        code = _error(emu)
        fit, left = [], tokens
        for n in new:
            fit.append(min(n, left))
            left -= fit[-1]
        before = [[int(x) for x in r] for r in torch.full((len(kept), 20), -1).tolist()]
        at = 0
        for b, n in enumerate(kept):
            for j in range(-(-n // 16)):
                before[b][j], at = 900 + at, at + 1
        want = ref.tables(kept, fit, before, list(range(800)), 16, tokens, taken)
        assert table.tolist() == want[0]
        for got, x in zip(plan[:4], want[1:5]):
            assert got.tolist() == x
        assert plan.taken.tolist() == [want[5]]
        assert code == (-1 if sum(new) > tokens else 0)
    run([0, 0, 0], [15, 15, 15], 20)
    run([0, 3, 16, 0], [40, 30, 70, 100], 64, taken=5)
    run([0, 3, 16, 0], [40, 30, 70, 100], 71)
    run([5, 5], [3, 50], 0)
    run([0, 3, 16, 0], [40, 30, 70, 100], 240)
    many = [(i * 11) % 9 for i in range(2500)]
    for tokens in (0, 1, 600, 5000, sum(many) - 1, sum(many)):
        run([0] * 2500, many, tokens) if tokens <= 600 else run([3] * 60, many[:60], min(tokens, sum(many[:60]) - 2))
