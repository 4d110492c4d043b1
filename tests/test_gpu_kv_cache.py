"""Page tables, slots and the store of keys and values in 8 bits, on the GPU,
against token by token Python: equal, not near."""
import gc
import math

import pytest

import kv_ref as ref
from gpu_util import emu_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def emu():
    yield emu_module()
    gc.collect()                                     # tensors that graphs and tracebacks still hold


def _error(emu):
    """The device's error word, which is cleared."""
    code = emu.emu_get_last_device_error()
    emu.emu_clear_device_error()
    return code


def _ints(x):
    import torch
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _held(kept, page, width, rng):
    """Tables of the tokens held, and the free pages, in random order."""
    need = [-(-k // page) for k in kept]
    order = list(range(sum(need) + 40 + len(kept) * width))
    rng.shuffle(order)
    table = [[order.pop() if j < n else -7 for j in range(width)] for n in need]
    return table, order, sum(need) + 40 + len(kept) * width


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("kept,new,behind", [
    ([0], [0], 0), ([0], [1], 0), ([15], [1], 2), ([16], [1], 0), ([0, 0, 0], [0, 0, 0], 4), ([5, 0, 100], [0, 33, 1], 7),
    ([31, 64, 63, 0], [300, 1, 2, 5], 0), ([0, 7], [1500, 700], 100), (list(range(50)), [1] * 50, 0),
    ([(i * 37) % 301 for i in range(1500)], [(i * 11) % 4 for i in range(1500)], 13),
    ([(i * 7) % 90 for i in range(3000)], [int(i % 50 == 49) for i in range(3000)], 0),
])
@pytest.mark.parametrize("taken", [None, 3])
def test_tables(emu, page, kept, new, behind, taken):
    import random
    import torch
    width = max(-(-(k + n) // page) for k, n in zip(kept, new)) + 2
    table, free, pages = _held(kept, page, width, random.Random(page))
    tokens = sum(new) + behind
    want = ref.tables(kept, new, table, free, page, tokens, taken or 0)
    dev = _ints(table)
    plan = emu.emu_kv_tables(_ints(kept), _ints(new), dev, _ints(free), pages, page, tokens,
                             None if taken is None else _ints([taken]))
    assert dev.tolist() == want[0]
    for got, x in zip((plan.starts, plan.lengths, plan.slots, plan.positions), want[1:5]):
        assert got.tolist() == x
    assert plan.taken.tolist() == [want[5]]
    assert _error(emu) == 0
    # again: the same places
    again = emu.emu_kv_tables(_ints(kept), _ints(new), dev, _ints(free), pages, page, tokens,
                              None if taken is None else _ints([taken]))
    assert all(torch.equal(a, b) for a, b in zip(plan, again)) and dev.tolist() == want[0]


def test_no_sequence(emu):
    import torch
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    plan = emu.emu_kv_tables(none, none, none.view(0, 4), none, 8, 16, 5)
    assert plan.starts.tolist() == [0] and plan.slots.tolist() == [-1] * 5 and plan.positions.tolist() == [0] * 5
    assert plan.taken.tolist() == [0] and plan.lengths.numel() == 0
    assert _error(emu) == 0


def test_tables_bad_values(emu):
    """Each is recorded, and hurts the sequence that it belongs to only."""
    def run(kept, new, table, free, pages=100, tokens=20, taken=None):
        dev = _ints(table)
        plan = emu.emu_kv_tables(_ints(kept), _ints(new), dev, _ints(free), pages, 16, tokens, taken)
        assert _error(emu) == -1
        return dev.tolist(), [x.tolist() for x in plan]
    # a negative length; more tokens than the table's row holds
    for k, n in ((-1, 3), (5, -2), (30, 3), (2 ** 31 - 1, 2 ** 31 - 1)):
        table, (starts, lengths, slots, positions, taken) = run([3, k, 0], [1, n, 2], [[7, -1], [8, 9], [-1, -1]], [50, 51])
        assert starts == [0, 1, 1, 3] and lengths == [4, 0, 2] and slots[:3] == [7 * 16 + 3, 800, 801]
        assert slots[3:] == [-1] * 17 and table == [[7, -1], [8, 9], [50, -1]] and taken == [1]
    # free pages run out, are outside the cache; the page held is
    table, (_, lengths, slots, positions, taken) = run([0, 0], [3, 3], [[-1], [-1]], [4])
    assert table == [[4], [-1]] and slots[:6] == [64, 65, 66, -1, -1, -1] and taken == [2] and lengths == [3, 3]
    assert positions[:6] == [0, 1, 2, 0, 1, 2]
    table, (_, _, slots, _, _) = run([0, 0], [3, 1], [[-1], [-1]], [100, 6])
    assert table == [[-1], [6]] and slots[:4] == [-1, -1, -1, 96]
    table, (_, _, slots, _, _) = run([3, 3], [1, 1], [[-1], [6]], [9])
    assert slots[:2] == [-1, 99]
    run([0], [1], [[-1]], [4, 5], taken=_ints([-1]))
    # more rows than the step has
    table, (starts, lengths, slots, _, _) = run([0, 0, 0], [15, 15, 15], [[-1], [-1], [-1]], [1, 2, 3])
    assert starts == [0, 15, 20, 20] and lengths == [15, 5, 0] and slots == list(range(16, 31)) + list(range(32, 37))


def _cache(pages, heads, page, D, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = [(torch.randn(pages, heads, page, D, generator=g, device="cuda") * 90).clamp(-448, 448).to(ref.F8)
             for _ in range(2)]
    scales = [torch.exp2(torch.randint(-9, -4, (pages, heads), generator=g, device="cuda").float()) for _ in range(2)]
    return codes[0], codes[1], scales[0], scales[1]


def _check_store(emu, k, v, cache, slots):
    import torch
    page = cache[0].size(2)
    want = [ref.store(x, c, s, slots, page) for x, c, s in ((k, cache[0], cache[2]), (v, cache[1], cache[3]))]
    assert emu.emu_kv_store(k, v, cache, slots) is None
    for (codes, scales), c, s in zip(want, cache[:2], cache[2:]):
        assert torch.equal(s.double().cpu(), scales)
        got = c.double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(codes))
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(codes))


RUNS = [[0], [5], [15, 16], list(range(16)), list(range(3, 40)), [-1, 7, 8, -1, 33, 80, 81, 82, -1], list(range(64, 192)),
        [100, 101, 48, 49, 50, 160], [-1, -1]]


def _one_run_a_page(slots, page):
    """What a call has to keep: a page's rows are neighbours, one after another."""
    led = [s // page for i, s in enumerate(slots)
           if s >= 0 and (i == 0 or slots[i - 1] != s - 1 or s % page == 0)]
    return len(set(led)) == len(led)


@pytest.mark.parametrize("type", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("runs,heads,page,D", [
    (i, *shape) for shape in [(1, 16, 16), (3, 32, 80), (8, 64, 128), (2, 128, 256), (1, 256, 96)]
    for i in range(len(RUNS)) if _one_run_a_page(RUNS[i], shape[1])])
@pytest.mark.parametrize("size", [-12, 0, 9])
def test_store(emu, type, heads, page, D, runs, size):
    import torch
    slots = _ints(RUNS[runs])
    pages = 256 // page + 2
    g = torch.Generator(device="cuda").manual_seed(runs)
    kv = torch.randn(len(RUNS[runs]), 2, heads, D, generator=g, device="cuda") * 2.0 ** size
    kv = kv.to(getattr(torch, type))
    _check_store(emu, kv[:, 0], kv[:, 1], _cache(pages, heads, page, D), slots)
    assert _error(emu) == 0


def test_store_many(emu):
    """As many rows as make one unit take several tokens, prompts and next tokens mixed, strided."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    kept = [(i * 13) % 70 for i in range(200)]
    new = [1 if i % 10 else 200 for i in range(200)]
    page, heads, D = 32, 6, 64
    table = torch.full((200, 10), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(2200, generator=g, device="cuda").to(torch.int32)
    held = [-(-k // page) for k in kept]
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    plan = emu.emu_kv_tables(_ints(kept), _ints(new), table, order[at:].contiguous(), 2200, page, sum(new) + 9)
    qkv = torch.randn(sum(new) + 9, (4 + 2 * heads) * D + 4, generator=g, device="cuda").to(torch.bfloat16)
    k = qkv[:, 4 * D + 4:(4 + heads) * D + 4].view(-1, heads, D)
    v = qkv[:, (4 + heads) * D + 1:(4 + 2 * heads) * D + 1].view(-1, heads, D)
    _check_store(emu, k, v, _cache(2200, heads, page, D), plan.slots)
    assert _error(emu) == 0


def test_store_borders(emu):
    """Largest values at the scale's border, zeros, subnormal and huge values, infinities and NaN."""
    import torch
    tops = [0.0, 1.0, 448.0, 448.0 * (1 + 2.0 ** -23), 447.99, 3.5, 3.5000002, 1.75, 1e-45, 1e-38, 2.0 ** -118, 448 * 2.0 ** -126,
            3.4e38, 2.0 ** 127, math.inf, -math.inf, math.nan]
    k = torch.zeros(len(tops), 1, 16, device="cuda")
    k[:, 0, 3] = torch.tensor(tops)
    k[:, 0, 5] = 0.3
    k[4:10, 0, 5] = 0.0
    v = torch.full_like(k, math.inf)
    v[:, 0, :8] = torch.linspace(-5, 5, 8, device="cuda")
    cache = _cache(len(tops), 1, 16, 16)
    _check_store(emu, k, v, cache, _ints([16 * i for i in range(len(tops))]))
    # behind them, in the same pages: larger and smaller ones
    for at, size in ((1, 1.0), (2, 1e6), (3, 1e-6)):
        _check_store(emu, k * size, k * (size / 3), cache, _ints([16 * i + at for i in range(len(tops))]))
    assert _error(emu) == 0


def test_store_slots_outside(emu):
    """Not stored, recorded; every other row is."""
    import torch
    cache = _cache(4, 2, 16, 32)
    k = torch.randn(5, 2, 32, device="cuda")
    _check_store(emu, k, k, cache, _ints([64, 3, -2, 2 ** 31 - 1, 20]))
    assert _error(emu) == -1


def test_store_and_tables_in_a_graph(emu):
    """A captured step: places, store; replayed token after token it fills the
    pages as single calls do."""
    import torch
    page, heads, D = 16, 2, 32
    kept, new = _ints([14, 0, 31]), _ints([1, 1, 1])
    taken = _ints([0])
    free = _ints(list(range(9, 0, -1)))
    table = _ints([[10, -1, -1, -1], [-1] * 4, [11, 12, -1, -1]])
    cache = _cache(13, heads, page, D)
    k, v = (torch.zeros(4, heads, D, device="cuda") for _ in range(2))

    def step():
        plan = emu.emu_kv_tables(kept, new, table, free, 13, page, 4, taken)
        emu.emu_kv_store(k, v, cache, plan.slots)
        kept.copy_(plan.lengths)
        taken.copy_(plan.taken)
    warm = [x.clone() for x in (kept, taken, table, *cache)]
    step()
    graph = torch.cuda.CUDAGraph()
    for x, y in zip((kept, taken, table, *cache), warm):
        x.copy_(y)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for x, y in zip((kept, taken, table, *cache), warm):
        x.copy_(y)
    g = torch.Generator(device="cuda").manual_seed(3)
    lengths, free_at = [14, 0, 31], 0
    rows, want = table.tolist(), [(warm[3 + i].double().cpu(), warm[5 + i].double().cpu()) for i in range(2)]
    for _ in range(20):
        k.copy_(torch.randn(k.shape, generator=g, device="cuda"))
        v.copy_(torch.randn(v.shape, generator=g, device="cuda") * 3)
        graph.replay()
        rows, _, lengths, slots, _, free_at = ref.tables(lengths, [1, 1, 1], rows, free.tolist(), page, 4, free_at)
        want = [ref.store(x, *w, torch.tensor(slots), page) for x, w in zip((k, v), want)]
    assert table.tolist() == rows and kept.tolist() == lengths and taken.tolist() == [free_at]
    for i in range(2):
        assert torch.equal(cache[i].double().cpu(), want[i][0]) and torch.equal(cache[2 + i].double().cpu(), want[i][1])
    assert _error(emu) == 0
