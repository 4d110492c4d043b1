"""The operators on keys and values kept in 8 bits without a GPU: the C entry
points refuse bad arguments before anything is launched (pointers are never
dereferenced), and the binding refuses tensors of the wrong kind."""
import struct

import pytest

torch = pytest.importorskip("torch")
Z = torch.zeros
F8 = torch.float8_e4m3fn
P = 1 << 20                                          # stands for a 16-byte aligned device pointer


@pytest.fixture(scope="module")
def layers():
    from fp32_emulated_gemm_split_gb300 import _build
    _build.build()
    from fp32_emulated_gemm_split_gb300 import layers as m
    return m


def _heads(data=P, heads=2, t=128, h=64):
    return struct.pack("4q", data or 0, heads, t, h)


def _cache(k=P, v=P, ks=P, vs=P, pages=8, heads=2, page=16, D=64):
    return struct.pack("8q", k or 0, v or 0, ks or 0, vs or 0, pages, heads, page, D)


BAD_CACHE = [dict(k=None), dict(v=P + 8), dict(ks=None), dict(vs=P + 2), dict(pages=-1), dict(pages=1 << 28), dict(heads=0),
             dict(heads=2000), dict(page=8), dict(page=48), dict(page=512), dict(D=8), dict(D=72), dict(D=272)]


def _tables(L, B=2, kept=P, new=P, pages=8, page=16, free=P, n_free=4, taken=P, table=P, width=4, T=6, starts=P, lengths=P,
            slots=P, positions=P, out=P + 64):
    return L.emu_kv_tables(B, kept, new, pages, page, free, n_free, taken, table, width, T, starts, lengths, slots,
                           positions, out, None)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(B=(1 << 20) + 1), dict(kept=None), dict(new=None), dict(pages=-1), dict(pages=1 << 27), dict(page=0),
    dict(page=24), dict(page=512), dict(free=None), dict(n_free=-1), dict(n_free=1 << 31), dict(table=None), dict(width=-1),
    dict(width=1 << 28), dict(T=-1), dict(T=1 << 25), dict(starts=None), dict(lengths=None), dict(slots=None),
    dict(positions=None), dict(out=None), dict(out=P),
])
def test_tables_refuses(layers, kw):
    assert _tables(layers._L(), **kw) == -1


def _store(L, dtype=0, T=3, k=None, v=None, slots=P, cache=None):
    return L.emu_kv_store(dtype, T, k or _heads(), v or _heads(), slots, cache or _cache(), None)


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(dtype=-1), dict(T=-1), dict(T=1 << 25), dict(k=_heads(None)),
                                dict(v=_heads(heads=1)), dict(k=_heads(t=1 << 50)), dict(slots=None)] +
                         [dict(cache=_cache(**c)) for c in BAD_CACHE])
def test_store_refuses(layers, kw):
    assert _store(layers._L(), **kw) == -1


def _attend(L, dtype=0, T=3, q=None, out=None, cache=None, B=2, table=P, width=4, starts=P, lengths=P, scale=0.1, window=0,
            most=0):
    return L.emu_kv_attention(dtype, T, q or _heads(heads=4, t=256), out or _heads(heads=4, t=256), cache or _cache(), B,
                              table, width, starts, lengths, scale, window, most, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(T=-1), dict(T=1 << 25), dict(q=_heads(heads=3)), dict(q=_heads(heads=0)), dict(out=_heads(heads=2)),
    dict(q=_heads(None, 4)), dict(out=_heads(None, 4)), dict(out=_heads(heads=4, h=1 << 41)), dict(B=-1), dict(B=1 << 21),
    dict(table=None), dict(width=-1), dict(width=1 << 27), dict(starts=None), dict(lengths=None), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(window=-1), dict(most=-1)] + [dict(cache=_cache(**c)) for c in BAD_CACHE])
def test_attention_refuses(layers, kw):
    assert _attend(layers._L(), **kw) == -1


def test_empty_calls_touch_nothing(layers):
    L = layers._L()
    assert _store(L, T=0, k=_heads(None), v=_heads(None), slots=None) == 0
    assert _attend(L, T=0, q=_heads(None, 4), out=_heads(None, 4)) == 0


# ---------------------------------------------------------------- binding --

def _kv(pages=8, heads=2, page=16, D=32):
    return (Z(pages, heads, page, D).to(F8), Z(pages, heads, page, D).to(F8), Z(pages, heads), Z(pages, heads))


def _with(i, x):
    c = list(_kv())
    c[i] = x
    return tuple(c)


BAD_KV = [
    (None, TypeError, "KvCache"), (_kv()[:3], TypeError, "KvCache"), (list(_kv()), TypeError, "KvCache"),
    (_with(0, Z(8, 2, 16, 32)), TypeError, "float8_e4m3fn"), (_with(1, Z(8, 2, 16, 48).to(F8)), ValueError, "pages x heads"),
    (_with(0, Z(8, 2, 32, 16).to(F8).transpose(2, 3)), ValueError, "contiguous"),
    (_with(2, Z(8, 2).half()), TypeError, "float32"), (_with(3, Z(8, 3)), ValueError, r"\(8, 2\)"),
    (_with(2, Z(2, 8).t()), ValueError, "contiguous"), (_kv(page=24), ValueError, "16, 32, 64"),
    (_kv(D=24), ValueError, "multiple of 16"), (_kv(D=272), ValueError, "up to 256"), (_with(1, None), TypeError, "cache.v"),
]


@pytest.mark.parametrize("cache,error,words", BAD_KV)
def test_bad_caches(layers, cache, error, words):
    with pytest.raises(error, match=words):
        layers.emu_kv_store(Z(3, 2, 32), Z(3, 2, 32), cache, Z(3).int())
    with pytest.raises(error, match=words):
        layers.emu_kv_attention(Z(3, 4, 32), cache, Z(2, 4).int(), Z(3).int(), Z(2).int())


@pytest.mark.parametrize("kw,error", [
    (dict(k=Z(3, 2, 32).double()), TypeError), (dict(k=Z(3, 64)), ValueError), (dict(v=Z(3, 2, 32).half()), TypeError),
    (dict(v=Z(2, 2, 32)), ValueError), (dict(k=Z(3, 3, 32)), ValueError), (dict(k=Z(3, 32, 2).transpose(1, 2)), ValueError),
    (dict(slots=Z(3).long()), ValueError), (dict(slots=Z(4).int()), ValueError), (dict(slots=None), ValueError),
    (dict(slots=Z(6).int()[::2]), ValueError), (dict(k=None), TypeError),
])
def test_store_binding_refuses(layers, kw, error):
    a = dict(k=Z(3, 2, 32), v=Z(3, 2, 32), cache=_kv(), slots=Z(3).int())
    a.update(kw)
    with pytest.raises(error):
        layers.emu_kv_store(**a)


@pytest.mark.parametrize("kw,error", [
    (dict(q=Z(3, 4, 32).double()), TypeError), (dict(q=Z(3, 3, 32)), ValueError), (dict(q=Z(3, 4, 16)), ValueError),
    (dict(q=Z(3, 128)), ValueError), (dict(q=Z(3, 0, 32)), ValueError), (dict(table=Z(3, 4).int()), ValueError),
    (dict(table=Z(2, 4).long()), ValueError), (dict(table=Z(4, 2).int().t()), ValueError), (dict(table=None), TypeError),
    (dict(starts=Z(2).int()), ValueError), (dict(starts=None), ValueError), (dict(lengths=Z(3).int()), ValueError),
    (dict(lengths=None), TypeError), (dict(lengths=Z(2)), ValueError), (dict(scale="x"), TypeError),
    (dict(window=0.5), TypeError), (dict(out=Z(3, 4, 32).half()), TypeError), (dict(out=Z(3, 2, 32)), ValueError),
    (dict(out=Z(1, 4, 32).expand(3, 4, 32)), ValueError),
])
def test_attention_binding_refuses(layers, kw, error):
    a = dict(q=Z(3, 4, 32), cache=_kv(), table=Z(2, 4).int(), starts=Z(3).int(), lengths=Z(2).int())
    a.update(kw)
    with pytest.raises(error):
        layers.emu_kv_attention(**a)


@pytest.mark.parametrize("kw,error", [
    (dict(kept=Z(2)), ValueError), (dict(kept=Z(3).int()), ValueError), (dict(new=None), TypeError),
    (dict(new=Z(4).int()[::2]), ValueError), (dict(table=Z(2, 4)), ValueError), (dict(table=Z(3, 4).int()), ValueError),
    (dict(free=Z(2, 2).int()), ValueError), (dict(free=Z(5)), ValueError), (dict(taken=Z(2).int()), ValueError),
    (dict(taken=3), TypeError), (dict(tokens=-1), ValueError), (dict(tokens=1 << 25), ValueError), (dict(page="x"), TypeError),
])
def test_tables_binding_refuses(layers, kw, error):
    a = dict(kept=Z(2).int(), new=Z(2).int(), table=Z(2, 4).int(), free=Z(5).int(), pages=8, page=16, tokens=6)
    a.update(kw)
    with pytest.raises(error):
        layers.emu_kv_tables(**a)


def test_cache_and_its_type(layers):
    import fp32_emulated_gemm_split_gb300 as emu
    c = emu.emu_kv_cache(5, 3, 48, page=32, device="cpu")
    assert isinstance(c, emu.KvCache) and isinstance(c, tuple)
    assert c.k.shape == c.v.shape == (5, 3, 32, 48) and c.k.dtype == F8 and c.k_scale.shape == (5, 3)
    assert not c.v.float().any() and not c.v_scale.any()
