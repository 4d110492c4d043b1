"""The binding of the layers' entry points refuses arguments with an error of
its own before it needs a GPU: types, shapes, strides, missing tensors, counts.
"""
import pytest
import torch


@pytest.fixture(scope="module")
def C():
    from fp32_emulated_gemm_split_gb300 import layers
    return layers._C()


def _packed(F=6, K=4):
    Wg, Wu = torch.zeros(F, K), torch.zeros(F, K)
    return Wg, Wu, torch.zeros(3, 512, 64, dtype=torch.int16), Wg._version, Wu._version


def _lora_packed(N=6, K=4):
    W = torch.zeros(N, K)
    return W, None, torch.zeros(3, N, 64, dtype=torch.int16), W._version


Z = torch.zeros


@pytest.mark.parametrize("args, error, words", [
    ((Z(3, 4).double(), Z(3, 4)), TypeError, "Wg must be float32"),
    ((Z(3, 4), Z(3, 5)), ValueError, r"Wu must be 3 x 4, got \(3, 5\)"),
    ((Z(3, 4), Z(4, 3).t()), ValueError, "unit stride"),
    ((Z(12), Z(3, 4)), ValueError, "M x K"),
    ((Z(3, 4), None), TypeError, "Wu must be a tensor"),
    ((3, Z(3, 4)), TypeError, "Wg must be a tensor, got int"),
    ((Z(1, 4).expand(3, 4), Z(3, 4)), ValueError, "rows overlap"),
    ((Z(3, 4),), TypeError, "expected 2 arguments"),
])
def test_pack_refuses(C, args, error, words):
    with pytest.raises(error, match=words):
        C.gated_pack(*args)


@pytest.mark.parametrize("X, error", [
    (Z(2, 5), ValueError), (Z(2, 4).half(), TypeError), (Z(4), ValueError), (None, TypeError),
])
def test_gated_refuses(C, X, error):
    with pytest.raises(error):
        C.gated(0, X, _packed(), False, None)
    with pytest.raises(error):
        C.gated_bwd(0, Z(2, 6), X, _packed(), Z(2, 6), Z(2, 6), True, True)


def test_gated_bwd_wants_the_saved_products_alike(C):
    with pytest.raises(ValueError, match="same row stride"):
        C.gated_bwd(0, Z(2, 6), Z(2, 4), _packed(), Z(2, 8)[:, :6], Z(2, 6), True, True)
    with pytest.raises(ValueError, match="G must be 2 x 6"):
        C.gated_bwd(0, Z(2, 6), Z(2, 4), _packed(), Z(2, 7), Z(2, 6), True, True)


def test_changed_weights_are_refused(C):
    packed = _packed()
    packed[1].add_(1)
    with pytest.raises(ValueError, match="pack again"):
        C.gated(0, Z(2, 4), packed, False, None)
    packed = _lora_packed()
    packed[0].add_(1)
    with pytest.raises(ValueError, match="pack again"):
        C.lora(Z(2, 4), packed, Z(1, 2, 4), Z(1, 6, 2), Z(2).int(), None, None)
    for wrong in (None, (), packed[:3]):
        with pytest.raises(TypeError):
            C.lora(Z(2, 4), wrong, Z(1, 2, 4), Z(1, 6, 2), Z(2).int(), None, None)
        with pytest.raises(TypeError):
            C.gated(0, Z(2, 4), wrong, False, None)


@pytest.mark.parametrize("kw, error", [
    (dict(A=Z(1, 2, 5)), ValueError), (dict(B=Z(1, 6, 3)), ValueError), (dict(B=Z(2, 6, 2)), ValueError),
    (dict(B=Z(6, 2)), ValueError), (dict(A=Z(1, 4, 2).transpose(1, 2)), ValueError), (dict(A=Z(1, 2, 4).half()), TypeError),
    (dict(index=None), ValueError), (dict(index=Z(2).long()), ValueError), (dict(index=Z(3).int()), ValueError),
    (dict(scale=Z(2)), ValueError), (dict(scale=Z(1).double()), ValueError),
])
def test_lora_refuses(C, kw, error):
    a = dict(A=Z(1, 2, 4), B=Z(1, 6, 2), index=Z(2).int(), scale=None)
    a.update(kw)
    with pytest.raises(error):
        C.lora(Z(2, 4), _lora_packed(), a["A"], a["B"], a["index"], a["scale"], None)


def test_lora_weights(C):
    with pytest.raises(ValueError, match="bias must be 6"):
        C.lora_weights(Z(6, 4), Z(4))
    with pytest.raises(ValueError, match="bias must be 6"):
        C.lora_weights(Z(6, 4), Z(12)[::2])


@pytest.mark.parametrize("kw, error", [
    (dict(q=Z(3, 2, 8).double()), TypeError), (dict(k=Z(3, 1, 8).half()), TypeError), (dict(k=Z(2, 1, 8)), ValueError),
    (dict(k=Z(3, 1, 6)), ValueError), (dict(q=Z(3, 16)), ValueError), (dict(q=Z(3, 8, 2).transpose(1, 2)), ValueError),
    (dict(wq=Z(4)), ValueError), (dict(wk=Z(8).half()), ValueError), (dict(sin=None), ValueError),
    (dict(cos=None), ValueError), (dict(cos=Z(9, 3)), ValueError), (dict(cos=Z(9, 4).half()), TypeError),
    (dict(positions=None), ValueError), (dict(positions=Z(3).long()), ValueError), (dict(positions=Z(2).int()), ValueError),
    (dict(eps="x"), TypeError), (dict(one=None), TypeError),
])
def test_qk_norm_refuses(C, kw, error):
    a = dict(q=Z(3, 2, 8), k=Z(3, 1, 8), wq=Z(8), wk=None, cos=Z(9, 4), sin=Z(9, 4), positions=Z(3).int(), eps=1e-6)
    q, k = a["q"], a["k"]
    one = kw.get("one", k)
    a.update({n: v for n, v in kw.items() if n != "one"})
    with pytest.raises(error):
        C.qk_norm_rope(*a.values(), False, q, one)
    with pytest.raises(error):
        C.qk_norm_rope_bwd(*a.values(), False, q, one)
