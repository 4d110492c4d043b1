"""include/emu_layers.h without a GPU: every bad argument is refused on the
host before anything is launched, and empty calls do nothing.  The pointers
are never dereferenced."""
import struct

import pytest

from fp32_emulated_gemm_split_gb300 import _build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def layers():
    _build.build()
    from fp32_emulated_gemm_split_gb300 import layers as m
    return m


P = 1 << 20                                          # stands for a 16-byte aligned device pointer


def _gated(L, act=0, M=4, F=8, K=16, X=P, ldx=16, Wg=P, ldwg=16, Wu=P, ldwu=16, Wp=P, ldwp=64, H=P, ldh=8,
           G=None, U=None, ldg=0):
    return L.emu_gated(act, M, F, K, X, ldx, Wg, ldwg, Wu, ldwu, Wp, ldwp, H, ldh, G, U, ldg, None)


@pytest.mark.parametrize("kw", [
    dict(act=-1), dict(act=5), dict(M=-1), dict(F=-1), dict(K=-1), dict(M=1 << 31), dict(F=1 << 30),
    dict(K=1 << 31, ldx=1 << 32, ldwp=1 << 32), dict(ldx=15), dict(ldh=7), dict(X=None), dict(H=None),
    dict(Wp=None), dict(Wp=P + 8), dict(ldwp=63), dict(ldwp=96), dict(K=65, ldx=65, ldwg=65, ldwu=65),
    dict(Wg=None), dict(Wu=None), dict(ldwg=15), dict(ldwu=15), dict(G=P), dict(U=P), dict(G=P, U=P, ldg=7),
])
def test_gated_refuses(layers, kw):
    assert _gated(layers._L(), **kw) == -1


def test_gated_pack_and_backward_refuse(layers):
    L = layers._L()
    pack = lambda F=8, K=16, Wg=P, ldg=16, Wu=P, ldu=16, Wp=P, ldp=64: L.emu_gated_pack(  # noqa: E731
        F, K, Wg, ldg, Wu, ldu, Wp, ldp, None)
    for kw in (dict(F=-1), dict(K=-1), dict(Wg=None), dict(Wu=None), dict(Wp=None), dict(Wp=P + 2), dict(ldg=15),
               dict(ldu=15), dict(ldp=16), dict(ldp=72)):
        assert pack(**kw) == -1, kw

    def bwd(act=0, M=4, F=8, K=16, dH=P, lddh=8, X=P, ldx=16, Wp=P, ldwp=64, G=P, U=P, ldg=8, dX=P, lddx=16, dW=P,
            lddw=16):
        return L.emu_gated_bwd(act, M, F, K, dH, lddh, X, ldx, Wp, ldwp, G, U, ldg, dX, lddx, dW, lddw, None)
    for kw in (dict(act=9), dict(M=-1), dict(dH=None), dict(X=None), dict(Wp=None), dict(G=None), dict(U=None),
               dict(lddh=7), dict(ldx=15), dict(ldg=7), dict(lddx=15), dict(lddw=15), dict(ldwp=70)):
        assert bwd(**kw) == -1, kw
    assert bwd(dX=None, dW=None) == 0


def test_gated_rows(layers):
    L = layers._L()
    assert [L.emu_gated_rows(f) for f in (0, 1, 32, 33, 5504)] == [0, 32, 32, 64, 5504]
    assert L.emu_gated_rows(-1) == -1 and L.emu_gated_rows(1 << 40) == -1


def test_empty_calls_touch_nothing(layers):
    L = layers._L()
    assert _gated(L, M=0, X=None, H=None) == 0 and _gated(L, F=0, H=None) == 0
    assert L.emu_gated_pack(0, 16, None, 16, None, 16, None, 64, None) == 0
    assert _lora(L, M=0, X=None, Y=None) == 0 and _lora(L, N=0, Y=None) == 0
    assert _qk(L, layers, T=0) == 0


def _lora(L, M=4, N=8, K=16, X=P, ldx=16, W=P, ldw=16, Wp=P, ldwp=16, bias=None, R=4, n=2, A=P, B=P, scale=None,
          index=P, Y=P, ldy=8):
    return L.emu_lora(M, N, K, X, ldx, W, ldw, Wp, ldwp, bias, R, n, A, B, scale, index, Y, ldy, None)


@pytest.mark.parametrize("kw", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(R=-1), dict(n=-1), dict(M=1 << 40), dict(N=1 << 40), dict(R=1 << 20),
    dict(n=1 << 24), dict(ldx=15), dict(ldy=7), dict(ldw=15), dict(X=None), dict(Y=None), dict(Wp=None),
    dict(Wp=P + 4), dict(ldwp=15), dict(ldwp=20), dict(A=None), dict(B=None), dict(index=None),
])
def test_lora_refuses(layers, kw):
    assert _lora(layers._L(), **kw) == -1


def _qk(L, m, dtype=0, T=3, D=64, rot=64, pairs=0, eps=1e-6, q=(P, 4, 256, 64), k=(P, 2, 128, 64), cos=P, sin=P,
        rows=100, pos=P, qo=(P, 4, 256, 64), ko=(P, 2, 128, 64)):
    heads = b"".join(struct.pack("4q", h[0] or 0, *h[1:]) for h in (q, k, qo, ko))
    return L.emu_qk_norm_rope(dtype, T, D, rot, pairs, eps, heads, None, None, cos, sin, rows, pos, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(dtype=-1), dict(T=-1), dict(T=1 << 31), dict(D=0), dict(D=513), dict(rot=63), dict(rot=66),
    dict(rot=-2), dict(pairs=2), dict(eps=-1.0), dict(eps=float("nan")), dict(q=(None, 4, 256, 64)),
    dict(q=(P, -1, 256, 64)), dict(qo=(P, 3, 256, 64)), dict(ko=(None, 2, 128, 64)), dict(cos=None),
    dict(sin=None), dict(pos=None), dict(rows=-1), dict(q=(P, 4, 1 << 50, 64)),
])
def test_qk_norm_refuses(layers, kw):
    assert _qk(layers._L(), layers, **kw) == -1
