"""rope_and_cache, gather_cache, paged_decode_mx4 without a GPU: argument errors
come back before anything is enqueued, and the binding refuses what it can see."""
import itertools
import os

import pytest
import torch

P = 0x10000
P8 = 0x10008
P2 = 0x10002


@pytest.fixture(scope="module")
def K():
    import int8_kv_cache_gb300 as K
    if not os.path.exists(K.library_path()):
        from int8_kv_cache_gb300 import build
        build.build()
    K.load()
    return K


def _append(K, **kw):
    a = dict(q=P, qs=512, k=P, ks=128, v=P, vs=128, pos=P, cs=P, mp=100, R=64, style=0, slots=P, T=4,
             Hq=8, Hkv=2, D=64, qo=P, kc=P, vc=P, cd=1, ns=128, bs=16, ksc=P, vsc=P, kind=1, flags=None)
    a.update(kw)
    return K.load().rope_and_cache(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["cs"], a["mp"], a["R"],
        a["style"], a["slots"], a["T"], a["Hq"], a["Hkv"], a["D"], a["qo"], a["kc"], a["vc"], a["cd"],
        a["ns"], a["bs"], a["ksc"], a["vsc"], a["kind"], a["flags"], None)


MX = dict(cd=4, vc=None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(Hq=-1), 1), (dict(D=0), 1), (dict(mp=-1), 1),
    (dict(ns=-1), 1), (dict(cd=0), 1), (dict(cd=5), 1), (dict(style=2), 1), (dict(kind=3), 1),
    (dict(R=-16), 1), (dict(R=80), 1), (dict(R=8), 2), (dict(D=72), 2), (dict(R=24), 2),
    (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1),
    (dict(pos=None), 1), (dict(cs=None), 1), (dict(kc=None), 1), (dict(vc=None), 1),
    (dict(ksc=None), 1), (dict(vsc=None), 1),
    (dict(qs=504), 1), (dict(ks=120), 1), (dict(vs=0), 1), (dict(qs=516), 3), (dict(ks=130), 3),
    (dict(vs=132), 3), (dict(q=P8), 3), (dict(qo=P8), 3), (dict(k=P8), 3), (dict(v=P2), 3),
    (dict(cs=P8), 3), (dict(pos=P2), 3), (dict(slots=P2), 3), (dict(kc=P8), 3), (dict(vc=P8), 3),
    (dict(flags=P2), 3), (dict(ksc=P8, kind=2), 3),
    (dict(MX, vc=P), 1), (dict(MX, bs=0), 1), (dict(MX, bs=24, ns=240), 2), (dict(MX, ns=120), 1),
    (dict(Hkv=1 << 26), 2), (dict(Hq=1 << 26), 2), (dict(MX, D=80, qs=640, ks=160, vs=160), 2), (dict(MX, R=48), 2), (dict(MX, R=16), 2),
])
def test_append_validation(K, kw, status):
    assert _append(K, **kw) == status


def test_append_of_nothing_is_ok(K):
    for cd in (1, 2, 3):
        assert _append(K, T=0, cd=cd) == 0
    assert _append(K, T=0, **MX) == 0
    assert _append(K, T=0, cd=2, ksc=None, vsc=None) == 0  # an fp16 cache takes no scales
    assert _append(K, T=0, q=None, qo=None, k=None, v=None, slots=None, pos=None, cs=None, kc=None, vc=None) == 0


def _gather(K, **kw):
    a = dict(slots=P, N=4, Hkv=2, D=64, kc=P, vc=P, cd=1, ns=128, bs=16, ksc=P, vsc=P, kind=1, ko=P, vo=P,
             flags=None)
    a.update(kw)
    return K.load().gather_cache(a["slots"], a["N"], a["Hkv"], a["D"], a["kc"], a["vc"], a["cd"], a["ns"],
                                 a["bs"], a["ksc"], a["vsc"], a["kind"], a["ko"], a["vo"], a["flags"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 1), (dict(Hkv=0), 1), (dict(D=0), 1), (dict(D=40), 2), (dict(cd=9), 1), (dict(ns=-5), 1),
    (dict(slots=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(ksc=None), 1), (dict(kind=0), 1),
    (dict(ko=P8), 3), (dict(vo=P8), 3), (dict(slots=P2), 3), (dict(kc=P8), 3), (dict(flags=P2), 3),
    (dict(MX, vc=P), 1), (dict(MX, bs=8), 2), (dict(MX, ns=100), 1), (dict(MX, D=96), 2),
    (dict(N=0), 0), (dict(ko=None, vo=None), 0),
])
def test_gather_validation(K, kw, status):
    assert _gather(K, **kw) == status


def _decode(K, **kw):
    a = dict(q=P, c=P, ks=P, vs=P, kind=1, bt=P, lens=P, B=2, Hq=4, Hkv=1, D=64, bs=16, mb=8, nb=20,
             sigma=0.125, sink=None, softcap=0.0, window=-1, ns=1, chunk=128, ws=None, wsb=0, out=P, lse=None,
             flags=None)
    a.update(kw)
    return K.load().paged_decode_mx4(
        a["q"], a["c"], a["ks"], a["vs"], a["kind"], a["bt"], a["lens"], a["B"], a["Hq"], a["Hkv"], a["D"],
        a["bs"], a["mb"], a["nb"], a["sigma"], a["sink"], a["softcap"], a["window"], a["ns"], a["chunk"],
        a["ws"], a["wsb"], a["out"], a["lse"], a["flags"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(mb=-1), 1), (dict(nb=-1), 1), (dict(bs=0), 1), (dict(ns=-1), 1), (dict(bs=24), 2),
    (dict(D=96), 2), (dict(Hq=5, Hkv=2), 1), (dict(Hq=17), 2), (dict(sigma=1.5), 2), (dict(sigma=-1.0), 1),
    (dict(sigma=float("nan")), 1), (dict(softcap=-1.0), 1), (dict(softcap=float("inf")), 1),
    (dict(window=-2), 1), (dict(kind=0), 1), (dict(ks=None), 1), (dict(q=None), 1), (dict(c=None), 1),
    (dict(lens=None), 1), (dict(bt=None), 1), (dict(q=P8), 3), (dict(c=P8), 3), (dict(out=P8), 3),
    (dict(lens=P2), 3), (dict(lse=P2), 3), (dict(sink=P2), 3), (dict(out=None), 1),
    (dict(ns=1, chunk=112), 1), (dict(ns=33, chunk=16), 1), (dict(ns=2, chunk=64), 4),
    (dict(ns=2, chunk=0), 4), (dict(ns=33, chunk=0), 1), (dict(ns=2, chunk=64, ws=P8, wsb=1 << 20), 3),
    (dict(mb=1 << 27, chunk=1 << 30), 2), (dict(B=1 << 27), 2),
    (dict(window=64, ns=1, chunk=64), 1),   # 64 < min(cap, window + 16)
    (dict(B=0), 0), (dict(B=0, window=64, chunk=80), 0),
])
def test_decode_validation(K, kw, status):
    assert _decode(K, **kw) == status


def test_the_other_calls_refuse_the_4_bit_cache(K):
    lib = K.load()
    assert lib.reshape_and_cache(P, P, P, 4, 2, 64, P, P, 100, P, P, 1, K.CACHE_MX4, None, None) == 1
    assert lib.paged_decode(P, P, P, K.CACHE_MX4, P, P, 1, P, P, 2, 4, 1, 64, 16, 8, 20, 0.125, None, 1, 128,
                            None, 0, P, None, None, None, None) == 1


def test_cache_size(K):
    for nb, bs, Hkv, D in itertools.product((1, 7), (16, 48, 64), (1, 8), (64, 128, 256)):
        shape = K.mx4_cache_shape(nb, bs, Hkv, D)
        assert shape == (nb, Hkv, bs // 16, 18 * D)
        # 16 tokens of 18 D bytes: 9 / 16 of a byte per key or value channel
        assert K.load().mx4_cache_bytes(nb, bs, Hkv, D) == nb * bs * Hkv * 2 * D * 9 // 16
    for bad in ((0, 16, 1, 64), (1, 24, 1, 64), (1, 16, 0, 64), (1, 16, 1, 96), (1, 0, 1, 64)):
        assert K.load().mx4_cache_bytes(*bad) == 0
        with pytest.raises(ValueError):
            K.mx4_cache_shape(*bad)


def test_binding_refuses_host_tensors(K, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    h = torch.zeros((2, 1, 64), dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    one = torch.ones(1)
    c8 = torch.zeros((16, 1, 64), dtype=torch.int8)
    mx = torch.zeros(K.mx4_cache_shape(1, 16, 1, 64), dtype=torch.uint8)
    for call in (lambda: K.rope_and_cache(h, h, h, i, None, i, c8, c8, one, one, 1),
                 lambda: K.rope_and_cache(h, h, h, i, None, i, mx, None, one, one, 1),
                 lambda: K.gather_cache(i, c8, c8, one, one, 1),
                 lambda: K.paged_decode_mx4(h, mx, one, one, 1, i[:, None], i, 0.1)):
        with pytest.raises(ValueError, match="current device"):
            call()
    with pytest.raises(TypeError):
        K.rope_and_cache(h, h, h, i, None, i, c8.float(), c8, one, one, 1)
    with pytest.raises(TypeError):
        K.paged_decode_mx4(h, mx.view(torch.int8), one, one, 1, i[:, None], i, 0.1)
