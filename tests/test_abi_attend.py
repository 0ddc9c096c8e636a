"""packed_prefill, paged_prefill and norm_rope_and_cache without a GPU: argument errors come back before anything
is enqueued, and the binding refuses what it can see."""
import itertools
import math
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


def _packed(K, **kw):
    a = dict(q=P, qs=512, k=P, ks=128, v=P, vs=128, starts=P, T=4, B=2, Hq=8, Hkv=2, D=64, sigma=0.125, sink=None,
             cap=0.0, window=-1, out=P, lse=None, flags=None)
    a.update(kw)
    return K.load().packed_prefill(*a.values(), None)


SHARED = [
    (dict(T=-1), 1), (dict(B=-1), 1), (dict(Hkv=0), 1), (dict(Hq=-1), 1), (dict(Hq=7), 1), (dict(D=0), 1),
    (dict(D=96), 2), (dict(D=512), 2), (dict(sigma=math.nan), 1), (dict(sigma=-1.0), 1),
    (dict(sigma=math.inf), 1), (dict(cap=-1.0), 1), (dict(cap=math.nan), 1),
    (dict(cap=math.inf), 1), (dict(window=-2), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(starts=None), 1),
    (dict(qs=504), 1), (dict(qs=516), 3), (dict(q=P8), 3), (dict(out=P8), 3), (dict(starts=P2), 3), (dict(lse=P2), 3),
    (dict(sink=P2), 3), (dict(flags=P2), 3),
    (dict(Hq=34, Hkv=2, qs=34 * 64), 2), (dict(sigma=1.5), 2),
    # a KV head's vectors are numbered in 32 bits
    (dict(T=1 << 29, qs=512), 2), (dict(T=(1 << 31) - 1, Hq=2), 2),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(k=None), 1), (dict(v=None), 1), (dict(ks=120), 1), (dict(vs=0), 1), (dict(ks=132), 3), (dict(vs=130), 3),
    (dict(k=P8), 3), (dict(v=P2), 3), (dict(ks=1 << 38), 2), (dict(vs=1 << 40), 2),
    (dict(T=0), 0), (dict(B=0), 0), (dict(T=0, q=None, k=None, v=None, starts=None, out=None), 0),
])
def test_packed_validation(K, kw, status):
    assert _packed(K, **kw) == status


def _paged(K, **kw):
    a = dict(q=P, qs=512, kc=P, vc=P, cd=1, ksc=P, vsc=P, kind=1, table=P, lens=P, starts=P, T=4, B=2, Hq=8, Hkv=2, D=64,
             bs=16, mb=8, nb=20, sigma=0.125, sink=None, cap=0.0, window=-1, ns=1, ws=None, wsb=0, out=P, lse=None, flags=None)
    a.update(kw)
    return K.load().paged_prefill(*a.values(), None)


MX = dict(cd=4, vc=None)


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(cd=0), 1), (dict(cd=5), 1), (dict(kind=0), 1), (dict(kind=3), 1), (dict(ksc=None), 1), (dict(vsc=None), 1),
    (dict(ksc=P8, kind=2), 3), (dict(kc=None), 1), (dict(vc=None), 1), (dict(lens=None), 1), (dict(table=None), 1),
    (dict(kc=P8), 3), (dict(vc=P8), 3), (dict(table=P2), 3), (dict(lens=P2), 3), (dict(bs=0), 1), (dict(bs=24), 2),
    (dict(bs=8), 2), (dict(mb=-1), 1), (dict(nb=-1), 1), (dict(ns=-1), 1), (dict(ns=1025), 1),
    (dict(mb=1 << 27), 2), (dict(nb=1 << 27), 2), (dict(MX, nb=1 << 31), 2), (dict(nb=1 << 40), 2),
    (dict(ns=2, ws=P8, wsb=1 << 30), 3), (dict(MX, vc=P), 1), (dict(MX, D=96), 2),
    (dict(T=0), 0), (dict(B=0), 0), (dict(T=0, cd=2, ksc=None, vsc=None), 0), (dict(MX, B=0), 0),
])
def test_paged_validation(K, kw, status):
    assert _paged(K, **kw) == status


def test_workspace(K):
    f = K.paged_prefill_workspace_bytes
    for D, n in itertools.product((64, 128, 256), (2, 3, 152, 1024)):
        # two partials per piece: 128 vectors (256 where sequences have about that many, but for head_dim 256) of D sums, a
        # maximum and a sum, in fp32
        assert f(4, 4, 8, 8, D, 4096, n) == n * 2 * 128 * (D + 2) * 4
        assert f(400, 1, 8, 8, D, 4096, n) == n * 2 * (128 if D == 256 else 256) * (D + 2) * 4
        assert f(4, 4, 8, 8, D, 4096, 1) == 0
    for bad in ((0, 4, 8, 8, 64, 4096, 2), (4, 0, 8, 8, 64, 4096, 2), (4, 4, 8, 3, 64, 4096, 2), (4, 4, 8, 8, 96, 4096, 2),
                (4, 4, 8, 8, 64, -1, 2), (4, 4, 8, 8, 64, 4096, 1025), (4, 4, 8, 8, 64, 4096, -1)):
        assert f(*bad) == 0


def _append(K, **kw):
    a = dict(q=P, qs=512, k=P, ks=128, v=P, vs=128, qw=P, kw=P, eps=1e-6, pos=P, cs=P, mp=100, R=64, style=0, slots=P, T=4,
             Hq=8, Hkv=2, D=64, qo=P, ko=None, kc=P, vc=P, cd=1, ns=128, bs=16, ksc=P, vsc=P, kind=1, flags=None)
    a.update(kw)
    return K.load().norm_rope_and_cache(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(Hkv=0), 1), (dict(D=0), 1), (dict(cd=0), 1), (dict(style=2), 1), (dict(kind=3), 1),
    (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1),
    (dict(qw=P8), 3), (dict(kw=P2), 3), (dict(ko=P8), 3), (dict(D=96, qs=768, ks=192, vs=192, R=0, cs=None), 2),
    (dict(R=80), 1), (dict(R=24), 2), (dict(q=None), 1), (dict(qo=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(slots=None), 1), (dict(pos=None), 1), (dict(cs=None), 1), (dict(kc=None), 1), (dict(vc=None), 1), (dict(ksc=None), 1),
    (dict(qs=504), 1), (dict(qs=516), 3), (dict(kc=P8), 3), (dict(MX, vc=P), 1), (dict(MX, bs=24, ns=240), 2),
    (dict(T=0), 0), (dict(MX, T=0), 0), (dict(T=0, qw=None, kw=None), 0),
])
def test_norm_append_validation(K, kw, status):
    assert _append(K, **kw) == status


def test_binding_refuses(K, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    h = torch.zeros((2, 1, 64), dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    one, w = torch.ones(1), torch.ones(64)
    c8 = torch.zeros((1, 16, 1, 64), dtype=torch.int8)
    mx = torch.zeros(K.mx4_cache_shape(1, 16, 1, 64), dtype=torch.uint8)
    for call in (lambda: K.packed_prefill(h, h, h, i, 0.1),
                 lambda: K.paged_prefill(h, c8, c8, one, one, 1, i[:1, None], i[:1], i, 0.1),
                 lambda: K.paged_prefill(h, mx, None, one, one, 1, i[:1, None], i[:1], i, 0.1),
                 lambda: K.norm_rope_and_cache(h, h, h, w, w, 1e-6, i, None, i, c8[0], c8[0], one, one, 1)):
        with pytest.raises(ValueError, match="current device"):
            call()
    with pytest.raises(TypeError):
        K.paged_prefill(h, c8.float(), c8, one, one, 1, i[:1, None], i[:1], i, 0.1)
    with pytest.raises(TypeError):
        K.packed_prefill(None, h, h, i, 0.1)
