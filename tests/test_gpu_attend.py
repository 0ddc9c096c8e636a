"""packed_prefill and paged_prefill on the GPU, against the definition in 64 bits (tests/attend64.py)."""
import math

import pytest
import torch

from attend64 import KINDS, attend64, bounds, cache_of, check, context_of, tables, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import int8_kv_cache_gb300 as K
    K.load()
    return K


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def firsts(new, first=0):
    s = [first]
    for n in new:
        s.append(s[-1] + n)
    return s


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def projection(g, T, Hq, Hkv, D, pad=0):
    """q, k, v as slices of one projection's output."""
    x = torch.randn((T, (Hq + 2 * Hkv) * D + pad), generator=g, device="cuda").half()
    q, k, v = x[:, :(Hq + 2 * Hkv) * D].unflatten(1, (-1, D)).split((Hq, Hkv, Hkv), dim=1)
    return q, k, v


def run_packed(K, q, k, v, starts, sigma, **kw):
    T, Hq, D = q.shape
    out = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.packed_prefill(q, k, v, ints(starts), sigma, out=out, lse=lse, flags=flags, **{a: b for a, b in kw.items() if b is not None})
    torch.cuda.synchronize()
    assert int(flags) == 0
    return out, lse


def packed_case(K, seed, new, Hq, Hkv, D, window=-1, softcap=0.0, sink=False, tail=0, head=0):
    g = gen(seed)
    starts = firsts(new, head)
    T = starts[-1] + tail
    q, k, v = projection(g, T, Hq, Hkv, D, pad=8)
    sk = torch.randn(Hq, generator=g, device="cuda") if sink else None
    sigma = D ** -0.5
    out, lse = run_packed(K, q, k, v, starts, sigma, head_sink=sk, window=window, softcap=softcap)
    ctx = lambda b: (k[starts[b]:starts[b + 1]].double(), v[starts[b]:starts[b + 1]].double(), None)
    ref = attend64(q, starts, new, ctx, sigma, window, softcap, sk)
    check(out, lse, ref, bounds(ref, D, max(new), False, softcap))
    outside = torch.ones(T, dtype=torch.bool, device="cuda")
    outside[starts[0]:starts[-1]] = False
    assert bool((out[outside] == 7).all()) and bool((lse[outside] == 7).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("new,Hq,Hkv", [
    ([1], 1, 1), ([17], 8, 2), ([128], 4, 4), ([129, 1, 127], 4, 2), ([5, 0, 300, 33, 0], 10, 2), ([515], 3, 3),
    ([256, 257], 12, 1), ([1, 2, 3, 4, 5, 6, 7] * 6, 16, 1),
])
def test_packed(K, D, new, Hq, Hkv):
    packed_case(K, 1, new, Hq, Hkv, D, tail=2, head=1 if len(new) > 1 else 0)


@pytest.mark.parametrize("D,Hq,Hkv,new", [(64, 16, 8, [1500, 1400, 700]), (128, 32, 8, [700, 1, 1300]), (128, 40, 8, [999]),
                                          (256, 12, 4, [1030]), (64, 8, 8, [2100, 260, 2049])])
def test_packed_many_tiles(K, D, Hq, Hkv, new):
    packed_case(K, 2, new, Hq, Hkv, D)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 15, 127, 128, 300])
def test_packed_window_cap_sink(K, D, window):
    packed_case(K, 3, [300, 45, 513], 6, 2, D, window=window, softcap=20.0, sink=True)


def paged_case(K, kind, seed, lens, new, Hq, Hkv, D, bs=16, per_channel=True, window=-1, softcap=0.0, sink=False,
               splits=0, ws=True, amplitude=1.0):
    g = gen(seed)
    table, pool = tables(g, lens, bs)
    c = cache_of(kind, g, pool, bs, Hkv, D, per_channel)
    starts = firsts(new)
    T = starts[-1] + 1
    q = (torch.randn((T, Hq + 1, D), generator=g, device="cuda") * amplitude).half()[:, :Hq]
    sk = torch.randn(Hq, generator=g, device="cuda") if sink else None
    out = torch.full((T, Hq, D), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    nbytes = K.paged_prefill_workspace_bytes(T, len(lens), Hq, Hkv, D, table.shape[1] * bs, splits)
    space = torch.full((max(nbytes // 4, 4),), math.nan, device="cuda") if ws else None
    K.paged_prefill(q, c["kc"], c["vc"], c["ks"], c["vs"], c["scale_kind"], table, ints(lens), ints(starts), D ** -0.5, sk,
                    num_splits=splits, workspace=space, out=out, lse=lse, flags=flags, softcap=softcap, window=window)
    torch.cuda.synchronize()
    assert int(flags) == 0
    k, v = values(c)
    ref = attend64(q, starts, lens, context_of(c, table, k, v), D ** -0.5, window, softcap, sk)
    check(out, lse, ref, bounds(ref, D, max(lens), per_channel and kind != "fp16", softcap), kind)
    assert bool((out[-1] == 7).all()) and bool((lse[-1] == 7).all())  # behind the last sequence


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,new,Hq,Hkv,bs", [
    ([1], [1], 2, 1, 16), ([300, 16, 129, 1], [1, 1, 1, 1], 8, 2, 16), ([700, 33, 0, 260], [4, 2, 0, 7], 10, 2, 48),
    ([513, 128], [140, 128], 4, 4, 64), ([1100], [300], 16, 1, 16),
])
def test_paged(K, kind, D, lens, new, Hq, Hkv, bs):
    for per_channel in (False, True):
        paged_case(K, kind, 4, lens, new, Hq, Hkv, D, bs, per_channel)
    paged_case(K, kind, 5, lens, new, Hq, Hkv, D, bs, splits=1, ws=False)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [2, 3, 7, 32, 400])
def test_paged_splits(K, kind, splits):
    paged_case(K, kind, 6, [1500, 7, 0, 640], [3, 7, 0, 40], 8, 2, 128, splits=splits, sink=True, window=700)
    paged_case(K, kind, 7, [2000, 90], [2, 60], 4, 1, 64, splits=splits, softcap=25.0)
    paged_case(K, kind, 8, [900, 333, 1], [9, 1, 1], 12, 2, 256, splits=splits)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,lens,new,Hq,Hkv", [(128, [2500, 1300], [1200, 1300], 32, 8), (64, [4000, 260], [2100, 255], 16, 8),
                                               (256, [1500], [1000], 24, 4)])
def test_paged_long_chunks(K, kind, D, lens, new, Hq, Hkv):
    paged_case(K, kind, 9, lens, new, Hq, Hkv, D)
