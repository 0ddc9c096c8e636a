"""rope_and_cache and gather_cache on the GPU.  What the append stores follows from
fp32 operations rounded one by one, so queries, codes and block scales are compared
bit for bit with the oracle; the read-back is the stored value times its scale,
rounded once."""
import numpy as np
import pytest
import torch

import oracle
from helpers import dev

pytestmark = pytest.mark.gpu

KINDS = ["int8", "e4m3", "fp16", "mx4"]


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import int8_kv_cache_gb300 as K
    K.load()
    return K


def angles(rng, max_pos, R):
    if R == 0:
        return None
    a = rng.uniform(-4, 4, (max_pos, R // 2))
    return np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)


def make(seed, kind, T, Hq, Hkv, D, R, per_channel, nb=9, bs=16, max_pos=61):
    """Rows, positions, slots (with padding and slots past the pool) and a cache
    holding random bytes."""
    rng = np.random.default_rng(seed)
    r = lambda H: (rng.standard_normal((T, H, D)) * np.exp(rng.uniform(-1, 1, (1, H, D)))).astype(np.float16)
    c = dict(q=r(max(Hq, 1))[:, :Hq], k=r(Hkv), v=r(Hkv), cs=angles(rng, max_pos, R), kind=kind,
             pos=rng.integers(0, max_pos, T).astype(np.int32), sk=2 if per_channel else 1)
    c["k"][0, 0, :8] = np.array([0.25, 0.75, -0.25, 1.25, 3000, -3000, 0, -0.0], np.float16)
    c["v"][T // 2, Hkv - 1, D - 8:] = np.array([1e-7, 0, 65504, -65504, 2.5, 3.5, 5, 0.1], np.float16)
    slots = rng.permutation(nb * bs)[:T].astype(np.int32)
    if T > 8:
        slots[3], slots[5], slots[6] = -1, -7, nb * bs + 4
        c["v"][1, 0, :4] = [np.nan, np.inf, -np.inf, 1]
    c["slots"] = slots
    top = {"int8": 1 / 40, "e4m3": 1 / 100, "mx4": 1.0, "fp16": 1.0}[kind]
    shape = (Hkv, D) if per_channel else (1,)
    c["ks"], c["vs"] = (np.exp(rng.uniform(-1, 1, shape)).astype(np.float32) * np.float32(top) for _ in range(2))
    if kind == "mx4":
        c["kc"], c["vc"] = rng.integers(0, 256, (nb, Hkv, bs // 16, 18 * D)).astype(np.uint8), None
    elif kind == "fp16":
        c["kc"], c["vc"] = (rng.standard_normal((nb, bs, Hkv, D)).astype(np.float16) for _ in range(2))
    else:
        dt = np.int8 if kind == "int8" else np.uint8
        c["kc"], c["vc"] = (rng.integers(0, 100, (nb, bs, Hkv, D)).astype(dt) for _ in range(2))
    return c


def stored(c, kr):
    """The caches after the append of the turned keys kr (fp32) and the values."""
    kind, v = c["kind"], c["v"].astype(np.float32)
    if kind == "mx4":
        return oracle.mx4_append(c["kc"], kr, v, c["slots"], c["ks"], c["vs"], c["sk"]), None
    out = []
    for cache, x, s in ((c["kc"], kr, c["ks"]), (c["vc"], v, c["vs"])):
        flat = cache.copy().reshape(-1, *cache.shape[-2:])
        for n, slot in enumerate(c["slots"]):
            if 0 <= slot < flat.shape[0]:
                for g in range(flat.shape[1]):
                    with np.errstate(over="ignore"):
                        flat[slot, g] = (x[n, g].astype(np.float16) if kind == "fp16" else
                                         (oracle.quantize_rows if kind == "int8" else oracle.quantize_rows_fp8)(
                                             x[n, g], s, c["sk"], g))
        out.append(flat.reshape(cache.shape))
    return out


def on_device(c, fused=False):
    d = {n: dev(c[n]) for n in ("pos", "slots", "ks", "vs", "kc", "vc", "cs")}
    if fused:
        T, D = c["q"].shape[0], c["q"].shape[2]
        qkv = torch.cat([dev(c[n]).flatten(1) for n in ("q", "k", "v")], dim=1)
        d["q"], d["k"], d["v"] = (x.unflatten(1, (-1, D)) for x in
                                  qkv.split([c[n].shape[1] * D for n in ("q", "k", "v")], dim=1))
    else:
        d["q"], d["k"], d["v"] = (dev(c[n]) for n in ("q", "k", "v"))
    return d


def append(K, c, d, **kw):
    scales = (None, None) if c["kind"] == "fp16" else (d["ks"], d["vs"])
    return K.rope_and_cache(d["q"], d["k"], d["v"], d["pos"], d["cs"], d["slots"], d["kc"], d["vc"], *scales, c["sk"],
                            **kw)


def check(K, c, interleaved, fused=False):
    d = on_device(c, fused)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = append(K, c, d, interleaved=interleaved, flags=flags)
    torch.cuda.synchronize()
    with np.errstate(all="ignore"):
        want_q = oracle.rotate(c["q"], c["cs"], c["pos"], interleaved).astype(np.float16)
        kr = oracle.rotate(c["k"], c["cs"], c["pos"], interleaved)
    np.testing.assert_array_equal(got.cpu().numpy().view(np.uint16), want_q.view(np.uint16))
    want_k, want_v = stored(c, kr)
    as_bits = lambda x: x.view(np.uint16) if x.dtype == np.float16 else x
    gk = d["kc"].cpu().numpy()
    if c["kind"] == "fp16":  # a NaN has many bit patterns
        nan = np.isnan(want_k)
        assert (np.isnan(gk) == nan).all()
        np.testing.assert_array_equal(as_bits(gk)[~nan], as_bits(want_k)[~nan])
        gv = d["vc"].cpu().numpy()
        nan = np.isnan(want_v)
        assert (np.isnan(gv) == nan).all()
        np.testing.assert_array_equal(as_bits(gv)[~nan], as_bits(want_v)[~nan])
    else:
        np.testing.assert_array_equal(gk, want_k)
        if want_v is not None:
            np.testing.assert_array_equal(d["vc"].cpu().numpy(), want_v)
    assert int(flags.item()) == (0x8 if (c["slots"] >= c["kc"].shape[0] * 16 * (
        c["kc"].shape[2] if c["kind"] == "mx4" else c["kc"].shape[1] // 16)).any() else 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("per_channel", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,R", [(4, 2, 64, 64), (8, 1, 128, 128), (6, 2, 256, 64), (3, 3, 128, 0)])
def test_bits(K, kind, interleaved, per_channel, Hq, Hkv, D, R):
    check(K, make(D + R + Hq, kind, 37, Hq, Hkv, D, R, per_channel), interleaved)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 2, 33])
def test_rows_of_one_projection(K, kind, T):
    # q, k and v are slices of one tensor: token strides larger than a row
    check(K, make(T, kind, T, 5, 1, 128, 96 if kind != "mx4" else 64, True), False, fused=True)


@pytest.mark.parametrize("kind,D,R,bs", [("int8", 80, 48, 16), ("e4m3", 96, 16, 32), ("fp16", 112, 112, 16),
                                         ("mx4", 64, 32, 48), ("mx4", 128, 96, 32), ("mx4", 256, 256, 64)])
def test_other_sizes(K, kind, D, R, bs):
    for il in (False, True):
        check(K, make(D, kind, 40, 2, 3, D, R, True, nb=5, bs=bs), il)


@pytest.mark.parametrize("D,R", [(64, 16), (64, 48), (128, 80), (256, 144)])
def test_blocks_of_a_range_that_is_no_multiple_of_32(K, D, R):
    check(K, make(D + R, "mx4", 40, 3, 2, D, R, True), True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
def test_many_tokens_store_what_few_at_a_time_store(K, kind, interleaved):
    # enough tokens for four query heads per thread and several tokens per thread, 6 heads (a
    # group and a half), in place; against calls of 90 tokens, one head per thread
    T = 8001
    c = make(21, kind, T, 6, 2, 64, 32, True, nb=510, max_pos=900)
    d, e = on_device(c), on_device(c)
    d["pos"][77], e["pos"][77] = 900, 900
    got = append(K, c, d, interleaved=interleaved, q_out=d["q"])
    for i in range(0, T, 90):
        f = {n: (x[i:i + 90] if n in ("q", "k", "v", "pos", "slots") else x) for n, x in e.items()}
        append(K, c, f, interleaved=interleaved, q_out=f["q"])
    for a, b in ((got, e["q"]), (d["kc"], e["kc"]), (d["vc"], e["vc"])):
        if a is not None:
            bits = lambda x: x.view(torch.int16) if x.dtype == torch.float16 else x
            assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("kind", KINDS)
def test_a_larger_batch(K, kind):
    # several tokens per thread: 1500 tokens against the oracle on every head
    c = make(9, kind, 1500, 2, 1, 64, 32, True, nb=100)
    check(K, c, False)


def test_no_rotation_stores_what_reshape_and_cache_stores(K):
    for kind in ("int8", "e4m3"):
        c = make(3, kind, 64, 4, 2, 128, 0, True)
        d, e = on_device(c), on_device(c)
        append(K, c, d)
        K.reshape_and_cache(e["k"], e["v"], e["slots"], e["kc"], e["vc"], e["ks"], e["vs"], c["sk"])
        assert torch.equal(d["kc"], e["kc"]) and torch.equal(d["vc"], e["vc"])


def test_queries_in_place_and_without_queries(K):
    c = make(4, "int8", 20, 4, 2, 64, 64, False)
    d, e = on_device(c), on_device(c)
    want = append(K, c, d)
    got = append(K, c, e, q_out=e["q"])
    assert got is e["q"] and torch.equal(got, want)
    f = on_device(c)
    f["q"] = None
    assert append(K, c, f) is None
    assert torch.equal(f["kc"], d["kc"]) and torch.equal(f["vc"], d["vc"])


def test_bad_positions_leave_their_token_out(K):
    c = make(5, "mx4", 12, 2, 1, 64, 64, True)
    c["slots"] = np.arange(12, dtype=np.int32)
    d = on_device(c)
    d["pos"][2], d["pos"][7] = 61, -1
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full_like(d["q"], 7.0)
    append(K, c, d, q_out=q_out, flags=flags)
    assert int(flags.item()) == K.FLAG_BAD_POSITION
    c["slots"][[2, 7]] = -1
    e = on_device(c)
    want = append(K, c, e)
    keep = [i for i in range(12) if i not in (2, 7)]
    assert torch.equal(q_out[keep], want[keep]) and (q_out[[2, 7]] == 7.0).all()
    assert torch.equal(d["kc"], e["kc"])
    # padding tokens may have any position: no flag
    flags.zero_()
    e["pos"][2] = -5
    append(K, c, e, flags=flags)
    assert int(flags.item()) == 0


def test_no_tokens(K):
    c = make(6, "mx4", 4, 2, 1, 64, 64, True)
    d = on_device(c)
    before = d["kc"].clone()
    d.update({n: d[n][:0] for n in ("q", "k", "v", "pos", "slots")})
    assert append(K, c, d).shape == (0, 2, 64)
    k, v = K.gather_cache(d["slots"], d["kc"], None, d["ks"], d["vs"], c["sk"])
    assert k.shape == v.shape == (0, 1, 64) and torch.equal(before, d["kc"])


def test_refusals_of_the_binding(K):
    c = make(7, "int8", 8, 4, 2, 64, 64, True)
    d = on_device(c)
    args = lambda **kw: [kw.get(n, d[n]) for n in ("q", "k", "v", "pos", "cs", "slots", "kc", "vc", "ks", "vs")]
    bad = [dict(k=d["k"][:, :1].contiguous()), dict(k=d["k"][:7].contiguous(), v=d["v"]), dict(pos=d["pos"][:5]),
           dict(slots=d["slots"][:5]), dict(ks=d["ks"][:1].contiguous()), dict(cs=d["cs"].t()),
           dict(vc=d["vc"][:4].contiguous()), dict(ks=None), dict(q=d["q"].transpose(0, 1)),
           dict(kc=d["kc"][..., :32]), dict(v=d["v"].transpose(1, 2).contiguous().transpose(1, 2))]
    for kw in bad:
        with pytest.raises((ValueError, AttributeError)):
            K.rope_and_cache(*args(**kw), 2)
    for kw in (dict(q=d["q"].float()), dict(pos=d["pos"].long()), dict(slots=d["slots"].long()),
               dict(cs=d["cs"].half()), dict(vc=d["vc"].view(torch.uint8))):
        with pytest.raises(TypeError):
            K.rope_and_cache(*args(**kw), 2)
    with pytest.raises(K.Int8KVError) as e:  # positions are needed to turn
        K.rope_and_cache(*args(pos=None), 2)
    assert e.value.status == 1
    with pytest.raises(ValueError):
        K.rope_and_cache(*args(q=None), 2, q_out=d["q"])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("per_channel", [False, True])
@pytest.mark.parametrize("D,Hkv,bs", [(64, 3, 16), (128, 2, 32), (256, 1, 48)])
def test_gather(K, kind, per_channel, D, Hkv, bs):
    rng = np.random.default_rng(D)
    c = make(D, kind, 8, 0, Hkv, D, 0, per_channel, nb=5, bs=bs)
    if kind == "mx4":  # scale bytes 0 .. 0x7E: everything but NaN
        for lo in (8 * D, 17 * D):
            c["kc"][..., lo:lo + D] = rng.integers(0, 0x7F, c["kc"][..., lo:lo + D].shape)
    slots = rng.integers(-2, 5 * bs + 2, 101).astype(np.int32)
    slots[0], slots[1] = 5 * bs - 1, 5 * bs
    d = on_device(c)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    scales = (None, None) if kind == "fp16" else (d["ks"], d["vs"])
    gk, gv = (x.cpu().numpy() for x in K.gather_cache(dev(slots), d["kc"], d["vc"], *scales, c["sk"], flags=flags))
    assert int(flags.item()) == 0x8
    for n, s in enumerate(slots):
        for g in range(Hkv):
            if not 0 <= s < 5 * bs:
                assert not gk[n, g].any() and not gv[n, g].any()
                continue
            if kind == "mx4":
                rows = oracle.mx4_row(c["kc"], s, g)
            else:
                rows = [x.reshape(-1, Hkv, D)[s, g].astype(np.float64) for x in (c["kc"], c["vc"])]
                if kind == "e4m3":
                    rows = [np.array([oracle.e4m3fn_value(int(b)) for b in r]) for r in rows]
            for got, r, sc in zip((gk, gv), rows, (c["ks"], c["vs"])):
                if kind != "fp16":
                    sc = np.broadcast_to(sc[0], (D,)) if c["sk"] == 1 else sc[g]
                    r = r.astype(np.float32) * sc.astype(np.float32)
                with np.errstate(over="ignore"):
                    np.testing.assert_array_equal(got[n, g], r.astype(np.float16))


@pytest.mark.parametrize("kind", ["mx4", "fp16"])
def test_append_then_gather_in_a_graph_on_another_stream(K, kind):
    # captured once, replayed on new rows: what it reads back is what an eager append stores
    c = make(11, kind, 33, 4, 2, 128, 64, True)
    c["slots"] = np.abs(c["slots"]) % 140
    c["slots"] = np.unique(c["slots"])[:30].astype(np.int32)
    for n in ("q", "k", "v", "pos"):
        c[n] = c[n][:len(c["slots"])]
    d = on_device(c)
    scales = (None, None) if kind == "fp16" else (d["ks"], d["vs"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        append(K, c, d)  # loads the kernels
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            q = append(K, c, d)
            k, v = K.gather_cache(d["slots"], d["kc"], d["vc"], *scales, c["sk"])
    for seed in (1, 2):
        torch.manual_seed(seed)
        for n in ("q", "k", "v"):
            d[n].copy_(torch.randn_like(d[n]))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        e = dict(d, kc=d["kc"].clone(), vc=None if d["vc"] is None else d["vc"].clone())
        q2 = append(K, c, e)
        k2, v2 = K.gather_cache(e["slots"], e["kc"], e["vc"], *scales, c["sk"])
        assert torch.equal(q, q2) and torch.equal(k, k2) and torch.equal(v, v2)
        # half a rounding step of the largest value away from the rows themselves
        if kind == "mx4":
            err = (v.float() - d["v"].float()).abs()
            assert (err <= d["v"].float().abs().amax() / 4).all()


def test_scales_of_another_shape_are_refused(K):
    # [D, Hkv] has as many values as [Hkv, D]
    for kind in ("int8", "mx4"):
        c = make(13, kind, 8, 4, 2, 64, 64, True)
        d = on_device(c)
        slots = torch.arange(4, dtype=torch.int32, device="cuda")
        turned = d["ks"].t().contiguous()
        before = d["kc"].clone()
        for kw in (dict(ks=turned), dict(vs=turned)):
            with pytest.raises(ValueError, match="_scale"):
                append(K, c, dict(d, **kw))
            e = dict(d, **kw)
            with pytest.raises(ValueError, match="_scale"):
                K.gather_cache(slots, d["kc"], d["vc"], e["ks"], e["vs"], 2)
            if kind == "mx4":
                lens = torch.ones(1, dtype=torch.int32, device="cuda")
                with pytest.raises(ValueError, match="_scale"):
                    K.paged_decode_mx4(d["q"][:1].contiguous(), d["kc"], e["ks"], e["vs"], 2, lens[:, None] * 0, lens, 0.1)
        assert torch.equal(before, d["kc"])
        # the same numbers in a row, or with dimensions of one, are taken
        want = K.gather_cache(slots, d["kc"], d["vc"], d["ks"], d["vs"], 2)
        for view in (lambda s: s.view(-1), lambda s: s.view(1, 2, 1, 64), lambda s: s.view(2, 64, 1)):
            got = K.gather_cache(slots, d["kc"], d["vc"], view(d["ks"]), view(d["vs"]), 2)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        one = make(14, kind, 8, 4, 1, 64, 64, True)  # one head: [D, 1] is [1, D]
        d = on_device(one)
        d["ks"] = d["ks"].t()
        append(K, one, dict(d, ks=d["ks"].contiguous()))


def test_other_threads_run_while_a_call_waits_for_the_queue(K):
    # calls behind a kernel that takes a while fill the queue of launches, and one waits for room in it
    import threading
    import time
    c = make(15, "int8", 4, 2, 1, 64, 64, True)
    d = on_device(c)
    append(K, c, d, q_out=d["q"])
    torch.cuda.synchronize()
    gaps, stop = [0.0], threading.Event()

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps[0] = max(gaps[0], now - last)
            last = now
    th = threading.Thread(target=tick)
    th.start()
    try:
        time.sleep(0.05)
        t0 = time.perf_counter()
        torch.cuda._sleep(800_000_000)  # cycles: 0.4 s or more
        for _ in range(3000):
            append(K, c, d, q_out=d["q"])
        waited = time.perf_counter() - t0
        torch.cuda.synchronize()
    finally:
        stop.set()
        th.join()
    if waited < 0.3:
        pytest.skip("the queue took every launch")
    # (one call waits for nearly all of it, once the queue is full)
    assert gaps[0] < waited / 2


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("per_channel", [False, True])
def test_scales_whose_reciprocal_overflows(K, kind, per_channel):
    # scales below 2^-128: 1 / scale is infinite in fp32 and x / scale need not be.  Keys turned by
    # cosines as small (nothing else brings an fp16 number down there); the codes are the quotients'
    rng = np.random.default_rng(12)
    T, Hkv, D, R = 24, 2, 64, 64
    c = make(12, kind, T, 1, Hkv, D, R, per_channel)
    c["k"] = rng.integers(-3, 4, (T, Hkv, D)).astype(np.float16)
    c["cs"] = (rng.integers(0, 100, c["cs"].shape) * 2.0 ** -140).astype(np.float32)
    c["ks"] = (rng.integers(1, 5, c["ks"].shape) * 2.0 ** -139).astype(np.float32)
    c["v"][1, 0, :4] = 1
    with np.errstate(all="ignore"):
        kr = oracle.rotate(c["k"], c["cs"], c["pos"], False)
        assert np.isinf(np.float32(1) / c["ks"]).all() and (np.abs(kr / c["ks"].max()) < 100).mean() > 0.5
    check(K, c, False)
