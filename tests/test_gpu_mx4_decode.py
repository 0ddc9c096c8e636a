"""paged_decode_mx4 on the GPU against attention over the cache's values in 64 bits.

Tolerances.  The cache's values are exact in the kernel's products.  What is rounded:
  - Q * k_scale to two fp16 numbers, where the scales are per channel (the first is half a step,
    2^-11, off, the second 2^-11 of that; 2^-20 with room for what the second loses below its
    smallest step): every score moves by at most e = 2^-20 E, E = max_t sigma sum_d |q_d K_t,d|;
    so the probabilities change by a factor within e^(+-2 e), and the lse by e;
  - the probabilities to fp16 (2^-11 each), with those below 2^-24 of the largest rounded
    to a multiple of 2^-32 at worst;
  - the sums in fp32: D products each of |.| summing to E, taken as D 2^-23 E on a score;
    the tanh of a softcap c to a few 2^-23 c;
  - the output to fp16 (2^-11).
With W = sum_t p_t |v_t|:  |dO| <= W (2^-11 + 2 (e + f)) (1 + 2^-6) + 2^-11 |O| + 2^-24,
f = (D + 16) 2^-23 (E + c) + 1e-6, and |dlse| <= e + f + 1e-6 |lse|."""
import numpy as np
import pytest
import torch

import oracle
from helpers import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import int8_kv_cache_gb300 as K
    K.load()
    return K


def case(seed, B, Hq, Hkv, D, bs, max_blocks, lens, per_channel=True, sink=False, sigma=None):
    rng = np.random.default_rng(seed)
    nb = B * max_blocks + 3
    cache = rng.integers(0, 256, (nb, Hkv, bs // 16, 18 * D)).astype(np.uint8)
    for lo in (8 * D, 17 * D):  # block scales of values around 1
        cache[..., lo:lo + D] = rng.integers(0x20, 0x36, cache[..., lo:lo + D].shape)
    table = rng.permutation(nb)[:B * max_blocks].reshape(B, max_blocks).astype(np.int32)
    shape = (Hkv, D) if per_channel else (1,)
    ks, vs = (np.exp(rng.uniform(-1, 1, shape)).astype(np.float32) for _ in range(2))
    return dict(q=rng.standard_normal((B, Hq, D)).astype(np.float16), cache=cache, ks=ks, vs=vs,
                sk=2 if per_channel else 1, table=table, lens=np.asarray(lens, np.int32),
                sigma=D ** -0.5 if sigma is None else sigma,
                sink=rng.standard_normal(Hq).astype(np.float32) if sink else None)


def on_device(c):
    return {n: dev(c[n]) for n in ("q", "cache", "ks", "vs", "table", "lens", "sink")}


def workspace(K, B, Hq, D, splits=32):
    return torch.full((splits * B * Hq * (D + 2),), float("nan"), device="cuda")


def run(K, c, d=None, ns=0, chunk=0, softcap=0.0, window=-1, flags=None, ws=None):
    d = d or on_device(c)
    B, Hq, D = c["q"].shape
    out = torch.full((B, Hq, D), float("nan"), dtype=torch.float16, device="cuda")
    lse = torch.full((B, Hq), float("nan"), device="cuda")
    K.paged_decode_mx4(d["q"], d["cache"], d["ks"], d["vs"], c["sk"], d["table"], d["lens"], c["sigma"], d["sink"],
                       num_splits=ns, chunk=chunk, workspace=workspace(K, B, Hq, D) if ws is None else ws, out=out,
                       lse=lse, flags=flags, softcap=softcap, window=window)
    torch.cuda.synchronize()
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def reference(c, softcap=0.0, window=-1):
    return oracle.mx4_paged_attention(c["q"], c["cache"], c["ks"], c["vs"], c["sk"], c["table"], c["lens"], c["sigma"],
                                      c["sink"], softcap, window)


def compare(c, got, ref, softcap=0.0, what=""):
    (o, l), (O, L, W, E) = got, ref
    D = c["q"].shape[2]
    e = 2.0 ** -20 * E if c["sk"] == 2 else 0.0 * E
    f = (D + 16) * 2.0 ** -23 * (E + softcap) + 1e-6
    tol = W * ((2.0 ** -11 + 2 * (e + f)) * (1 + 2.0 ** -6))[..., None] + 2.0 ** -11 * np.abs(O) + 2.0 ** -24
    assert np.isfinite(o).all(), what
    bad = np.abs(o - O) - tol
    assert (bad <= 0).all(), f"{what}: worst {bad.max()} over a tolerance at {np.unravel_index(bad.argmax(), bad.shape)}"
    assert (np.isneginf(l) == np.isneginf(L)).all(), what
    fin = np.isfinite(L)
    off = np.abs(l[fin] - L[fin]) - (e + f + 1e-6 * np.abs(np.where(fin, L, 0)))[fin]
    assert (off <= 0).all(), f"{what}: lse off by {off.max()} over its tolerance"


SHAPES = [(4, 1, 64), (8, 8, 64), (16, 1, 64), (8, 1, 128), (24, 2, 128), (10, 2, 128), (4, 2, 256), (24, 2, 256),
          (16, 1, 256), (3, 3, 256)]


@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("per_channel", [False, True])
def test_heads(K, Hq, Hkv, D, per_channel):
    # lengths of zero and one, ends inside a tile, on a tile, inside a block, and the whole capacity
    lens = [0, 1, 15, 16, 17, 100, 211, 288]
    c = case(Hq + D, 8, Hq, Hkv, D, 32, 9, lens, per_channel, sink=True)
    ref = reference(c)
    for ns, chunk in ((0, 0), (1, 288), (2, 144), (7, 48), (18, 16), (2, 0), (5, 0), (32, 0)):
        compare(c, run(K, c, ns=ns, chunk=chunk), ref, what=f"{ns} splits of {chunk}")


@pytest.mark.parametrize("bs", [16, 48, 64, 128])
def test_block_sizes(K, bs):
    c = case(bs, 3, 8, 2, 128, bs, 512 // bs, [511 // bs * bs, 1, 333])
    ref = reference(c)
    for ns, chunk in ((0, 0), (1, 512), (4, 128), (9, 0)):
        compare(c, run(K, c, ns=ns, chunk=chunk), ref, what=f"{ns} splits of {chunk}")


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 16, 1), (256, 6, 2)])
@pytest.mark.parametrize("softcap,window", [(0.0, 0), (0.0, 15), (0.0, 100), (5.0, -1), (2.0, 63), (0.0, 5000)])
def test_softcap_and_window(K, D, Hq, Hkv, softcap, window):
    c = case(D + window, 6, Hq, Hkv, D, 16, 20, [0, 1, 64, 101, 317, 320], sink=True)
    ref = reference(c, softcap, window)
    span = K.window_span(320, window)
    for ns, chunk in ((0, 0), (1, (span + 15) // 16 * 16), (4, 0), (32, 0)):
        compare(c, run(K, c, ns=ns, chunk=chunk, softcap=softcap, window=window), ref, softcap,
                f"{ns} splits of {chunk}")


def test_lengths_outside_the_capacity(K):
    c = case(1, 3, 8, 2, 64, 16, 5, [-4, 81, 1 << 30])
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = reference(c)
    for ns, chunk in ((1, 80), (3, 0)):
        flags.zero_()
        compare(c, run(K, c, ns=ns, chunk=chunk, flags=flags), ref)
        assert int(flags.item()) == K.FLAG_LEN_CLAMPED


def test_bad_blocks_are_not_attended(K):
    c = case(2, 3, 8, 2, 128, 16, 12, [190, 100, 20])
    c["table"][0, 3], c["table"][0, 11], c["table"][1, 0] = -1, c["cache"].shape[0], -(1 << 31)
    c["table"][2, 0] = c["table"][2, 1] = 1 << 30  # all of a sequence
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = reference(c)
    assert np.isneginf(ref[1][2]).all()
    for ns, chunk in ((1, 192), (4, 48), (6, 0)):
        flags.zero_()
        compare(c, run(K, c, ns=ns, chunk=chunk, flags=flags), ref)
        assert int(flags.item()) == K.FLAG_BAD_BLOCK
    # entries past the live length are not looked at
    c["table"][:] = 0
    c["lens"][:] = 16
    c["table"][:, 1:] = -1
    flags.zero_()
    compare(c, run(K, c, flags=flags), reference(c))
    assert int(flags.item()) == 0


def test_stale_bytes_past_the_end_do_not_count(K):
    # NaN block scales behind the last token, in the same tile, for keys and values
    c = case(3, 2, 8, 1, 64, 16, 4, [37, 5])
    ref = reference(c)
    D = 64
    for b, n in enumerate(c["lens"]):
        blk, off = int(c["table"][b, n // 16]), int(n % 16)
        for lo in (8 * D, 17 * D):
            c["cache"][blk, :, 0, lo + off * (D // 16): lo + D] = 0x7F
    for ns, chunk in ((1, 64), (2, 0), (4, 16)):
        compare(c, run(K, c, ns=ns, chunk=chunk), ref)


def test_large_common_score_and_one_dominant_token(K):
    c = case(4, 2, 8, 2, 128, 16, 16, [256, 250], per_channel=False, sigma=1.0)
    c["q"] = (c["q"].astype(np.float32) * 60).astype(np.float16)
    ref = reference(c)
    assert np.abs(ref[1]).max() > 2000  # scores far beyond exp's range
    for ns, chunk in ((1, 256), (5, 0), (16, 16)):
        compare(c, run(K, c, ns=ns, chunk=chunk), ref)


def test_scales_of_any_size(K):
    # per-channel key scales over eight decades, beyond fp16 on both sides; values near the fp16 maximum
    c = case(5, 2, 8, 2, 128, 16, 8, [128, 77], sigma=1e-4)
    rng = np.random.default_rng(0)
    c["ks"] = np.exp(rng.uniform(np.log(1e-6), np.log(1e6), c["ks"].shape)).astype(np.float32)
    c["q"] = (c["q"].astype(np.float32) / c["ks"].repeat(4, 0)[None]).clip(-6e4, 6e4).astype(np.float16)
    c["vs"] = (c["vs"] * 900).astype(np.float32)
    ref = reference(c)
    for ns, chunk in ((1, 128), (3, 0)):
        compare(c, run(K, c, ns=ns, chunk=chunk), ref)


def test_zero_queries_give_the_mean_of_the_values(K):
    c = case(6, 1, 4, 1, 64, 16, 8, [100])
    c["q"][:] = 0
    o, l = run(K, c, ns=4, chunk=0)
    rows = np.stack([oracle.mx4_row(c["cache"], c["table"][0, t // 16] * 16 + t % 16, 0)[1] for t in range(100)]) * c["vs"][0]
    tol = (2.0 ** -11 + 2.0 ** -11) * np.abs(rows).mean(0) + 1e-6
    assert (np.abs(o[0] - rows.mean(0)) <= tol).all()
    np.testing.assert_allclose(l, np.log(100), atol=1e-6)


def test_partials_join_with_split_combine(K):
    c = case(7, 4, 8, 2, 128, 16, 20, [300, 17, 0, 320], sink=True)
    d = on_device(c)
    want = run(K, c, d, ns=6, chunk=0)
    ws = workspace(K, 4, 8, 128, 6)
    r = K.paged_decode_mx4(d["q"], d["cache"], d["ks"], d["vs"], 2, d["table"], d["lens"], c["sigma"], num_splits=6,
                           workspace=ws, partials_only=True)
    assert r is None
    n = 4 * 2 * 6 * 4
    out = K.split_combine(ws[:n * 128].view(8, 6, 4, 128), ws[n * 128:n * 129].view(8, 6, 4), ws[n * 129:].view(8, 6, 4),
                          8, 2, d["sink"])
    assert np.array_equal(out.double().cpu().numpy().reshape(4, 8, 128), want[0])


def test_plan_is_what_the_automatic_call_uses(K):
    for B, cap_blocks, lens in ((2, 4, [60, 3]), (3, 64, [1000, 20, 512]), (1, 128, [2048])):
        c = case(B, B, 8, 2, 64, 16, cap_blocks, lens)
        d = on_device(c)
        ns, chunk, wsb, wave = K.decode_plan(K.PATH_PAGED, K.CACHE_MX4, cap_blocks * 16, B, 8, 2, 64, K.GEOM_BALANCED)
        assert wave >= 148 and wsb == K.split_workspace_bytes(B * 2, ns, 4, 64)
        ws = torch.empty(max(wsb // 4, 4), device="cuda")
        a, b = run(K, c, d, ws=ws), run(K, c, d, ns=ns, chunk=chunk, ws=ws)
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
        if ns > 1:
            with pytest.raises(K.Int8KVError) as e:
                run(K, c, d, ws=torch.empty(wsb // 4 - 4, device="cuda"))
            assert e.value.status == 4


@pytest.mark.parametrize("B,Hkv", [(33, 1), (150, 2), (700, 1)])
def test_large_batches(K, B, Hkv):
    rng = np.random.default_rng(B)
    c = case(B, B, 2 * Hkv, Hkv, 64, 16, 6, rng.integers(0, 97, B))
    compare(c, run(K, c), reference(c))
    compare(c, run(K, c, ns=32, chunk=0), reference(c))


@pytest.mark.parametrize("Hq,D", [(4, 64), (12, 64), (4, 128), (7, 128), (16, 128), (3, 256), (8, 256), (13, 256)])
@pytest.mark.parametrize("per_channel", [False, True])
def test_pieces_of_many_rows_and_of_few(K, Hq, D, per_channel):
    # the partial slots of 50 rows fill any GPU, those of one to three do not
    rng = np.random.default_rng(Hq)
    c = case(Hq * D, 50, Hq, 1, D, 16, 14, rng.integers(0, 225, 50), per_channel)
    c["lens"][:3] = [224, 0, 193]
    ref = reference(c, window=199)
    compare(c, run(K, c, ns=32, chunk=0, window=199), ref)
    for B in (1, 3):
        part = dict(c, q=c["q"][:B], table=c["table"][:B], lens=c["lens"][:B])
        for ns in (3, 14, 31):
            compare(part, run(K, part, ns=ns, chunk=0, window=199), [x[:B] for x in ref], what=f"{B} {ns}")


@pytest.mark.parametrize("B,D,Hq,Hkv", [(160, 64, 8, 2), (256, 64, 4, 2), (257, 64, 4, 2), (97, 128, 16, 4), (81, 128, 48, 4),
                                        (50, 256, 8, 8)])
def test_one_cta_per_row_for_more_rows_than_are_resident(K, B, D, Hq, Hkv):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 60, B)
    lens[rng.permutation(B)[:12]] = [1024, 1023, 1024, 512, 511, 0, -7, 1 << 30, 900, 1, 16, 17]
    c = case(B, B, Hq, Hkv, D, 64, 16, lens)
    ref = reference(c)
    compare(c, run(K, c, ns=1, chunk=1024), ref)
    compare(c, run(K, c), ref)
    c["lens"][:] = 33  # all alike, then all empty
    compare(c, run(K, c, ns=1, chunk=1024), reference(c))
    c["lens"][:] = 0
    compare(c, run(K, c, ns=1, chunk=1024), reference(c))


@pytest.mark.parametrize("B,D,Hq,Hkv", [(90, 64, 12, 4), (160, 64, 48, 4), (50, 128, 24, 8), (90, 128, 32, 2), (160, 128, 44, 4),
                                        (80, 256, 20, 2), (60, 256, 12, 4), (130, 256, 48, 4)])
@pytest.mark.parametrize("per_channel", [False, True])
def test_one_cta_per_row_over_a_longer_span(K, B, D, Hq, Hkv, per_channel):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 40, B)
    lens[rng.permutation(B)[:5]] = [1200, 1199, 0, 500, 1041]
    c = case(B, B, Hq, Hkv, D, 16, 75, lens, per_channel, sink=True)
    compare(c, run(K, c, ns=1, chunk=1200), reference(c))
    compare(c, run(K, c, softcap=3.0, window=30), reference(c, 3.0, 30), 3.0)


def reference_on_device(c, d, rows, window=-1):
    """Attention of some sequences in 64 bits with torch on the device."""
    bs, D, Hkv = c["cache"].shape[2] * 16, c["q"].shape[2], c["cache"].shape[1]
    lut = torch.tensor(oracle.e2m1_value(np.arange(16)), device="cuda")
    e4 = torch.tensor([oracle.e4m3fn_value(i) for i in range(128)] + [0.0] * 128, device="cuda", dtype=torch.float64)

    def values(rec, base):
        codes = rec[..., base:base + 8 * D].unflatten(-1, (16, D // 2)).int()
        s = e4[rec[..., base + 8 * D:base + 9 * D].unflatten(-1, (16, D // 16)).int()]
        v = lut[torch.stack((codes & 15, codes >> 4), -1).flatten(-2)]
        return (v.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)  # [blocks, Hkv, tiles, 16, D]
    out = []
    for b in rows:
        n = int(c["lens"][b])
        rec = d["cache"][d["table"][b, :-(-n // bs)].long()]
        k, v = (values(rec, x).permute(0, 2, 3, 1, 4).reshape(-1, Hkv, D)[:n] for x in (0, 9 * D))
        k, v = k * d["ks"].double(), v * d["vs"].double()
        s = torch.einsum("hgd,thd->hgt", d["q"][b].double().view(Hkv, -1, D), k) * c["sigma"]
        E = (torch.einsum("hgd,thd->hgt", d["q"][b].double().view(Hkv, -1, D).abs(), k.abs()) * c["sigma"]).amax(-1)
        if window >= 0:
            s[..., :max(0, n - 1 - window)] = float("-inf")
        p = torch.softmax(s, -1)
        f = lambda x: x.reshape(-1, D).cpu().numpy()
        out.append((f(torch.einsum("hgt,thd->hgd", p, v)), torch.logsumexp(s, -1).flatten().cpu().numpy(),
                    f(torch.einsum("hgt,thd->hgd", p, v.abs())), E.flatten().cpu().numpy()))
    return [np.stack(x) for x in zip(*out)]


@pytest.mark.parametrize("B,Hq,Hkv,D,lo,hi", [(16, 32, 8, 128, 512, 8192), (1, 4, 1, 128, 131072, 131072),
                                              (2, 16, 1, 256, 20000, 40000), (3, 5, 5, 64, 9000, 30000)])
def test_long_contexts(K, B, Hq, Hkv, D, lo, hi):
    rng = np.random.default_rng(D)
    lens = rng.integers(lo, hi + 1, B)
    c = case(0, B, Hq, Hkv, D, 16, 1, lens)
    mb = -(-hi // 16)
    nb = B * mb
    g = torch.Generator(device="cuda").manual_seed(1)
    d = on_device(c)
    d["cache"] = torch.randint(0, 256, (nb, Hkv, 1, 18 * D), generator=g, device="cuda", dtype=torch.uint8)
    for x in (8 * D, 17 * D):
        d["cache"][..., x:x + D] = torch.randint(0x20, 0x36, (nb, Hkv, 1, D), generator=g, device="cuda", dtype=torch.uint8)
    d["table"] = torch.randperm(nb, generator=g, device="cuda").view(B, mb).int()
    c["cache"] = np.empty((nb, Hkv, 1, 0))
    rows = sorted(set((0, B // 2, B - 1)))
    for window in (-1, 4095):
        want = reference_on_device(c, d, rows, window)
        for ns, chunk in ((0, 0), (32, -(-hi // 32 // 16) * 16 + 16)):
            o, l = run(K, c, d, ns=ns, chunk=chunk, window=window)
            compare(dict(c, q=c["q"][rows]), (o[rows], l[rows]), want, what=f"{window} {ns}")


def test_cache_beyond_32_bit_offsets(K):
    # 5 GB of records: the last blocks lie past 2^32 bytes
    D, Hkv = 256, 8
    nb = (5 << 30) // (Hkv * 18 * D)
    c = case(8, 2, 16, Hkv, D, 16, 4, [64, 50], sink=False)
    d = on_device(c)
    small = d["cache"]
    d["cache"] = torch.zeros((nb, Hkv, 1, 18 * D), dtype=torch.uint8, device="cuda")
    at = torch.tensor([nb - 1 - i for i in range(small.shape[0])], device="cuda")
    d["cache"][at] = small
    d["table"] = (nb - 1 - d["table"]).int()
    ref = reference(c)
    for ns, chunk in ((1, 64), (2, 0)):
        compare(c, run(K, c, d, ns=ns, chunk=chunk), ref)
    slots = d["table"][0, :1] * 16 + torch.arange(16, device="cuda", dtype=torch.int32)
    k, v = K.gather_cache(slots, d["cache"], None, d["ks"], d["vs"], 2)
    want = oracle.mx4_row(c["cache"], int(c["table"][0, 0]) * 16 + 7, 5)
    np.testing.assert_array_equal(k[7, 5].cpu().numpy(), (want[0].astype(np.float32) * c["ks"][5]).astype(np.float16))


def test_two_graphs_and_an_eager_call_with_one_workspace(K):
    # replayed in turn on one stream with new lengths and queries
    cs = [case(20 + i, 4, 8, 2, 128, 16, 40, [600, 5, 0, 333]) for i in range(2)]
    ds = [on_device(c) for c in cs]
    ws = workspace(K, 4, 8, 128)
    outs, graphs = [], []
    s = torch.cuda.Stream()
    for c, d in zip(cs, ds):
        with torch.cuda.stream(s):
            out = torch.empty_like(d["q"])
            call = lambda: K.paged_decode_mx4(d["q"], d["cache"], d["ks"], d["vs"], 2, d["table"], d["lens"], c["sigma"],
                                              workspace=ws, out=out)
            call()
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                call()
        outs.append(out)
        graphs.append(g)
    for lens in ([640, 1, 17, 2], [3, 640, 100, 0]):
        for c, d in zip(cs, ds):
            c["lens"] = np.asarray(lens, np.int32)
            d["lens"].copy_(dev(c["lens"]))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, d, out in zip(cs, ds, outs):
            want = run(K, c, d, ws=ws)
            assert np.array_equal(out.double().cpu().numpy(), want[0])
            compare(c, want, reference(c))


def test_same_bits_every_time(K):
    c = case(30, 8, 16, 2, 128, 16, 64, [1000, 30, 700, 1024, 512, 0, 8, 900], sink=True)
    d = on_device(c)
    first = run(K, c, d)
    for _ in range(5):
        again = run(K, c, d)
        assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])


def test_a_serving_loop_appends_and_attends(K):
    """The operators together: a prompt is appended, then token after token is rotated,
    appended and attended, against the same in 64 bits over the rows read back."""
    torch.manual_seed(0)
    B, Hq, Hkv, D, R, bs, mb = 3, 8, 2, 128, 64, 16, 6
    ang = torch.rand(96, R // 2, device="cuda", dtype=torch.float64) * 6
    cs = torch.cat((ang.cos(), ang.sin()), 1).float()
    cache = torch.zeros(K.mx4_cache_shape(B * mb, bs, Hkv, D), dtype=torch.uint8, device="cuda")
    table = torch.randperm(B * mb, device="cuda").view(B, mb).int()
    one = torch.ones(1, device="cuda")
    lens = torch.tensor([40, 1, 17], dtype=torch.int32, device="cuda")
    sigma = D ** -0.5

    def slots_of(b, pos):
        return (table[b, pos // bs] * bs + pos % bs).int()
    for b, n in enumerate(lens.tolist()):
        pos = torch.arange(n, device="cuda")
        kv = torch.randn(n, 2 * Hkv, D, device="cuda").half()
        K.rope_and_cache(None, kv[:, :Hkv], kv[:, Hkv:], pos.int(), cs, slots_of(b, pos), cache, None, one, one, 1)
    ws = workspace(K, B, Hq, D)
    for step in range(20):
        qkv = torch.randn(B, Hq + 2 * Hkv, D, device="cuda").half()
        slots = slots_of(torch.arange(B, device="cuda"), lens.long())
        q = K.rope_and_cache(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], lens, cs, slots, cache, None, one, one, 1)
        lens = lens + 1
        out = K.paged_decode_mx4(q, cache, one, one, 1, table, lens, sigma, workspace=ws)
        if step % 6:
            continue
        for b, n in enumerate(lens.tolist()):
            pos = torch.arange(n, device="cuda")
            k, v = K.gather_cache(slots_of(b, pos), cache, None, one, one, 1)
            k, v = k.double(), v.double()  # exact: 6 significant bits at a scale of 1
            s = torch.einsum("hgd,thd->hgt", q[b].double().view(Hkv, -1, D), k) * sigma
            p = torch.softmax(s, -1)
            want = torch.einsum("hgt,thd->hgd", p, v).reshape(Hq, D)
            W = torch.einsum("hgt,thd->hgd", p, v.abs()).reshape(Hq, D)
            tol = 2.0 ** -10 * W + 2.0 ** -11 * want.abs() + 1e-5
            assert ((out[b].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("per_channel", [False, True])
def test_a_head_that_is_not_finite_spoils_itself_only(K, per_channel):
    c = case(40, 2, 8, 1, 128, 16, 40, [600, 33], per_channel)
    ref = reference(c)
    c["q"][0, 2, 5], c["q"][0, 6, 7] = np.nan, np.inf
    good = np.ones((2, 8), bool)
    good[0, [2, 6]] = False
    for ns, chunk in ((0, 0), (1, 640), (5, 0), (10, 64)):
        o, l = run(K, c, ns=ns, chunk=chunk)
        assert np.isnan(o[0, [2, 6]]).all()
        pick = lambda x: x[good][None]
        compare(dict(c, q=c["q"][good][None]), (pick(o), pick(l)), [pick(x) for x in ref], what=f"{ns} splits of {chunk}")


def test_very_negative_scores_and_late_maxima(K):
    # all scores far below zero; then rows whose scores climb towards the end, in steps beyond the room
    c = case(41, 2, 4, 1, 64, 16, 40, [640, 500], per_channel=False, sigma=1.0)
    c["q"] = (np.abs(c["q"].astype(np.float32)) * 20).astype(np.float16)
    D = 64
    for b in range(2):
        for t in range(640):
            blk, r = c["table"][b, t // 16], t % 16
            row = c["cache"][blk, 0, 0]
            row[r * D // 2:(r + 1) * D // 2] = 0xAA  # code -1.0 in every channel
            row[8 * D + r * D // 16:8 * D + (r + 1) * D // 16] = 0x38 - (t // 100 if b else 0)
    ref = reference(c)
    assert ref[1].max() < -100
    for ns, chunk in ((0, 0), (1, 640), (3, 0), (40 // 2, 32)):
        compare(c, run(K, c, ns=ns, chunk=chunk), ref, what=f"{ns} splits of {chunk}")


def test_an_explicit_stream(K):
    c = case(42, 4, 8, 2, 128, 16, 20, [300, 17, 0, 320])
    d = on_device(c)
    want = run(K, c, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = workspace(K, 4, 8, 128)
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        out = K.paged_decode_mx4(d["q"], d["cache"], d["ks"], d["vs"], 2, d["table"], d["lens"], c["sigma"],
                                 workspace=ws, stream=stream)
        slots = torch.arange(40, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        k, v = K.gather_cache(slots, d["cache"], None, d["ks"], d["vs"], 2, stream=stream)
        s.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), want[0])
        k2, v2 = K.gather_cache(slots, d["cache"], None, d["ks"], d["vs"], 2)
        assert torch.equal(k, k2) and torch.equal(v, v2)


def test_two_streams_at_once(K):
    # two batches decoded concurrently, each with its own workspace, many times
    cs = [case(50 + i, 3, 16, 2, 128, 16, 60, [900, 100, 960]) for i in range(2)]
    ds = [on_device(c) for c in cs]
    wants = [run(K, c, d) for c, d in zip(cs, ds)]
    ss = [torch.cuda.Stream() for _ in cs]
    wss = [workspace(K, 3, 16, 128) for _ in cs]
    outs = [[], []]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (c, d, s, ws) in enumerate(zip(cs, ds, ss, wss)):
            with torch.cuda.stream(s):
                outs[i].append(K.paged_decode_mx4(d["q"], d["cache"], d["ks"], d["vs"], 2, d["table"], d["lens"],
                                                  c["sigma"], workspace=ws))
    torch.cuda.synchronize()
    for o, w in zip(outs, wants):
        assert all(np.array_equal(x.double().cpu().numpy(), w[0]) for x in o)


@pytest.mark.parametrize("per_channel", [False, True])
def test_lse_of_a_head_that_is_not_finite(K, per_channel):
    # NaN whichever way the work is cut, as the outputs are
    c = case(43, 2, 8, 1, 128, 16, 40, [600, 33], per_channel)
    c["q"][0, 2, 5], c["q"][0, 6, 7], c["q"][1, 1, 9] = np.nan, np.inf, -np.inf
    bad = np.zeros((2, 8), bool)
    bad[0, [2, 6]] = bad[1, 1] = True
    for ns, chunk in ((0, 0), (1, 640), (2, 0), (5, 0), (8, 0), (10, 64), (32, 0)):
        o, l = run(K, c, ns=ns, chunk=chunk)
        assert np.isnan(l[bad]).all(), (ns, chunk)
        assert np.isnan(o[bad]).all(), (ns, chunk)
        assert np.isfinite(l[~bad]).all() and np.isfinite(o[~bad]).all(), (ns, chunk)


@pytest.mark.parametrize("D,per_channel", [(64, False), (128, False), (256, False), (128, True)])
@pytest.mark.parametrize("inf", [np.inf, -np.inf])
def test_an_infinite_query_whose_scores_all_have_one_sign(K, D, per_channel, inf):
    # every key has the same sign in the channel, so every score is +inf or every one -inf
    c = case(44 + D, 2, 4, 1, D, 16, 8, [128, 20], per_channel)
    c["cache"][..., :8 * D] = 0x22  # code 1.0 in every channel of every key
    ref = reference(c)
    c["q"][0, 1, 3] = inf
    bad = np.zeros((2, 4), bool)
    bad[0, 1] = True
    for ns, chunk in ((0, 0), (1, 128), (2, 0), (5, 0), (4, 32)):
        o, l = run(K, c, ns=ns, chunk=chunk)
        assert np.isnan(o[bad]).all() and np.isnan(l[bad]).all(), (ns, chunk)
        pick = lambda x: x[~bad][None]
        compare(dict(c, q=c["q"][~bad][None]), (pick(o), pick(l)), [pick(x) for x in ref], what=f"{ns} splits of {chunk}")


@pytest.mark.parametrize("window", [-1, 1 << 30])
def test_the_longest_sequence(K, window):
    # 2^31 - 32 tokens, as many as positions of 32 bits take: a table that names one block over and over.
    # Zero queries and values of 1 make every sum exact: the mean is 1, the lse log of the tokens
    D, tiles, mb = 64, 6 * 8191, 2731
    n = 16 * tiles * mb
    assert n == 2 ** 31 - 32
    cache = torch.zeros((1, 1, tiles, 18 * D), dtype=torch.uint8, device="cuda")
    cache[..., 9 * D:17 * D] = 0x22
    cache[..., 17 * D:] = 0x38
    one = torch.ones(1, device="cuda")
    q = torch.zeros((1, 2, D), dtype=torch.float16, device="cuda")
    table = torch.zeros((1, mb), dtype=torch.int32, device="cuda")
    ws = workspace(K, 1, 2, D)
    for length in (n, n - 500):
        live = length if window < 0 else min(length, window + 1)
        lens = torch.tensor([length], dtype=torch.int32, device="cuda")
        for ns in (32, 31, 0):
            lse = torch.empty((1, 2), device="cuda")
            out = K.paged_decode_mx4(q, cache, one, one, 1, table, lens, 0.125, num_splits=ns, workspace=ws, lse=lse,
                                     window=window)
            assert (out == 1).all()
            # (the logarithm of 2^31 / 32, and its sum with 8 log 2 and the pieces': a few steps of 2^-20)
            assert (lse.double() - np.log(live)).abs().max().item() <= 1e-5, (length, ns)
