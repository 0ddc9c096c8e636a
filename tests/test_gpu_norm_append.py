"""norm_rope_and_cache on the GPU: the normed and turned queries and keys against 64 bits, and the stored codes
against those of every value that fp32's roundings allow."""
import numpy as np
import pytest
import torch

import oracle.mx4 as mx4

pytestmark = pytest.mark.gpu

KINDS = ["int8", "e4m3", "fp16", "mx4"]
EPS = 1e-5
# The norm and the turn in fp32: the sum of D squares of fp16 values (exact products, at most D / 16 + 20 roundings of
# 2^-24 below), its mean, eps, the root (half of their error) and two products, then two products and a sum of the turn:
# below 24 roundings of 2^-24, relative to |a| + |b| of a pair.
OFF = 24 * 2.0 ** -24


@pytest.fixture(scope="module")
def K():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import int8_kv_cache_gb300 as K
    K.load()
    return K


def make(seed, kind, T, Hq, Hkv, D, R, per_channel, nb=40, bs=16, max_pos=91):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"

    def randn(*s):
        return torch.randn(s, generator=g, device=dev)

    x = torch.empty((T, Hq + 2 * Hkv, D), dtype=torch.float16, device=dev)
    x.copy_(randn(T, Hq + 2 * Hkv, D) * torch.exp(2 * randn(T, Hq + 2 * Hkv, 1)))
    x[0, 0] = 0  # a head of zeros: eps alone
    x[-1, Hq, :] = 60000.0
    c = dict(q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:], kind=kind, kind_of_scale=2 if per_channel else 1)
    a = torch.rand((max_pos, max(R // 2, 1)), generator=g, device=dev) * 8 - 4
    c["cs"] = torch.cat((a.cos(), a.sin()), 1).float().contiguous() if R else None
    c["pos"] = torch.randint(0, max_pos, (T,), generator=g, device=dev, dtype=torch.int32)
    c["slots"] = torch.randperm(nb * bs, generator=g, device=dev)[:T].int()
    if T > 4:
        c["slots"][2] = -1
    c["qw"], c["kw"] = (1 + 0.3 * randn(D) for _ in range(2))
    shape = (Hkv, D) if per_channel else (1,)
    top = {"int8": 1 / 40, "e4m3": 1 / 100, "mx4": 1.0, "fp16": 1.0}[kind]
    c["ks"], c["vs"] = (torch.exp(torch.rand(shape, generator=g, device=dev) * 2 - 1) * top for _ in range(2))
    if kind == "mx4":
        c["kc"], c["vc"] = torch.zeros((nb, Hkv, bs // 16, 18 * D), dtype=torch.uint8, device=dev), None
    else:
        dt = {"int8": torch.int8, "e4m3": torch.uint8, "fp16": torch.float16}[kind]
        c["kc"], c["vc"] = (torch.zeros((nb, bs, Hkv, D), dtype=dt, device=dev) for _ in range(2))
    return c


def exact(x, w, cs, pos, interleaved):
    """The normed and turned heads in 64 bits, and |a| + |b| of each channel's pair."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()
    y, size = x.clone(), x.abs()
    if cs is not None:
        R = cs.shape[1]
        t = cs.double()[pos.long()][:, None]
        co, si = t[..., :R // 2], t[..., R // 2:]
        i = torch.arange(R // 2, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        y[..., a], y[..., b] = x[..., a] * co - x[..., b] * si, x[..., b] * co + x[..., a] * si
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def within(got, ref, size):
    bound = 2.0 ** -11 * ref.abs() + 1.01 * OFF * size + 2.0 ** -25
    # fp16 ends at 65504 and its step there is 32: what reaches 65520 is an infinity
    inf = torch.isinf(got)
    assert (ref.abs() + 1.01 * OFF * size >= 65520)[inf].all() and (torch.sign(got) == torch.sign(ref))[inf].all()
    assert (ref.abs() - 1.01 * OFF * size < 65520)[~inf].all()
    off = torch.where(inf, 0.0, (got.double() - ref).abs())
    assert (off <= bound).all(), f"{(off / bound).max():.3f} times the bound off"


def e2m1(y):
    """Nearest e2m1 values, ties to the even code."""
    return torch.from_numpy(mx4.e2m1_value(mx4.e2m1_encode(y.cpu().numpy()))).to(y.device)


def codes(kind, y):
    if kind == "int8":
        return torch.round(y).clamp(-127, 127)
    return y.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()


def check_stored(c, y, size, is_v, off=OFF):
    """The cache's rows at the slots are codes of values within `off` of y (rounding is monotonic)."""
    sel = c["slots"].long() >= 0
    slots, y, size = c["slots"].long()[sel], y[sel], size[sel]
    scale = (c["vs"] if is_v else c["ks"]).double()
    cache = c["vc"] if is_v and c["kind"] != "mx4" else c["kc"]
    D = y.shape[-1]
    if c["kind"] == "mx4":
        bs = cache.shape[2] * 16
        at = (slots // bs, slice(None), slots % bs // 16)
        rec = cache[at]  # [T, Hkv, 18 D]
        tok = slots % 16
        base = 9 * D if is_v else 0
        code = rec[..., base:base + 8 * D].unflatten(-1, (16, D // 2))[torch.arange(len(slots)), :, tok].cpu().numpy()
        sb = rec[..., base + 8 * D:base + 9 * D].unflatten(-1, (16, D // 16))[torch.arange(len(slots)), :, tok]
        got = torch.from_numpy(mx4.e2m1_value(mx4.unpack(code))).to(y.device)
        s = sb.view(torch.float8_e4m3fn).double()
        z, zs = (y / scale).unflatten(-1, (-1, 16)), (size / scale).unflatten(-1, (-1, 16))
        slack = off + 4 * 2.0 ** -24  # the reciprocals' and the products' roundings
        top = (z.abs().amax(-1) / 6, zs.amax(-1) * slack / 6 + z.abs().amax(-1) * 2.0 ** -22)
        for sign, cmp in ((-1, torch.ge), (1, torch.le)):
            assert cmp(s, (top[0] + sign * top[1]).clamp(0, 448).float().to(torch.float8_e4m3fn).double()).all()
        zero = s[..., None] == 0
        sv = torch.where(zero, 1.0, s[..., None])
        lo, hi = ((z + d * (zs * slack + z.abs() * 2.0 ** -22)) / sv for d in (-1, 1))
        got = got.unflatten(-1, (-1, 16))
        assert torch.where(zero, got == 0, (got >= e2m1(lo)) & (got <= e2m1(hi))).all()
        return
    raw = cache.flatten(0, 1)[slots]
    if c["kind"] == "fp16":
        return within(raw, y, size if not is_v else torch.zeros_like(size))
    got = raw.double() if c["kind"] == "int8" else raw.view(torch.float8_e4m3fn).double()
    z, zs = y / scale, size / scale
    d = zs * off + z.abs() * 2.0 ** -23
    assert ((got >= codes(c["kind"], z - d)) & (got <= codes(c["kind"], z + d))).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,R", [(1, 1, 1, 64, 64), (7, 8, 2, 128, 128), (37, 5, 1, 128, 64), (19, 24, 2, 256, 128),
                                          (600, 10, 2, 64, 32), (5, 4, 4, 256, 0), (530, 32, 8, 128, 128)])
def test_against_64_bits(K, kind, interleaved, T, Hq, Hkv, D, R):
    c = make(T + D, kind, T, Hq, Hkv, D, R, per_channel=T % 2 == 1)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k = K.norm_rope_and_cache(c["q"], c["k"], c["v"], c["qw"], c["kw"], EPS, c["pos"], c["cs"], c["slots"], c["kc"],
                                 c["vc"], c["ks"], c["vs"], c["kind_of_scale"], interleaved=interleaved, flags=flags,
                                 return_keys=True)
    assert int(flags) == 0
    within(q, *exact(c["q"], c["qw"], c["cs"], c["pos"], interleaved))
    ky, ksize = exact(c["k"], c["kw"], c["cs"], c["pos"], interleaved)
    within(k, ky, ksize)
    check_stored(c, ky, ksize, False)
    check_stored(c, c["v"].double(), c["v"].double().abs(), True, off=2.0 ** -24)


@pytest.mark.parametrize("kind", KINDS)
def test_without_weights_it_is_the_plain_append(K, kind):
    a, b = (make(3, kind, 45, 6, 2, 128, 64, True) for _ in range(2))
    q = K.rope_and_cache(a["q"], a["k"], a["v"], a["pos"], a["cs"], a["slots"], a["kc"], a["vc"], a["ks"], a["vs"], 2)
    q2, none = K.norm_rope_and_cache(b["q"], b["k"], b["v"], None, None, EPS, b["pos"], b["cs"], b["slots"], b["kc"],
                                     b["vc"], b["ks"], b["vs"], 2)
    assert none is None and torch.equal(q, q2) and torch.equal(a["kc"], b["kc"])
    q3, k3 = K.norm_rope_and_cache(b["q"], b["k"], b["v"], None, None, EPS, b["pos"], b["cs"], b["slots"], b["kc"],
                                   b["vc"], b["ks"], b["vs"], 2, return_keys=True)
    assert torch.equal(q, q3) and torch.equal(a["kc"], b["kc"]) and (kind == "mx4" or torch.equal(a["vc"], b["vc"]))
    within(k3, *exact(b["k"], None, b["cs"], b["pos"], False))


@pytest.mark.parametrize("kind", KINDS)
def test_one_weight_no_query_and_in_place(K, kind):
    c = make(5, kind, 33, 4, 2, 128, 128, False)
    ky, ksize = exact(c["k"], c["kw"], c["cs"], c["pos"], False)
    qy, qsize = exact(c["q"], None, c["cs"], c["pos"], False)
    k, q = c["k"].contiguous(), c["q"].contiguous()
    q_out, k_out = K.norm_rope_and_cache(q, k, c["v"], None, c["kw"], EPS, c["pos"], c["cs"], c["slots"], c["kc"], c["vc"],
                                         c["ks"], c["vs"], 1, q_out=q, k_out=k)
    assert q_out is q and k_out is k
    within(q, qy, qsize)
    within(k, ky, ksize)
    check_stored(c, ky, ksize, False)
    nothing, k2 = K.norm_rope_and_cache(None, c["k"], c["v"], c["qw"], c["kw"], EPS, c["pos"], c["cs"], c["slots"], c["kc"],
                                        c["vc"], c["ks"], c["vs"], 1, return_keys=True)
    assert nothing is None and torch.equal(k2, k)


@pytest.mark.parametrize("kind", KINDS)
def test_skipped_tokens(K, kind):
    """A bad position leaves its rows alone; a slot past the pool or below zero stores nothing, and its queries and
    keys are still given."""
    c = make(6, kind, 24, 4, 2, 64, 64, False)
    c["pos"][5], c["pos"][9] = 91, -1
    c["slots"][9], c["slots"][7], c["slots"][11] = -1, 40 * 16, -3
    q_out, k_out = torch.full((24, 4, 64), 7.0, device="cuda").half(), torch.full((24, 2, 64), 7.0, device="cuda").half()
    before = c["kc"].clone()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    K.norm_rope_and_cache(c["q"], c["k"], c["v"], c["qw"], c["kw"], EPS, c["pos"], c["cs"], c["slots"], c["kc"], c["vc"],
                          c["ks"], c["vs"], 1, q_out=q_out, k_out=k_out, flags=flags)
    assert int(flags) == K.FLAG_BAD_POSITION | K.FLAG_BAD_SLOT
    skipped = [5, 9]
    assert bool((q_out[skipped] == 7).all()) and bool((k_out[skipped] == 7).all())
    rest = [i for i in range(24) if i not in skipped]
    pos = c["pos"].clamp(0, 90)
    for got, x, w in ((q_out, c["q"], c["qw"]), (k_out, c["k"], c["kw"])):
        y, size = exact(x, w, c["cs"], pos, False)
        within(got[rest], y[rest], size[rest])
    if kind != "mx4":
        written = torch.zeros(40 * 16, dtype=torch.bool, device="cuda")
        written[[int(s) for i, s in enumerate(c["slots"]) if i not in skipped and 0 <= s < 640]] = True
        assert torch.equal(c["kc"].flatten(0, 1)[~written], before.flatten(0, 1)[~written])


def test_values_that_are_no_numbers(K):
    c = make(7, "int8", 12, 4, 2, 128, 0, False)
    c["q"][3, 1, 5] = float("nan")
    c["q"][4, 2, 6] = float("inf")
    c["k"][5, 0, 7] = float("nan")
    q, k = K.norm_rope_and_cache(c["q"], c["k"], c["v"], c["qw"], c["kw"], EPS, None, None, c["slots"], c["kc"], c["vc"],
                                 c["ks"], c["vs"], 1, return_keys=True)
    assert bool(q[3, 1].isnan().all()) and bool(q[3, 0].isfinite().all()) and bool(q[2, 1].isfinite().all())
    assert bool(q[4, 2, 6].isnan()) and bool((q[4, 2, 7:] == 0).all())
    assert bool(k[5, 0].isnan().all()) and bool(k[5, 1].isfinite().all())
    assert bool((c["kc"].flatten(0, 1)[c["slots"][5].long(), 0] == 0).all())


def test_captured(K):
    c = make(8, "int8", 20, 4, 2, 128, 128, True)
    q_out, k_out = torch.empty((20, 4, 128), dtype=torch.float16, device="cuda"), torch.empty((20, 2, 128), dtype=torch.float16, device="cuda")

    def call(stream=None):
        K.norm_rope_and_cache(c["q"], c["k"], c["v"], c["qw"], c["kw"], EPS, c["pos"], c["cs"], c["slots"], c["kc"], c["vc"],
                              c["ks"], c["vs"], 2, q_out=q_out, k_out=k_out, stream=stream)
    call()
    torch.cuda.synchronize()
    want = q_out.clone(), k_out.clone(), c["kc"].clone()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
    for x in (q_out, k_out, c["kc"]):
        x.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (q_out, k_out, c["kc"])))
