"""The cache-side operators of a serving step, as cases to be timed and compared: the append of new rows with
their position rotation (``rope_and_cache``), the read-back of cache rows (``gather_cache``) and the decode of one
new token over a paged 4-bit cache (``paged_decode_mx4``).  ``run`` computes them from elementary torch operations,
or, where ``own`` is true, with the package's calls.

MX4, the 4-bit cache: uint8 [num_blocks, Hkv, block_size / 16, 18 * D].  One record holds 16 tokens of one KV head:
K codes [16, D / 2] (e2m1, the even channel in the low nibble), K block scales [16, D / 16] (e4m3), V codes [16, D / 2],
V block scales [16, D / 16].  value = scale * block scale * e2m1 value, scale one number or one per (head, channel).
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
PER_TENSOR, PER_CHANNEL = 1, 2  # scale kinds, as the package numbers them


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a batch: 16 new tokens at their own positions, into an int8 cache
        dict(name="append_decode_int8", op="append", T=16, Hq=32, Hkv=8, D=128, R=128, kind="int8", per_channel=True,
             interleaved=False, max_pos=8192, chunked=False),
        # a prompt of 8192 tokens into an int8 cache, from one fused projection
        dict(name="append_prompt_int8", op="append", T=8192, Hq=32, Hkv=8, D=128, R=128, kind="int8", per_channel=True,
             interleaved=False, max_pos=16384, chunked=True),
        # the largest: 32768 prompt tokens of several requests into the 4-bit cache
        dict(name="append_prompt_mx4", op="append", T=32768, Hq=32, Hkv=8, D=128, R=128, kind="mx4", per_channel=False,
             interleaved=False, max_pos=131072, chunked=True),
        # an odd chunk of a small-headed model, adjacent channels rotated in pairs, float8 cache
        dict(name="append_chunk_e4m3", op="append", T=2049, Hq=16, Hkv=2, D=64, R=64, kind="e4m3", per_channel=False,
             interleaved=True, max_pos=4096, chunked=True),
        # wide heads of which a quarter is rotated, values kept in fp16
        dict(name="append_partial_fp16", op="append", T=517, Hq=24, Hkv=2, D=256, R=64, kind="fp16", per_channel=False,
             interleaved=False, max_pos=32768, chunked=True),
        # a cached prefix of 16384 tokens read back for a dense prefill over it
        dict(name="gather_prefix_mx4", op="gather", N=16384, Hkv=8, D=128, kind="mx4", per_channel=True),
        # a few int8 rows with padding among them
        dict(name="gather_rows_int8", op="gather", N=129, Hkv=2, D=256, kind="int8", per_channel=True),
        # one sequence with a short context: latency
        dict(name="decode_one_short", op="decode", B=1, Hq=32, Hkv=8, D=128, lo=300, hi=300, per_channel=False, sink=False,
             softcap=0.0, window=-1, len_seed=1),
        # a ragged batch under a sink: the repository's paged decode workload
        dict(name="decode_ragged", op="decode", B=16, Hq=32, Hkv=8, D=128, lo=512, hi=8192, per_channel=True, sink=True,
             softcap=0.0, window=-1, len_seed=2),
        # equal contexts, few KV heads: the repository's deep-context workload
        dict(name="decode_deep", op="decode", B=16, Hq=16, Hkv=2, D=128, lo=2600, hi=2600, per_channel=True, sink=False,
             softcap=0.0, window=-1, len_seed=3),
        # long documents
        dict(name="decode_long", op="decode", B=16, Hq=32, Hkv=8, D=128, lo=8192, hi=32768, per_channel=False, sink=False,
             softcap=0.0, window=-1, len_seed=4),
        # a whole step of wide heads: append the new token's row, then attend it and a window before it
        dict(name="step_wide_window", op="step", B=8, Hq=24, Hkv=2, D=256, R=128, lo=1, hi=4097, per_channel=True, sink=True,
             softcap=30.0, window=2047, len_seed=5, interleaved=False),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "append", "gather", "decode", "decode", "step"))
    D = rng.choice((64, 128, 128, 256))
    Hkv = rng.choice((1, 2, 4, 8))
    Hq = Hkv * rng.choice((1, 2, 4, 5, 8, 12, 16))
    if op == "append":
        T = _log_uniform(rng, 1, max(1, min(32768, (32768 * 48 * 128) // ((Hq + 2 * Hkv) * D))))
        kind = rng.choice(("int8", "e4m3", "fp16", "mx4", "mx4"))
        R = rng.choice([r for r in (0, 32, 64, 128, 256) if r <= D])
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, D=D, R=R, kind=kind, per_channel=rng.random() < 0.5,
                    interleaved=rng.random() < 0.4, max_pos=T + rng.randrange(1, 65536), chunked=rng.random() < 0.5)
    if op == "gather":
        return dict(op=op, N=_log_uniform(rng, 1, 16384), Hkv=Hkv, D=D, kind=rng.choice(("int8", "e4m3", "fp16", "mx4", "mx4")),
                    per_channel=rng.random() < 0.5)
    B = _log_uniform(rng, 1, 160)
    top = max(2, min(32768, (16 * 20480 * 8 * 128) // (B * Hkv * D)))
    hi = _log_uniform(rng, 1, top)
    lo = rng.choice((hi, max(1, hi // 16), 0 if op == "decode" and hi >= 64 and B > 2 else 1))
    case = dict(op=op, B=B, Hq=Hq, Hkv=Hkv, D=D, lo=min(lo, hi), hi=hi, per_channel=rng.random() < 0.5, sink=rng.random() < 0.5,
                softcap=rng.choice((0.0, 0.0, 30.0)), window=rng.choice((-1, -1, rng.randrange(0, 4096))),
                len_seed=rng.randrange(1 << 20))
    if op == "step":
        case.update(R=rng.choice([r for r in (32, 64, 128, 256) if r <= D]), interleaved=rng.random() < 0.4)
    return case


def _lens(case):
    """The live lengths (new token included): the case's own, so that the work is known without a seed."""
    r = random.Random(case["len_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


_ELEM = {"int8": 1.0, "e4m3": 1.0, "fp16": 2.0, "mx4": 0.5625}  # bytes of one cached value


def _append_bytes(T, Hq, Hkv, D, R, kind):
    return T * (Hq * D * 4 + 2 * Hkv * D * 2 + 2 * Hkv * D * _ELEM[kind] + 4 * R + 8)


def work(case):
    if case["op"] == "append":  # rows in, rotated queries and cache rows out, and the cached values as read back
        T, Hkv, D = case["T"], case["Hkv"], case["D"]
        rows = _append_bytes(T, case["Hq"], Hkv, D, case["R"], case["kind"])
        return {"bytes": rows + T * 4 * Hkv * D, "flops": 3.0 * T * (case["Hq"] + Hkv) * case["R"]}
    if case["op"] == "gather":
        n = case["N"] * 2 * case["Hkv"] * case["D"]
        return {"bytes": n * (_ELEM[case["kind"]] + 2) + 4 * case["N"], "flops": n}
    w = case["window"]
    live = sum(n if w < 0 else min(n, w + 1) for n in _lens(case))
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    bytes_ = live * Hkv * 2 * D * _ELEM["mx4"] + 4 * B * Hq * D + live / 4
    if case["op"] == "step":
        bytes_ += _append_bytes(B, Hq, Hkv, D, case["R"], "mx4") - 2 * B * Hq * D
    return {"bytes": bytes_, "flops": 4.0 * D * Hq * live}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rotate(x, cs, positions, interleaved):
    """x [T, H, D]; cs [max_pos, R]: cosines of the R / 2 angles, then sines.  fp32, every product and sum rounded once."""
    x = x.float()
    if cs is None:
        return x
    R = cs.shape[1]
    t = cs[positions.long()]
    c, s = t[:, None, :R // 2], t[:, None, R // 2:]
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        rot = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        rot = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return torch.cat((rot, x[..., R:]), dim=-1)


def _mx4_codes(x, scale):
    """fp32 [..., D] -> (codes [..., D] in 0..15, e4m3 block scales [..., D / 16])."""
    y = (x * (1.0 / scale)).unflatten(-1, (-1, 16))
    s = (y.abs().amax(-1) * (1.0 / 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()[..., None]
    q = torch.where(sf > 0, y * (1.0 / torch.where(sf > 0, sf, 1.0)), torch.zeros_like(y))
    a = q.abs()
    # ties to the even code: the half-way points 0.25, 1.25, 2.5 and 5 go down, 0.75, 1.75 and 3.5 go up
    m = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
         + (a >= 3.5).int() + (a > 5.0).int())
    return (m + 8 * (q < 0).int()).flatten(-2).to(torch.uint8), s


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpack(b):
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=b.device)
    n = torch.stack((b & 15, b >> 4), dim=-1).flatten(-2)
    return lut[n.int()]


def _fields(rec, D):
    """Views of the fields of records [..., 18 D]: K codes, K scales, V codes, V scales."""
    kc = rec[..., :8 * D].unflatten(-1, (16, D // 2))
    ks = rec[..., 8 * D:9 * D].unflatten(-1, (16, D // 16))
    vc = rec[..., 9 * D:17 * D].unflatten(-1, (16, D // 2))
    vs = rec[..., 17 * D:].unflatten(-1, (16, D // 16))
    return kc, ks, vc, vs


def _mx4_values(codes, scales):
    """Packed codes [..., D / 2] and scale bytes [..., D / 16] -> fp32 values [..., D] (without the outer scale)."""
    s = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (_unpack(codes).unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _mx4_rows(cache, slots, D):
    """The fields of the cache at token slots [N]: ([N, Hkv, D / 2], [N, Hkv, D / 16]) of K and of V."""
    bs = cache.shape[2] * 16
    slots = slots.long()
    blk, off = slots // bs, slots % bs
    at = (blk, slice(None), off // 16, off % 16)
    return tuple(f[at] for f in _fields(cache, D))


def _plain_append(st):
    q, k, v = st["q"], st["k"], st["v"]
    qr = _rotate(q, st["cs"], st["positions"], st["interleaved"]).half()
    kr = _rotate(k, st["cs"], st["positions"], st["interleaved"])
    vr = v.float()
    slots, D = st["slots"].long(), k.shape[-1]
    if st["kind"] == "mx4":
        cache = st["k_cache"]
        bs = cache.shape[2] * 16
        blk, off = slots // bs, slots % bs
        at = (blk, slice(None), off // 16, off % 16)
        fkc, fks, fvc, fvs = _fields(cache, D)
        for x, sc, fc, fs in ((kr, st["k_scale"], fkc, fks), (vr, st["v_scale"], fvc, fvs)):
            c, s = _mx4_codes(x, sc)
            fc[at] = _pack(c)
            fs[at] = s.view(torch.uint8)
        return qr
    for x, sc, cache in ((kr, st["k_scale"], st["k_cache"]), (vr, st["v_scale"], st["v_cache"])):
        flat = cache.view(-1, *cache.shape[-2:])
        if st["kind"] == "int8":
            flat[slots] = (x / sc).round().clamp(-127, 127).to(torch.int8)
        elif st["kind"] == "e4m3":
            flat.view(torch.uint8)[slots] = (x / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            flat[slots] = x.half()
    return qr


def _plain_gather(st):
    slots = st["slots"].long()
    good = (slots >= 0)[:, None, None]
    at = slots.clamp(min=0)
    if st["kind"] == "mx4":
        kc, ks, vc, vs = _mx4_rows(st["k_cache"], at, st["D"])
        k, v = _mx4_values(kc, ks) * st["k_scale"], _mx4_values(vc, vs) * st["v_scale"]
    elif st["kind"] == "fp16":
        k, v = (st[c].view(-1, *st[c].shape[-2:])[at].float() for c in ("k_cache", "v_cache"))
    else:
        k, v = (st[c].view(-1, *st[c].shape[-2:]).view(torch.uint8)[at].view(st[c].dtype).float() * st[s]
                for c, s in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
    return torch.where(good, k, 0.0).half(), torch.where(good, v, 0.0).half()


def _plain_decode(st, q):
    cache, table, lens = st["k_cache"], st["table"], st["lens"]
    B, Hq, D = q.shape
    nb, Hkv, tiles, _ = cache.shape
    mb = table.shape[1]
    rec = cache[table.clamp(min=0).long()]  # [B, mb, Hkv, tiles, 18 D]
    rec = rec.transpose(1, 2).reshape(B, Hkv, mb * tiles, 18 * D)
    kc, ks, vc, vs = _fields(rec, D)
    k = _mx4_values(kc, ks).reshape(B, Hkv, mb * tiles * 16, D)
    qs = q.float().view(B, Hkv, Hq // Hkv, D)
    if st["per_channel"]:
        qs = qs * st["k_scale"][None, :, None, :]
    s = torch.matmul(qs, k.transpose(-1, -2)) * st["sigma"]
    del k
    if not st["per_channel"]:
        s = s * st["k_scale"]
    if st["softcap"] > 0:
        s = st["softcap"] * torch.tanh(s / st["softcap"])
    t = torch.arange(s.shape[-1], device=s.device)[None, None, None, :]
    n = lens.long()[:, None, None, None]
    live = t < n
    if st["window"] >= 0:
        live = live & (t >= n - 1 - st["window"])
    s = torch.where(live, s, float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    v = _mx4_values(vc, vs).reshape(B, Hkv, mb * tiles * 16, D)
    o = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    o = o * (st["v_scale"][None, :, None, :] if st["per_channel"] else st["v_scale"])
    if st["sink"] is not None:
        z = st["sink"].view(1, Hkv, -1, 1) - (m + torch.log(l))
        o = torch.where(l > 0, o / (1.0 + torch.exp(z)), o)
    return o.view(B, Hq, D).half()


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _angles(max_pos, R, device):
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=device) / R)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), dim=1).float()


def _scales(g, kind, Hkv, D, per_channel, std):
    """k or v scale as calibration gives it: the amplitude of each channel (or of all) over what the cache type holds."""
    if kind == "fp16":
        return None
    top = {"int8": 4.5 / 127, "e4m3": 4.5 / 448, "mx4": 1.0}[kind]
    return (std * top).contiguous() if per_channel else torch.full((1,), top, device=std.device)


def _empty_cache(kind, blocks, bs, Hkv, D, device):
    if kind == "mx4":
        return torch.zeros((blocks, Hkv, bs // 16, 18 * D), dtype=torch.uint8, device=device), None
    dt = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "fp16": torch.float16}[kind]
    return tuple(torch.zeros((blocks, bs, Hkv, D), dtype=torch.uint8 if kind == "e4m3" else dt, device=device).view(dt)
                 for _ in range(2))


def _channel_std(g, Hkv, D, per_channel):
    """Channel amplitudes: some channels are several times larger than others where the scales are per channel."""
    u = torch.rand((Hkv, D), generator=g, device=g.device)
    return torch.exp((u * 2 - 1) * math.log(2.0)) if per_channel else torch.ones((Hkv, D), device=g.device)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    bs = 16
    Hkv, D, op, pc = case["Hkv"], case["D"], case["op"], case["per_channel"]
    kind = case.get("kind", "mx4")
    std_k, std_v = _channel_std(g, Hkv, D, pc), _channel_std(g, Hkv, D, pc)
    st = dict(op=op, kind=kind, D=D, k_scale=_scales(g, kind, Hkv, D, pc, std_k), v_scale=_scales(g, kind, Hkv, D, pc, std_v),
              per_channel=pc, scale_kind=PER_CHANNEL if pc else PER_TENSOR)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def rows(T, Hq):
        """New rows as one projection leaves them: q, k and v side by side, [T, (Hq + 2 Hkv) D]."""
        qkv = torch.empty((T, (Hq + 2 * Hkv) * D), dtype=torch.float16, device=dev)
        st["q"], st["k"], st["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split((Hq * D, Hkv * D, Hkv * D), dim=1))
        st["q"].copy_(randn(T, Hq, D))
        st["k"].copy_(randn(T, Hkv, D) * std_k)
        st["v"].copy_(randn(T, Hkv, D) * std_v)

    if op == "append":
        T, R = case["T"], case["R"]
        rows(T, case["Hq"])
        blocks = -(-T // bs) + 2
        st["k_cache"], st["v_cache"] = _empty_cache(kind, blocks, bs, Hkv, D, dev)
        if case["chunked"]:  # consecutive positions; consecutive tokens fill scattered blocks
            p0 = int(torch.randint(0, case["max_pos"] - T + 1, (1,), generator=g, device=dev))
            st["positions"] = torch.arange(p0, p0 + T, device=dev, dtype=torch.int32)
            table = torch.randperm(blocks, generator=g, device=dev)
            t = torch.arange(T, device=dev)
            st["slots"] = (table[t // bs] * bs + t % bs).int()
        else:  # one token of each of T sequences
            st["positions"] = torch.randint(0, case["max_pos"], (T,), generator=g, device=dev, dtype=torch.int32)
            st["slots"] = torch.randperm(blocks * bs, generator=g, device=dev)[:T].int()
        st["cs"] = _angles(case["max_pos"], R, dev) if R else None
        st["interleaved"] = case["interleaved"]
        return st
    if op == "gather":
        N = case["N"]
        blocks = -(-N // bs) + 1
        st["k_cache"], st["v_cache"] = _empty_cache(kind, blocks, bs, Hkv, D, dev)
        fill = dict(st, q=randn(blocks * bs, 1, D).half(), k=(randn(blocks * bs, Hkv, D) * std_k).half(),
                    v=(randn(blocks * bs, Hkv, D) * std_v).half(), cs=None, positions=None, interleaved=False,
                    slots=torch.arange(blocks * bs, device=dev))
        _plain_append(fill)
        table = torch.randperm(blocks, generator=g, device=dev)
        t = torch.arange(N, device=dev)
        slots = (table[t // bs] * bs + t % bs).int()
        st["slots"] = torch.where(torch.rand((N,), generator=g, device=dev) < 0.02, torch.full_like(slots, -1), slots)
        return st
    # decode / step: B sequences over a pool of randomly placed blocks
    B, Hq = case["B"], case["Hq"]
    lens = _lens(case)
    need = [-(-n // bs) for n in lens]
    mb = max(max(need), 1)
    pool = max(sum(need), 1)
    st["k_cache"], st["v_cache"] = _empty_cache("mx4", pool, bs, Hkv, D, dev)
    step = 4096  # blocks filled at a time
    for b0 in range(0, pool, step):
        n = min(step, pool - b0) * bs
        _plain_append(dict(st, q=randn(1, 1, D), k=(randn(n, Hkv, D) * std_k).half(), v=(randn(n, Hkv, D) * std_v).half(),
                           cs=None, positions=None, interleaved=False, slots=torch.arange(b0 * bs, b0 * bs + n, device=dev)))
    perm = torch.randperm(pool, generator=g, device=dev).int()
    table = torch.full((B, mb), -1, dtype=torch.int32, device=dev)
    owner = torch.arange(mb, device=dev)[None, :] < torch.tensor(need, device=dev)[:, None]
    table[owner] = perm[:sum(need)]
    st.update(table=table, lens=torch.tensor(lens, dtype=torch.int32, device=dev), sigma=D ** -0.5, softcap=case["softcap"],
              window=case["window"], sink=randn(Hq) if case["sink"] else None)
    # scratch a serving loop keeps: the largest the decode asks for (32 splits of each row)
    st["workspace"] = torch.empty(32 * B * Hq * (D + 2), dtype=torch.float32, device=dev)
    rows(B, Hq)
    if op == "decode":
        st["q"] = st["q"].contiguous()
        return st
    st["positions"] = st["lens"] - 1
    last = st["positions"].long()
    st["slots"] = (table[torch.arange(B, device=dev), last // bs].long() * bs + last % bs).int()
    st["cs"] = _angles(case["hi"], case["R"], dev)
    st["interleaved"] = case["interleaved"]
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    st = state
    if own:
        import int8_kv_cache_gb300 as K

        if st["op"] in ("append", "step"):
            q = K.rope_and_cache(st["q"], st["k"], st["v"], st["positions"], st["cs"], st["slots"], st["k_cache"],
                                 st["v_cache"], st["k_scale"], st["v_scale"], st["scale_kind"],
                                 interleaved=st["interleaved"])
        if st["op"] in ("append", "gather"):
            k, v = K.gather_cache(st["slots"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"],
                                  st["scale_kind"])
            return (q, k, v) if st["op"] == "append" else (k, v)
        out = K.paged_decode_mx4(q if st["op"] == "step" else st["q"], st["k_cache"], st["k_scale"], st["v_scale"],
                                 st["scale_kind"], st["table"], st["lens"], st["sigma"], st["sink"],
                                 workspace=st["workspace"], softcap=st["softcap"], window=st["window"])
        return (q, out) if st["op"] == "step" else out
    if st["op"] == "gather":
        return _plain_gather(st)
    if st["op"] == "append":
        q = _plain_append(st)
        return (q,) + _plain_gather(st)
    if st["op"] == "step":
        q = _plain_append(st)
        return q, _plain_decode(st, q)
    return _plain_decode(st, st["q"])


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _grid_round(x, mant, emin, top):
    """Nearest value with `mant` mantissa bits after the leading one, exponents >= emin, magnitude <= top."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=emin).double() - mant)
    return (torch.round(x / step) * step).clamp(-top, top)


def _exact_rotation(x, positions, R, interleaved):
    x = x.double()
    if R == 0:
        return x
    out = x.clone()
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=x.device) / R)
    ang = positions.double()[:, None, None] * inv
    first = torch.arange(R // 2, device=x.device) * (2 if interleaved else 1)
    second = first + (1 if interleaved else R // 2)
    out[..., first] = x[..., first] * ang.cos() - x[..., second] * ang.sin()
    out[..., second] = x[..., second] * ang.cos() + x[..., first] * ang.sin()
    return out


def _exact_stored(x, scale, kind):
    """The value that the cache keeps of x, in 64 bits."""
    if kind == "fp16":
        return x.half().double()
    y = x / scale.double()
    if kind == "int8":
        return torch.round(y).clamp(-127, 127) * scale.double()
    if kind == "e4m3":
        return _grid_round(y, 3, -6, 448.0) * scale.double()
    b = y.reshape(*y.shape[:-1], -1, 16)
    s = _grid_round(b.abs().max(-1, keepdim=True).values / 6.0, 3, -6, 448.0)
    c = _grid_round(b / s.clamp(min=1e-300), 1, 0, 6.0)
    return (c * s).reshape(y.shape) * scale.double()


def _exact_record(rec, D):
    """(K, V) [..., 16, D] of records in 64 bits, from the bits of the codes and scales."""
    rec = rec.to(torch.int32)

    def nibbles(b):
        n = torch.empty((*b.shape, 2), dtype=torch.int32, device=b.device)
        n[..., 0], n[..., 1] = b % 16, b // 16
        return n.reshape(*b.shape[:-1], -1)

    def e2m1(n):
        e, m = (n % 8) // 2, (n % 2).double()
        mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
        return torch.where(n >= 8, -mag, mag)

    def e4m3(n):
        e, m = n // 8, (n % 8).double()
        return torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))

    def at(i, n, shape):
        return rec[..., i:i + n].reshape(*rec.shape[:-1], *shape)

    k = e2m1(nibbles(at(0, 8 * D, (16, D // 2))))
    ks = e4m3(at(8 * D, D, (16, D // 16)))
    v = e2m1(nibbles(at(9 * D, 8 * D, (16, D // 2))))
    vs = e4m3(at(17 * D, D, (16, D // 16)))
    return k * ks.repeat_interleave(16, -1), v * vs.repeat_interleave(16, -1)


def _exact_attention(st, q, lens, row_values):
    """q [B, Hq, D] in 64 bits; row_values(b) gives sequence b's keys and values [n, Hkv, D] (outer scales applied)."""
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k, v = row_values(b, n)
        lo = 0 if st["window"] < 0 else max(0, n - 1 - st["window"])
        k, v = k[lo:n], v[lo:n]
        Hkv = k.shape[1]
        s = torch.einsum("hgd,thd->hgt", q[b].reshape(Hkv, -1, q.shape[-1]), k) * st["sigma"]
        if st["softcap"] > 0:
            s = st["softcap"] * torch.tanh(s / st["softcap"])
        lse = torch.logsumexp(s, -1)
        o = torch.einsum("hgt,thd->hgd", torch.exp(s - lse[..., None]), v)
        if st["sink"] is not None:
            o = o * torch.sigmoid(lse - st["sink"].double().view(Hkv, -1))[..., None]
        out[b] = o.reshape(q.shape[1:])
    return out


def exact(case, seed):
    st = prepare(case, seed)
    D, kind = st["D"], st["kind"]
    slots = st["slots"].long() if "slots" in st else None
    if case["op"] == "append":
        q = _exact_rotation(st["q"], st["positions"], case["R"], case["interleaved"])
        k = _exact_rotation(st["k"], st["positions"], case["R"], case["interleaved"])
        return q, _exact_stored(k, st["k_scale"], kind), _exact_stored(st["v"].double(), st["v_scale"], kind)
    if case["op"] == "gather":
        keep = (slots >= 0).double()[:, None, None]
        at = slots.clamp(min=0)
        if kind == "mx4":
            k, v = _exact_record(st["k_cache"], D)  # [blocks, Hkv, 1, 16, D]
            k, v = (x.transpose(1, 2).transpose(2, 3).reshape(-1, case["Hkv"], D)[at] for x in (k, v))
        else:
            k, v = (st[c].double().reshape(-1, case["Hkv"], D)[at] for c in ("k_cache", "v_cache"))
        if kind != "fp16":
            k, v = k * st["k_scale"].double(), v * st["v_scale"].double()
        return k * keep, v * keep
    lens = _lens(case)
    if sum(lens) * case["Hkv"] * D > 16 * 40000 * 8 * 128:
        return None
    q = st["q"].double()
    if case["op"] == "step":
        q = _exact_rotation(st["q"], st["positions"], case["R"], case["interleaved"])
        knew = _exact_rotation(st["k"], st["positions"], case["R"], case["interleaved"])
        knew = _exact_stored(knew, st["k_scale"], "mx4")
        vnew = _exact_stored(st["v"].double(), st["v_scale"], "mx4")

    def row_values(b, n):
        rec = st["k_cache"][st["table"][b, :-(-n // 16)].long()]  # [nblk, Hkv, 1, 18 D]
        k, v = (x.permute(0, 2, 3, 1, 4).reshape(-1, case["Hkv"], D) for x in _exact_record(rec, D))
        k, v = k * st["k_scale"].double(), v * st["v_scale"].double()
        if case["op"] == "step":
            k[n - 1], v[n - 1] = knew[b], vnew[b]
        return k, v

    # a query is attended as the rotation leaves it: rounded to fp16
    out = _exact_attention(st, q.half().double(), lens, row_values)
    return (q, out) if case["op"] == "step" else out
