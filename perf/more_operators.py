"""The prompt side of a serving step, as cases to be timed and compared: attention over whole prompts packed one after
another (``packed_prefill``), attention of a chunk of new tokens over a paged cache (``paged_prefill``), and the append of
new rows whose queries and keys are normed per head and turned by their positions (``norm_rope_and_cache``).  ``run``
computes them from elementary torch operations, or, where ``own`` is true, with the package's calls.

Attention: token i of a sequence's n new ones sits at position p = L - n + i of its L tokens and attends the positions
[max(0, p - window), p] (window < 0: [0, p]); scores are scaled, capped to softcap tanh(s / softcap) where a cap is given,
and a head's sink logit joins the sum of the softmax.  Query heads are grouped over the KV heads.

Caches: int8, e4m3 or fp16 [num_blocks, block_size, Hkv, D], times a scale (one, or one per head and channel; fp16 has
none); or MX4, uint8 [num_blocks, Hkv, block_size / 16, 18 * D], whose records hold 16 tokens of one KV head: K codes
[16, D / 2] (e2m1, the even channel in the low nibble), K block scales [16, D / 16] (e4m3), V codes, V block scales, and
value = scale * block scale * e2m1 value.

Norm: y = x / sqrt(mean(x^2) + eps) * weight over the D channels of a head, before the rotation.
"""
import math
import random

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
PER_TENSOR, PER_CHANNEL = 1, 2  # scale kinds, as the package numbers them
EPS = 1e-6
BLOCK = 16  # tokens of a cache block
SCRATCH = 64 << 20  # bytes of scratch that a serving loop keeps


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one short prompt: latency
        dict(name="packed_one_short", op="packed", B=1, lo=17, hi=17, Hq=32, Hkv=8, D=128, window=-1, softcap=0.0, sink=False,
             len_seed=1),
        # a batch of prompts of different lengths, one after another
        dict(name="packed_ragged", op="packed", B=16, lo=64, hi=2048, Hq=32, Hkv=8, D=128, window=-1, softcap=0.0, sink=False,
             len_seed=2),
        # the largest: one long document
        dict(name="packed_long", op="packed", B=1, lo=16384, hi=16384, Hq=32, Hkv=8, D=128, window=-1, softcap=0.0, sink=False,
             len_seed=3),
        # wide heads, few KV heads, a sliding window, capped scores and a sink
        dict(name="packed_wide_window", op="packed", B=3, lo=1000, hi=4097, Hq=24, Hkv=2, D=256, window=1023, softcap=30.0,
             sink=True, len_seed=4),
        # four proposed tokens of each sequence checked at once over a ragged batch, as the repository's paged decode workload
        dict(name="paged_verify_int8", op="paged", B=16, nlo=4, nhi=4, lo=512, hi=8192, Hq=32, Hkv=8, D=128, kind="int8",
             per_channel=True, window=-1, softcap=0.0, sink=True, len_seed=5),
        # the last chunk of a long prompt that is taken in chunks
        dict(name="paged_chunk_int8", op="paged", B=1, nlo=2048, nhi=2048, lo=16384, hi=16384, Hq=32, Hkv=8, D=128, kind="int8",
             per_channel=True, window=-1, softcap=0.0, sink=False, len_seed=6),
        # chunks and single tokens in one batch over the 4-bit cache
        dict(name="paged_mixed_mx4", op="paged", B=12, nlo=1, nhi=512, lo=600, hi=8192, Hq=32, Hkv=8, D=128, kind="mx4",
             per_channel=False, window=-1, softcap=0.0, sink=False, len_seed=7),
        # one new token of each of equal contexts, few KV heads: the repository's deep-context workload
        dict(name="paged_single_fp16", op="paged", B=16, nlo=1, nhi=1, lo=2600, hi=2600, Hq=16, Hkv=2, D=128, kind="fp16",
             per_channel=False, window=-1, softcap=0.0, sink=False, len_seed=8),
        # odd chunks of a small-headed model over a float8 cache
        dict(name="paged_chunk_e4m3", op="paged", B=4, nlo=300, nhi=1001, lo=1001, hi=4096, Hq=16, Hkv=2, D=64, kind="e4m3",
             per_channel=False, window=-1, softcap=0.0, sink=False, len_seed=9),
        # one decode step's rows: latency
        dict(name="norm_decode_int8", op="norm", T=16, Hq=32, Hkv=8, D=128, R=128, kind="int8", per_channel=True,
             interleaved=False, max_pos=8192, chunked=False),
        # prompt tokens of several requests into the 4-bit cache, from one fused projection
        dict(name="norm_prompt_mx4", op="norm", T=16384, Hq=32, Hkv=8, D=128, R=128, kind="mx4", per_channel=False,
             interleaved=False, max_pos=131072, chunked=True),
        # a layer's cache side: the chunks of a batch appended, then attended over what the cache holds
        dict(name="step_wide_int8", op="step", B=4, nlo=200, nhi=300, lo=1000, hi=8192, Hq=24, Hkv=2, D=256, R=64, kind="int8",
             per_channel=True, interleaved=True, window=-1, softcap=0.0, sink=False, len_seed=10),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("packed", "packed", "paged", "paged", "paged", "norm", "step"))
    D = rng.choice((64, 128, 128, 256))
    Hkv = rng.choice((1, 2, 4, 8))
    Hq = Hkv * rng.choice((1, 2, 4, 5, 8, 12, 16))
    case = dict(op=op, Hq=Hq, Hkv=Hkv, D=D)
    kind = rng.choice(("int8", "int8", "e4m3", "fp16", "mx4"))
    if op in ("norm", "step"):
        case.update(R=rng.choice([r for r in (32, 64, 128, 256) if r <= D]), interleaved=rng.random() < 0.4)
    if op == "norm":
        T = _log_uniform(rng, 1, min(16384, (16384 * 48 * 128) // ((Hq + 2 * Hkv) * D)))
        return dict(case, T=T, kind=kind, per_channel=rng.random() < 0.5, max_pos=T + rng.randrange(1, 65536),
                    chunked=rng.random() < 0.5)
    case.update(window=rng.choice((-1, -1, -1, rng.randrange(0, 4096))), softcap=rng.choice((0.0, 0.0, 0.0, 30.0)),
                sink=rng.random() < 0.3, len_seed=rng.randrange(1 << 20))
    room = (1 << 32) * 128 // (max(D, 128) * Hq)  # products of a batch's longest chunk and context, for each head
    if op == "packed":
        B = _log_uniform(rng, 1, 48)
        hi = _log_uniform(rng, 1, max(2, min(16384, math.isqrt(room // B), (1 << 27) // (B * (Hq + 2 * Hkv) * D) * 2)))
        return dict(case, B=B, lo=max(1, hi // rng.choice((1, 4, 16))), hi=hi)
    B = _log_uniform(rng, 1, 64)
    hi = _log_uniform(rng, 1, max(2, min(32768, (16 * 20480 * 8 * 128) // (B * Hkv * D))))
    few = _log_uniform(rng, 1, 16)
    nhi = min(hi, rng.choice((1, few, _log_uniform(rng, 1, 4096))), max(1, room // (B * hi)))
    return dict(case, B=B, nlo=max(1, nhi // rng.choice((1, 4, 16))), nhi=nhi, lo=max(nhi, hi // rng.choice((1, 4, 16))), hi=hi,
                kind=kind, per_channel=rng.random() < 0.5)


def _lens(case):
    """(lengths, new tokens of each sequence): the case's own, so that the work is known without a seed."""
    r = random.Random(case["len_seed"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    return lens, lens if case["op"] == "packed" else [r.randint(case["nlo"], min(case["nhi"], n)) for n in lens]


_ELEM = {"int8": 1.0, "e4m3": 1.0, "fp16": 2.0, "mx4": 0.5625}  # bytes of one cached value


def _append_work(T, Hq, Hkv, D, R, kind):
    rows = T * (Hq * D * 4 + 2 * Hkv * D * 2 + 2 * Hkv * D * _ELEM[kind] + 4 * R + 8)
    return rows, T * (Hq + Hkv) * (4.0 * D + 3.0 * R)


def _pairs(lens, new, window):
    """Attended (token, position) pairs, and the positions that some token of a sequence attends."""
    pairs = live = 0
    for L, n in zip(lens, new):
        w = L if window < 0 else window + 1
        full = max(0, min(n, L - w))  # tokens that see a whole window
        pairs += full * w + sum(range(L - n + 1, L + 1)) - sum(range(L - full + 1, L + 1))
        live += min(L, n - 1 + w)
    return pairs, live


def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "norm":  # rows in, turned queries, keys and cache rows out, and the cached values as read back
        b, f = _append_work(case["T"], Hq, Hkv, D, case["R"], case["kind"])
        return {"bytes": b + case["T"] * Hkv * D * 6, "flops": f}
    lens, new = _lens(case)
    T = sum(new)
    pairs, live = _pairs(lens, new, case["window"])
    kind = "fp16" if case["op"] == "packed" else case["kind"]
    b, f = 4 * T * Hq * D + 2 * live * Hkv * D * _ELEM[kind], 4.0 * D * Hq * pairs
    if case["op"] == "step":
        rows, more = _append_work(T, Hq, Hkv, D, case["R"], kind)
        b, f = b + rows - 2 * T * Hq * D, f + more
    return {"bytes": b, "flops": f}


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _normed(x, weight):
    x = x.float()
    return x * (1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)) * weight


def _rotate(x, cs, positions, interleaved):
    """x [T, H, D] fp32; cs [max_pos, R]: cosines of the R / 2 angles, then sines."""
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


def _fields(rec, D):
    """Views of the fields of records [..., 18 D]: K codes, K scales, V codes, V scales."""
    kc = rec[..., :8 * D].unflatten(-1, (16, D // 2))
    ks = rec[..., 8 * D:9 * D].unflatten(-1, (16, D // 16))
    vc = rec[..., 9 * D:17 * D].unflatten(-1, (16, D // 2))
    vs = rec[..., 17 * D:].unflatten(-1, (16, D // 16))
    return kc, ks, vc, vs


def _mx4_values(codes, scales):
    """Packed codes [..., D / 2] and scale bytes [..., D / 16] -> fp32 values [..., D] (without the outer scale)."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
    x = lut[torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).int()]
    s = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _place(cache, slots):
    """Where the tokens of `slots` are in the fields of an MX4 cache."""
    bs = cache.shape[2] * 16
    blk, off = slots // bs, slots % bs
    return blk, slice(None), off // 16, off % 16


def _store(st, slots, k, v):
    """fp32 rows [T, Hkv, D] into the cache in its type."""
    kind, D = st["kind"], k.shape[-1]
    if kind == "mx4":
        at = _place(st["k_cache"], slots)
        kc, ks, vc, vs = _fields(st["k_cache"], D)
        for x, scale, fc, fs in ((k, st["k_scale"], kc, ks), (v, st["v_scale"], vc, vs)):
            c, s = _mx4_codes(x, scale)
            fc[at] = c[..., 0::2] | (c[..., 1::2] << 4)
            fs[at] = s.view(torch.uint8)
        return
    for x, scale, cache in ((k, st["k_scale"], st["k_cache"]), (v, st["v_scale"], st["v_cache"])):
        flat = cache.view(-1, *cache.shape[-2:])
        if kind == "int8":
            flat[slots] = (x / scale).round().clamp(-127, 127).to(torch.int8)
        elif kind == "e4m3":
            flat.view(torch.uint8)[slots] = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            flat[slots] = x.half()


def _rows(st, slots):
    """The cache's rows at slots [...], as fp32 values [..., Hkv, D] with their scales."""
    if st["kind"] == "mx4":
        at = _place(st["k_cache"], slots.reshape(-1))
        kc, ks, vc, vs = (f[at] for f in _fields(st["k_cache"], st["D"]))
        k, v = _mx4_values(kc, ks) * st["k_scale"], _mx4_values(vc, vs) * st["v_scale"]
        return k.unflatten(0, slots.shape), v.unflatten(0, slots.shape)
    if st["kind"] == "fp16":
        return tuple(st[c].view(-1, *st[c].shape[-2:])[slots].float() for c in ("k_cache", "v_cache"))
    return tuple(st[c].view(-1, *st[c].shape[-2:]).view(torch.uint8)[slots].view(st[c].dtype).float() * st[s]
                 for c, s in (("k_cache", "k_scale"), ("v_cache", "v_scale")))


def _plain_append(st):
    q = _rotate(_normed(st["q"], st["q_weight"]), st["cs"], st["positions"], st["interleaved"]).half()
    k = _rotate(_normed(st["k"], st["k_weight"]), st["cs"], st["positions"], st["interleaved"])
    _store(st, st["slots"].long(), k, st["v"].float())
    return q, k.half()


def _plain_attention(st, q, k, v):
    """q [T, Hq, D] packed; k, v [B, L, Hkv, D] fp32, padded at the end -> [T, Hq, D]."""
    lens, starts = st["lens"].long(), st["starts"].long()
    T, Hq, D = q.shape
    B, L, Hkv, _ = k.shape
    n = starts[1:] - starts[:-1]
    N = st["longest"]
    i = torch.arange(N, device=q.device)
    real = i[None, :] < n[:, None]  # [B, N]
    src = torch.where(real, starts[:-1, None] + i, 0)
    x = q[src].float().unflatten(2, (Hkv, -1)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)  # [B, Hkv, G N, D]
    s = torch.matmul(x, k.permute(0, 2, 3, 1)).mul_(st["sigma"])
    if st["softcap"] > 0:
        s = s.div_(st["softcap"]).tanh_().mul_(st["softcap"])
    s = s.unflatten(2, (-1, N))  # [B, Hkv, G, N, L]
    p = (lens - n)[:, None] + i  # positions of the new tokens
    t = torch.arange(L, device=q.device)
    dead = t[None, None, :] > p[:, :, None]
    if st["window"] >= 0:
        dead |= t[None, None, :] < p[:, :, None] - st["window"]
    s.masked_fill_(dead[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    e = s.sub_(m).exp_()
    l = e.sum(-1, keepdim=True)
    if st["sink"] is not None:
        l = l + torch.exp(st["sink"].view(1, Hkv, -1, 1, 1) - m) * (l > 0)
    o = torch.matmul(e.flatten(2, 3), v.transpose(1, 2)).unflatten(2, (-1, N)) / torch.where(l > 0, l, 1.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, N, Hq, D)[real].half()


def _padded(x, starts, longest):
    """Packed rows [T, H, D] -> [B, longest, H, D] fp32, padded with row 0's."""
    starts = starts.long()
    i = torch.arange(longest, device=x.device)
    at = starts[:-1, None] + i
    return x[torch.where(at < starts[1:, None], at, 0)].float()


def _plain_paged(st, q):
    t = torch.arange(st["table"].shape[1] * BLOCK, device=q.device)
    slots = st["table"].clamp(min=0).long()[:, t // BLOCK] * BLOCK + t % BLOCK
    return _plain_attention(st, q, *_rows(st, slots))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _angles(max_pos, R, device):
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=device) / R)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat((a.cos(), a.sin()), dim=1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, Hq, Hkv, D = case["op"], case["Hq"], case["Hkv"], case["D"]
    kind, pc = case.get("kind", "fp16"), case.get("per_channel", False)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    # channel amplitudes: some channels are several times larger than others where the scales are per channel
    amp_k, amp_v = (torch.exp((torch.rand((Hkv, D), generator=g, device=dev) * 2 - 1) * math.log(2.0)) if pc
                    else torch.ones((Hkv, D), device=dev) for _ in range(2))
    # scales as calibration gives them: the amplitude of each channel (or of all) over what the cache type holds
    top = {"int8": 4.5 / 127, "e4m3": 4.5 / 448, "mx4": 1.0, "fp16": 1.0}[kind]
    scale = [None if kind == "fp16" else (a * top).contiguous() if pc else torch.full((1,), top, device=dev)
             for a in (amp_k, amp_v)]
    st = dict(op=op, kind=kind, D=D, k_scale=scale[0], v_scale=scale[1], scale_kind=PER_CHANNEL if pc else PER_TENSOR)

    def rows(T):
        """New rows as one projection leaves them: q, k and v side by side, [T, (Hq + 2 Hkv) D]."""
        qkv = torch.empty((T, (Hq + 2 * Hkv) * D), dtype=torch.float16, device=dev)
        st["q"], st["k"], st["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split((Hq * D, Hkv * D, Hkv * D), dim=1))
        st["q"].copy_(randn(T, Hq, D))
        st["k"].copy_(randn(T, Hkv, D) * amp_k)
        st["v"].copy_(randn(T, Hkv, D) * amp_v)

    def cache(blocks):
        if kind == "mx4":
            st["k_cache"], st["v_cache"] = torch.zeros((blocks, Hkv, BLOCK // 16, 18 * D), dtype=torch.uint8, device=dev), None
        else:
            dt = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn, "fp16": torch.float16}[kind]
            raw = torch.float16 if kind == "fp16" else torch.uint8
            st["k_cache"], st["v_cache"] = (torch.zeros((blocks, BLOCK, Hkv, D), dtype=raw, device=dev).view(dt)
                                            for _ in range(2))

    def norm_inputs(max_pos):
        # the norm brings every head to about one per channel, and its weight to the channel's amplitude
        st["q_weight"], st["k_weight"] = 1.0 + 0.1 * randn(D), (1.0 + 0.1 * randn(D)) * amp_k[0]
        st["cs"], st["interleaved"] = _angles(max_pos, case["R"], dev), case["interleaved"]

    if op == "norm":
        T = case["T"]
        rows(T)
        blocks = -(-T // BLOCK) + 2
        cache(blocks)
        norm_inputs(case["max_pos"])
        if case["chunked"]:  # consecutive positions; consecutive tokens fill scattered blocks
            p0 = int(torch.randint(0, case["max_pos"] - T + 1, (1,), generator=g, device=dev))
            st["positions"] = torch.arange(p0, p0 + T, device=dev, dtype=torch.int32)
            table, t = torch.randperm(blocks, generator=g, device=dev), torch.arange(T, device=dev)
            st["slots"] = (table[t // BLOCK] * BLOCK + t % BLOCK).int()
        else:  # one token of each of T sequences
            st["positions"] = torch.randint(0, case["max_pos"], (T,), generator=g, device=dev, dtype=torch.int32)
            st["slots"] = torch.randperm(blocks * BLOCK, generator=g, device=dev)[:T].int()
        return st
    lens, new = _lens(case)
    T = sum(new)
    rows(T)
    st.update(lens=torch.tensor(lens, dtype=torch.int32, device=dev), sigma=D ** -0.5, window=case["window"],
              starts=torch.tensor([0] + new, device=dev).cumsum(0).int(), longest=max(new), softcap=case["softcap"],
              sink=randn(Hq) if case["sink"] else None)
    if op == "packed":
        return st
    # B sequences over a pool of randomly placed blocks
    need = [-(-n // BLOCK) for n in lens]
    pool = sum(need)
    cache(pool)
    step = 4096  # blocks filled at a time
    for b in range(0, pool, step):
        n = min(step, pool - b) * BLOCK
        _store(st, torch.arange(b * BLOCK, b * BLOCK + n, device=dev), randn(n, Hkv, D) * amp_k, randn(n, Hkv, D) * amp_v)
    table = torch.full((case["B"], max(need)), -1, dtype=torch.int32, device=dev)
    owner = torch.arange(max(need), device=dev)[None, :] < torch.tensor(need, device=dev)[:, None]
    table[owner] = torch.randperm(pool, generator=g, device=dev).int()
    st.update(table=table, workspace=torch.empty(SCRATCH // 4, dtype=torch.float32, device=dev))
    if op == "paged":
        st["q"] = st["q"].contiguous()
        return st
    norm_inputs(case["hi"])
    seq = torch.repeat_interleave(torch.arange(case["B"], device=dev), torch.tensor(new, device=dev))
    p = torch.arange(T, device=dev) - st["starts"].long()[seq] + (st["lens"].long() - torch.tensor(new, device=dev))[seq]
    st["positions"] = p.int()
    st["slots"] = (table[seq, p // BLOCK].long() * BLOCK + p % BLOCK).int()
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    st = state
    if own:
        import int8_kv_cache_gb300 as K

        if st["op"] == "packed":
            return K.packed_prefill(st["q"], st["k"], st["v"], st["starts"], st["sigma"], st["sink"], softcap=st["softcap"],
                                    window=st["window"])
        q = st["q"]
        if st["op"] in ("norm", "step"):
            q, k = K.norm_rope_and_cache(q, st["k"], st["v"], st["q_weight"], st["k_weight"], EPS, st["positions"], st["cs"],
                                         st["slots"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"],
                                         st["scale_kind"], interleaved=st["interleaved"], return_keys=st["op"] == "norm")
        if st["op"] == "norm":
            return (q, k) + K.gather_cache(st["slots"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"],
                                           st["scale_kind"])
        out = K.paged_prefill(q, st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["scale_kind"], st["table"],
                              st["lens"], st["starts"], st["sigma"], st["sink"], workspace=st["workspace"],
                              softcap=st["softcap"], window=st["window"])
        return (q, out) if st["op"] == "step" else out
    if st["op"] == "packed":
        return _plain_attention(st, st["q"], *(_padded(x, st["starts"], st["longest"]) for x in (st["k"], st["v"])))
    if st["op"] == "paged":
        return _plain_paged(st, st["q"])
    q, k = _plain_append(st)
    if st["op"] == "step":
        return q, _plain_paged(st, q)
    return (q, k) + tuple(x.half() for x in _rows(st, st["slots"].long()))


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _grid_round(x, mant, emin, top):
    """Nearest value with `mant` mantissa bits after the leading one, exponents >= emin, magnitude <= top."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=emin).double() - mant)
    return (torch.round(x / step) * step).clamp(-top, top)


def _exact_head(x, weight, positions, R, interleaved):
    x = x.double()
    x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()
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

    k, ks = e2m1(nibbles(at(0, 8 * D, (16, D // 2)))), e4m3(at(8 * D, D, (16, D // 16)))
    v, vs = e2m1(nibbles(at(9 * D, 8 * D, (16, D // 2)))), e4m3(at(17 * D, D, (16, D // 16)))
    return k * ks.repeat_interleave(16, -1), v * vs.repeat_interleave(16, -1)


def _exact_context(st, b, L, Hkv):
    """Sequence b's keys and values [L, Hkv, D] in 64 bits, from the cache."""
    D, blocks = st["D"], st["table"][b, :-(-L // BLOCK)].long()
    if st["kind"] == "mx4":
        k, v = (x.permute(0, 2, 3, 1, 4).reshape(-1, Hkv, D)[:L] for x in _exact_record(st["k_cache"][blocks], D))
    else:
        raw = torch.float16 if st["kind"] == "fp16" else torch.uint8
        k, v = (st[c].view(raw)[blocks].view(st[c].dtype).double().reshape(-1, Hkv, D)[:L] for c in ("k_cache", "v_cache"))
    if st["kind"] != "fp16":
        k, v = k * st["k_scale"].double().reshape(-1, 1 if st["k_scale"].numel() == 1 else D), \
            v * st["v_scale"].double().reshape(-1, 1 if st["v_scale"].numel() == 1 else D)
    return k, v


def _exact_attention(st, q, lens, new, context):
    """q [T, Hq, D] in 64 bits; context(b) gives sequence b's keys and values [L, Hkv, D]."""
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    first = 0
    for b, (L, n) in enumerate(zip(lens, new)):
        k, v = context(b)
        G = q.shape[1] // k.shape[1]
        some = max(1, (1 << 27) // (L * G))  # tokens at a time
        for i in range(0, n, some):
            m = min(some, n - i)
            hi = L - n + i + m  # no token of these attends further
            pos = torch.arange(hi - m, hi, device=q.device)[:, None]
            t = torch.arange(hi, device=q.device)[None, :]
            seen = (t <= pos) & (t >= pos - st["window"]) if st["window"] >= 0 else t <= pos
            for h in range(q.shape[1]):
                s = q[first + i:first + i + m, h] @ k[:hi, h // G].T * st["sigma"]
                if st["softcap"] > 0:
                    s = st["softcap"] * torch.tanh(s / st["softcap"])
                s = torch.where(seen, s, -math.inf)
                lse = torch.logsumexp(s, -1, keepdim=True)
                if st["sink"] is not None:
                    lse = torch.logaddexp(lse, st["sink"][h].double())
                out[first + i:first + i + m, h] = torch.exp(s - lse) @ v[:hi, h // G]
        first += n
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "step"):
        q = _exact_head(st["q"], st["q_weight"], st["positions"], case["R"], case["interleaved"])
        k = _exact_head(st["k"], st["k_weight"], st["positions"], case["R"], case["interleaved"])
        ks, vs = _exact_stored(k, st["k_scale"], st["kind"]), _exact_stored(st["v"].double(), st["v_scale"], st["kind"])
    if op == "norm":
        return q, k, ks, vs
    lens, new = _lens(case)
    first = [sum(new[:b]) for b in range(len(new))]

    def context(b):
        n, L = new[b], lens[b]
        if op == "packed":
            return tuple(st[x][first[b]:first[b] + n].double() for x in ("k", "v"))
        k, v = _exact_context(st, b, L, case["Hkv"])
        if op == "step":
            k[L - n:], v[L - n:] = ks[first[b]:first[b] + n], vs[first[b]:first[b] + n]
        return k, v

    if op == "step":  # a query is attended as it leaves the append: rounded to fp16
        return q, _exact_attention(st, q.half().double(), lens, new, context)
    return _exact_attention(st, st["q"].double(), lens, new, context)
