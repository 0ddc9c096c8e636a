"""Causal attention of new tokens in 64 bits, with the bounds that the kernels' roundings give, and caches of
random codes together with the values that they stand for.  Plain torch, row by row from the definition."""
import math

import torch

import oracle.mx4 as mx4

KINDS = ["int8", "e4m3", "fp16", "mx4"]


def attend64(q, starts, lens, context, sigma, window=-1, softcap=0.0, sink=None):
    """q [T, Hq, D]; starts [B + 1], lens [B] (lists); context(b) -> keys, values [L, Hkv, D] in 64 bits, and a
    truth value for each position that may be attended (or None).  Returns out [T, Hq, D], lse [T, Hq] (rows of
    no sequence: NaN), and for the bounds spread[T, Hq, D] = the weighted mean of |V| and terms[T, Hq] =
    max_t sigma sum_d |q_d K[t, d]|."""
    T, Hq, D = q.shape
    nan = math.nan
    out = torch.full((T, Hq, D), nan, dtype=torch.float64, device=q.device)
    lse, spread = out[..., 0].clone(), out.clone()
    terms = torch.zeros_like(lse)
    for b, L in enumerate(lens):
        s0, n = starts[b], starts[b + 1] - starts[b]
        if n == 0:
            continue
        k, v, ok = context(b)
        k, v = k[:L], v[:L]
        G = Hq // k.shape[1]
        pos = torch.arange(L - n, L, device=q.device)[:, None]
        t = torch.arange(L, device=q.device)[None, :]
        seen = t <= pos
        if window >= 0:
            seen &= t >= pos - window
        if ok is not None:
            seen &= ok[None, :L]
        for h in range(Hq):
            x = q[s0:s0 + n, h].double()
            kh, vh = k[:, h // G], v[:, h // G]
            s = sigma * (x @ kh.T)
            if softcap > 0:
                s = softcap * torch.tanh(s / softcap)
            s = torch.where(seen, s, -math.inf)
            m = s.amax(-1, keepdim=True) if L else torch.full((n, 1), -math.inf, dtype=torch.float64, device=q.device)
            some = seen.any(-1, keepdim=True)
            e = torch.where(seen, torch.exp(s - torch.where(some, m, 0.0)), 0.0)
            l = e.sum(-1, keepdim=True)
            w = e / torch.where(some, l, 1.0)
            # a value that is not finite reaches the rows that attend it alone
            fin = torch.isfinite(vh)
            o = w @ torch.where(fin, vh, 0.0)
            for t0 in (~fin.all(-1)).nonzero().flatten().tolist():
                hit = seen[:, t0]
                o[hit] += torch.where(fin[t0], 0.0, vh[t0])
            z = torch.where(some, m + torch.log(l), -math.inf)
            if sink is not None:
                o = torch.where(some, o * torch.sigmoid(z - sink[h].double()), o)
            out[s0:s0 + n, h], lse[s0:s0 + n, h] = o, z[:, 0]
            spread[s0:s0 + n, h] = w @ torch.where(fin, vh, 0.0).abs()
            a = torch.where(torch.isfinite(kh), kh, 0.0).abs()
            terms[s0:s0 + n, h] = torch.where(seen, sigma * (x.abs() @ a.T), 0.0).amax(-1) if L else 0.0
    return out, lse, spread, terms


def bounds(ref, D, longest, folds, softcap=0.0):
    """(|out - ref|, |lse - ref|) of attend64's answer: the output's rounding to fp16 (2^-11 of it, half a step of
    2^-24 below the smallest normal) and the probabilities' (2^-11 of each: of the mean of |V|); a score's error d
    moves its weight by e^d, and the mean by 2 d: 2^-11 of each term where a scale per channel is folded into fp16
    queries (twice 2^-12 where the sum of the terms is not aligned), and fp32's 2^-24 for the products' sum in
    D / 16 + 4 steps, truncated (2^-23 each), the exponent's argument (three roundings of at most the score's
    size) and 2^-22 of the exponential; the sums over the positions in longest / 16 steps of 2^-23, and another 2^-23
    for each of at most 8 rescalings and merges.  A cap's tanh adds four roundings of its size."""
    out, lse, spread, terms = ref
    d = terms * ((2.0 ** -11 if folds else 0.0) + (D / 16 + 4 + 3) * 2.0 ** -23) + softcap * 2.0 ** -21 + 2.0 ** -22
    sums = (longest / 16 + 8) * 2.0 ** -23
    fin = torch.where(torch.isfinite(out), out, 0.0).abs()
    o = 2.0 ** -11 * fin + spread * (2.0 ** -11 + sums + 2 * d[..., None]) * 1.01 + 2.0 ** -25
    return o, d + sums + 2.0 ** -22 * lse.abs().nan_to_num(0, 0, 0) + 2.0 ** -22


def check(got, got_lse, ref, bound, what=""):
    out, lse = ref[0], ref[1]
    live = ~torch.isnan(ref[2][..., 0])  # rows of some sequence
    g, r, b = got.double()[live], out[live], bound[0][live]
    odd = ~torch.isfinite(r)
    assert torch.equal(torch.isnan(g), torch.isnan(r)), f"{what}: NaN where none belongs, or none where one does"
    assert torch.equal(g[odd & ~torch.isnan(r)], r[odd & ~torch.isnan(r)]), f"{what}: infinities differ"
    err = ((g - r).abs() / b)[~odd]
    assert err.numel() == 0 or err.max() <= 1.0, f"{what}: an output is {err.max():.3f} times its bound off"
    if got_lse is not None:
        g, r, b = got_lse.double()[live], lse[live], bound[1][live]
        assert torch.equal(torch.isinf(g), torch.isinf(r)), f"{what}: empty rows differ"
        fin = torch.isfinite(r)
        err = ((g - r).abs() / b)[fin]
        assert err.numel() == 0 or err.max() <= 1.0, f"{what}: an lse is {err.max():.3f} times its bound off"


def cache_of(kind, g, blocks, bs, Hkv, D, per_channel):
    """A pool of random codes: the caches, scales and scale kind as the calls take them, and the values of its
    rows [blocks * bs, Hkv, D] in 64 bits."""
    dev = g.device

    def rand(*s):
        return torch.rand(s, generator=g, device=dev)

    shape = (Hkv, D) if per_channel else (1,)
    amp = {"int8": 1 / 40, "e4m3": 1 / 16, "mx4": 1.0, "fp16": 1.0}[kind]
    ks, vs = (torch.exp(rand(*shape) * 2 - 1) * amp for _ in range(2))
    c = dict(kind=kind, scale_kind=2 if per_channel else 1, ks=ks, vs=vs, bs=bs)
    if kind == "mx4":
        rec = torch.randint(0, 256, (blocks, Hkv, bs // 16, 18 * D), generator=g, device=dev, dtype=torch.uint8)
        for at in (8 * D, 17 * D):  # block scales 2^-2 .. 2
            rec[..., at:at + D] = torch.randint(40, 57, (blocks, Hkv, bs // 16, D), generator=g, device=dev, dtype=torch.uint8)
        c.update(kc=rec, vc=None)
    elif kind == "int8":
        c.update({x: torch.randint(-128, 128, (blocks, bs, Hkv, D), generator=g, device=dev, dtype=torch.int8) for x in ("kc", "vc")})
    else:
        dt = torch.float16 if kind == "fp16" else torch.float8_e4m3fn
        x = [torch.randn((blocks, bs, Hkv, D), generator=g, device=dev) * (1 if kind == "fp16" else 16) for _ in range(2)]
        c.update(kc=x[0].to(dt), vc=x[1].to(dt))
    if kind == "fp16":
        c.update(ks=None, vs=None)
    return c


def values(c):
    """K and V of a pool's rows in 64 bits, scales applied."""
    if c["kind"] == "mx4":
        rec = c["kc"].cpu().numpy()
        nb, Hkv, tiles, _ = rec.shape
        D = rec.shape[3] // 18

        def part(at):
            codes = torch.from_numpy(mx4.e2m1_value(mx4.unpack(rec[..., at:at + 8 * D].reshape(nb, Hkv, tiles, 16, D // 2))))
            b = rec[..., at + 8 * D:at + 9 * D].reshape(nb, Hkv, tiles, 16, D // 16)
            s = torch.from_numpy(mx4.e4m3_values(b & 127)).masked_fill(torch.from_numpy((b & 127) == 127), math.nan)
            x = codes * s.repeat_interleave(16, -1)
            return x.permute(0, 2, 3, 1, 4).reshape(-1, Hkv, D).to(c["kc"].device)
        k, v = part(0), part(9 * D)
    else:
        k, v = (c[x].double().flatten(0, 1) for x in ("kc", "vc"))
        if c["kind"] == "fp16":
            return k, v
    return k * c["ks"].double(), v * c["vs"].double()


def tables(g, lens, bs, spare=3):
    """A block table of scattered blocks for sequences of these lengths (unused entries -1), and the pool's size."""
    need = [-(-n // bs) for n in lens]
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=g, device=g.device).int()
    t = torch.full((len(lens), max(max(need), 1) + 1), -1, dtype=torch.int32, device=g.device)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, pool


def context_of(c, table, k, v):
    """context(b) for attend64 over a pool's values."""
    bs = c["bs"]

    def context(b):
        t = torch.arange(table.shape[1] * bs, device=table.device)
        blk = table[b].long()[t // bs]
        ok = (blk >= 0) & (blk < k.shape[0] // bs)
        rows = torch.where(ok, blk, 0) * bs + t % bs
        return k[rows], v[rows], ok
    return context
