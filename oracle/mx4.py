"""The 4-bit cache, the position rotation and the rotating append, in plain NumPy.

TEST INFRASTRUCTURE ONLY (see ``oracle/attention.py``).

A record of 18 D bytes holds 16 tokens of one KV head: K codes [16, D / 2] (e2m1,
the even channel in the low nibble), K block scales [16, D / 16] (e4m3fn), V codes
and V block scales likewise.  What the append stores is fixed by fp32 operations
that are each rounded once, so it is compared bit for bit; attention over the cache
is evaluated in 64 bits.
"""
from __future__ import annotations

import numpy as np

from .attention import attend, apply_head_sink, live_length, window_start, _sink_of
from .quantize import e4m3fn_encode

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
_F1 = np.float32(1.0)


def e2m1_value(code):
    """Values of codes 0 .. 15 (bit 3: sign)."""
    c = np.asarray(code)
    return np.where(c & 8, -E2M1[c & 7], E2M1[c & 7])


def e2m1_encode(v):
    """Nearest code of each value, ties to the even code, saturated to +-6."""
    v = np.asarray(v, np.float64)
    a = np.minimum(np.abs(v), 6.0)
    hi = np.clip(np.searchsorted(E2M1, a, side="left"), 1, 7)  # E2M1[hi - 1] < a <= E2M1[hi]
    lo = hi - 1
    dl, dh = a - E2M1[lo], E2M1[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def e4m3_values(b):
    """Values of non-negative e4m3fn bytes."""
    b = np.asarray(b).astype(np.int64)
    e, m = b >> 3, b & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def _scale_of(scale, scale_kind, g, D):
    s = np.asarray(scale, np.float32)
    return np.broadcast_to(s.reshape(-1)[0], (D,)) if scale_kind == 1 else s[g]


def mx4_encode(x, scale):
    """(codes [D], scale bytes [D / 16]) of one row x [D] (fp32), scale [D]."""
    with np.errstate(all="ignore"):
        y = (np.asarray(x, np.float32) * (_F1 / np.asarray(scale, np.float32))).astype(np.float32)
        y = np.where(np.isnan(y), np.float32(0), y).reshape(-1, 16)
        amax = np.abs(y).max(-1)
        t = (amax * np.float32(1.0 / 6.0)).astype(np.float32)
        sb = np.array([e4m3fn_encode(float(v)) for v in t], np.uint8)
        sv = e4m3_values(sb).astype(np.float32)
        r = np.where(sv > 0, _F1 / np.where(sv > 0, sv, _F1), np.float32(0)).astype(np.float32)
        q = np.where(sv[:, None] > 0, (y * r[:, None]).astype(np.float32), np.float32(0))
    return e2m1_encode(q).reshape(-1), sb


def pack(codes):
    c = np.asarray(codes, np.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def unpack(b):
    b = np.asarray(b, np.uint8)
    return np.stack((b & 15, b >> 4), axis=-1).reshape(*b.shape[:-1], -1)


def mx4_row(cache, slot, g):
    """(K, V) [D] in 64 bits of one slot and KV head of a cache [num_blocks, Hkv,
    block_size / 16, 18 D], outer scales not applied."""
    nb, Hkv, tiles, rec = cache.shape
    D, bs = rec // 18, 16 * tiles
    blk, off = divmod(int(slot), bs)
    r, t = cache[blk, g, off // 16], off % 16
    out = []
    for base in (0, 9 * D):
        codes = unpack(r[base + t * (D // 2): base + (t + 1) * (D // 2)])
        sc = r[base + 8 * D + t * (D // 16): base + 8 * D + (t + 1) * (D // 16)]
        out.append(e2m1_value(codes) * np.repeat(e4m3_values(sc), 16))
    return out


def mx4_store(cache, slot, g, v_part, codes, scales):
    """Write one row (K, or V with v_part) into the cache, in place."""
    nb, Hkv, tiles, rec = cache.shape
    D, bs = rec // 18, 16 * tiles
    blk, off = divmod(int(slot), bs)
    r, t, base = cache[blk, g, off // 16], off % 16, 9 * D if v_part else 0
    r[base + t * (D // 2): base + (t + 1) * (D // 2)] = pack(codes)
    r[base + 8 * D + t * (D // 16): base + 8 * D + (t + 1) * (D // 16)] = scales


def rotate(x, cos_sin, positions, interleaved):
    """x [T, H, D] turned by the angles of its positions; fp32, each product and
    sum rounded once."""
    x = np.asarray(x).astype(np.float32).copy()
    if cos_sin is None:
        return x
    R = cos_sin.shape[1]
    h = R // 2
    for n, p in enumerate(positions):
        c, s = cos_sin[p, :h], cos_sin[p, h:]
        ia = np.arange(0, R, 2) if interleaved else np.arange(h)
        ib = ia + (1 if interleaved else h)
        a, b = x[n][:, ia].copy(), x[n][:, ib].copy()
        x[n][:, ia] = (a * c).astype(np.float32) - (b * s).astype(np.float32)
        x[n][:, ib] = (b * c).astype(np.float32) + (a * s).astype(np.float32)
    return x


def mx4_append(cache, k, v, slots, k_scale, v_scale, scale_kind):
    """Rows k, v [T, Hkv, D] (fp32, rotated) into a copy of the cache."""
    out = cache.copy()
    nb, Hkv, tiles, rec = out.shape
    D = rec // 18
    for n, slot in enumerate(slots):
        if slot < 0 or slot >= nb * tiles * 16:
            continue
        for g in range(Hkv):
            for part, x, sc in ((False, k, k_scale), (True, v, v_scale)):
                c, s = mx4_encode(x[n, g], _scale_of(sc, scale_kind, g, D))
                mx4_store(out, slot, g, part, c, s)
    return out


def mx4_paged_attention(q, cache, k_scale, v_scale, scale_kind, block_table, seq_lens, sigma,
                        sink=None, softcap=0.0, window=-1):
    """(O, lse, W, E) in 64 bits: outputs [B, Hq, D], log-sum-exps [B, Hq], and for
    tolerances W = sum_t p_t |v_t| [B, Hq, D] and E = max_t sigma sum_d |q_d K_t,d| [B, Hq].
    Positions of a block outside the cache are not attended."""
    B, Hq, D = q.shape
    nb, Hkv, tiles, _ = cache.shape
    bs, G = 16 * tiles, Hq // Hkv
    cap = block_table.shape[1] * bs
    O = np.zeros((B, Hq, D))
    W = np.zeros((B, Hq, D))
    lse = np.full((B, Hq), -np.inf)
    E = np.zeros((B, Hq))
    for b in range(B):
        L = live_length(int(seq_lens[b]), cap)
        pos = [t for t in range(window_start(L, window), L)
               if 0 <= block_table[b, t // bs] < nb]
        if not pos:
            continue
        for g in range(Hkv):
            rows = [mx4_row(cache, block_table[b, t // bs] * bs + t % bs, g) for t in pos]
            ks = _scale_of(k_scale, scale_kind, g, D).astype(np.float64)
            vs = _scale_of(v_scale, scale_kind, g, D).astype(np.float64)
            Km = np.stack([r[0] for r in rows]) * ks
            Vm = np.stack([r[1] for r in rows]) * vs
            for h in range(g * G, (g + 1) * G):
                qh = q[b, h].astype(np.float64)
                o, e = attend(qh, Km, Vm, sigma, softcap=softcap)
                s = sigma * (Km @ qh)
                E[b, h] = (sigma * (np.abs(Km) @ np.abs(qh))).max()
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                W[b, h] = np.exp(s - e) @ np.abs(Vm)
                lse[b, h] = e
                O[b, h] = apply_head_sink(o, e, _sink_of(sink, h))
    return O, lse, W, E
