"""The oracle of the 4-bit cache and the rotating append, pinned by hand cases and
by independent forms (no GPU)."""
import numpy as np
import pytest

import oracle


def test_e2m1_codes_and_ties():
    vals = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert oracle.e2m1_value(np.arange(8)).tolist() == vals
    assert oracle.e2m1_value(np.arange(8, 16)).tolist() == [-v for v in vals]
    for c, v in enumerate(vals):
        assert oracle.e2m1_encode(v) == c and (c == 0 or oracle.e2m1_encode(-v) == c + 8)
    # half-way points go to the even code
    for v, c in ((0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)):
        assert oracle.e2m1_encode(v) == c
        below, above = oracle.e2m1_encode(np.nextafter(v, 0)), oracle.e2m1_encode(np.nextafter(v, 9))
        assert above == below + 1 and c in (below, above) and c % 2 == 0
    assert oracle.e2m1_encode(1e30) == 7 and oracle.e2m1_encode(-np.inf) == 15
    # nearest: no other value is nearer
    x = np.random.default_rng(0).uniform(-7, 7, 4000)
    got = oracle.e2m1_value(oracle.e2m1_encode(x))
    grid = np.array(vals + [-v for v in vals])
    best = np.abs(np.clip(x, -6, 6)[:, None] - grid).min(1)
    np.testing.assert_allclose(np.abs(got - np.clip(x, -6, 6)), best, atol=1e-12)


def test_mx4_row_by_hand():
    x = np.zeros(32, np.float32)
    x[:16] = [6, -6, 3, 1, 0.5, 0, 2.4, 2.6, 5, -5, 4.9, 5.1, 0.2, -0.3, 1.5, 1.25]
    x[16:] = 1e-5  # max / 6 rounds to a scale of 0: the block is stored as zeros
    codes, s = oracle.mx4_encode(x, np.ones(32, np.float32))
    assert s.tolist() == [0x38, 0]  # 1.0 and 0
    assert oracle.e2m1_value(codes[:16]).tolist() == [6, -6, 3, 1, .5, 0, 2, 3, 4, -4, 4, 6, 0, -.5,
                                                      1.5, 1]
    assert not codes[16:].any()
    x[3], x[5] = np.nan, np.inf
    codes, s = oracle.mx4_encode(x, np.ones(32, np.float32))
    assert s[0] == 0x7E and codes[3] == 0 and codes[5] == 7


def test_mx4_store_and_read_back():
    rng = np.random.default_rng(1)
    D, Hkv = 64, 2
    cache = rng.integers(0, 256, (3, Hkv, 2, 18 * D)).astype(np.uint8)
    before = cache.copy()
    x = rng.standard_normal((2, D)).astype(np.float32)
    kc, ksc = oracle.mx4_encode(x[0], np.ones(D, np.float32))
    vc, vsc = oracle.mx4_encode(x[1], np.ones(D, np.float32))
    slot = 1 * 32 + 21  # block 1, record 1, token 5
    oracle.mx4_store(cache, slot, 1, False, kc, ksc)
    oracle.mx4_store(cache, slot, 1, True, vc, vsc)
    k, v = oracle.mx4_row(cache, slot, 1)
    assert np.abs(k - x[0]).max() <= np.abs(x[0]).max() / 6 * 1.1
    assert np.abs(v - x[1]).max() <= np.abs(x[1]).max() / 6 * 1.1
    changed = np.argwhere(cache != before)
    assert set(map(tuple, changed[:, :3])) == {(1, 1, 1)}
    # bytes of token 5 only: codes at 5 D/2, scales at 8D + 5 D/16, values 9D further
    ok = set()
    for base in (0, 9 * D):
        ok |= set(range(base + 5 * D // 2, base + 6 * D // 2))
        ok |= set(range(base + 8 * D + 5 * D // 16, base + 8 * D + 6 * D // 16))
    assert set(changed[:, 3]) <= ok


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(2)
    D, R, T = 64, 32, 5
    x = rng.standard_normal((T, 3, D)).astype(np.float16)
    ang = rng.uniform(-3, 3, (40, R // 2))
    cs = np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)
    pos = rng.integers(0, 40, T)
    y = oracle.rotate(x, cs, pos, interleaved).astype(np.float64)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    z = x[..., a].astype(np.float64) + 1j * x[..., b]
    w = z * np.exp(1j * ang[pos])[:, None]
    np.testing.assert_allclose(y[..., a], w.real, atol=2e-6)
    np.testing.assert_allclose(y[..., b], w.imag, atol=2e-6)
    np.testing.assert_array_equal(y[..., R:], x[..., R:])


def test_attention_over_records_is_attention_over_their_values():
    rng = np.random.default_rng(3)
    D, Hkv, Hq, bs, nb = 64, 2, 4, 16, 6
    cache = np.zeros((nb, Hkv, 1, 18 * D), np.uint8)
    k = rng.standard_normal((nb * bs, Hkv, D)).astype(np.float32)
    v = rng.standard_normal((nb * bs, Hkv, D)).astype(np.float32)
    one = np.ones(1, np.float32)
    cache = oracle.mx4_append(cache, k, v, np.arange(nb * bs), one, one, 1)
    q = rng.standard_normal((1, Hq, D)).astype(np.float16)
    table = np.array([[4, 0, 2, -1]], np.int32)
    sink = rng.standard_normal(Hq).astype(np.float32)
    O, lse, W, _ = oracle.mx4_paged_attention(q, cache, one, one, 1, table, np.array([37]), 0.125,
                                              sink, window=20)
    slots = [int(table[0, t // 16]) * 16 + t % 16 for t in range(16, 37)]
    for h in range(Hq):
        rows = [oracle.mx4_row(cache, s, h // 2) for s in slots]
        K, V = np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])
        s = 0.125 * K @ q[0, h].astype(np.float64)
        p = np.exp(s)
        want = p @ V / (p.sum() + np.exp(float(sink[h])))
        np.testing.assert_allclose(O[0, h], want, rtol=1e-10, atol=1e-12)
        np.testing.assert_allclose(lse[0, h], np.log(p.sum()), rtol=1e-12)
    assert (W >= np.abs(O) - 1e-12).all()
