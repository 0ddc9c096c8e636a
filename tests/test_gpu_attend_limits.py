"""paged_prefill and packed_prefill at the ends of what they accept, against the definition in 64 bits (attend64.py)."""
import math

import pytest
import torch

from attend64 import attend64, bounds, cache_of, check, context_of, tables, values
from test_gpu_attend import K, firsts, gen, ints, paged_case, projection, run_packed  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["int8", "mx4"])
@pytest.mark.parametrize("bs", [16, 128])
@pytest.mark.parametrize("splits", [1, 3])
def test_a_sequence_that_ends_just_below_2_31(K, kind, bs, splits):
    """The longest context there is: a table that repeats a few pages, and a window, so that little is attended.  Steps
    over pages that go past its end must not wrap (nor read the table in front of it)."""
    blocks = (2 ** 31 - 1 - 512) // bs
    L, D, Hq, n, window = blocks * bs, 64, 4, 5, 1000
    g = gen(60)
    c = cache_of(kind, g, 7, bs, 1, D, True)
    table = torch.randint(0, 7, (1, blocks), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn((n, Hq, D), generator=g, device="cuda").half()
    out, lse = torch.empty_like(q), torch.empty((n, Hq), device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    nbytes = K.paged_prefill_workspace_bytes(n, 1, Hq, 1, D, L, splits)
    space = torch.full((max(nbytes // 4, 4),), math.nan, device="cuda")
    K.paged_prefill(q, c["kc"], c["vc"], c["ks"], c["vs"], 2, table, ints([L]), ints([0, n]), 0.125, num_splits=splits,
                    workspace=space, out=out, lse=lse, flags=flags, window=window)
    torch.cuda.synchronize()
    assert int(flags) == 0
    # the window's pages alone: the same distances between positions
    tail = -(-(window + n) // bs) * bs
    t = torch.arange(tail, device="cuda")
    rows = table[0, blocks - tail // bs:].long()[t // bs] * bs + t % bs
    k, v = values(c)
    ref = attend64(q, [0, n], [tail], lambda b: (k[rows], v[rows], None), 0.125, window)
    check(out, lse, ref, bounds(ref, D, window, True), kind)


@pytest.mark.parametrize("kind", ["int8", "fp16"])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 2, 2), (128, 3, 1), (256, 2, 1)])
def test_pieces_that_hold_nothing_for_some_lanes_of_a_warp(K, kind, D, Hq, Hkv):
    """A narrow window, blocks that begin inside a warp's 32 vectors, last vectors of a tile that are not there: the
    lanes of a warp write their partials, or nothing, side by side."""
    for window in (0, 3):
        for lens, new in (([403], [200]), ([403, 77], [19, 70])):
            paged_case(K, kind, 61, lens, new, Hq, Hkv, D, splits=9, window=window)


def capped_bounds(ref, D, starts, lens, context, cap):
    """Those of scores without a cap, and a cap's own error relative to the score: its series is cut off at 2^-21.5 and
    has four roundings; beyond a quarter of the cap c, tanh is above 0.2449 and 2^-21 of c off at most (the exponential
    and the reciprocal 2^-22 and 2^-23, of a slope of at most 1/2 and 1; four roundings): 2^-18.9 of the score.  Caps up to
    128 are taken so for all scores: 2^-21 of the cap.
    Scores of some tens leave weights far below the largest one, w = 1 (so the sum of all is 1 at least).  They are held
    as fp16 numbers w 2^8 or larger ones, whose half steps below the smallest normal are 2^-25: 2^-33 of the largest
    weight for each value attended.  (It shows where the values of the large weights are zeros.)"""
    o, z = bounds(ref, D, max(lens), False)
    d = ref[3] * 2.0 ** -18.9 + (cap * 2.0 ** -21 if cap <= 128 else 0.0)
    o = o + ref[2] * 2 * d[..., None] * 1.01
    for b, L in enumerate(lens):
        v = context(b)[1][:L].abs().sum(0)
        rows = slice(starts[b], starts[b + 1])
        o[rows] += 2.0 ** -33 * v.repeat_interleave(o.shape[1] // v.shape[0], 0)
    return o, z + d


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap", [0.25, 4.0, 30.0, 128.0, 300.0, 1e4, 1e5, 1e6, 3e38])
def test_caps_small_and_far_above_the_scores(K, D, cap):
    """c tanh(s / c) is s where c is far above it."""
    g = gen(62)
    new = [300, 45]
    starts = firsts(new)
    q, k, v = projection(g, starts[-1], 4, 2, D)
    q = q * 8  # scores of some tens
    ctx = lambda b: (k[starts[b]:starts[b + 1]].double(), v[starts[b]:starts[b + 1]].double(), None)  # noqa: E731,B023
    ref = attend64(q, starts, new, ctx, D ** -0.5, softcap=cap)
    out, lse = run_packed(K, q, k, v, starts, D ** -0.5, softcap=cap)
    check(out, lse, ref, capped_bounds(ref, D, starts, new, ctx, cap))
    lens, new, bs = [400, 300, 77], [70, 1, 3], 16
    starts = firsts(new)
    for kind in ("int8", "mx4"):
        table, pool = tables(g, lens, bs)
        c = cache_of(kind, g, pool, bs, 2, D, False)
        q = (torch.randn((starts[-1], 4, D), generator=g, device="cuda") * 4).half()
        ctx = context_of(c, table, *values(c))
        ref = attend64(q, starts, lens, ctx, D ** -0.5, softcap=cap)
        for splits in (1, 5):
            out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
            n = K.paged_prefill_workspace_bytes(starts[-1], 3, 4, 2, D, table.shape[1] * bs, splits)
            K.paged_prefill(q, c["kc"], c["vc"], c["ks"], c["vs"], 1, table, ints(lens), ints(starts), D ** -0.5,
                            num_splits=splits, workspace=torch.empty(n // 4 + 4, device="cuda"), out=out, lse=lse, softcap=cap)
            check(out, lse, ref, capped_bounds(ref, D, starts, lens, ctx, cap), kind)
