"""paged_prefill and packed_prefill at the ends of what they accept, against the definition in 64 bits (attend64.py)."""
import math

import pytest
import torch

from attend64 import attend64, bounds, cache_of, check, values
from test_gpu_attend import K, gen, ints, paged_case  # noqa: F401

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
