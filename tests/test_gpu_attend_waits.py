"""The dense causal attention where a copy or a hand-over does not come (tests/attend_withheld.cu: waits of 20 ms): the
kernel returns, nothing that was made of what did not come is given out as a result, and the flag tells."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

from attend64 import attend64, bounds, check
from test_gpu_attend import gen, ints

pytestmark = pytest.mark.gpu

NONE, Q, KEYS, VALUES, P0, P1 = -1, 0, 1, 2, 3, 4
F16, INT8 = 0, 1
TIMEOUT = 0x20


@pytest.fixture(scope="module")
def withheld(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from int8_kv_cache_gb300 import build
    # (its own copies of the launchers' statics: those of the library belong to other kernels of the same names)
    here = os.path.dirname(os.path.abspath(__file__))
    so = str(tmp_path_factory.mktemp("withheld") / "withheld.so")
    subprocess.run([build.nvcc()] + build.ARCH + ["-O3", "-std=c++17", "--expt-relaxed-constexpr", "-I",
                   os.path.join(build.ROOT, "include"), "-shared", "-Xcompiler", "-fPIC,-fvisibility=hidden,-fno-gnu-unique",
                   os.path.join(here, "attend_withheld.cu"), "-o", so], check=True, capture_output=True)
    f = ctypes.CDLL(so).attend_withheld
    i, p = ctypes.c_int, ctypes.c_void_p
    f.argtypes = [i] * 6 + [p] * 7 + [i] * 7 + [p] * 6
    f.restype = i
    return f


def at(x):
    return None if x is None else x.data_ptr()


class Prompt:
    """A prompt of 300 tokens, 3 heads, by one CTA: items by falling length, (the last tile, head 0), ..."""
    T, H = 300, 3

    def __init__(self, f, D, two):
        g = gen(70)
        self.f, self.D, self.two, self.M = f, D, two, 256 if two else 128
        self.q, self.k, self.v = (torch.randn((self.T, self.H, D), generator=g, device="cuda").half() for _ in range(3))
        self.tiles = -(-self.T // self.M)
        self.items = [(t, h) for t in reversed(range(self.tiles)) for h in range(self.H)]

    def run(self, what, item, block):
        out, lse = torch.full_like(self.q, 7.0), torch.full((self.T, self.H), 7.0, device="cuda")
        flags, starts = torch.zeros(1, dtype=torch.int32, device="cuda"), ints([0, self.T])
        torch.cuda.synchronize()
        assert self.f(what, item, block, F16, self.two, 0, at(self.q), at(self.k), at(self.v), None, None, None, at(starts),
                      self.T, 1, self.H, self.H, self.D, 0, 0, at(out), at(lse), at(flags), None, None, None) == 0
        return out, lse, int(flags)

    def rows(self, item):
        t, h = self.items[item]
        return slice(t * self.M, (t + 1) * self.M), h


@pytest.mark.parametrize("D,two", [(128, 1), (128, 0), (256, 0)])
def test_a_prompt(withheld, D, two):
    p = Prompt(withheld, D, two)
    clean = p.run(NONE, 0, 0)
    assert clean[2] == 0
    ref = attend64(p.q, [0, p.T], [p.T], lambda b: (p.k.double(), p.v.double(), None), 1 / 16)
    check(clean[0], clean[1], ref, bounds(ref, D, p.T, False))
    last = len(p.items) - 1
    for what in (KEYS, VALUES, Q, P0):
        for item in (0, last - 1, last):
            for block in {0, p.items[item][0] * (2 if two else 1)}:  # the first one, and a later one
                if what == Q and block:
                    continue
                out, lse, flags = p.run(what, item, block)
                where = f"{what}, item {item}, block {block}"
                assert flags == TIMEOUT, where
                for i in range(last + 1):
                    r, h = p.rows(i)
                    if i < item:
                        assert torch.equal(out[r, h], clean[0][r, h]) and torch.equal(lse[r, h], clean[1][r, h]), where
                    elif i == item and two and what == P0:  # (the other tile may have been done)
                        assert bool(out[r, h][:128].isnan().all() & lse[r, h][:128].isnan().all()), where
                    else:
                        assert bool(out[r, h].isnan().all() & lse[r, h].isnan().all()), where
    assert torch.equal(p.run(NONE, 0, 0)[0], clean[0])


def test_the_second_tile_alone(withheld):
    """Its rows are NaN and the flag is raised also where the first one had been written by then."""
    p = Prompt(withheld, 128, 1)
    clean = p.run(NONE, 0, 0)
    last = len(p.items) - 1
    for block in (0, 1):
        out, lse, flags = p.run(P1, last, block)
        assert flags == TIMEOUT
        r, h = p.rows(last)
        assert bool(out[r, h][128:].isnan().all() & lse[r, h][128:].isnan().all())
        first = out[r, h][:128]
        done = ~first.isnan().any(-1)
        assert torch.equal(first[done], clean[0][r, h][:128][done])


@pytest.mark.parametrize("two", [0, 1])
@pytest.mark.parametrize("pieces", [0, 3])
def test_a_quantised_cache(withheld, two, pieces):
    """Whole, rows are NaN; in pieces, the partials say so: a maximum of infinity and a sum that is NaN."""
    L, n, D = 700, 64, 128
    g = gen(71)
    blocks = -(-L // 16)
    k, v = (torch.randint(-128, 128, (blocks, 16, 1, D), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    scale, table = torch.full((1,), 0.02, device="cuda"), torch.randperm(blocks, generator=g, device="cuda").int()
    q = torch.randn((n, 1, D), generator=g, device="cuda").half()
    M = 256 if two else 128
    lens, starts = ints([L]), ints([0, n])

    def run(what, block):
        out, lse = torch.full_like(q, 7.0), torch.full((n, 1), 7.0, device="cuda")
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        acc = torch.full((2 * max(pieces, 1), M, D), 7.0, device="cuda")
        m, l = (torch.full((2 * max(pieces, 1), M), 7.0, device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        assert withheld(what, 0, block, INT8, two, pieces, at(q), at(k), at(v), at(scale), at(table), at(lens), at(starts), n,
                        1, 1, 1, D, blocks, blocks, at(out), at(lse), at(flags), at(acc), at(m), at(l)) == 0
        return out, lse, int(flags), m, l

    out, lse, flags, m, l = run(NONE, 0)
    assert flags == 0 and (pieces > 0 or bool(out.isfinite().all()))
    for what in (KEYS, VALUES, Q, P0):
        for block in (0, 1) if what != Q else (0,):
            out, lse, flags, m, l = run(what, block)
            assert flags == TIMEOUT, (what, block)
            if pieces == 0:
                assert bool(out.isnan().all() & lse.isnan().all()), (what, block)
            else:
                for s in (1, 2, 4):
                    assert bool((m[s, :n] == math.inf).all() & l[s, :n].isnan().all()), (what, block, s)
