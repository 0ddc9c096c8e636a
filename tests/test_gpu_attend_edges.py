"""packed_prefill and paged_prefill where they can go wrong: values that are no numbers, bad pages and lengths, rows that
attend nothing, long strides, streams, graphs, shared workspaces, and a run with norm_rope_and_cache; against 64 bits."""
import math

import pytest
import torch

from attend64 import KINDS, attend64, bounds, cache_of, check, context_of, tables, values
from test_gpu_attend import K, firsts, gen, ints, paged_case, projection, run_packed  # noqa: F401

pytestmark = pytest.mark.gpu


class Paged:
    """A batch over a pool of random codes; edit its parts, then run() and check()."""

    def __init__(self, kind, seed, lens, new, Hq, Hkv, D, bs=16, per_channel=True):
        g = self.g = gen(seed)
        self.kind, self.lens, self.new, self.D, self.bs, self.per_channel = kind, list(lens), list(new), D, bs, per_channel
        self.table, self.pool = tables(g, lens, bs)
        self.c = cache_of(kind, g, self.pool, bs, Hkv, D, per_channel)
        self.starts = firsts(new)
        self.q = torch.randn((self.starts[-1], Hq, D), generator=g, device="cuda").half()
        self.sigma = D ** -0.5

    def row(self, b, t):
        """(block, place in it) of position t of sequence b."""
        return int(self.table[b, t // self.bs]), t % self.bs

    def run(self, K, splits=0, ws=True, window=-1, softcap=0.0, lens=None, starts=None, flag=0, stream=None, **kw):
        c, T = self.c, self.q.shape[0]
        self.window, self.softcap = window, softcap
        out = torch.full(self.q.shape, 7.0, dtype=torch.float16, device="cuda")
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        Hq, Hkv = self.q.shape[1], c["kc"].shape[1 if self.kind == "mx4" else 2]
        nbytes = K.paged_prefill_workspace_bytes(T, len(self.lens), Hq, Hkv, self.D, self.table.shape[1] * self.bs, splits)
        space = torch.full((max(nbytes // 4, 4),), math.nan, device="cuda") if ws else None
        K.paged_prefill(self.q, c["kc"], c["vc"], c["ks"], c["vs"], c["scale_kind"], self.table, ints(lens or self.lens),
                        ints(starts or self.starts), self.sigma, num_splits=splits, workspace=space, out=out, lse=lse,
                        flags=flags, softcap=softcap, window=window, stream=stream, **kw)
        torch.cuda.synchronize()
        assert int(flags) == flag
        return out, lse

    def reference(self, starts=None):
        k, v = values(self.c)
        return attend64(self.q, starts or self.starts, self.lens, context_of(self.c, self.table, k, v), self.sigma, self.window,
                        self.softcap)

    def check(self, out, lse, starts=None):
        ref = self.reference(starts)
        folds = self.per_channel and self.kind != "fp16"
        check(out, lse, ref, bounds(ref, self.D, max(max(self.lens), 1), folds, self.softcap), self.kind)


def spoil(p, part, b, t, g, d, value=math.nan):
    """A value of a paged batch that is no number (fp16: the value given; MX4: the block scale of 16 channels)."""
    blk, r = p.row(b, t)
    if p.kind == "fp16":
        p.c[part][blk, r, g, d] = value
    elif p.kind == "e4m3":
        p.c[part].view(torch.uint8)[blk, r, g, d] = 0x7F if value == value else 0xFF
    else:
        at = (0 if part == "kc" else 9 * p.D) + 8 * p.D + (r % 16) * (p.D // 16) + d // 16
        p.c["kc"][blk, g, r // 16, at] = 0x7F


@pytest.mark.parametrize("kind", ["fp16", "e4m3", "mx4"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("splits", [1, 5])
def test_values_that_are_no_numbers(K, kind, D, splits):
    """In V: a masked one reaches no row, an attended one each row that attends it and none else."""
    for lens, new, Hq, Hkv in (([300, 40, 200], [90, 40, 1], 8, 2), ([400], [300], 8, 2)):
        p = Paged(kind, 20, lens, new, Hq, Hkv, D)
        for b, L in enumerate(lens):
            for t in {L - 1, L - 2, max(L - new[b], 0) + new[b] // 2, max(L - new[b] - 1, 0)}:
                spoil(p, "vc", b, t, (b + t) % Hkv, (7 * t) % D, math.inf if t % 2 else -math.inf)
        p.check(*p.run(K, splits))
        p.check(*p.run(K, splits, window=20))


@pytest.mark.parametrize("kind", ["fp16", "e4m3", "mx4"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_keys_that_are_no_numbers(K, kind, D):
    """In K: the rows that attend it are NaN, the others what they were."""
    p = Paged(kind, 21, [300, 200], [90, 1], 8, 2, D)
    clean = p.run(K, 1)
    spoil(p, "kc", 0, 270, 1, 5)
    for splits in (1, 4):
        out, lse = p.run(K, splits)
        bad = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
        bad[60:90, 4:] = True  # from position 270 on, of the heads of KV head 1
        assert torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad) and torch.equal(lse.isnan(), bad)
        if splits == 1:
            assert torch.equal(out[~bad], clean[0][~bad]) and torch.equal(lse[~bad], clean[1][~bad])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_packed_values_that_are_no_numbers(K, D):
    new = [200, 1, 300, 64]
    starts = firsts(new)
    q, k, v = projection(gen(22), starts[-1], 8, 2, D)
    for t, x in ((199, math.inf), (150, math.nan), (200, -math.inf), (201, math.nan), (501, math.inf), (340, 65504.0)):
        v[t, t % 2, (3 * t) % D] = x
    ctx = lambda b: (k[starts[b]:starts[b + 1]].double(), v[starts[b]:starts[b + 1]].double(), None)  # noqa: E731
    for window in (-1, 0, 33):
        ref = attend64(q, starts, new, ctx, D ** -0.5, window)
        out, lse = run_packed(K, q, k, v, starts, D ** -0.5, window=window)
        check(out, lse, ref, bounds(ref, D, max(new), False))
    # a prompt's own rows alone count: the one before it is all NaN
    v[200:501], k[200:501] = 1.0, 1.0
    want = run_packed(K, q, k, v, starts, D ** -0.5)
    v[:200], k[:200] = math.nan, math.nan
    got = run_packed(K, q, k, v, starts, D ** -0.5)
    assert torch.equal(got[0][200:], want[0][200:]) and torch.equal(got[1][200:], want[1][200:])
    assert bool(got[0][:200].isnan().all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_queries_that_are_no_numbers(K, kind, value):
    for D, Hq, new in ((64, 4, [80, 3]), (128, 4, [150, 3]), (256, 4, [9, 70])):
        p = Paged(kind, 23, [300, 90], new, Hq, 2, D)
        clean = p.run(K, 1)
        p.q[2, 3, D - 1] = value
        out, lse = p.run(K, 1)
        assert bool(out[2, 3].isnan().all()) and bool(lse[2, 3].isnan())
        keep = torch.ones_like(lse, dtype=torch.bool)
        keep[2, 3] = False
        assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", [16, 48, 64])
@pytest.mark.parametrize("splits", [1, 6])
def test_bad_pages(K, kind, bs, splits):
    """Positions of a page out of range are skipped, and the flag tells."""
    for D, new in ((64, [100, 1, 2]), (128, [100, 1, 2]), (256, [30, 1, 2])):
        p = Paged(kind, 24, [500, 260, 2], new, 8, 2, D, bs)
        p.table[0, 1], p.table[0, 420 // bs], p.table[1, 0], p.table[2, 0] = -1, p.pool, -(1 << 31), (1 << 31) - 1
        p.check(*p.run(K, splits, flag=K.FLAG_BAD_BLOCK))
        # a page that no row attends is not looked at
        p = Paged(kind, 24, [500, 260], [3, 1], 8, 2, D, bs)
        p.table[:, 0] = -7
        p.check(*p.run(K, splits, window=100))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [1, 4])
def test_rows_that_attend_nothing(K, kind, splits):
    """More new tokens than the sequence has: the first ones lie before its beginning."""
    p = Paged(kind, 25, [200, 130, 3, 10], [250, 130, 9, 1], 4, 2, 128)
    p.lens = [200, 0, 3, 10]
    p.check(*p.run(K, splits))
    p.check(*p.run(K, splits, window=0))


@pytest.mark.parametrize("splits", [1, 4])
def test_a_window_wider_than_any_sequence(K, splits):
    """The widest there is, where a tile's first tokens lie before the sequence's beginning."""
    for D, new in ((64, [250, 20]), (128, [250, 20]), (256, [60, 20])):
        p = Paged("fp16", 40, [40, 300], new, 4, 2, D)
        p.check(*p.run(K, splits, window=(1 << 31) - 1))


@pytest.mark.parametrize("splits", [1, 4])
def test_lengths_and_starts_out_of_range(K, splits):
    p = Paged("int8", 26, [100, 64, 60], [10, 20, 5], 4, 2, 128)
    p.table = torch.where(p.table < 0, 0, p.table)
    cap = p.table.shape[1] * 16
    given = [cap + 1000, -5, 60]
    out, lse = p.run(K, splits, lens=given, flag=K.FLAG_LEN_CLAMPED)
    p.lens = [cap, 0, 60]
    p.check(out, lse)
    # starts that fall, or leave the rows of q: rows 5 .. 9, none, and 3 .. 34; rows that two sequences have are one's or
    # the other's
    p = Paged("int8", 27, [100, 64, 60], [10, 20, 5], 4, 2, 128)
    out, lse = p.run(K, splits, starts=[5, 10, 3, 1 << 30], flag=K.FLAG_LEN_CLAMPED)
    assert bool((out[:3] == 7).all()) and bool((lse[:3] == 7).all()) and bool(torch.isfinite(out[5:10]).all())
    p.table, p.lens = p.table[2:], [60]
    ref = p.reference([3, 35])
    ref[2][5:10] = math.nan
    check(out, lse, ref, bounds(ref, 128, 60, True))


@pytest.mark.parametrize("kind", KINDS)
def test_scales_of_either_sign(K, kind):
    if kind == "fp16":
        pytest.skip("an fp16 cache takes no scales")
    for per_channel in (False, True):
        for D, new in ((64, [300]), (128, [3, 200]), (256, [40])):
            p = Paged(kind, 28, [300, 220][:len(new)], new, 8, 2, D, per_channel=per_channel)
            p.c["ks"].view(-1)[::2] *= -1
            p.c["vs"].view(-1)[::3] *= -1
            p.check(*p.run(K, 1))
            p.c["ks"].view(-1)[0] = 0
            p.c["vs"].view(-1)[-1] = 0
            p.check(*p.run(K, 3))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_scale_of_zero(K, D):
    """softmax_scale 0: the mean of the values attended."""
    p = Paged("fp16", 29, [300, 77], [200, 1], 4, 2, D)
    p.sigma = 0.0
    p.check(*p.run(K, 1))
    p.check(*p.run(K, 3, softcap=5.0))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", [48, 80, 272])
def test_windows_and_page_sizes(K, kind, bs):
    for D, splits in ((64, 1), (128, 1), (128, 5), (256, 2)):
        paged_case(K, kind, 30, [1000, 129, 600], [300, 1, 7], 8, 2, D, bs, window=130, softcap=15.0, sink=True, splits=splits)


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences(K, kind):
    """More than are sorted by length, and more than a warp's worth of them."""
    g = torch.Generator().manual_seed(31)
    lens = torch.randint(0, 200, (300,), generator=g).tolist()
    new = [min(int(n), L) for n, L in zip(torch.randint(0, 6, (300,), generator=g), lens)]
    for splits in (0, 1):
        paged_case(K, kind, 31, lens, new, 4, 2, 64, splits=splits)
    paged_case(K, kind, 32, lens[:129], new[:129], 6, 1, 128, splits=1, window=50)


def test_many_prompts(K):
    g = torch.Generator().manual_seed(33)
    new = torch.randint(0, 150, (200,), generator=g).tolist()
    starts = firsts(new)
    q, k, v = projection(gen(33), starts[-1], 4, 2, 64)
    ctx = lambda b: (k[starts[b]:starts[b + 1]].double(), v[starts[b]:starts[b + 1]].double(), None)  # noqa: E731
    for window in (-1, 40):
        ref = attend64(q, starts, new, ctx, 0.125, window)
        check(*run_packed(K, q, k, v, starts, 0.125, window=window), ref, bounds(ref, 64, max(new), False))


def test_caches_past_32_bits(K):
    """Pages whose codes begin past 2^32 bytes."""
    for kind, D, Hkv in (("int8", 128, 8), ("fp16", 64, 8), ("mx4", 128, 8)):
        bs, per = 16, Hkv * D * 16  # values of a page
        blocks = (1 << 32) // (per * 9 // 8 if kind == "mx4" else per) + 64
        p = Paged(kind, 34, [300, 40], [140, 1], 2 * Hkv, Hkv, D, bs)
        big = {}
        for x in ("kc", "vc"):
            if p.c[x] is None:
                big[x] = None
                continue
            big[x] = torch.empty((blocks,) + p.c[x].shape[1:], dtype=p.c[x].dtype, device="cuda")
            big[x][-p.pool:].copy_(p.c[x])
        small, table = dict(p.c), p.table.clone()
        p.c.update(big)
        p.table = torch.where(table >= 0, table + (blocks - p.pool), -1)
        got = [p.run(K, s) for s in (1, 3)]
        p.c, p.table = small, table
        for out, lse in got:
            p.check(out, lse)


def test_packed_strides_past_32_bits(K):
    T, D = 9000, 64
    stride = 1 << 19
    base = torch.empty(T * stride, dtype=torch.float16, device="cuda")  # 9.4 GB
    g = gen(35)
    new = [4000, 4999]
    starts = firsts(new)
    q, k, v = (base[8 * i * D:].as_strided((T, h, D), (stride, D, 1)) for i, h in ((0, 2), (1, 1), (2, 1)))
    for x in (q, k, v):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    got = run_packed(K, q, k, v, starts, 0.125)
    want = run_packed(K, q.contiguous(), k.contiguous(), v.contiguous(), starts, 0.125)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_workspace_too_small(K):
    p = Paged("int8", 36, [2000, 900], [1, 3], 8, 2, 128)
    whole = p.run(K, 1, ws=False)
    for none in (p.run(K, 0, ws=False),):
        assert torch.equal(none[0], whole[0]) and torch.equal(none[1], whole[1])
    c = p.c
    args = (p.q, c["kc"], c["vc"], c["ks"], c["vs"], 2, p.table, ints(p.lens), ints(p.starts), p.sigma)
    need = K.paged_prefill_workspace_bytes(4, 2, 8, 2, 128, p.table.shape[1] * 16, 4)
    for ws in (None, torch.empty(need // 4 - 1, device="cuda")):
        with pytest.raises(K.Int8KVError):
            K.paged_prefill(*args, num_splits=4, workspace=ws)
    out = K.paged_prefill(*args, workspace=torch.empty(16, device="cuda"))
    assert torch.equal(out, whole[0])


def test_calls_repeat_themselves(K):
    """The same call gives the same bits."""
    for kind in KINDS:
        p = Paged(kind, 37, [900, 700, 3], [200, 1, 3], 8, 2, 128)
        for splits in (1, 9):
            a = p.run(K, splits)
            for _ in range(5):
                b = p.run(K, splits)
                assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_streams(K):
    """An explicit stream, the current one, and two at once with a workspace each."""
    p = Paged("int8", 38, [900, 700], [200, 2], 8, 2, 128)
    want = p.run(K, 0)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = p.run(K, 0, stream=s1)
    assert torch.equal(got[0], want[0])
    with torch.cuda.stream(s2):
        got = p.run(K, 0)
    assert torch.equal(got[0], want[0])
    c = p.c
    args = (p.q, c["kc"], c["vc"], c["ks"], c["vs"], 2, p.table, ints(p.lens), ints(p.starts), p.sigma)
    torch.cuda.synchronize()
    nbytes = K.paged_prefill_workspace_bytes(p.q.shape[0], 2, 8, 2, 128, p.table.shape[1] * 16)
    spaces = [torch.empty(nbytes // 4, device="cuda") for _ in range(2)]
    outs = [torch.empty((20,) + tuple(p.q.shape), dtype=torch.float16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for s, ws, out in zip((s1, s2), spaces, outs):
            K.paged_prefill(*args, workspace=ws, out=out[i], stream=s)
    torch.cuda.synchronize()
    for out in outs:
        assert bool((out == want[0]).all())


def test_graphs(K):
    """Two captured graphs that share a workspace, replayed in turn on other inputs than those they were captured on."""
    batches = [Paged(kind, 39 + i, lens, new, 8, 2, 128) for i, (kind, lens, new) in enumerate(
        (("int8", [900, 700], [200, 2]), ("e4m3", [1500, 40], [1, 1])))]
    nbytes = max(K.paged_prefill_workspace_bytes(p.q.shape[0], 2, 8, 2, 128, p.table.shape[1] * 16) for p in batches)
    ws = torch.empty(nbytes // 4, device="cuda")
    want = [p.run(K) for p in batches]
    graphs, outs, queries = [], [], []
    for p in batches:
        c = p.c
        q = torch.zeros_like(p.q)
        out = torch.empty_like(q)
        args = (q, c["kc"], c["vc"], c["ks"], c["vs"], 2, p.table, ints(p.lens), ints(p.starts), p.sigma)
        K.paged_prefill(*args, workspace=ws, out=out)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            K.paged_prefill(*args, workspace=ws, out=out)
        p.args = args
        graphs.append(gr)
        outs.append(out)
        queries.append(q)
    for p, q in zip(batches, queries):
        q.copy_(p.q)
    for _ in range(4):
        for gr, out, w in zip(graphs, outs, want):
            out.fill_(0)
            ws.fill_(math.nan)
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, w[0])
    for _ in range(4):  # back to back, one after the other
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out, w[0])


@pytest.mark.parametrize("kind", KINDS)
def test_a_prompt_its_next_chunk_and_single_tokens(K, kind):
    """norm_rope_and_cache, packed_prefill over the prompts' own keys, then chunks and single tokens over the cache."""
    Hq, Hkv, D, R, bs = 8, 2, 128, 64, 16
    g = gen(50)
    total = [150, 37, 260]
    table, pool = tables(g, [t + 80 for t in total], bs)
    c = cache_of(kind, g, pool, bs, Hkv, D, True)
    if kind == "fp16":
        c["ks"] = c["vs"] = None
    else:
        c["ks"] *= 4  # normed keys are a few units wide
    qw, kw = (1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
    angle = torch.rand((400, R // 2), generator=g, device="cuda") * 6 - 3
    cs = torch.cat((angle.cos(), angle.sin()), 1).contiguous()
    sigma = D ** -0.5
    have = [0, 0, 0]
    # prompts; chunks for two of them; single tokens
    for step, new in enumerate((total, [40, 0, 33], [1, 1, 1], [1, 1, 1])):
        starts = firsts(new)
        T = starts[-1]
        q, k, v = projection(g, T, Hq, Hkv, D)
        pos = torch.cat([torch.arange(a, a + n) for a, n in zip(have, new)]).int().cuda()
        seq = torch.cat([torch.full((n,), b) for b, n in enumerate(new)]).cuda()
        slots = (table[seq, (pos // bs).long()] * bs + pos % bs).int()
        qo, ko = K.norm_rope_and_cache(q, k, v, qw, kw, 1e-6, pos, cs, slots, *(
            (c["kc"], None) if kind == "mx4" else (c["kc"].view(-1, Hkv, D), c["vc"].view(-1, Hkv, D))),
            c["ks"], c["vs"], c["scale_kind"], return_keys=True)
        have = [a + n for a, n in zip(have, new)]
        out, lse = torch.empty_like(qo), torch.empty((T, Hq), device="cuda")
        if step == 0:
            K.packed_prefill(qo, ko, v, ints(starts), sigma, out=out, lse=lse)
            ctx = lambda b: (ko[starts[b]:starts[b + 1]].double(), v[starts[b]:starts[b + 1]].double(), None)  # noqa: E731,B023
            folds = False
        else:
            ws = torch.empty(max(K.paged_prefill_workspace_bytes(T, 3, Hq, Hkv, D, table.shape[1] * bs) // 4, 4), device="cuda")
            K.paged_prefill(qo, c["kc"], c["vc"], c["ks"], c["vs"], c["scale_kind"], table, ints(have), ints(starts), sigma,
                            workspace=ws, out=out, lse=lse)
            ctx = context_of(c, table, *values(c))
            folds = kind != "fp16"
        ref = attend64(qo, starts, have, ctx, sigma)
        check(out, lse, ref, bounds(ref, D, max(have), folds), f"{kind}, step {step}")
        # what the norm and the turn made of the queries: fp16's rounding and fp32's
        x = q.double()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * qw.double()
        co, si = (t[pos.long()][:, None].double() for t in cs.split(R // 2, 1))
        a, b = y[..., :R // 2], y[..., R // 2:R]
        y = torch.cat((a * co - b * si, b * co + a * si, y[..., R:]), -1)
        size = torch.cat((a.abs() + b.abs(),) * 2 + (y[..., R:].abs(),), -1)
        assert bool(((qo.double() - y).abs() <= 2.0 ** -11 * y.abs() + 24 * 2.0 ** -24 * 1.01 * size + 2.0 ** -25).all())
