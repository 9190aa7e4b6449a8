"""Attention of sequences that share a prefix in the paged cache, on an
MI355X, against plain float64 forms."""
import math

import pytest
import torch

import attention_ref as ref
from test_gpu_attention_sinks import Paged, check_rows, cu_of, plain, randn

pytestmark = pytest.mark.gpu

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_07_amd as mod
    mod.lib()
    return mod


class Call:
    """Groups of sequences: pre[m] prefix keys, own[n] own keys, lq[n] new
    tokens; cuts: first sequence of each group and the end of the last."""

    def __init__(self, g, pre, cuts, lq, own, Hq, Hk, d, page, dtype, f8, seed=0, packed=False, tail=0):
        self.pre, self.cuts, self.lq, self.own = pre, cuts, lq, own
        self.d, self.dtype, self.f8 = d, dtype, f8
        # one cache: the prefixes' rows and the sequences'
        self.c = Paged(g, list(pre) + list(own), Hk, d, page, dtype, f8, seed)
        M = len(pre)
        cut = lambda t, rows: t[:, :max(1, -(-max(rows) // page))].contiguous()
        self.prefix_table, self.table = cut(self.c.table[:M], pre).cuda(), cut(self.c.table[M:], own).cuda()
        self.prefix_lens, self.lens = self.c.lens[:M].clone(), self.c.lens[M:].clone()
        self.groups = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        self.cu = cu_of(lq) if packed else None
        shape = (1, sum(lq) + tail, Hq, d) if packed else (len(lq), lq[0], Hq, d)
        self.q = randn(seed + 77, shape, dtype)

    def run(self, g, one=False, **kw):
        groups = None if one else self.groups
        o, lse = torch.full_like(self.q, 7.0), torch.full(self.q.shape[:3], 7.0, device="cuda")
        g.attn_paged_prefix(self.q, self.c.k, self.c.v, self.prefix_table, self.prefix_lens, self.table, self.lens,
                            cu_groups=groups, cu_seqlens=self.cu, out=o, lse=lse, **self.c.scales(), **kw)
        torch.cuda.synchronize()
        return o, lse

    def group_of(self, n):
        for m in range(len(self.pre)):
            if self.cuts[m] <= n < self.cuts[m + 1]:
                return m

    def check(self, o, lse):
        flat = lambda x: x.reshape(-1, *x.shape[2:])
        o, lse, q = flat(o), flat(lse), flat(self.q)
        t0 = 0
        for n, lq in enumerate(self.lq):
            t = slice(t0, t0 + lq)
            t0 += lq
            m = self.group_of(n)
            k, v = self.c.rows[len(self.pre) + n]
            own = k.shape[0]
            dead = max(0, lq - own)
            assert (o[t][:dead] == 0).all() and (lse[t][:dead] == -math.inf).all(), n
            if lq == dead:
                continue
            if m is not None:
                k, v = torch.cat((self.c.rows[m][0], k)), torch.cat((self.c.rows[m][1], v))
            check_rows(o[t][dead:], lse[t][dead:], q[t][dead:], k, v, 0, 0, self.dtype, self.d,
                       f"seq {n} group {m} new {lq} own {own}", self.f8)
        assert (o[t0:] == 7.0).all() and (lse[t0:] == 7.0).all(), "rows behind the last sequence were written"


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("d,page,Hq,Hk", [(128, 64, 8, 2), (64, 16, 3, 3), (128, 128, 5, 1), (64, 256, 16, 2)])
def test_prefix_decode(g, d, page, Hq, Hk, f8, dtype):
    """One group of all sequences, single tokens: few rows and many."""
    for N, P in ((1, 1), (3, 130), (20, 517), (70, 300)):
        print(f"prefix decode N={N} P={P} Hq={Hq} Hk={Hk} d={d} page={page} f8={f8} {dtype}", flush=True)
        own = [1 + (37 * n) % 90 for n in range(N)]
        c = Call(g, [P], [0, N], [1] * N, own, Hq, Hk, d, page, dtype, f8, seed=N)
        a = c.run(g, one=True)
        c.check(*a)
        # the same as an explicit group
        assert all(torch.equal(x, y) for x, y in zip(a, c.run(g)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("f8", [False, True])
def test_prefix_groups(g, f8, dtype):
    """Several groups, empty ones and empty prefixes among them; sequences of
    no group; padding (no own keys); more new tokens than own keys."""
    for T in (1, 3, 40):
        print(f"prefix groups T={T} f8={f8} {dtype}", flush=True)
        own = [5, 200, T, 0, 64, max(T - 2, 0), 33 + T, 1, T + 1, 129, 77, T]
        pre = [300, 65, 0, 1, 128]
        c = Call(g, pre, [1, 4, 4, 6, 9, 10], [T] * len(own), own, 8, 2, 128, 64, dtype, f8, seed=T)
        c.check(*c.run(g))
        c = Call(g, pre, [1, 4, 4, 6, 9, 10], [T] * len(own), own, 8, 2, 128, 64, dtype, f8, seed=T, packed=True, tail=3)
        c.check(*c.run(g))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("f8", [False, True])
def test_prefix_chunk(g, f8, dtype):
    """A new request's chunk among single tokens, packed, with empty sequences."""
    lq = [1, 1, 333, 0, 1, 50, 1, 0]
    own = [40, 300, 400, 7, 1, 50, 20, 0]
    print(f"prefix chunk f8={f8} {dtype}", flush=True)
    for cuts, pre in (([0, 8], [700]), ([0, 3, 8], [260, 513])):
        c = Call(g, pre, cuts, lq, own, 12, 4, 128, 32, dtype, f8, seed=len(pre), packed=True, tail=11)
        c.check(*c.run(g, one=len(pre) == 1))


def test_prefix_many_groups(g):
    """More groups than a wave has lanes, some of no sequence."""
    M = 150
    sizes = [(7 * m * m + 3) % 4 for m in range(M)]
    cuts = [0] + torch.tensor(sizes).cumsum(0).tolist()
    N = cuts[-1]
    print(f"prefix many groups N={N}", flush=True)
    c = Call(g, [(11 * m) % 70 for m in range(M)], cuts, [1] * N, [1 + n % 9 for n in range(N)], 4, 2, 64, 16, BF16, False,
             seed=6)
    c.check(*c.run(g))


def test_prefix_long(g):
    """Keys of both kinds in parts."""
    print("prefix long", flush=True)
    c = Call(g, [5000], [0, 9], [1] * 9, [1500 + 100 * n for n in range(9)], 16, 4, 128, 64, BF16, True, seed=8)
    c.check(*c.run(g, one=True))
    c = Call(g, [4000, 100], [0, 2, 4], [2] * 4, [900, 2, 17, 400], 16, 1, 128, 64, BF16, False, seed=9)
    c.check(*c.run(g))


@pytest.mark.parametrize("dtype,f8", [(BF16, False), (BF16, True), (F32, False)])
def test_prefix_equals_whole_tables(g, dtype, f8):
    """The same rows through attn_paged with the prefix's pages in every table
    (a prefix of whole pages): equal within the roundings of either."""
    page, P, N, Hk, d = 16, 160, 6, 2, 64
    own = [3, 50, 17, 1, 90, 33]
    c = Call(g, [P], [0, N], [1] * N, own, 8, Hk, d, page, dtype, f8, seed=11)
    o, lse = c.run(g)
    table = torch.cat((c.prefix_table.expand(N, -1), c.table), 1).contiguous()
    o2, lse2 = g.attn_paged(c.q, c.c.k, c.c.v, table, c.lens + P, want_lse=True, **c.c.scales())
    c.check(o2, lse2)
    c.check(o, lse)


@pytest.mark.parametrize("f8", [False, True])
def test_prefix_odd_values_and_entries(g, f8):
    """Table entries outside the cache stand for zeros, those behind a length
    are not read; NaN in a page none sees stays there, in a prefix reaches its
    group alone; a row whose own scores are all -inf still has its prefix."""
    page, Hk, d, N = 16, 2, 64, 6
    own = [20, 5, 40, 33, 1, 16]
    c = Call(g, [100, 50], [0, 3, 6], [1] * N, own, 4, Hk, d, page, BF16, f8, seed=12)
    o0, lse0 = c.run(g)
    c.check(o0, lse0)
    nan_page = c.c.spare
    c.c.poison(nan_page)
    # behind the lengths
    c.prefix_table[1, 4:] = nan_page
    c.table[4, 1:] = nan_page
    o, lse = c.run(g)
    assert torch.equal(o, o0) and torch.equal(lse, lse0)
    # a NaN page in one prefix
    save = c.prefix_table.clone()
    c.prefix_table[0, 2] = nan_page
    o, lse = c.run(g)
    assert o[:3].isnan().all() and torch.equal(o[3:], o0[3:]) and torch.equal(lse[3:], lse0[3:])
    # entries outside the cache: pages of zeros
    for bad in (-1, 2 ** 31 - 1, c.c.k.shape[0]):
        c.prefix_table.copy_(save)
        c.prefix_table[0, 2] = bad
        k, v = (x.clone() for x in c.c.rows[0])
        rows = c.c.rows[0]
        k[2 * page:3 * page], v[2 * page:3 * page] = 0.0, 0.0
        c.c.rows[0] = (k, v)
        c.check(*c.run(g))
        c.c.rows[0] = rows


def test_prefix_rows_of_no_finite_score(g):
    """Own keys of -inf scores: the prefix alone; nothing finite at all: o = 0, lse = -inf."""
    page, Hk, d, N = 16, 1, 64, 3
    c = Call(g, [40], [0, N], [1] * N, [4, 1, 20], 2, Hk, d, page, F32, False, seed=13)
    c.q.abs_()
    far = torch.full((d,), -math.inf, device="cuda")
    for i in range(1, N + 1):
        n = c.own[i - 1]
        s = c.c.slots(i, n)
        c.c.k[s // page, :, s % page] = far
    o, lse = c.run(g)
    for n in range(N):
        k, v = c.c.rows[0]
        check_rows(o[n], lse[n], c.q[n], k, v, 0, 0, F32, d, f"seq {n}", False)
    s = c.c.slots(0, 40)
    c.c.k[s // page, :, s % page] = far
    o, lse = c.run(g)
    assert (o == 0).all() and (lse == -math.inf).all()


def test_prefix_tables_of_no_pages(g):
    N, Hk, d, page = 3, 2, 64, 16
    kc, vc = (torch.full((2, Hk, page, d), math.nan, dtype=BF16, device="cuda") for _ in range(2))
    q = randn(1, (N, 1, 4, d), BF16)
    none = torch.empty((N, 0), dtype=torch.int32, device="cuda")
    lens = torch.tensor([5, 0, 9], dtype=torch.int32, device="cuda")
    o, lse = g.attn_paged_prefix(q, kc, vc, none[:1], lens[:1].clone(), none, lens, want_lse=True)
    assert (o == 0).all() and (lse == -math.inf).all()


def test_prefix_bad_groups(g):
    """cu_groups that fall, or lie outside the sequences: any result for those, nothing else is written, no fault."""
    N = 5
    c = Call(g, [70, 33, 20], [0, 2, 3, 5], [1] * N, [9, 4, 30, 1, 2], 4, 2, 64, 16, BF16, False, seed=14, packed=True,
             tail=6)
    for bad in ([0, 4, 1, 5], [-9, 2 ** 30, 3, 2 ** 31 - 1], [5, 5, 5, 5], [3, 2, 1, 0]):
        c.groups.copy_(torch.tensor(bad, dtype=torch.int32))
        o, lse = c.run(g)
        assert (o[:, N:] == 7.0).all() and (lse[:, N:] == 7.0).all()


def test_prefix_runs_streams_and_graphs(g):
    """The same bits every run and on another stream; a captured step among
    eager work, with lengths and groups that change between replays; calls at
    once on workspaces of their own."""
    N, M = 24, 2
    c = Call(g, [300, 700], [0, 9, N], [1] * N, [1 + 13 * n % 200 for n in range(N)], 16, 4, 128, 64, BF16, True, seed=15)
    need = g.attn_paged_prefix_workspace_bytes(c.q, c.c.k, c.prefix_table, c.table)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    want = c.run(g, workspace=ws)
    c.check(*want)
    ws.fill_(127)
    assert all(torch.equal(x, y) for x, y in zip(want, c.run(g, workspace=ws)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = c.run(g)
    here = c.run(g, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(want, other, here))
    o, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:3], device="cuda")

    def step():
        g.attn_paged_prefix(c.q, c.c.k, c.c.v, c.prefix_table, c.prefix_lens, c.table, c.lens, cu_groups=c.groups, out=o,
                            lse=lse, workspace=ws, **c.c.scales())
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        c.prefix_lens.sub_(17 * i)
        c.groups[1] += i
        c.q.mul_(1.25)
        step()
        eager = o.clone(), lse.clone()
        o.zero_()
        lse.zero_()
        ws.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, eager[0]) and torch.equal(lse, eager[1]), i


def test_serving_with_a_shared_prompt(g):
    """As it is used: the common prompt appended once (normed and rotated),
    requests that decode behind it, each step's tokens appended and attended;
    equal to attention over every request's whole sequence."""
    P, N, steps, Hq, Hk, d, page = 100, 5, 6, 8, 2, 128, 16
    fr = g.rope_frequencies(d)
    wq, wk = (1.0 + 0.1 * randn(80 + i, (d,), F32) for i in range(2))
    per = -(-steps // page)
    pages = -(-P // page) + N * per
    kc, vc = (torch.zeros((pages, Hk, page, d), dtype=BF16, device="cuda") for _ in range(2))
    ptab = torch.arange(-(-P // page), dtype=torch.int32, device="cuda")[None]
    tab = (-(-P // page) + torch.arange(N * per, dtype=torch.int32, device="cuda")).reshape(N, per)
    plen = torch.tensor([P], dtype=torch.int32, device="cuda")

    def project(seed, shape):
        x = randn(seed, (*shape, Hq + 2 * Hk, d), BF16)
        return x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:]

    q0, k0, v0 = project(90, (1, P))
    pos0 = torch.arange(P, dtype=torch.int32, device="cuda")[None]
    g.kv_cache_append(q0, k0, v0, torch.arange(P, device="cuda"), kc, vc, fr, wq, wk, positions=pos0)
    _, kr0 = g.qk_norm_rope(q0.contiguous(), k0.contiguous(), fr, wq, wk, pos0)
    ks, vs = [kr0.expand(N, -1, -1, -1)], [v0.expand(N, -1, -1, -1)]
    for t in range(steps):
        q, k, v = project(91 + t, (N, 1))
        pos = torch.full((N, 1), P + t, dtype=torch.int32, device="cuda")
        slots = tab[:, t // page].long() * page + t % page
        qr = g.kv_cache_append(q, k, v, slots, kc, vc, fr, wq, wk, positions=pos)
        lens = torch.full((N,), t + 1, dtype=torch.int32, device="cuda")
        o, lse = g.attn_paged_prefix(qr, kc, vc, ptab, plen, tab, lens, want_lse=True)
        q2, k2 = g.qk_norm_rope(q.contiguous(), k.contiguous(), fr, wq, wk, pos)
        assert torch.equal(qr, q2)
        ks.append(k2)
        vs.append(v)
        kk, vv = torch.cat(ks, 1), torch.cat(vs, 1)
        for n in range(N):
            r = plain(q2[n].double(), kk[n].double(), vv[n].double(), 0, 0)
            ref.check_attn({"o": o[n], "lse": lse[n]}, r, BF16, kk.shape[1], d, f"step {t} request {n}")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,f8", [(BF16, False), (BF16, True), (F32, False), (F32, True)])
def test_prefix_odd_values_and_entries_many_rows(g, dtype, f8, d):
    """The same with tiles of 128 rows: entries outside the cache, odd pages behind the length, NaN that one group sees."""
    page, Hk, N = 16, 2, 90
    own = [1 + 7 * n % 40 for n in range(N)]
    print(f"prefix odd, many rows d={d} {dtype} f8={f8}", flush=True)
    c = Call(g, [300, 190], [0, 50, N], [1] * N, own, 8, Hk, d, page, dtype, f8, seed=21)
    o0, lse0 = c.run(g)
    c.check(o0, lse0)
    c.c.poison(c.c.spare)
    c.prefix_table[1, 12:] = c.c.spare
    o, lse = c.run(g)
    assert torch.equal(o, o0) and torch.equal(lse, lse0)
    rows = c.c.rows[0]
    k, v = (x.clone() for x in rows)
    for p, bad in ((2, -1), (7, 2 ** 31 - 1), (18, c.c.k.shape[0])):
        c.prefix_table[0, p] = bad
        k[p * page:(p + 1) * page], v[p * page:(p + 1) * page] = 0.0, 0.0
    c.c.rows[0] = (k, v)
    c.check(*c.run(g))
    c.prefix_table[0, 5] = c.c.spare
    o, lse = c.run(g)
    assert o[:50].isnan().all() and torch.equal(o[50:], o0[50:]) and torch.equal(lse[50:], lse0[50:])


@pytest.mark.parametrize("power", [-100, 60])
def test_prefix_scales(g, power):
    """Quantised rows of very small and large scales, for few rows and many."""
    page, Hk, d, P = 16, 1, 64, 200
    for N in (3, 70):
        print(f"prefix scales 2^{power} N={N}", flush=True)
        c = Call(g, [P], [0, N], [1] * N, [3] * N, 4, Hk, d, page, BF16, True, seed=22)
        # every other row of the prefix's values, and its keys one way (scores of size 1 need the other in q)
        s = c.c.slots(0, P)
        e = torch.arange(P, device="cuda") % 2 * power
        c.c.vs[s // page, :, s % page] = (c.c.vs[s // page, :, s % page].int() + e[:, None]).to(torch.uint8)
        k, v = c.c.rows[0]
        c.c.rows[0] = (k, v * torch.exp2(e.double())[:, None, None])
        c.check(*c.run(g))


def test_prefix_offsets_past_32_bits(g):
    """A cache of 5 GiB (bfloat16) and 2.5 GiB (e4m3), prefix and own keys in its last pages."""
    Hk, page, d, P = 8, 64, 128, 150
    pages = 5 * (1 << 30) // (Hk * page * d * 2)
    for cdt in (BF16, F8):
        kc, vc = (torch.empty((pages, Hk, page, d), dtype=cdt, device="cuda") for _ in range(2))
        ks, vs = (torch.empty((pages, Hk, page), dtype=torch.uint8, device="cuda") for _ in range(2)) \
            if cdt == F8 else (None, None)
        ptab = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device="cuda")
        for N in (2, 40):
            tab = (pages - 4 - torch.arange(N, dtype=torch.int32, device="cuda"))[:, None].contiguous()
            lens = torch.arange(1, N + 1, dtype=torch.int32, device="cuda")
            t = torch.arange(P, device="cuda")
            slots = [ptab[0, t // page].long() * page + t % page]
            slots += [tab[n, 0].long() * page + torch.arange(n + 1, device="cuda") for n in range(N)]
            rows = []
            for i, s in enumerate(slots):
                k, v = (randn(200 + 2 * i + j, (s.numel(), Hk, d), BF16) for j in range(2))
                g.kv_cache_write(k, v, s, kc, vc, ks, vs)
                rows.append(tuple(x.double() for x in g.kv_cache_read(s, kc, vc, ks, vs)))
            q = randn(199, (N, 1, 16, d), BF16)
            print(f"prefix large cache {cdt} N={N}", flush=True)
            o, lse = g.attn_paged_prefix(q, kc, vc, ptab, torch.tensor([P], dtype=torch.int32, device="cuda"), tab, lens,
                                         k_scale=ks, v_scale=vs, want_lse=True)
            for n in range(N):
                kk, vv = (torch.cat((rows[0][j], rows[1 + n][j])) for j in range(2))
                check_rows(o[n], lse[n], q[n], kk, vv, 0, 0, BF16, d, f"seq {n}", cdt == F8)
        del kc, vc, ks, vs
        torch.cuda.empty_cache()


def test_prefix_two_calls_at_once(g):
    """Two calls on two streams, each on its own workspace, many times over."""
    calls = [Call(g, [900], [0, 33], [1] * 33, [1 + 5 * n for n in range(33)], 8, 2, 128, 64, BF16, f8, seed=23 + f8)
             for f8 in (False, True)]
    want = [c.run(g, one=True) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    outs = []
    for i in range(8):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                outs.append(g.attn_paged_prefix(c.q, c.c.k, c.c.v, c.prefix_table, c.prefix_lens, c.table, c.lens,
                                                want_lse=True, **c.c.scales()))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(outs):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


@pytest.mark.parametrize("dtype,f8", [(BF16, False), (BF16, True), (F32, False), (F32, True)])
@pytest.mark.parametrize("d", [64, 128])
def test_prefix_tile_shapes_together(g, d, dtype, f8):
    """Every pair of the prefixes' and the own keys' tiles (32 or 128 rows; 16, 32 or 128)."""
    print(f"prefix tile shapes d={d} {dtype} f8={f8}", flush=True)
    # 32 rows over the prefixes (more groups than rows would need), 128 over the own keys
    c = Call(g, [90, 0, 40, 7, 200], [0, 0, 1, 1, 2, 2], [40, 40], [60, 41], 2, 2, d, 32, dtype, f8, seed=31)
    c.check(*c.run(g))
    # 32 and 32 (packed), 32 and 16
    for packed in (True, False):
        c = Call(g, [130, 60, 5], [0, 1, 2, 3], [2] * 3, [33, 2, 150], 8, 2, d, 16, dtype, f8, seed=32, packed=packed)
        c.check(*c.run(g))
    # 128 and 16, 128 and 32 (packed), 128 and 128
    for T, packed in ((1, False), (1, True), (20, False), (20, True)):
        c = Call(g, [333], [0, 48], [T] * 48, [T + n % 30 for n in range(48)], 8, 2, d, 64, dtype, f8, seed=33, packed=packed)
        c.check(*c.run(g, one=True))


def test_prefix_scale_and_defaults(g):
    """A scale of its own, and outputs and workspace that the call makes."""
    c = Call(g, [100], [0, 9], [1] * 9, [1 + n for n in range(9)], 4, 2, 64, 16, F32, False, seed=34)
    c.q.mul_(0.3 * 8)  # scale 0.3 on the same scores as 1 / 8 on these
    o, lse = c.run(g)
    q = c.q / (0.3 * 8)
    o2, lse2 = g.attn_paged_prefix(q, c.c.k, c.c.v, c.prefix_table, c.prefix_lens, c.table, c.lens, scale=0.3, want_lse=True)
    o3, none = g.attn_paged_prefix(q, c.c.k, c.c.v, c.prefix_table, c.prefix_lens, c.table, c.lens, scale=0.3)
    assert none is None and torch.equal(o2, o3)
    assert (o2 - o).abs().max() < 1e-5 and (lse2 - lse).abs().max() < 1e-5


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("N", [3, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_prefix_ends_inside_pages(g, d, N, f8, dtype):
    """Prefixes that end inside a tile and a page, of every page size and shape of the
    rows: what the page holds behind the last key does not reach a row, and an infinite
    value of the last key reaches all of its group's."""
    for page, pre in ((16, [70, 1, 250]), (32, [33, 520, 31]), (256, [65, 300, 1030])):
        c = Call(g, pre, [0, N // 3, N - 1, N], [1] * N, [n % 7 for n in range(N)], 8, 2, d, page, dtype, f8, seed=page + N)
        c.check(*c.run(g))
        for m, n in enumerate(pre):
            slot, end = int(c.c.slots(m, n)[-1]), n % page
            p = slot // page
            if end:
                if f8:
                    c.c.ks[p, :, end:], c.c.vs[p, :, end:] = 255, 255
                else:
                    c.c.k[p, :, end:], c.c.v[p, :, end:] = math.nan, math.nan
        o0, lse0 = c.run(g)
        c.check(o0, lse0)
        if not f8:
            p = int(c.c.slots(1, pre[1])[-1])
            c.c.v[p // page, 1, p % page, 3] = math.inf
            o, lse = c.run(g)
            t0, t1 = N // 3, N - 1
            assert torch.equal(lse, lse0) and torch.equal(o[:t0], o0[:t0]) and torch.equal(o[t1:], o0[t1:])
            # (a sequence without own keys has its token at position -1: it sees nothing)
            seen = [math.inf if n % 7 else 0. for n in range(t0, t1)]
            assert (o[t0:t1, 0, 4:, 3] == torch.tensor(seen, device="cuda")[:, None]).all(), (page, d)
            o[t0:t1, :, 4:, 3] = o0[t0:t1, :, 4:, 3]
            assert torch.equal(o, o0), (page, d)
