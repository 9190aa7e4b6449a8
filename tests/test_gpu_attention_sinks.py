"""Attention with a sliding window and first tokens that stay visible (sinks),
over whole sequences with gradients and over the paged cache, on an MI355X,
against plain float64 forms with bounds counted from the roundings each kernel
makes."""
import math

import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import gated_delta_rule_07_amd as mod
    mod.lib()
    return mod


def randn(seed, shape, dtype):
    gn = torch.Generator(device="cuda")
    gn.manual_seed(seed)
    return torch.randn(shape, generator=gn, device="cuda").to(dtype)


def cu_of(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


def plain(q, k, v, window, sinks, do=None):
    """One sequence by the definition: q [Lq, Hq, d] at the last positions, k,
    v [Lk, Hk, d], float64; the dict that ``attention_ref.check_attn`` takes
    (o, lse, gradients, and the magnitudes the bounds are made of)."""
    (lq, Hq, d), (lk, Hk, _) = q.shape, k.shape
    G, scale = Hq // Hk, d ** -0.5
    kk, vv = (x.repeat_interleave(G, 1).transpose(0, 1) for x in (k, v))
    qq = q.transpose(0, 1)
    i, j = torch.arange(lk - lq, lk, device=q.device)[:, None], torch.arange(lk, device=q.device)[None]
    vis = j <= i
    if window:
        vis = vis & ((j > i - window) | (j < sinks))
    s = torch.where(vis, qq @ kk.transpose(1, 2) * scale, float("-inf"))
    lse = torch.logsumexp(s, -1)
    p = torch.where(vis & (lse[..., None] > float("-inf")), torch.exp(s - lse[..., None]), 0.0)
    vf = torch.where(torch.isfinite(vv), vv, 0.0)
    r = {"o": p @ vf, "lse": lse, "o_abs": p @ vf.abs(),
         "s_abs": (qq.abs() @ kk.nan_to_num(0.0, 0.0, 0.0).abs().transpose(1, 2) * scale).amax().item()}
    if do is not None:
        dd = do.transpose(0, 1)
        ds = p * (dd @ vv.transpose(1, 2) - (dd * r["o"]).sum(-1, keepdim=True))
        dd_abs = (dd.abs() * (r["o"].abs() + r["o_abs"])).sum(-1, keepdim=True)
        w = ds.abs() + p * dd_abs
        mag = p * (dd.abs() @ vv.abs().transpose(1, 2) + dd_abs)
        fold = lambda x: x.reshape(Hk, G, lk, d).sum(1)
        for n, a in (("dq", ds), ("dq_abs", w), ("dq_mag", mag)):
            r[n] = a @ (kk if n == "dq" else kk.abs()) * scale
        for n, a in (("dk", ds), ("dk_abs", w), ("dk_mag", mag)):
            r[n] = fold(a.transpose(1, 2) @ (qq if n == "dk" else qq.abs()) * scale)
        r["dv"], r["dv_abs"] = fold(p.transpose(1, 2) @ dd), fold(p.transpose(1, 2) @ dd.abs())
        r["dv_mag"] = r["dv_abs"]
    return {n: x.transpose(0, 1) if torch.is_tensor(x) else x for n, x in r.items()}


def run(g, lens, Hq, Hk, d, dtype, window, sinks, packed=True, bwd=True, seed=0, tail=0):
    print(f"sinks lens={lens} Hq={Hq} Hk={Hk} d={d} {dtype} window={window} sinks={sinks} packed={packed}", flush=True)
    B, T = (1, sum(lens) + tail) if packed else (len(lens), lens[0])
    q, k, v, do = (randn(4 * seed + i, (B, T, h, d), dtype) for i, h in enumerate((Hq, Hk, Hk, Hq)))
    kw = dict(cu_seqlens=cu_of(lens) if packed else None, window=window, sinks=sinks)
    o, lse = torch.full_like(q, 7.0), torch.full((B, T, Hq), 7.0, device="cuda")
    g.attn_fwd(q, k, v, out=o, lse=lse, **kw)
    gr = {n: torch.full_like(x, 7.0) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    if bwd:
        g.attn_bwd(q, k, v, o, lse, do, out=gr, **kw)
    torch.cuda.synchronize()
    flat = lambda x: x.reshape(-1, *x.shape[2:])
    q, k, v, do, o, lse = (flat(x) for x in (q, k, v, do, o, lse))
    gr = {n: flat(x) for n, x in gr.items()}
    t0 = 0
    for n in lens:
        t = slice(t0, t0 + n)
        t0 += n
        if n == 0:
            continue
        r = plain(q[t].double(), k[t].double(), v[t].double(), window, sinks, do[t].double() if bwd else None)
        got = {"o": o[t], "lse": lse[t]}
        if bwd:
            got.update({m: x[t] for m, x in gr.items()})
        ref.check_attn(got, r, dtype, n, d, f"len {n}")
    for x in (o, lse) + (tuple(gr.values()) if bwd else ()):
        assert (x[t0:] == 7.0).all(), "rows behind the last sequence were written"


# (window, sinks): one of each, sinks that fill tiles or not, sinks next to the window, more sinks than window
PAIRS = [(1, 1), (2, 3), (31, 4), (64, 32), (100, 33), (7, 64), (50, 130), (299, 1), (1000, 5)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", PAIRS)
def test_sinks_packed(g, window, sinks, dtype):
    run(g, [300, 7, 0, 161, 1], 6, 2, 64, dtype, window, sinks, seed=window, tail=19)
    run(g, [33, 420], 4, 1, 128, dtype, window, sinks, seed=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", PAIRS)
def test_sinks_fixed(g, window, sinks, dtype):
    run(g, [257, 257], 4, 1, 128, dtype, window, sinks, packed=False, seed=window)
    run(g, [200] * 3, 5, 5, 64, dtype, window, sinks, packed=False, seed=sinks)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
def test_sinks_many_rows(g, dtype, d):
    """Tiles of 128 rows, and rows behind the window of many tiles that several workgroups share."""
    T = 2000 if dtype == BF16 else 1100
    run(g, [T, T], 16, 4, d, dtype, 333, 4, packed=False, seed=1)
    run(g, [T, 3, T - 77], 16, 8, d, dtype, 200, 70, seed=2, tail=3)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sinks_key_tiles_of_128(g, dtype):
    """Whole key tiles in the backward (many sequences and kv heads)."""
    run(g, [1024] * 8, 8, 8, 64, dtype, 100, 9, packed=False, seed=3)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
def test_sinks_one_kv_head(g, dtype, d):
    """Many query heads on one kv head: key tiles whose rows several workgroups share, joined with the sinks' sums."""
    run(g, [700, 0, 411, 33], 16, 1, d, dtype, 90, 40, seed=4, tail=5)
    run(g, [1030], 35, 1, d, dtype, 64, 3, packed=False, seed=5)
    run(g, [700, 0, 411, 33], 67, 1, d, dtype, 256, 128, seed=6, tail=5)


def test_sinks_many_sequences(g):
    lens = [(7 * i * i + 3) % 41 if i % 5 else 0 for i in range(150)]
    run(g, lens, 4, 2, 64, BF16, 9, 3, seed=7, tail=2)
    run(g, lens, 4, 2, 128, F32, 5, 20, seed=8)


def test_sinks_long(g):
    run(g, [4096], 4, 1, 128, BF16, 1024, 4, packed=False, seed=9)
    run(g, [4096], 4, 2, 128, BF16, 100, 1000, packed=False, seed=10)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sinks_that_hide_nothing_more(g, dtype):
    """No sinks is the window alone, and window and sinks that cover the sequence are plain attention, bit for bit."""
    q, k, v, do = (randn(i, (1, 300, h, 64), dtype) for i, h in enumerate((6, 2, 2, 6)))

    def both(**kw):
        o, lse = g.attn_fwd(q, k, v, **kw)
        gr = g.attn_bwd(q, k, v, o, lse, do, **kw)
        return [o, lse] + [gr[n] for n in ("dq", "dk", "dv")]
    for a, b in ((dict(window=90, sinks=0), dict(window=90)), (dict(sinks=12), {}), (dict(window=90, sinks=210), {}),
                 (dict(window=90, sinks=2 ** 40), {}), (dict(window=2 ** 40, sinks=3), {})):
        for x, y in zip(both(**a), both(**b)):
            assert torch.equal(x, y), (a, b)


def test_sinks_gradients_by_differences(g):
    """float32 gradients against central differences of the forward in float64."""
    lens, window, sinks, d = [40], 6, 3, 64
    q, k, v, do = (randn(20 + i, (1, 40, h, d), F32) for i, h in enumerate((2, 1, 1, 2)))
    o, lse = g.attn_fwd(q, k, v, window=window, sinks=sinks)
    gr = g.attn_bwd(q, k, v, o, lse, do, window=window, sinks=sinks)

    def loss(q, k, v):
        return (plain(q[0], k[0], v[0], window, sinks)["o"] * do[0].double()).sum().item()
    x = {n: t.double() for n, t in (("q", q), ("k", k), ("v", v))}
    h = 1e-5
    for n in x:
        for t in (0, 2, 3, 20, 39):
            for c in (0, 37):
                at = (0, t, 0, c)
                up, dn = (dict(x, **{n: x[n].clone()}) for _ in range(2))
                up[n][at] += h
                dn[n][at] -= h
                num = (loss(**up) - loss(**dn)) / (2 * h)
                # the difference quotient's own error: h^2 and 2^-52 of the loss over h
                assert abs(gr["d" + n][at].item() - num) < 2e-4 * max(1.0, abs(num)), (n, t, c)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sinks_odd_values(g, dtype):
    """Infinities and NaN between the sinks and a row's window do not reach
    it; in a sink they reach every later row of its sequence."""
    T, window, sinks = 400, 50, 6
    q, k, v = (randn(30 + i, (1, T, h, 128), dtype) for i, h in enumerate((4, 2, 2)))
    o0, lse0 = g.attn_fwd(q, k, v, window=window, sinks=sinks)
    for bad in (math.nan, math.inf):
        k2, v2 = k.clone(), v.clone()
        k2[0, 100, :, 3] = bad
        v2[0, 101, :, 5] = bad
        v2[0, 7, :, 9] = bad
        o, lse = g.attn_fwd(q, k2, v2, window=window, sinks=sinks)
        clean = [t for t in range(T) if not (100 <= t < 101 + window or 7 <= t < 7 + window)]
        assert torch.equal(o[0, clean], o0[0, clean]) and torch.equal(lse[0, clean], lse0[0, clean])
        assert not torch.isfinite(o[0, 101, :, 5]).any()
        v3 = v.clone()
        v3[0, sinks - 1, :, 9] = bad
        o, lse = g.attn_fwd(q, k, v3, window=window, sinks=sinks)
        assert not torch.isfinite(o[0, sinks - 1:, :, 9]).any()
        rest = [c for c in range(128) if c != 9]
        assert torch.equal(o[..., rest], o0[..., rest]) and torch.equal(lse, lse0)


def test_sinks_runs_streams_and_graphs(g):
    """The same bits every run, on another stream, and from a captured step replayed among eager work."""
    lens, kw = [300, 41, 700], dict(window=64, sinks=5)
    T = sum(lens)
    q, k, v, do = (randn(40 + i, (1, T, h, 128), BF16) for i, h in enumerate((8, 2, 2, 8)))
    cu = cu_of(lens)
    need = g.attn_bwd_workspace_bytes(1, T, 8, 2, 128, BF16, sinks=5, num_seqs=3)
    assert need > g.attn_bwd_workspace_bytes(1, T, 8, 2, 128, BF16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((1, T, 8), device="cuda")
    gr = {n: torch.empty_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v))}

    def step():
        g.attn_fwd(q, k, v, cu_seqlens=cu, out=o, lse=lse, **kw)
        g.attn_bwd(q, k, v, o, lse, do, cu_seqlens=cu, workspace=ws, out=gr, **kw)
        return [o, lse, *gr.values()]
    want = [x.clone() for x in step()]
    ws.fill_(255)
    for x, y in zip(step(), want):
        assert torch.equal(x, y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ws.fill_(127)
        got = [x.clone() for x in step()]
    torch.cuda.current_stream().wait_stream(s)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    q0 = q.clone()
    for i in range(3):
        q.copy_(q0 * (1 + i))
        eager = [x.clone() for x in step()]
        for x in (o, lse, *gr.values()):
            x.zero_()
        ws.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((o, lse, *gr.values()), eager):
            assert torch.equal(x, y), i


# ------------------------------------------------------------------ the cache
class Paged:
    """Sequences of lk keys in a shuffled paged cache, and their values in float64."""

    def __init__(self, g, lk, Hk, d, page, dtype, f8, seed, max_pages=None):
        need = [-(-n // page) for n in lk]
        total = sum(need) + 4
        order = torch.randperm(total, generator=torch.Generator().manual_seed(seed))
        mp = max(max(need), 1) + 1 if max_pages is None else max_pages
        self.table = torch.full((len(lk), mp), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n].to(torch.int32)
            at += n
        self.spare = int(order[-1])
        self.lk, self.page, self.Hk, self.d = lk, page, Hk, d
        cdt = F8 if f8 else dtype
        self.k, self.v = (torch.zeros((total, Hk, page, d), device="cuda").to(cdt) for _ in range(2))
        self.ks, self.vs = ((torch.full((total, Hk, page), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
                            if f8 else (None, None))
        self.rows = []
        for i, n in enumerate(lk):
            slots = self.slots(i, n)
            k, v = (randn(1000 * seed + 2 * i + j, (n, Hk, d), dtype) for j in range(2))
            g.kv_cache_write(k, v, slots, self.k, self.v, k_scale=self.ks, v_scale=self.vs)
            kr, vr = g.kv_cache_read(slots, self.k, self.v, k_scale=self.ks, v_scale=self.vs, dtype=F32 if f8 else dtype)
            self.rows.append((kr.double(), vr.double()))
        self.lens = torch.tensor(lk, dtype=torch.int32, device="cuda")

    def slots(self, i, n):
        j = torch.arange(n)
        return (self.table[i].long()[j // self.page] * self.page + j % self.page).cuda()

    def args(self):
        return self.k, self.v, self.table.cuda(), self.lens

    def scales(self):
        return dict(k_scale=self.ks, v_scale=self.vs)

    def poison(self, page):
        """A page of NaN (quantised: rows whose exponent byte says NaN)."""
        if self.ks is None:
            self.k[page], self.v[page] = math.nan, math.nan
        else:
            self.ks[page], self.vs[page] = 255, 255


def check_rows(o, lse, q, k, v, window, sinks, dtype, d, label, f8):
    """Rows of one sequence against the definition; rows at negative positions see nothing."""
    lq, lk = q.shape[0], k.shape[0]
    dead = max(0, lq - lk)
    assert (o[:dead] == 0).all() and (lse[:dead] == -math.inf).all(), label
    if lq > dead:
        r = plain(q[dead:].double(), k, v, window, sinks)
        ref.check_attn({"o": o[dead:], "lse": lse[dead:]}, r, dtype, lk, d, label)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("T,G", [(1, 1), (1, 4), (4, 4), (3, 8), (40, 2)])
def test_sinks_paged(g, T, G, f8, dtype):
    """Decode tiles (T G <= 16), 32-row and 128-row tiles; pages of the gap are
    freed (no entry, an entry far outside, a page of NaN)."""
    Hk = 2
    for page, d, window, sinks in ((16, 128, 100, 4), (64, 64, 33, 20), (128, 128, 300, 130), (32, 64, 17, 32), (16, 128, 5, 1)):
        lk = [1, 1200, 0, sinks, sinks + window, sinks + window + T, 777, 2]
        print(f"paged sinks T={T} G={G} f8={f8} {dtype} page={page} d={d} window={window} sinks={sinks}", flush=True)
        c = Paged(g, lk, Hk, d, page, dtype, f8, seed=page + T)
        c.poison(c.spare)
        for i, n in enumerate(lk):
            first = max(0, n - T + 1 - window)
            for p in range(-(-sinks // page), first // page):
                c.table[i, p] = (-1, c.spare, 2 ** 30)[p % 3]
        q = randn(T, (len(lk), T, Hk * G, d), dtype)
        kw = dict(window=window, sinks=sinks, want_lse=True, **c.scales())
        o, lse = g.attn_paged(q, *c.args(), **kw)
        torch.cuda.synchronize()
        for i, n in enumerate(lk):
            check_rows(o[i], lse[i], q[i], *c.rows[i], window, sinks, dtype, d, f"keys {n}", f8)
        # packed, the same rows
        cu = torch.arange(len(lk) + 1, dtype=torch.int32, device="cuda") * T
        o2, lse2 = g.attn_paged(q.reshape(1, -1, Hk * G, d), *c.args(), cu_seqlens=cu, **kw)
        for i, n in enumerate(lk):
            check_rows(o2.reshape(o.shape)[i], lse2.reshape(lse.shape)[i], q[i], *c.rows[i], window, sinks, dtype, d,
                       f"packed, keys {n}", f8)


@pytest.mark.parametrize("f8", [False, True])
def test_sinks_paged_chunk(g, f8):
    """A prompt's chunk of many rows among single tokens, keys in parts."""
    lq, lk, Hk, d, page = [600, 1, 1, 90], [2500, 3000, 40, 90], 4, 128, 64
    for dtype, window, sinks in ((BF16, 512, 4), (BF16, 100, 200), (F32, 300, 17)):
        print(f"paged sinks chunk {dtype} f8={f8} window={window} sinks={sinks}", flush=True)
        c = Paged(g, lk, Hk, d, page, dtype, f8, seed=5)
        q = randn(3, (1, sum(lq) + 5, 4 * Hk, d), dtype)
        o, lse = torch.full_like(q, 7.0), torch.full(q.shape[:3], 7.0, device="cuda")
        g.attn_paged(q, *c.args(), cu_seqlens=cu_of(lq), window=window, sinks=sinks, out=o, lse=lse, **c.scales())
        torch.cuda.synchronize()
        t0 = 0
        for i, n in enumerate(lq):
            t = slice(t0, t0 + n)
            t0 += n
            check_rows(o[0, t], lse[0, t], q[0, t], *c.rows[i], window, sinks, dtype, d, f"new {n}, keys {lk[i]}", f8)
        assert (o[0, t0:] == 7.0).all() and (lse[0, t0:] == 7.0).all()


def test_sinks_prompt_then_decode(g):
    """A layer as it is used: a prompt by whole-sequence attention, then decode
    over the cache, each step equal (within the roundings) to the prompt form
    on the longer sequence."""
    T, steps, Hq, Hk, d, page, window, sinks = 150, 40, 8, 2, 128, 16, 48, 4
    q, k, v = (randn(50 + i, (1, T + steps, h, d), BF16) for i, h in enumerate((Hq, Hk, Hk)))
    whole, _ = g.attn_fwd(q, k, v, window=window, sinks=sinks)
    pages = -(-(T + steps) // page)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    kc, vc = (torch.zeros((pages, Hk, page, d), dtype=BF16, device="cuda") for _ in range(2))
    at = torch.arange(T + steps)
    slots = (table.long()[at // page] * page + at % page).cuda()
    g.kv_cache_write(k[0, :T], v[0, :T], slots[:T], kc, vc)
    tb = table[None].cuda()
    for t in range(T, T + steps):
        g.kv_cache_write(k[0, t:t + 1], v[0, t:t + 1], slots[t:t + 1], kc, vc)
        lens = torch.tensor([t + 1], dtype=torch.int32, device="cuda")
        o, _ = g.attn_paged(q[:, t:t + 1], kc, vc, tb, lens, window=window, sinks=sinks)
        r = plain(q[0, t:t + 1].double(), k[0, :t + 1].double(), v[0, :t + 1].double(), window, sinks)
        for x in (o[0], whole[0, t:t + 1]):
            ref.check_attn({"o": x}, r, BF16, t + 1, d, f"step {t}")


def test_sinks_offsets_past_32_bits(g):
    """Tensors of 4 GiB each: one sequence of 2^17 tokens x 128 heads, whose
    last rows see the first keys; the sinks' gradients are sums over all rows."""
    H, d, T, window, sinks, n = 128, 128, (1 << 17) + 70, 64, 4, 70
    gn = torch.Generator(device="cuda")
    gn.manual_seed(60)
    q, k, v, do = (torch.randn((1, T, H, d), generator=gn, device="cuda", dtype=BF16) for _ in range(4))
    print("sinks large tensors: forward", flush=True)
    o, lse = g.attn_fwd(q, k, v, window=window, sinks=sinks)
    keys = torch.cat((torch.arange(sinks), torch.arange(T - n - window + 1, T))).cuda()
    kk, vv = k[0, keys].double(), v[0, keys].double()
    # those rows and keys as a sequence of their own
    r = plain(q[0, T - n:].double(), kk, vv, window, sinks)
    ref.check_attn({"o": o[0, T - n:], "lse": lse[0, T - n:]}, r, BF16, keys.numel(), d, "last rows")
    print("sinks large tensors: backward", flush=True)
    gr = g.attn_bwd(q, k, v, o, lse, do, window=window, sinks=sinks)
    # the sinks' gradients by the formula from the forward's o and lse, a block of rows at a time
    want = {m: torch.zeros((sinks, H, d), dtype=torch.float64, device="cuda") for m in ("dk", "dv", "dk_abs", "dv_abs")}
    for t in range(0, T, 1 << 13):
        rows = slice(t, min(t + (1 << 13), T))
        qq, dd, oo = (x[0, rows].double() for x in (q, do, o))
        delta = (dd * oo).sum(-1)
        pos = torch.arange(T, device="cuda")[rows]
        for j in range(sinks):
            p = torch.exp((qq * k[0, j].double()).sum(-1) * d ** -0.5 - lse[0, rows].double())
            p = torch.where(pos[:, None] >= j, p, 0.0)
            ds = p * ((dd * v[0, j].double()).sum(-1) - delta) * d ** -0.5
            want["dv"][j] += (p[..., None] * dd).sum(0)
            want["dk"][j] += (ds[..., None] * qq).sum(0)
            want["dv_abs"][j] += (p[..., None] * dd.abs()).sum(0)
            want["dk_abs"][j] += (ds.abs()[..., None] * qq.abs()).sum(0)
    for m in ("dk", "dv"):
        # half a step of the weights as operands and of the output; in float32 a product of 128 terms inside each
        # weight and a sum of up to 2^17 rows in parts of at most 2^12
        bound = ref.step(BF16) * want[m].abs() + (1.01 * ref.step(BF16) + 2.0 ** -11) * want[m + "_abs"]
        ref.check(gr[m][0, :sinks], want[m], bound, m)
    assert all(torch.isfinite(x).all() for x in gr.values())


def test_sinks_two_calls_at_once(g):
    """Forward and backward of two sizes on two streams, each on its own workspace."""
    sets = []
    for i, (T, Hk, d) in enumerate(((500, 2, 128), (900, 1, 64))):
        x = [randn(70 + 4 * i + j, (1, T, h, d), BF16) for j, h in enumerate((4 * Hk, Hk, Hk, 4 * Hk))]
        ws = torch.empty(g.attn_bwd_workspace_bytes(1, T, 4 * Hk, Hk, d, BF16, sinks=5), dtype=torch.uint8, device="cuda")
        sets.append((x, ws))

    def step(x, ws):
        q, k, v, do = x
        o, lse = g.attn_fwd(q, k, v, window=40, sinks=5)
        gr = g.attn_bwd(q, k, v, o, lse, do, window=40, sinks=5, workspace=ws)
        return [o, lse, gr["dq"], gr["dk"], gr["dv"]]
    want = [step(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(step(*s))
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(x, want[i % 2]))


def test_sinks_scale_and_defaults(g):
    q, k, v = (randn(90 + i, (1, 200, h, 64), F32) for i, h in enumerate((4, 2, 2)))
    o, lse = g.attn_fwd(q * (0.3 * 8), k, v, window=30, sinks=3)
    o2, lse2 = g.attn_fwd(q, k, v, window=30, sinks=3, scale=0.3)
    o3, none = g.attn_fwd(q, k, v, window=30, sinks=3, scale=0.3, want_lse=False)
    assert none is None and torch.equal(o2, o3)
    assert (o2 - o).abs().max() < 1e-5 and (lse2 - lse).abs().max() < 1e-5


@pytest.mark.parametrize("f8", [False, True])
def test_sinks_decode_in_a_graph(g, f8):
    """A captured decode step replayed while the sequences grow past their window, its workspace shared with another graph."""
    Hq, Hk, d, page, window, sinks = 8, 2, 128, 16, 40, 3
    c = Paged(g, [200, 37, 90], Hk, d, page, BF16, f8, seed=91)
    q = randn(92, (3, 1, Hq, d), BF16)
    table = c.table.cuda()
    lens = torch.tensor([100, 10, 43], dtype=torch.int32, device="cuda")
    ws = torch.empty(max(1, g.attn_paged_workspace_bytes(q, c.k, table, None, window, sinks),
                         g.attn_paged_workspace_bytes(q, c.k, table)), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for _ in range(2)]
    lses = [torch.empty((3, 1, Hq), device="cuda") for _ in range(2)]
    calls = [dict(window=window, sinks=sinks), dict()]

    def step(i):
        g.attn_paged(q, c.k, c.v, table, lens, out=outs[i], lse=lses[i], workspace=ws, **c.scales(), **calls[i])
    graphs = []
    for i in range(2):
        step(i)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            step(i)
    for t in range(4):
        lens.add_(9)
        want = []
        for i in range(2):
            step(i)
            want.append((outs[i].clone(), lses[i].clone()))
        for i in (0, 1, 0):
            outs[i].zero_()
            ws.fill_(t)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], want[i][0]) and torch.equal(lses[i], want[i][1]), (t, i)
        for i, n in enumerate(lens.tolist()):
            n = min(n, c.lk[i])
            if lens[i] <= c.lk[i]:
                check_rows(outs[0][i], lses[0][i], q[i], c.rows[i][0][:n], c.rows[i][1][:n], window, sinks, BF16, d,
                           f"step {t} sequence {i}", f8)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("f8", [False, True])
def test_sinks_decode_workgroups(g, f8, d):
    """Decode's workgroups of 12 waves, of 4 with keys in parts, and of 4 where there are many sequences."""
    Hk, page = 2, 32
    for N, T, top, window, sinks in ((6, 1, 900, 500, 4), (6, 2, 400, 30, 37), (3, 1, 4000, 2000, 20), (3, 4, 3000, 1500, 5),
                                     (140, 1, 300, 64, 5), (140, 3, 200, 130, 40)):
        print(f"sinks decode N={N} T={T} window={window} sinks={sinks} d={d} f8={f8}", flush=True)
        lk = [max(0, top - 37 * n % (top + 1)) for n in range(N)]
        lk[1] = 0
        c = Paged(g, lk, Hk, d, page, BF16, f8, seed=N + T)
        c.poison(c.spare)
        for i, n in enumerate(lk):
            c.table[i, -(-sinks // page):max(0, n - T + 1 - window) // page] = c.spare
        q = randn(N, (N, T, 4 * Hk, d), BF16)
        assert (g.attn_paged_workspace_bytes(q, c.k, c.table, None, window, sinks) > 0) == (window > 200)
        o, lse = g.attn_paged(q, *c.args(), window=window, sinks=sinks, want_lse=True, **c.scales())
        torch.cuda.synchronize()
        for i, n in enumerate(lk):
            check_rows(o[i], lse[i], q[i], *c.rows[i], window, sinks, BF16, d, f"keys {n}", f8)
