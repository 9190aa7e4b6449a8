"""Attention operators of a hybrid stack on an MI355X, against plain float64
forms (tests/attention_ref.py) with bounds counted from the roundings each
kernel makes."""
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


def gen(seed):
    x = torch.Generator(device="cuda")
    x.manual_seed(seed)
    return x


def randn(gn, shape, dtype):
    return torch.randn(shape, generator=gn, device="cuda").to(dtype)


def cu_of(lens):
    return torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ whole sequences
def run_attn(g, lens, Hq, Hk, d, dtype, window, packed, bwd, seed=0, tail=0):
    gn = gen(seed)
    B, T = (1, sum(lens) + tail) if packed else (len(lens), lens[0])
    q, k, v, do = (randn(gn, (B, T, h, d), dtype) for h in (Hq, Hk, Hk, Hq))
    cu = cu_of(lens) if packed else None
    o = torch.full_like(q, 7.0)
    lse = torch.full((B, T, Hq), 7.0, device="cuda")
    g.attn_fwd(q, k, v, cu_seqlens=cu, window=window, out=o, lse=lse)
    gr = {n: torch.full_like(x, 7.0) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    if bwd:
        g.attn_bwd(q, k, v, o, lse, do, cu_seqlens=cu, window=window, out=gr)
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
        r = ref.attn(q[t].double(), k[t].double(), v[t].double(), window, d ** -0.5, do[t].double() if bwd else None)
        got = {"o": o[t], "lse": lse[t]}
        if bwd:
            got.update({m: x[t] for m, x in gr.items()})
        ref.check_attn(got, r, dtype, n, d, f"len {n}")
    for x in (o, lse) + (tuple(gr.values()) if bwd else ()):
        assert (x[t0:] == 7.0).all(), "rows behind the last sequence were written"


LENS = [[1], [2, 1], [31, 32, 33], [127, 1, 0, 129, 64], [300], [0, 65, 0], [513, 100]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("i", range(len(LENS)))
def test_attn_packed(g, i, d, dtype):
    Hq, Hk = [(4, 4), (4, 2), (6, 2), (3, 1), (8, 1), (5, 5), (8, 2)][i]
    print(f"attn packed lens={LENS[i]} Hq={Hq} Hk={Hk} d={d} {dtype}", flush=True)
    run_attn(g, LENS[i], Hq, Hk, d, dtype, 0, True, True, seed=i, tail=37)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [1, 2, 31, 64, 100, 299, 1000])
def test_attn_window(g, window, dtype):
    print(f"attn window={window} {dtype}", flush=True)
    run_attn(g, [300, 7, 161], 6, 2, 64, dtype, window, True, True, seed=window)
    run_attn(g, [257, 257], 4, 1, 128, dtype, window, False, True, seed=window)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
def test_attn_fixed_lengths(g, dtype, d):
    for B, T, Hq, Hk in ((1, 1, 1, 1), (3, 1, 4, 2), (2, 128, 2, 2), (9, 70, 8, 8), (1, 700, 16, 4), (5, 33, 9, 3)):
        print(f"attn fixed B={B} T={T} Hq={Hq} Hk={Hk} d={d} {dtype}", flush=True)
        run_attn(g, [T] * B, Hq, Hk, d, dtype, 0, False, True, seed=T)


def test_attn_many_sequences(g):
    """More sequences than a wave has lanes, empty ones among them."""
    lens = [(7 * i * i + 3) % 41 if i % 5 else 0 for i in range(150)]
    print("attn many sequences", flush=True)
    run_attn(g, lens, 4, 2, 64, BF16, 0, True, True, seed=3)
    run_attn(g, lens, 4, 2, 64, BF16, 9, True, True, seed=4)


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
def test_attn_one_kv_head(g, dtype, d):
    """Many query heads on one kv head: few key tiles with many rows, shared
    by several workgroups."""
    print(f"attn one kv head d={d} {dtype}", flush=True)
    run_attn(g, [700, 0, 411, 33], 16, 1, d, dtype, 0, True, True, seed=8, tail=5)
    run_attn(g, [700, 0, 411, 33], 35, 1, d, dtype, 90, True, True, seed=9, tail=5)
    run_attn(g, [130], 67, 1, d, dtype, 0, False, True, seed=10)


def test_attn_long(g):
    """A long sequence (rows of 64 key tiles) with a window and without."""
    print("attn long 4096", flush=True)
    run_attn(g, [4096], 4, 1, 128, BF16, 0, False, True, seed=5)
    run_attn(g, [4096], 4, 2, 128, BF16, 2048, False, True, seed=6)


def test_offsets_past_32_bits(g):
    """Tensors of 4 GiB each and more: packed sequences of zeros, then one of
    70 tokens behind 2^24 rows."""
    Hq = Hk = 128
    d, n, lead, N = 128, 70, 1 << 17, 1 << 8
    T = lead + n
    gn = gen(55)

    def tensor():
        x = torch.zeros((1, T, Hq, d), dtype=BF16, device="cuda")
        x[0, lead:] = randn(gn, (n, Hq, d), BF16)
        return x

    cu = torch.arange(0, lead + 1, lead // N, dtype=torch.int32, device="cuda")
    cu = torch.cat([cu, torch.tensor([T], dtype=torch.int32, device="cuda")])
    q, k, v, do = (tensor() for _ in range(4))
    print("large tensors: forward", flush=True)
    o, lse = g.attn_fwd(q, k, v, cu)
    last = [x[0, lead:].double() for x in (q, k, v)]
    r = ref.attn(*last, 0, d ** -0.5)
    ref.check_attn({"o": o[0, lead:], "lse": lse[0, lead:]}, r, BF16, n, d, "last sequence")
    assert (o[0, :lead] == 0).all()
    print("large tensors: backward", flush=True)
    gr = g.attn_bwd(q, k, v, o, lse, do, cu)
    small = [x[:, lead:].contiguous() for x in (q, k, v, o, lse, do)]
    want = g.attn_bwd(*small)
    for name, x in gr.items():
        # (other workgroup shapes: the sums' order differs, 70 terms at most)
        y = want[name].double()
        assert (x[0, lead:].double() - y[0]).abs().max() <= 2 ** -7 * y.abs().max(), name
        assert (x[0, :lead] == 0).all(), name
    print("large tensors: norm and rotation", flush=True)
    f = g.rope_frequencies(d)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    q2, k2 = g.qk_norm_rope(q, k, f, positions=pos)
    s2 = g.qk_norm_rope(small[0], small[1], f, positions=pos[:, lead:].contiguous())
    assert torch.equal(q2[:, lead:], s2[0]) and torch.equal(k2[:, lead:], s2[1])
    gr = g.qk_norm_rope_bwd(q, k, f, do, do, positions=pos)
    w = g.qk_norm_rope_bwd(small[0], small[1], f, small[5], small[5], positions=pos[:, lead:].contiguous())
    assert torch.equal(gr["dq"][:, lead:], w["dq"]) and torch.equal(gr["dk"][:, lead:], w["dk"])
    del gr, w, q, k, v, do, o, q2, k2
    torch.cuda.empty_cache()


def test_attn_gradients_against_differences(g):
    """dL along random directions, L = sum(o * do): the kernels' gradients
    against central differences of the float64 definition.  The definition's
    third derivative leaves an error of order eps^2 = 1e-8; the float32
    gradients' own error is bounded as in check_attn, far below 1e-4 of the
    directional derivative's terms."""
    gn = gen(11)
    T, Hq, Hk, d, W = 77, 4, 2, 64, 30
    q, k, v, do = (randn(gn, (1, T, h, d), F32) for h in (Hq, Hk, Hk, Hq))
    o, lse = g.attn_fwd(q, k, v, window=W)
    gr = g.attn_bwd(q, k, v, o, lse, do, window=W)
    base = [x[0].double() for x in (q, k, v)]

    def loss(xs):
        return (ref.attn(*xs, W, d ** -0.5)["o"] * do[0].double()).sum()

    for i, n in enumerate(("dq", "dk", "dv")):
        u = torch.randn(base[i].shape, generator=gn, device="cuda", dtype=torch.float64)
        e = 1e-4
        up, dn = [list(base) for _ in range(2)]
        up[i], dn[i] = base[i] + e * u, base[i] - e * u
        want = ((loss(up) - loss(dn)) / (2 * e)).item()
        terms = gr[n][0].double() * u
        assert abs(terms.sum().item() - want) <= 1e-4 * terms.abs().sum().item(), n


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attn_large_scores(g, dtype):
    """Scores of hundreds: one key takes all the weight."""
    gn = gen(12)
    T, d = 200, 64
    q, k, v = (randn(gn, (1, T, 2, d), dtype) * 30 for _ in range(3))
    o, lse = g.attn_fwd(q, k, v)
    r = ref.attn(q[0].double(), k[0].double(), v[0].double(), 0, d ** -0.5)
    # a score's float32 error is absolute in exp's argument: float32_part
    # counts it by s_abs
    ref.check_attn({"o": o[0], "lse": lse[0]}, r, dtype, T, d, "large")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("window", [0, 40])
def test_attn_nonfinite_values_reach_only_their_rows(g, bad, window, dtype):
    gn = gen(13)
    T, at, d = 210, 101, 128
    q, k, v = randn(gn, (1, T, 4, d), dtype), randn(gn, (1, T, 2, d), dtype), randn(gn, (1, T, 2, d), dtype)
    clean, _ = g.attn_fwd(q, k, v, window=window)
    for which in ("k", "v"):
        k2, v2 = k.clone(), v.clone()
        (k2 if which == "k" else v2)[0, at, 0, 5] = bad
        o, _ = g.attn_fwd(q, k2, v2, window=window)
        see = torch.zeros(T, dtype=torch.bool, device="cuda")
        see[at:(at + window if window else T)] = True
        # rows that do not see the key, and the other kv head: the same bits
        assert torch.equal(o[0, ~see], clean[0, ~see]), which
        assert torch.equal(o[0, :, 2:], clean[0, :, 2:]), which
        if which == "v":
            x = o[0, see][:, :2, 5].float()
            want = torch.full_like(x, bad)
            assert torch.equal(torch.isnan(x), torch.isnan(want))
            assert (torch.isnan(want) | (x == want)).all()
            rest = [c for c in range(d) if c != 5]
            a, b = o[0][:, :, rest].double(), clean[0][:, :, rest].double()
            # the same weights: the sums may differ by the order of a term
            assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -9).all()


def test_attn_same_bits_every_run_and_stream(g):
    gn = gen(14)
    q, k, v, do = (randn(gn, (2, 333, h, 128), BF16) for h in (8, 2, 2, 8))

    def both():
        o, lse = g.attn_fwd(q, k, v, window=150)
        gr = g.attn_bwd(q, k, v, o, lse, do, window=150)
        return [o, lse, gr["dq"], gr["dk"], gr["dv"]]

    a = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = both()
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


# ---------------------------------------------------------- norm and rotation
ROPE = [
    # B, T, Hq, Hk, d, rot, inter, far, norm, weights
    (1, 1, 1, 1, 64, 64, False, 0, True, True),
    (2, 33, 6, 2, 128, 128, False, 1 << 20, True, True),
    (3, 17, 5, 3, 128, 64, True, 1 << 24, True, False),
    (2, 129, 16, 4, 64, 16, False, 4096, True, True),
    (1, 70, 3, 1, 64, 24, True, 100, False, False),
    (1, 1000, 9, 9, 128, 8, False, 7, True, True),
    (4, 5, 2, 2, 128, 0, False, 0, True, True),
    (1, 2500, 16, 4, 128, 128, False, 0, True, True),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("i", range(len(ROPE)))
def test_qk_norm_rope(g, i, dtype):
    B, T, Hq, Hk, d, rot, inter, far, norm, weights = ROPE[i]
    print(f"rope {ROPE[i]} {dtype}", flush=True)
    gn = gen(100 + i)
    q, k = randn(gn, (B, T, Hq, d), dtype), randn(gn, (B, T, Hk, d), dtype)
    gq, gk = randn(gn, (B, T, Hq, d), dtype), randn(gn, (B, T, Hk, d), dtype)
    wq, wk = (torch.randn(d, generator=gn, device="cuda") for _ in range(2)) if weights else (None, None)
    freqs = g.rope_frequencies(rot) if rot else None
    pos = None
    if far:
        pos = torch.randint(-far, far, (B, T), generator=gn, device="cuda").to(torch.int32)
    kw = dict(wq=wq, wk=wk, positions=pos, interleaved=inter, norm=norm, eps=1e-5)
    oq, ok = g.qk_norm_rope(q, k, freqs, **kw)
    gr = g.qk_norm_rope_bwd(q, k, freqs, gq, gk, **kw)
    torch.cuda.synchronize()
    p = pos if pos is not None else torch.arange(T, device="cuda").expand(B, T)
    h = ref.step(dtype)
    for n, x, w, y, gy in (("q", q, wq, oq, gq), ("k", k, wk, ok, gk)):
        xd = x.double().requires_grad_()
        wd = None if w is None else w.double().requires_grad_()
        one = torch.ones(d, dtype=torch.float64, device="cuda", requires_grad=True)
        want = ref.rope(xd, wd if wd is not None else (one if norm else None), freqs, p, inter, norm, 1e-5)
        # half a step of the output; in float32 a dozen roundings of the row's
        # largest value, and the sine's and cosine's error: 2^-25 of a turn
        # (2^-22.3 radians) and 2 ulp
        big = want.detach().abs().amax(-1, keepdim=True)
        f = 2.0 ** -20
        ref.check(y, want.detach(), h * want.detach().abs() + f * big, n)
        (want * gy.double()).sum().backward()
        # the gradient's terms reach |u| (1 + |xh| mean|u xh| / |u|): the
        # row's largest |dy w r| times d in the worst case, in practice the
        # largest term; bounded by the row's sums
        r = 1.0 / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-5) if norm else torch.ones_like(big)
        u = gy.double().abs().amax(-1, keepdim=True) * (1.0 if w is None else w.double().abs().amax()) * 2
        xh = x.double().abs().amax(-1, keepdim=True) * r if norm else 0.0
        ref.check(gr["d" + n], xd.grad, h * xd.grad.abs() + f * r * u * (1.0 + xh * xh), "d" + n)
        if norm:
            gw = (wd if wd is not None else one).grad
            # float32 sums: per channel one rounding a row of the partial sums
            terms = (gy.double().abs().amax(-1, keepdim=True) * 2 * x.double().abs() * r).sum((0, 1, 2))
            ref.check(gr["dw" + n], gw, 2.0 ** -19 * terms, "dw" + n)


def test_qk_norm_rope_in_place_and_default_positions(g):
    gn = gen(7)
    q, k = randn(gn, (2, 40, 4, 64), BF16), randn(gn, (2, 40, 2, 64), BF16)
    fr = g.rope_frequencies(64)
    a = g.qk_norm_rope(q, k, fr)
    pos = torch.arange(40, device="cuda", dtype=torch.int32).expand(2, 40).contiguous()
    b = g.qk_norm_rope(q, k, fr, positions=pos)
    q2, k2 = q.clone(), k.clone()
    g.qk_norm_rope(q2, k2, fr, out=(q2, k2))
    for x, y, z in zip(a, b, (q2, k2)):
        assert torch.equal(x, y) and torch.equal(x, z)
    # the backward into the gradient's own buffers
    gq, gk = randn(gn, q.shape, BF16), randn(gn, k.shape, BF16)
    r = g.qk_norm_rope_bwd(q, k, fr, gq, gk)
    r2 = g.qk_norm_rope_bwd(q, k, fr, gq, gk, out={"dq": gq, "dk": gk})
    assert all(torch.equal(r[n], r2[n]) for n in ("dq", "dk", "dwq", "dwk"))


def test_qk_norm_rope_empty(g):
    q, k = torch.empty((2, 0, 4, 64), device="cuda"), torch.empty((2, 0, 2, 64), device="cuda")
    fr = g.rope_frequencies(64)
    out = {n: torch.full((64,), 5.0, device="cuda") for n in ("dwq", "dwk")}
    r = g.qk_norm_rope_bwd(q, k, fr, q.clone(), k.clone(), out=out)
    assert (r["dwq"] == 0).all() and (r["dwk"] == 0).all()
    assert g.qk_norm_rope(q, k, fr)[0].shape == q.shape


# -------------------------------------------------------------------- cache
def make_cache(g, gn, pages, Hk, page, d, dtype, cdt):
    """Caches filled with values (a quantised one through the operator), and
    what they stand for in float64, [pages * page, Hk, d]."""
    n = pages * page
    k, v = randn(gn, (n, Hk, d), dtype), randn(gn, (n, Hk, d), dtype)
    kc, vc = (torch.zeros((pages, Hk, page, d), device="cuda").to(cdt) for _ in range(2))
    ks = vs = None
    if cdt == F8:
        ks, vs = (torch.zeros((pages, Hk, page), dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.arange(n, device="cuda")
    g.kv_cache_write(k, v, slots, kc, vc, ks, vs)
    if cdt == F8:
        k, v = ref.quantise(k.double())[0], ref.quantise(v.double())[0]
    return kc, vc, ks, vs, k.double(), v.double()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,page,Hk,n", [(64, 16, 1, 1), (128, 64, 4, 333), (128, 256, 3, 1000), (64, 128, 5, 77)])
@pytest.mark.parametrize("f8", [False, True])
def test_kv_cache_write_read(g, d, page, Hk, n, dtype, f8):
    print(f"cache d={d} page={page} Hk={Hk} n={n} {dtype} f8={f8}", flush=True)
    gn = gen(n + d)
    pages = -(-n // page) + 2
    mul = torch.exp(6 * torch.randn((n, Hk, 1), generator=gn, device="cuda"))
    k, v = (randn(gn, (n, Hk, d), F32) * mul).to(dtype), (randn(gn, (n, Hk, d), F32) / mul).to(dtype)
    k[0, 0] = 0
    if n > 10:
        v[3, 0, 7] = math.inf
        k[4, 0, 1] = math.nan
        v[5, 0, 2] = -math.inf
        k[6, 0] = k[6, 0] * 2.0 ** -110
        v[7, 0, :] = 448.0          # the largest code exactly
        v[8, 0, :] = 449.0
    slots = torch.randperm(pages * page, generator=gn, device="cuda")[:n]
    if n > 10:
        slots[2], slots[9] = -1, pages * page  # skipped
    cdt = F8 if f8 else dtype
    poison = 1.5
    kc, vc = (torch.full((pages, Hk, page, d), poison, device="cuda").to(cdt) for _ in range(2))
    ks, vs = (torch.full((pages, Hk, page), 9, dtype=torch.uint8, device="cuda") for _ in range(2)) if f8 else (None, None)
    g.kv_cache_write(k, v, slots, kc, vc, ks, vs)
    rk, rv = g.kv_cache_read(slots, kc, vc, ks, vs, dtype=dtype)
    torch.cuda.synchronize()
    ok = (slots >= 0) & (slots < pages * page)
    for x, r, c, s in ((k, rk, kc, ks), (v, rv, vc, vs)):
        want = x.double()
        if f8:
            want, byte = ref.quantise(want)
            pg, off = slots[ok] // page, slots[ok] % page
            assert torch.equal(s[pg, :, off], byte[ok])
        want = want.to(dtype)
        same = (r == want) | (torch.isnan(r) & torch.isnan(want))
        assert same[ok].all()
        assert (r[~ok] == 0).all()
        # rows of no slot keep what they held
        free = torch.ones(pages * page, dtype=torch.bool, device="cuda")
        free[slots[ok]] = False
        f = free.nonzero()[:, 0]
        assert (c.float()[f // page, :, f % page] == poison).all()
        if f8:
            assert (s[f // page, :, f % page] == 9).all()


# -------------------------------------------------------------- paged attention
def run_paged(g, lq, lk, Hq, Hk, d, page, dtype, cdt, window, packed, seed=0, spare=2, tail=0, poison=False):
    gn = gen(seed)
    need = [-(-n // page) for n in lk]
    pages = sum(need) + spare
    kc, vc, ks, vs, kd, vd = make_cache(g, gn, pages, Hk, page, d, dtype, cdt)
    perm = torch.randperm(pages, generator=gn, device="cuda").tolist()
    table = torch.full((len(lk), max(max(need), 1) + 1), -5 if poison else 0, dtype=torch.int32)
    at, used = 0, []
    for i, n in enumerate(need):
        table[i, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        used.append(perm[at:at + n])
        at += n
    if poison:
        # whatever no query sees: pages of no sequence, rows behind a
        # sequence's end, entries before the window
        free = torch.ones((pages, page), dtype=torch.bool, device="cuda")
        for i, n in enumerate(lk):
            first = max(0, n - lq[i] - window + 1) if window else 0
            for j in range(n):
                if j >= first:
                    free[used[i][j // page], j % page] = False
            table[i, :first // page] = 1 << 30
        bad = free[:, None, :].expand(pages, Hk, page)
        for c, s in ((kc, ks), (vc, vs)):
            if s is not None:
                s[bad] = 255
                c.view(torch.uint8)[bad] = 0x7f
            else:
                c[bad] = math.nan
    T = sum(lq) + tail
    q = randn(gn, (1, T, Hq, d) if packed else (len(lq), lq[0], Hq, d), dtype)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device="cuda")
    g.attn_paged(q, kc, vc, table.cuda(), torch.tensor(lk, dtype=torch.int32, device="cuda"),
                 cu_seqlens=cu_of(lq) if packed else None, k_scale=ks, v_scale=vs, window=window, out=out, lse=lse)
    torch.cuda.synchronize()
    q, out, lse = (x.reshape(-1, *x.shape[2:]) for x in (q, out, lse))
    t0 = 0
    for i, (a, n) in enumerate(zip(lq, lk)):
        t = slice(t0, t0 + a)
        t0 += a
        rows = torch.tensor([used[i][j // page] * page + j % page for j in range(n)], dtype=torch.long, device="cuda")
        r = ref.attn(q[t].double(), kd[rows], vd[rows], window, d ** -0.5)
        ref.check_attn({"o": out[t], "lse": lse[t]}, r, dtype, n, d, f"new {a} of {n}")
    assert (out[t0:] == 7.0).all() and (lse[t0:] == 7.0).all(), "rows behind the last sequence were written"


CACHES = [(BF16, BF16), (BF16, F8), (F32, F32), (F32, F8)]


@pytest.mark.parametrize("dtype,cdt", CACHES)
@pytest.mark.parametrize("d", [64, 128])
def test_paged_decode(g, d, dtype, cdt):
    for Hq, Hk, page, window, lk in ((4, 2, 16, 0, [1, 15, 16, 17, 300]), (8, 1, 64, 50, [64, 1, 65, 2000]),
                                     (6, 2, 128, 0, [129]), (3, 3, 32, 1, [40, 1]), (16, 4, 256, 0, [5000, 3]),
                                     (40, 1, 16, 0, [90, 33])):
        print(f"paged decode Hq={Hq} Hk={Hk} page={page} window={window} lk={lk} d={d} {dtype} {cdt}", flush=True)
        run_paged(g, [1] * len(lk), lk, Hq, Hk, d, page, dtype, cdt, window, False, seed=page, poison=True)


@pytest.mark.parametrize("dtype,cdt", CACHES)
def test_paged_chunk(g, dtype, cdt):
    for lq, lk, Hq, Hk, d, page, window in (([100], [100], 4, 2, 64, 16, 0), ([130], [1000], 4, 1, 128, 64, 0),
                                            ([33], [333], 6, 2, 64, 32, 77), ([260], [3000], 2, 2, 128, 128, 1000)):
        print(f"paged chunk lq={lq} lk={lk} Hq={Hq} Hk={Hk} d={d} page={page} W={window} {dtype} {cdt}", flush=True)
        run_paged(g, lq, lk, Hq, Hk, d, page, dtype, cdt, window, False, seed=d, poison=True)


@pytest.mark.parametrize("dtype,cdt", CACHES)
@pytest.mark.parametrize("d", [64, 128])
def test_paged_mixed_batch(g, d, dtype, cdt):
    """One chunk among single tokens, an empty sequence, and fewer keys than
    new tokens (rows that see nothing)."""
    for window in (0, 60):
        print(f"paged mixed d={d} W={window} {dtype} {cdt}", flush=True)
        run_paged(g, [1, 150, 0, 1, 5, 3, 2], [700, 420, 33, 1, 5, 1, 0], 8, 2, d, 32, dtype, cdt, window, True,
                  seed=9, tail=13, poison=True)


def test_paged_several_tokens_each(g):
    """Speculative steps: a few new tokens a sequence, both kernel shapes."""
    for t in (2, 4, 8, 9):
        print(f"paged T={t}", flush=True)
        run_paged(g, [t] * 3, [t, 50, 700], 8, 2, 128, 16, BF16, F8, 0, False, seed=t, poison=True)


def test_paged_nonfinite_values_reach_only_their_rows(g):
    gn = gen(21)
    page, d, n, lq, at = 16, 64, 200, 70, 160
    for cdt in (BF16, F8):
        kc, vc, ks, vs, _, _ = make_cache(g, gn, 13, 2, page, d, BF16, cdt)
        table = torch.arange(13, dtype=torch.int32, device="cuda")[None]
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        q = randn(gn, (1, lq, 4, d), BF16)
        kw = dict(k_scale=ks, v_scale=vs)
        clean, _ = g.attn_paged(q, kc, vc, table, lens, **kw)
        x = torch.zeros((1, 2, d), dtype=BF16, device="cuda")
        x[0, 0, 3] = math.inf
        kk, _ = g.kv_cache_read(torch.tensor([at], device="cuda"), kc, vc, ks, vs)
        g.kv_cache_write(kk, x, torch.tensor([at], device="cuda"), kc, vc, ks, vs)
        o, _ = g.attn_paged(q, kc, vc, table, lens, **kw)
        first = at - (n - lq)
        assert torch.equal(o[0, :first], clean[0, :first])
        seen = o[0, first:, :2].float()
        assert (torch.isnan(seen).all() if cdt == F8 else (seen[..., 3] == math.inf).all())


def test_paged_offsets_past_32_bits(g):
    """Caches of 5 GiB each (bfloat16) and 2.5 GiB (e4m3): the sequence's keys
    lie in the last pages.  Only those are ever touched."""
    Hk, page, d, n, T = 8, 64, 128, 150, 40
    pages = 5 * (1 << 30) // (Hk * page * d * 2)
    for cdt in (BF16, F8):
        gn = gen(51)
        kc, vc = (torch.empty((pages, Hk, page, d), dtype=cdt, device="cuda") for _ in range(2))
        ks, vs = (torch.empty((pages, Hk, page), dtype=torch.uint8, device="cuda") for _ in range(2)) \
            if cdt == F8 else (None, None)
        k, v = randn(gn, (n, Hk, d), BF16), randn(gn, (n, Hk, d), BF16)
        table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32, device="cuda")
        t = torch.arange(n, device="cuda")
        slots = table[0, t // page].long() * page + t % page
        print(f"paged large cache {cdt} pages={pages}", flush=True)
        g.kv_cache_write(k, v, slots, kc, vc, ks, vs)
        rk, rv = g.kv_cache_read(slots, kc, vc, ks, vs)
        if cdt == F8:
            k, v = (ref.quantise(x.double())[0] for x in (k, v))
        assert torch.equal(rk.double(), k.double()) and torch.equal(rv.double(), v.double())
        lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        for t_new in (1, T):
            q = randn(gn, (1, t_new, 16, d), BF16)
            o, lse = g.attn_paged(q, kc, vc, table, lens, k_scale=ks, v_scale=vs, want_lse=True)
            r = ref.attn(q[0].double(), k.double(), v.double(), 0, d ** -0.5)
            ref.check_attn({"o": o[0], "lse": lse[0]}, r, BF16, n, d, f"new {t_new}")
        del kc, vc, ks, vs
        torch.cuda.empty_cache()


def test_paged_table_of_no_pages(g):
    """A batch that holds no keys yet: every query sees nothing."""
    gn = gen(53)
    for dtype, cdt in CACHES:
        for shape in ((3, 1, 4, 64), (2, 40, 4, 64)):
            kc, vc, ks, vs, _, _ = make_cache(g, gn, 2, 2, 16, 64, dtype, cdt)
            q = randn(gn, shape, dtype)
            table = torch.empty((shape[0], 0), dtype=torch.int32, device="cuda")
            lens = torch.full((shape[0],), 7, dtype=torch.int32, device="cuda")
            o, lse = g.attn_paged(q, kc, vc, table, lens, k_scale=ks, v_scale=vs, want_lse=True)
            assert (o == 0).all() and (lse == -math.inf).all()


def test_paged_entries_outside_the_cache_stand_for_zeros(g):
    gn = gen(52)
    Hk, page, d, n = 2, 16, 64, 100
    for dtype, cdt in CACHES:
        for T, Hq in ((1, 4), (9, 4), (60, 4)):
            kc, vc, ks, vs, kd, vd = make_cache(g, gn, 8, Hk, page, d, dtype, cdt)
            table = torch.arange(8, dtype=torch.int32, device="cuda")[None].clone()
            kd, vd = kd.clone(), vd.clone()
            for at, e in ((1, 8), (3, -1), (4, 1 << 30)):
                table[0, at] = e
                kd[at * page:(at + 1) * page] = 0
                vd[at * page:(at + 1) * page] = 0
            print(f"paged bad entries T={T} {dtype} {cdt}", flush=True)
            q = randn(gn, (1, T, Hq, d), dtype)
            o, lse = g.attn_paged(q, kc, vc, table, torch.tensor([n], dtype=torch.int32, device="cuda"), k_scale=ks,
                                  v_scale=vs, want_lse=True)
            r = ref.attn(q[0].double(), kd[:n], vd[:n], 0, d ** -0.5)
            ref.check_attn({"o": o[0], "lse": lse[0]}, r, dtype, n, d, f"new {T}")


# ------------------------------------------------------- as they are used
def layer_weights(gn, d, Hq, Hk):
    return torch.rand(d, generator=gn, device="cuda") + 0.5, torch.rand(d, generator=gn, device="cuda") + 0.5


@pytest.mark.parametrize("f8", [False, True])
def test_hybrid_layer_prompt_then_decode(g, f8):
    """A window layer over a prompt, its cache, then single tokens: each
    token's output equals whole-sequence attention over everything so far."""
    gn = gen(31)
    B, T, steps, Hq, Hk, d, page, W = 3, 150, 5, 8, 2, 128, 16, 64
    n = T + steps
    q0, k0, v = (randn(gn, (B, n, h, d), BF16) for h in (Hq, Hk, Hk))
    wq, wk = layer_weights(gn, d, Hq, Hk)
    fr = g.rope_frequencies(d, scaling="yarn", factor=4.0, original_length=2048)
    pos = torch.arange(n, device="cuda", dtype=torch.int32).expand(B, n).contiguous()
    per = -(-n // page)
    table = torch.randperm(B * per, generator=gn, device="cuda").to(torch.int32).reshape(B, per)
    cdt = F8 if f8 else BF16
    kc, vc = (torch.zeros((B * per, Hk, page, d), device="cuda").to(cdt) for _ in range(2))
    ks, vs = (torch.zeros((B * per, Hk, page), dtype=torch.uint8, device="cuda") for _ in range(2)) if f8 else (None, None)

    def slots(t0, t1):
        t = torch.arange(t0, t1, device="cuda")
        return (table[:, t // page].long() * page + t % page).reshape(-1).contiguous()

    cut = lambda x, t0, t1: x[:, t0:t1].contiguous()
    q, k = g.qk_norm_rope(cut(q0, 0, T), cut(k0, 0, T), fr, wq, wk, cut(pos, 0, T))
    g.attn_fwd(q, k, cut(v, 0, T), window=W)
    g.kv_cache_write(k, cut(v, 0, T), slots(0, T), kc, vc, ks, vs)
    outs = []
    for t in range(T, n):
        q, k = g.qk_norm_rope(cut(q0, t, t + 1), cut(k0, t, t + 1), fr, wq, wk, cut(pos, t, t + 1))
        g.kv_cache_write(k, cut(v, t, t + 1), slots(t, t + 1), kc, vc, ks, vs)
        lens = torch.full((B,), t + 1, dtype=torch.int32, device="cuda")
        outs.append(g.attn_paged(q, kc, vc, table, lens, k_scale=ks, v_scale=vs, window=W)[0])
    outs = torch.cat(outs, 1)
    # the same through whole-sequence attention on what the cache holds
    qa, ka = g.qk_norm_rope(q0, k0, fr, wq, wk, pos)
    kr, vr = g.kv_cache_read(slots(0, n), kc, vc, ks, vs)
    kr, vr = (x.reshape(B, n, Hk, d) for x in (kr, vr))
    if not f8:
        assert torch.equal(kr, ka) and torch.equal(vr, v)
    o, _ = g.attn_fwd(qa, kr, vr, window=W)
    for b in range(B):
        r = ref.attn(qa[b, T:].double(), kr[b].double(), vr[b].double(), W, d ** -0.5)
        ref.check_attn({"o": outs[b]}, r, BF16, n, d, "decode")
        ref.check_attn({"o": o[b, T:]}, r, BF16, n, d, "whole")


def replay(fn, outputs, between, reps=3):
    """fn captured; every replay's outputs against the eager ones, bit for bit."""
    fn()
    torch.cuda.synchronize()
    want = [x.clone() for x in outputs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        fn()
    for r in range(reps):
        for x in outputs:
            x.zero_()
        gr.replay()
        between()
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(outputs, want)):
            assert torch.equal(x, y), f"replay {r}, output {i}"


def test_training_step_in_a_graph(g):
    gn = gen(41)
    B, T, Hq, Hk, d, W = 2, 260, 4, 2, 64, 100
    q0, k0, v, do = (randn(gn, (B, T, h, d), BF16) for h in (Hq, Hk, Hk, Hq))
    wq, wk = layer_weights(gn, d, Hq, Hk)
    fr = g.rope_frequencies(d)
    q, k, o = torch.empty_like(q0), torch.empty_like(k0), torch.empty_like(q0)
    lse = torch.empty((B, T, Hq), device="cuda")
    ga = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v)}
    gb = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dwq": torch.empty(d, device="cuda"),
          "dwk": torch.empty(d, device="cuda")}
    wa = torch.empty(g.attn_bwd_workspace_bytes(B, T, Hq, Hk, d), dtype=torch.uint8, device="cuda")
    wb = torch.empty(g.lib().gdn2_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hk, d), dtype=torch.uint8, device="cuda")

    def step():
        g.qk_norm_rope(q0, k0, fr, wq, wk, out=(q, k))
        g.attn_fwd(q, k, v, window=W, out=o, lse=lse)
        g.attn_bwd(q, k, v, o, lse, do, window=W, workspace=wa, out=ga)
        g.qk_norm_rope_bwd(q0, k0, fr, ga["dq"], ga["dk"], wq, wk, workspace=wb, out=gb)

    print("graph: training step", flush=True)
    replay(step, [o, lse, ga["dv"], *gb.values()], lambda: g.attn_fwd(q0, k0, v))


def test_two_calls_at_once(g):
    """Calls on two streams, each with a workspace of its own, and two graphs
    that take turns on one workspace, give the serial results."""
    gn = gen(63)
    B, T, Hq, Hk, d = 1, 1500, 8, 1, 128
    x = [[randn(gn, (B, T, h, d), BF16) for h in (Hq, Hk, Hk, Hq)] for _ in range(2)]
    kc, vc, _, _, _, _ = make_cache(g, gn, 200, Hk, 16, d, BF16, BF16)
    table = torch.arange(200, dtype=torch.int32, device="cuda").view(2, 100).contiguous()
    lens = torch.tensor([1600, 999], dtype=torch.int32, device="cuda")
    qd = [randn(gn, (2, 1, Hq, d), BF16) for _ in range(2)]
    need = max(g.attn_bwd_workspace_bytes(B, T, Hq, Hk, d), g.attn_paged_workspace_bytes(qd[0], kc, table))
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]

    def step(i, w):
        q, k, v, do = x[i]
        o, lse = g.attn_fwd(q, k, v, window=700)
        gr = g.attn_bwd(q, k, v, o, lse, do, window=700, workspace=w)
        od, _ = g.attn_paged(qd[i], kc, vc, table, lens, workspace=w)
        return [o, lse, gr["dq"], gr["dk"], gr["dv"], od]

    want = [step(i, ws[0]) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [None, None]
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = step(i, ws[i])
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(i, ws[0]))
        graphs.append(graph)
    for _ in range(3):
        for i in range(2):
            for t in outs[i]:
                t.fill_(7.0)
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[i], want[i]))


def test_decode_step_in_a_graph(g):
    gn = gen(42)
    N, Hq, Hk, d, page, n = 4, 8, 2, 128, 32, 900
    per = -(-n // page)
    kc, vc, ks, vs, _, _ = make_cache(g, gn, N * per, Hk, page, d, BF16, F8)
    table = torch.randperm(N * per, generator=gn, device="cuda").to(torch.int32).reshape(N, per)
    lens = torch.tensor([900, 33, 512, 1], dtype=torch.int32, device="cuda")
    last = (lens - 1).long()
    slots = table.gather(1, (last // page)[:, None])[:, 0].long() * page + last % page
    q0, k0, v = (randn(gn, (N, 1, h, d), BF16) for h in (Hq, Hk, Hk))
    fr = g.rope_frequencies(d)
    pos = (lens - 1)[:, None].contiguous()
    q, k, o = torch.empty_like(q0), torch.empty_like(k0), torch.empty_like(q0)
    ws = torch.empty(max(1, g.attn_paged_workspace_bytes(q, kc, table)), dtype=torch.uint8, device="cuda")

    def step():
        g.qk_norm_rope(q0, k0, fr, positions=pos, out=(q, k))
        g.kv_cache_write(k, v, slots, kc, vc, ks, vs)
        g.attn_paged(q, kc, vc, table, lens, k_scale=ks, v_scale=vs, out=o, workspace=ws)

    print("graph: decode step", flush=True)
    replay(step, [o], lambda: g.attn_paged(q0, kc, vc, table, lens, k_scale=ks, v_scale=vs))
