"""Attention operators on an MI355X at the edges of what their documentation
allows.  Bounds as in test_gpu_attention.py."""
import math

import pytest
import torch

import attention_ref as ref
from test_gpu_attention import BF16, CACHES, F8, F32, g, gen, make_cache, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cdt", CACHES)
@pytest.mark.parametrize("T", [1, 9, 60])
def test_paged_bad_entries_beside_a_page_of_nan(g, T, dtype, cdt):
    """Entries outside the cache stand for zeros whatever the cache's pages
    hold: page 0 (no sequence's) is NaN throughout, its scales too."""
    gn = gen(71)
    Hq, Hk, page, d, n, pages = 4, 2, 16, 64, 133, 9
    kc, vc, ks, vs, kd, vd = make_cache(g, gn, pages, Hk, page, d, dtype, cdt)
    for c, s in ((kc, ks), (vc, vs)):
        if s is not None:
            s[0] = 255
            c.view(torch.uint8)[0] = 0x7f
        else:
            c[0] = math.nan
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].clone()
    kd, vd = kd.clone(), vd.clone()
    for at, e in ((0, -1), (1, pages), (4, 1 << 30), (8, -(1 << 31))):
        table[0, at] = e
        kd[at * page:(at + 1) * page] = 0
        vd[at * page:(at + 1) * page] = 0
    print(f"paged bad entries, page 0 of NaN, T={T} {dtype} {cdt}", flush=True)
    q = randn(gn, (1, T, Hq, d), dtype)
    o, lse = g.attn_paged(q, kc, vc, table, torch.tensor([n], dtype=torch.int32, device="cuda"), k_scale=ks, v_scale=vs,
                          want_lse=True)
    r = ref.attn(q[0].double(), kd[:n], vd[:n], 0, d ** -0.5)
    ref.check_attn({"o": o[0], "lse": lse[0]}, r, dtype, n, d, f"new {T}")


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 63])
def test_window_past_the_range_of_an_int(g, window):
    """A window longer than every sequence hides nothing, however long it is."""
    gn = gen(73)
    q, k, v, do = (randn(gn, (1, 300, h, 64), BF16) for h in (4, 2, 2, 4))
    o, lse = g.attn_fwd(q, k, v)
    gr = g.attn_bwd(q, k, v, o, lse, do)
    ow, lw = g.attn_fwd(q, k, v, window=window)
    gw = g.attn_bwd(q, k, v, o, lse, do, window=window)
    assert torch.equal(o, ow) and torch.equal(lse, lw)
    assert all(torch.equal(gr[n], gw[n]) for n in gr)
    kc, vc, _, _, _, _ = make_cache(g, gn, 20, 2, 16, 64, BF16, BF16)
    table = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([300], dtype=torch.int32, device="cuda")
    for t in (1, 40):
        x = q[:, :t].contiguous()
        assert g.attn_paged_workspace_bytes(x, kc, table, window=window) == g.attn_paged_workspace_bytes(x, kc, table)
        want, _ = g.attn_paged(x, kc, vc, table, lens)
        got, _ = g.attn_paged(x, kc, vc, table, lens, window=window)
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_cache_rows_of_the_smallest_exponents(g, dtype):
    """Rows down to the format's smallest scale, 2^-126, whose codes are
    multiples of 2^-135: exact in float32 always, in bfloat16 (smallest
    subnormal 2^-133) from e = -124 up and rounded once below."""
    gn = gen(74)
    d, page, Hk = 64, 16, 2
    es = torch.arange(-131, -115, device="cuda")
    n = es.numel()
    top = torch.exp2(es.double() + 8.5)[:, None, None]     # a row's largest value: between 448 2^(e-1) and 448 2^e
    x = torch.rand((n, Hk, d), generator=gn, device="cuda", dtype=torch.float64) * 2 - 1
    x[..., 0] = 1
    k = (x * top).to(dtype)
    kc, vc = (torch.zeros((1, Hk, page, d), device="cuda").to(F8) for _ in range(2))
    ks, vs = (torch.zeros((1, Hk, page), dtype=torch.uint8, device="cuda") for _ in range(2))
    slots = torch.arange(n, device="cuda")
    g.kv_cache_write(k, k, slots, kc, vc, ks, vs)
    val, byte = ref.quantise(k.double())
    assert torch.equal(ks[0].t(), byte) and torch.equal(vs[0].t(), byte)
    e = byte.int() - 127
    assert e.min() == -126 and e.max() > -120
    for y in g.kv_cache_read(slots, kc, vc, ks, vs, dtype=F32):
        assert torch.equal(y.double(), val)
    for y in g.kv_cache_read(slots, kc, vc, ks, vs, dtype=BF16):
        off = (y.double() - val).abs()
        assert (off[e >= -124] == 0).all()
        assert (off <= 2.0 ** -134).all()
        # (rows that were bfloat16: a multiple of 2^-133 is 4 m steps of 2^-135,
        # and rounding that to a code's grid, steps of 1, 2, 4, .., leaves a
        # multiple of 4: always exact)
        assert (off > 0).any() == (dtype == F32)


@pytest.mark.parametrize("Hq,Hk,T", [(1 << 15, 1 << 15, 130), (1 << 15, 1, 3), (1 << 15, 1 << 12, 40)])
def test_most_query_heads(g, Hq, Hk, T):
    """2^15 query heads, each its own kv head or sharing: some heads of every
    part against float64."""
    gn = gen(75)
    d, G = 64, Hq // Hk
    print(f"most heads Hq={Hq} Hk={Hk} T={T}", flush=True)
    q, k, v, do = (randn(gn, (1, T, h, d), BF16) for h in (Hq, Hk, Hk, Hq))
    o, lse = g.attn_fwd(q, k, v)
    gr = g.attn_bwd(q, k, v, o, lse, do)
    for h in sorted({0, Hk // 2, Hk - 1}):
        hq = slice(h * G, (h + 1) * G)
        r = ref.attn(q[0, :, hq].double(), k[0, :, h:h + 1].double(), v[0, :, h:h + 1].double(), 0, d ** -0.5,
                     do[0, :, hq].double())
        ref.check_attn({"o": o[0, :, hq], "lse": lse[0, :, hq], "dq": gr["dq"][0, :, hq]}, r, BF16, T, d, f"head {h}")
        # a kv head's gradients sum T G terms, not T
        ref.check_attn({"o": o[0, :, hq], "dk": gr["dk"][0, :, h:h + 1], "dv": gr["dv"][0, :, h:h + 1]}, r, BF16, T * G, d,
                       f"kv head {h}")


def test_cache_slots_read_twice_and_far_away(g):
    """A slot may be read more than once; slots far outside read as zeros and
    are not written."""
    gn = gen(76)
    Hk, page, d, n = 3, 16, 128, 40
    for dtype, cdt in CACHES:
        kc, vc, ks, vs, kd, vd = make_cache(g, gn, 4, Hk, page, d, dtype, cdt)
        far = [-(1 << 63), -(1 << 32), -1, 4 * page, 1 << 31, 1 << 32, (1 << 32) + 5, (1 << 63) - 1]
        slots = torch.cat([torch.tensor(far, device="cuda"), torch.arange(n, device="cuda"), torch.full((n,), 7, device="cuda")])
        keep = [x.clone() for x in (kc.view(torch.uint8), vc.view(torch.uint8))]
        x = randn(gn, (len(far), Hk, d), dtype)
        g.kv_cache_write(x, x, slots[:len(far)].contiguous(), kc, vc, ks, vs)
        assert torch.equal(kc.view(torch.uint8), keep[0]) and torch.equal(vc.view(torch.uint8), keep[1])
        for y, c in zip(g.kv_cache_read(slots, kc, vc, ks, vs, dtype=dtype), (kd, vd)):
            m = len(far)
            assert (y[:m] == 0).all()
            assert torch.equal(y[m:m + n].double(), c[:n])
            assert torch.equal(y[m + n:].double(), c[7].expand(n, Hk, d))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B", [1, 32])
def test_rows_whose_scores_are_all_minus_infinity(g, B, dtype):
    """Such a row counts as one that sees nothing: o = 0, lse = -inf, in the
    32-row and the 128-row kernels and over the cache."""
    gn = gen(77)
    T, Hq, Hk, d, n = 210, 16, 4, 64, 3
    q, k, v = (randn(gn, (B, T, h, d), dtype) for h in (Hq, Hk, Hk))
    q[:, :, :, 5] = 1
    k[:, :n, :, 5] = -math.inf
    o, lse = g.attn_fwd(q, k, v)
    assert (o[:, :n] == 0).all() and (lse[:, :n] == -math.inf).all()
    r = ref.attn(q[0, n:].double(), k[0, n:].double(), v[0, n:].double(), 0, d ** -0.5)
    ref.check_attn({"o": o[0, n:], "lse": lse[0, n:]}, r, dtype, T, d, "rows that see other keys")
    kc, vc = (torch.zeros((B, Hk, 16, d), device="cuda").to(dtype) for _ in range(2))
    slots = (torch.arange(B, device="cuda")[:, None] * 16 + torch.arange(n, device="cuda")).reshape(-1)
    kn, vn = (x[:, :n].contiguous() for x in (k, v))
    g.kv_cache_write(kn, vn, slots, kc, vc)
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    for t in (1, n, 60):   # (60: rows without any key too)
        lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
        o, lse = g.attn_paged(q[:, :t].contiguous(), kc, vc, table, lens, want_lse=True)
        assert (o == 0).all() and (lse == -math.inf).all()
