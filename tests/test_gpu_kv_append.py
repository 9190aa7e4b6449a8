"""The cache append (norm, rotation and write of new tokens in one pass) on an
MI355X, against the formulas in float64 and against the calls it stands for."""
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


def cache(pages, Hk, page, d, dtype, f8, fill=3.0):
    kv = [torch.full((pages, Hk, page, d), fill, device="cuda").to(F8 if f8 else dtype) for _ in range(2)]
    sc = [torch.full((pages, Hk, page), 99, dtype=torch.uint8, device="cuda") if f8 else None for _ in range(2)]
    return kv, sc


def rows_of(c, slots):
    """Rows [n, Hk, ...] of a cache [pages, Hk, page, ...] (of bytes for codes)."""
    page = c.shape[2]
    c = c.view(torch.uint8) if c.dtype == F8 else c
    return c[slots // page, :, slots % page]


# B, T, Hq, Hk, d, rot, interleaved, far, norm, weights, page, layout
CASES = [
    (1, 1, 1, 1, 64, 64, False, 0, True, True, 16, "apart"),
    (5, 1, 16, 4, 128, 128, False, 1 << 22, True, True, 64, "fused"),
    (2, 33, 6, 3, 64, 32, True, 1 << 15, True, False, 32, "fused"),
    (3, 7, 5, 5, 128, 16, True, 100, False, False, 128, "gaps"),
    (1, 300, 8, 2, 128, 64, False, 9, True, True, 256, "fused"),
    (2, 19, 3, 1, 64, 0, False, 0, True, True, 16, "gaps"),
    (4, 1, 4, 4, 64, 8, False, 50, True, True, 16, "gaps"),
    (1, 2500, 16, 4, 128, 128, False, 0, True, True, 64, "fused"),
    (1, 9, 71, 9, 64, 64, True, 1 << 30, True, True, 16, "apart"),
]


def tensors(gn, B, T, Hq, Hk, d, dtype, layout):
    if layout == "apart":
        return [randn(gn, (B, T, h, d), dtype) for h in (Hq, Hk, Hk)]
    extra = 0 if layout == "fused" else 3
    x = randn(gn, (B, T, Hq + 2 * Hk + extra, d), dtype)
    return [x[:, :, a:a + n] for a, n in ((0, Hq), (Hq, Hk), (Hq + Hk, Hk))]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_append(g, i, f8, dtype):
    B, T, Hq, Hk, d, rot, inter, far, norm, weights, page, layout = CASES[i]
    print(f"append {CASES[i]} f8={f8} {dtype}", flush=True)
    gn = gen(i)
    q, k, v = tensors(gn, B, T, Hq, Hk, d, dtype, layout)
    wq, wk = (1.0 + 0.3 * torch.randn(d, generator=gn, device="cuda") for _ in range(2)) if weights else (None, None)
    freqs = g.rope_frequencies(rot) if rot else None
    pos = torch.randint(-far, far, (B, T), generator=gn, device="cuda").to(torch.int32) if far else None
    pages = -(-B * T // page) + 3
    slots = torch.randperm(pages * page, generator=gn, device="cuda")[:B * T]
    if B * T > 4:
        slots[1], slots[3] = -1, pages * page  # outside the cache: their queries only
    (kc, vc), (ks, vs) = cache(pages, Hk, page, d, dtype, f8)
    kw = dict(wq=wq, wk=wk, positions=pos, interleaved=inter, norm=norm, eps=1e-5)
    before = [x.clone() for x in (q, k, v)]
    o = g.kv_cache_append(q, k, v, slots, kc, vc, freqs, k_scale=ks, v_scale=vs, **kw)
    torch.cuda.synchronize()
    assert o.is_contiguous() and all(torch.equal(x, y) for x, y in zip((q, k, v), before))
    # q as the norm and rotation alone leave it, bit for bit
    kr_call = [x.contiguous() for x in (q, k)]
    oq, ok = g.qk_norm_rope(*kr_call, freqs, **kw)
    assert torch.equal(o, oq)
    live = (slots >= 0) & (slots < pages * page)
    at = slots[live]
    p = pos if pos is not None else torch.arange(T, device="cuda").expand(B, T)
    want = ref.rope(k.double(), None if wk is None else wk.double(), freqs, p, inter, norm, 1e-5).reshape(-1, Hk, d)[live]
    want_v = v.double().reshape(-1, Hk, d)[live]
    # a dozen roundings of the row's largest value, and the sine's and cosine's error (2^-25 of a turn and 2 ulp)
    big = 2.0 ** -20 * want.abs().amax(-1, keepdim=True)
    if not f8:
        ref.check(rows_of(kc, at), want, ref.step(dtype) * want.abs() + big, "keys")
        assert torch.equal(rows_of(kc, at), ok.reshape(-1, Hk, d)[live])
        assert torch.equal(rows_of(vc, at), v.reshape(-1, Hk, d)[live])
    else:
        val, byte = ref.quantise(want_v)
        assert torch.equal(rows_of(vs, at), byte)
        rk, rv = g.kv_cache_read(at, kc, vc, ks, vs, dtype=F32)
        assert torch.equal(rv.double(), val)
        # keys: the smallest scale that holds the row (by float32's error the other one at the border), then half a
        # step of the code: 2^-4 of a value of 2^-6 times the scale and more, 2^-10 times the scale below
        e = rows_of(ks, at).double()[..., None] - 127
        amax = want.abs().amax(-1, keepdim=True)
        tight = (amax <= 448 * torch.exp2(e) * (1 + 2.0 ** -19)) & \
            ((amax > 448 * torch.exp2(e - 1) * (1 - 2.0 ** -19)) | (e <= -126) | (amax == 0))
        assert tight.all()
        ref.check(rk, want, torch.maximum(want.abs() * 2.0 ** -4, torch.exp2(e - 10)) * (1 + 2.0 ** -18) + big, "keys")
    # nothing else was written
    for c, fill in ((kc, 3.0), (vc, 3.0), (ks, 99), (vs, 99)):
        if c is None:
            continue
        left = torch.ones(pages * page, dtype=torch.bool, device="cuda")
        left[at] = False
        left = left.nonzero()[:, 0]
        assert (rows_of(c, left) == rows_of(torch.full_like(c.float(), fill).to(c.dtype), left)).all()


@pytest.mark.parametrize("f8", [False, True])
def test_append_in_place(g, f8):
    """q's output in its own place in the projection, and into a view with other distances."""
    gn = gen(70)
    B, T, Hq, Hk, d, page = 2, 21, 8, 2, 128, 16
    x = randn(gn, (B, T, Hq + 2 * Hk, d), BF16)
    fr = g.rope_frequencies(d)
    slots = torch.arange(B * T, device="cuda")
    outs = []
    for how in ("new", "place", "view"):
        y = x.clone()
        q, k, v = y[:, :, :Hq], y[:, :, Hq:Hq + Hk], y[:, :, Hq + Hk:]
        (kc, vc), (ks, vs) = cache(4, Hk, page, d, BF16, f8)
        wide = torch.full((B, T, Hq + 5, d), 7.0, dtype=BF16, device="cuda")
        out = {"new": None, "place": q, "view": wide[:, :, 2:Hq + 2]}[how]
        o = g.kv_cache_append(q, k, v, slots, kc, vc, fr, k_scale=ks, v_scale=vs, out=out)
        outs.append([o, kc.view(torch.uint8), vc.view(torch.uint8)] + ([ks, vs] if f8 else []))
        if how == "place":
            assert torch.equal(y[:, :, Hq:], x[:, :, Hq:])
        if how == "view":
            assert (wide[:, :, :2] == 7).all() and (wide[:, :, Hq + 2:] == 7).all()
    for a, b in ((0, 1), (0, 2)):
        assert all(torch.equal(s, t) for s, t in zip(outs[a], outs[b]))


def test_append_odd_rows(g):
    """Rows of zeros, of infinities and NaN: as the norm and the write treat them; other rows are not touched."""
    gn = gen(71)
    T, Hq, Hk, d, page = 40, 4, 2, 64, 16
    q, k, v = (randn(gn, (1, T, h, d), F32) for h in (Hq, Hk, Hk))
    slots, fr = torch.arange(T, device="cuda"), g.rope_frequencies(d)
    clean = []
    for f8 in (False, True):
        (kc, vc), (ks, vs) = cache(3, Hk, page, d, F32, f8)
        g.kv_cache_append(q, k, v, slots, kc, vc, fr, k_scale=ks, v_scale=vs)
        clean.append((kc, vc, ks, vs))
    k2, v2 = k.clone(), v.clone()
    k2[0, 3, 0], v2[0, 3, 0] = 0.0, 0.0
    k2[0, 5, 1, 7], v2[0, 6, 0, 1] = math.nan, math.inf
    for f8, (kc0, vc0, ks0, vs0) in zip((False, True), clean):
        (kc, vc), (ks, vs) = cache(3, Hk, page, d, F32, f8)
        g.kv_cache_append(q, k2, v2, slots, kc, vc, fr, k_scale=ks, v_scale=vs)
        rk, rv = g.kv_cache_read(slots, kc, vc, ks, vs, dtype=F32)
        rk0, rv0 = g.kv_cache_read(slots, kc0, vc0, ks0, vs0, dtype=F32)
        assert (rk[3, 0] == 0).all() and (rv[3, 0] == 0).all()
        assert rk[5, 1].isnan().all()
        assert rv[6, 0].isnan().all() if f8 else (rv[6, 0, 1] == math.inf and torch.equal(rv[6, 0, 2:], rv0[6, 0, 2:]))
        for r, r0, odd in ((rk, rk0, [(3, 0), (5, 1)]), (rv, rv0, [(3, 0), (6, 0)])):
            keep = torch.ones((T, Hk), dtype=torch.bool, device="cuda")
            for t, h in odd:
                keep[t, h] = False
            assert torch.equal(r[keep], r0[keep])
        if f8:
            assert ks[0, 1, 5] == 255 and vs[0, 0, 6] == 255 and ks[0, 0, 3] == 127


def test_append_no_tokens(g):
    (kc, vc), _ = cache(2, 2, 16, 64, BF16, False)
    q, k = torch.empty((1, 0, 4, 64), dtype=BF16, device="cuda"), torch.empty((1, 0, 2, 64), dtype=BF16, device="cuda")
    o = g.kv_cache_append(q, k, k, torch.empty(0, dtype=torch.int64, device="cuda"), kc, vc, g.rope_frequencies(64))
    assert o.shape == q.shape and (kc == 3).all() and (vc == 3).all()


def test_append_offsets_past_32_bits(g):
    """Token strides, and cache rows, that pass 32 bits in bytes and values."""
    gn = gen(72)
    T, Hq, Hk, d, page = 5, 2, 1, 128, 64
    stride = (1 << 30) + 64
    buf = torch.empty(4 * stride + (Hq + 2 * Hk) * d, dtype=BF16, device="cuda")
    x = buf.as_strided((1, T, Hq + 2 * Hk, d), (T * stride, stride, d, 1))
    x.copy_(randn(gn, (1, T, Hq + 2 * Hk, d), BF16))
    pages = (5 << 30) // (Hk * page * d * 2)
    (kc, vc) = (torch.empty((pages, Hk, page, d), dtype=BF16, device="cuda") for _ in range(2))
    slots = torch.arange(pages * page - T, pages * page, device="cuda")
    fr = g.rope_frequencies(d)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:]
    print("append far strides", flush=True)
    o = g.kv_cache_append(q, k, v, slots, kc, vc, fr)
    oq, ok = g.qk_norm_rope(q.contiguous(), k.contiguous(), fr)
    assert torch.equal(o, oq)
    assert torch.equal(rows_of(kc, slots), ok[0]) and torch.equal(rows_of(vc, slots), v[0])


def test_append_in_a_graph_and_on_streams(g):
    gn = gen(73)
    B, T, Hq, Hk, d, page = 8, 1, 16, 4, 128, 16
    x = randn(gn, (B, T, Hq + 2 * Hk, d), BF16)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:]
    fr = g.rope_frequencies(d)
    pos = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    slots = torch.arange(B, device="cuda") * 3
    (kc, vc), (ks, vs) = cache(3, Hk, page, d, BF16, True)
    out = torch.empty((B, T, Hq, d), dtype=BF16, device="cuda")

    held = [out, kc.view(torch.uint8), vc.view(torch.uint8), ks, vs]

    def step():
        g.kv_cache_append(q, k, v, slots, kc, vc, fr, positions=pos, k_scale=ks, v_scale=vs, out=out)

    def clear():
        for t in held:
            t.zero_()

    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_(randn(gn, x.shape, BF16))
        pos.add_(1)
        slots.add_(1)
        clear()
        step()
        want = [t.clone() for t in held]
        clear()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(t, w) for t, w in zip(held, want)), i
        clear()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t, w) for t, w in zip(held, want)), i


@pytest.mark.parametrize("dtype,f8", [(BF16, False), (F32, True)])
def test_append_without_norm_and_rotation(g, dtype, f8):
    """Neither norm nor rotation: the write, from any distance between tokens."""
    gn = gen(74)
    x = randn(gn, (2, 9, 8, 64), dtype)
    q, k, v = x[:, :, :4], x[:, :, 4:6], x[:, :, 6:]
    slots = torch.arange(18, device="cuda") * 2
    (kc, vc), (ks, vs) = cache(4, 2, 16, 64, dtype, f8)
    (kc2, vc2), (ks2, vs2) = cache(4, 2, 16, 64, dtype, f8)
    o = g.kv_cache_append(q, k, v, slots, kc, vc, None, norm=False, k_scale=ks, v_scale=vs)
    g.kv_cache_write(k.contiguous(), v.contiguous(), slots, kc2, vc2, k_scale=ks2, v_scale=vs2)
    assert torch.equal(o, q)
    assert torch.equal(kc.view(torch.uint8), kc2.view(torch.uint8)) and torch.equal(vc.view(torch.uint8), vc2.view(torch.uint8))
    assert not f8 or (torch.equal(ks, ks2) and torch.equal(vs, vs2))
