"""Refusals of the attention operators that need no GPU: every bad argument is
answered with the documented status before anything is launched, by the
product library and by its host-checked build; and the rotation's
frequencies against their definitions."""
import ctypes
import math
import os

import pytest
import torch

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every case fails first
F32, BF16, F8 = 0, 1, 2
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module", params=["libgdn2.so", "libgdn2_hostcheck.so"])
def L(request):
    import gated_delta_rule_07_amd as g
    path = os.path.join(os.path.dirname(g.LIB_PATH), request.param)
    if not os.path.exists(path):
        pytest.fail(f"{request.param} is not built (run __graft_entry__.build())")
    return g.lib() if request.param == "libgdn2.so" else g.configure(ctypes.CDLL(path))


def rope(L, bwd=False, q=FAKE, wq=FAKE, freqs=FAKE, pos=FAKE, B=2, T=8, Hq=4, Hk=2, d=64, rot=64, eps=1e-6, dt=BF16,
         flags=0, out=FAKE, dw=FAKE, ws=FAKE, ws_bytes=1 << 40):
    head = (q, FAKE, wq, wq, freqs, pos)
    sizes = (B, T, Hq, Hk, d, rot, eps, dt, flags)
    if bwd:
        return L.gdn2_qk_norm_rope_bwd(*head, FAKE, FAKE, *sizes, out, FAKE, dw, dw, ws, ws_bytes, None)
    return L.gdn2_qk_norm_rope_fwd(*head, *sizes, out, FAKE, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_rope_refusals(L, bwd):
    def r(**kw):
        return rope(L, bwd, **kw)
    assert r(dt=F8) == 2 and r(dt=7) == 2
    assert r(d=32) == 2 and r(d=96) == 2 and r(d=256) == 2
    assert r(rot=4) == 2 and r(rot=72) == 2 and r(rot=-8) == 2
    assert r(rot=0) == 1 and r(freqs=None) == 1
    assert r(B=0) == 1 and r(T=-1) == 1 and r(Hq=0) == 1 and r(Hk=-1) == 1
    assert r(flags=4) == 1
    assert r(flags=2) == 1                       # weights without the norm
    assert r(eps=-1.0) == 1 and r(eps=math.nan) == 1
    assert r(q=None) == 1 and r(q=FAKE + 8) == 1 and r(wq=FAKE + 4) == 1 and r(out=FAKE + 2) == 1
    assert r(B=BIG, T=BIG) == 2 and r(T=1 << 24, Hq=16) == 2 and r(Hq=BIG, Hk=BIG) == 2
    if bwd:
        assert r(ws_bytes=16) == 3 and r(ws=None) == 3
        assert r(flags=2, wq=None) == 1          # weight gradients without the norm
    else:
        assert r(T=0) == 0


def test_rope_workspace_bytes(L):
    f = L.gdn2_qk_norm_rope_bwd_workspace_bytes
    assert f(8, 4096, 16, 4, 128) == 1024 * 2 * 128 * 4
    assert 0 < f(1, 1, 1, 1, 64) <= 1024 * 2 * 64 * 4
    assert f(BIG, BIG, 1, 1, 64) == 0 and f(1, 8, 1, 1, 32) == 0 and f(0, 8, 1, 1, 64) == 0


def fwd(L, q=FAKE, cu=None, B=2, T=64, Hq=4, Hk=2, d=64, N=0, window=0, scale=0.125, dt=BF16, o=FAKE, lse=FAKE):
    return L.gdn2_attn_fwd(q, FAKE, FAKE, cu, B, T, Hq, Hk, d, N, window, scale, dt, o, lse, None)


def bwd(L, q=FAKE, cu=None, B=2, T=64, Hq=4, Hk=2, d=64, N=0, window=0, scale=0.125, dt=BF16, o=FAKE, lse=FAKE,
        ws=FAKE, ws_bytes=1 << 40):
    return L.gdn2_attn_bwd(q, FAKE, FAKE, o, lse, FAKE, cu, B, T, Hq, Hk, d, N, window, scale, dt, FAKE, FAKE, FAKE, ws,
                           ws_bytes, None)


@pytest.mark.parametrize("f", [fwd, bwd])
def test_attn_refusals(L, f):
    assert f(L, dt=F8) == 2 and f(L, dt=5) == 2
    assert f(L, d=16) == 2 and f(L, d=32) == 2 and f(L, d=192) == 2
    assert f(L, Hq=5) == 1 and f(L, Hk=0) == 1 and f(L, Hq=2, Hk=4) == 1
    assert f(L, B=0) == 1 and f(L, T=-1) == 1 and f(L, N=-1) == 1
    assert f(L, N=2) == 1 and f(L, cu=FAKE, N=2) == 1 and f(L, cu=FAKE, B=1, N=0) == 1
    assert f(L, window=-1) == 1
    for s in (0.0, -1.0, math.inf, math.nan):
        assert f(L, scale=s) == 1
    assert f(L, q=None) == 1 and f(L, q=FAKE + 8) == 1 and f(L, o=None) == 1 and f(L, lse=FAKE + 4) == 1
    assert f(L, cu=FAKE + 4, B=1, N=2) == 1
    assert f(L, T=1, B=1, Hq=1 << 16, Hk=1) == 2
    assert f(L, B=BIG, T=BIG) == 2 and f(L, T=1 << 24) == 2 and f(L, B=1, cu=FAKE, N=BIG) == 2
    assert f(L, T=0) == 0
    assert L.gdn2_last_error() == b""
    if f is bwd:
        assert f(L, lse=None) == 1
        assert f(L, ws_bytes=2 * 64 * 4 * 8 - 1) == 3 and f(L, ws=None) == 3


def test_attn_bwd_workspace_bytes(L):
    f = L.gdn2_attn_bwd_workspace_bytes
    assert f(2, 64, 4, 2, 64) == 2 * 64 * 4 * 8
    assert f(2, 64, 5, 2, 64) == 0 and f(BIG, BIG, 4, 2, 64) == 0 and f(1, 64, 4, 2, 48) == 0
    assert L.gdn2_last_error() == b""


def paged(L, q=FAKE, ks=None, vs=None, table=FAKE, lens=FAKE, cu=None, B=2, T=1, Hq=4, Hk=2, d=64, N=0, pages=10,
          page=16, mp=5, window=0, scale=0.125, dt=BF16, cdt=BF16, o=FAKE, lse=None, ws=FAKE, ws_bytes=1 << 40):
    return L.gdn2_attn_paged(q, FAKE, FAKE, ks, vs, table, lens, cu, B, T, Hq, Hk, d, N, pages, page, mp, window, scale,
                             dt, cdt, o, lse, ws, ws_bytes, None)


def test_paged_refusals(L):
    assert paged(L, dt=F8) == 2 and paged(L, dt=F32, cdt=BF16) == 2 and paged(L, cdt=9) == 2
    assert paged(L, cdt=F8) == 1 and paged(L, cdt=F8, ks=FAKE) == 1 and paged(L, ks=FAKE, vs=FAKE) == 1
    assert paged(L, d=32) == 2 and paged(L, page=8) == 2 and paged(L, page=48) == 2 and paged(L, page=512) == 2
    assert paged(L, pages=0) == 1 and paged(L, pages=1 << 27) == 1
    assert paged(L, mp=-1) == 2 and paged(L, mp=(1 << 24) + 1) == 2
    assert paged(L, Hq=3) == 1 and paged(L, B=0) == 1 and paged(L, T=-1) == 1
    assert paged(L, N=2) == 1 and paged(L, cu=FAKE, B=1) == 1 and paged(L, cu=FAKE, B=2, N=2) == 1
    assert paged(L, window=-3) == 1 and paged(L, scale=0.0) == 1
    assert paged(L, q=None) == 1 and paged(L, table=None) == 1 and paged(L, lens=FAKE + 4) == 1
    assert paged(L, o=FAKE + 8) == 1
    assert paged(L, mp=1000, ws_bytes=100) == 3 and paged(L, mp=1000, ws=None) == 3
    assert paged(L, T=0) == 0


def test_paged_workspace_bytes(L):
    f = L.gdn2_attn_paged_workspace_bytes
    n = f(1, 1, 16, 4, 128, 0, 16, 1000, 0)
    assert n > 0 and n % (16 * 129 * 4) == 0          # parts x (o and lse) of 16 rows
    assert f(1, 1, 16, 4, 128, 0, 16, 1, 0) == 0      # one page: nothing to split
    assert f(4096, 1, 16, 4, 128, 0, 16, 1000, 0) == 0  # rows enough
    assert f(1, 1, 16, 4, 48, 0, 16, 1000, 0) == 0 and f(1, 0, 16, 4, 128, 0, 16, 1000, 0) == 0
    assert f(1, BIG, 16, 4, 128, 0, 16, BIG, BIG) == 0


def cache(L, read=False, k=FAKE, slots=FAKE, n=5, Hk=2, d=64, pages=4, page=16, dt=BF16, cdt=BF16, kc=FAKE, ks=None,
          vs=None):
    if read:
        return L.gdn2_kv_cache_read(slots, n, Hk, d, pages, page, dt, cdt, kc, FAKE, ks, vs, k, FAKE, None)
    return L.gdn2_kv_cache_write(k, FAKE, slots, n, Hk, d, pages, page, dt, cdt, kc, FAKE, ks, vs, None)


@pytest.mark.parametrize("read", [False, True])
def test_cache_refusals(L, read):
    def c(**kw):
        return cache(L, read, **kw)
    assert c(dt=F8, cdt=F8, ks=FAKE, vs=FAKE) == 2 and c(cdt=F32) == 2
    assert c(cdt=F8) == 1 and c(ks=FAKE, vs=FAKE) == 1 and c(cdt=F8, vs=FAKE) == 1
    assert c(d=48) == 2 and c(page=1) == 2 and c(pages=0) == 1 and c(pages=BIG) == 1
    assert c(n=-1) == 1 and c(Hk=0) == 1 and c(n=BIG) == 2 and c(n=1 << 25, Hk=2) == 2
    assert c(k=None) == 1 and c(k=FAKE + 8) == 1 and c(kc=FAKE + 1) == 1 and c(slots=None) == 1 and c(slots=FAKE + 4) == 1
    assert c(n=0) == 0


def test_binding_takes_device_tensors_only():
    import gated_delta_rule_07_amd as g
    q, k = torch.zeros((1, 4, 4, 64)), torch.zeros((1, 4, 2, 64))
    with pytest.raises(ValueError, match="device"):
        g.attn_fwd(q, k, k)
    with pytest.raises(ValueError, match="device"):
        g.qk_norm_rope(q, k, None)
    with pytest.raises(ValueError, match="device"):
        g.kv_cache_read(torch.zeros(1, dtype=torch.int64), k, k)


def test_rope_frequencies():
    import gated_delta_rule_07_amd as g
    f = g.rope_frequencies(64, device="cpu")
    j = torch.arange(32, dtype=torch.float64)
    assert f.dtype == torch.float64 and torch.allclose(f, 10000.0 ** (-2 * j / 64), rtol=1e-15, atol=0)
    lin = g.rope_frequencies(64, scaling="linear", factor=8.0, device="cpu")
    assert torch.equal(lin, f / 8)
    ntk = g.rope_frequencies(64, scaling="ntk", factor=8.0, device="cpu")
    assert ntk[0] == 1.0 and math.isclose(ntk[-1].item(), f[-1].item() / 8, rel_tol=1e-12)
    yarn = g.rope_frequencies(64, scaling="yarn", factor=8.0, original_length=4096, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(yarn[turns >= 32], f[turns >= 32])
    assert torch.allclose(yarn[turns <= 1], f[turns <= 1] / 8, rtol=1e-15, atol=0)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (yarn[mid] < f[mid]).all() and (yarn[mid] > f[mid] / 8).all()
    for kw in (dict(rotary_dim=12), dict(rotary_dim=0), dict(rotary_dim=64, scaling="x"),
               dict(rotary_dim=64, scaling="yarn", factor=2.0),
               dict(rotary_dim=64, scaling="yarn", factor=2.0, original_length=4096, beta_fast=1.0), dict(rotary_dim=64, scaling="linear", factor=0.0)):
        with pytest.raises(ValueError):
            g.rope_frequencies(device="cpu", **kw)
