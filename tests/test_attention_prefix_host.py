"""Refusals and workspace sizes of shared-prefix attention, without a GPU."""
import ctypes
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


def prefix(L, q=FAKE, ks=None, vs=None, ptab=FAKE, plens=FAKE, groups=None, table=FAKE, lens=FAKE, cu=None, B=2, T=1,
           Hq=4, Hk=2, d=64, N=0, M=1, pages=10, page=16, mpp=5, mp=5, scale=0.125, dt=BF16, cdt=BF16, o=FAKE, lse=None,
           ws=FAKE, ws_bytes=1 << 40):
    return L.gdn2_attn_paged_prefix(q, FAKE, FAKE, ks, vs, ptab, plens, groups, table, lens, cu, B, T, Hq, Hk, d, N, M,
                                    pages, page, mpp, mp, scale, dt, cdt, o, lse, ws, ws_bytes, None)


def test_refusals(L):
    def r(**kw):
        return prefix(L, **kw)
    assert r(dt=F8) == 2 and r(dt=F32, cdt=BF16) == 2 and r(cdt=9) == 2
    assert r(cdt=F8) == 1 and r(cdt=F8, ks=FAKE) == 1 and r(ks=FAKE, vs=FAKE) == 1
    assert r(d=32) == 2 and r(page=8) == 2 and r(page=512) == 2 and r(pages=0) == 1 and r(pages=1 << 27) == 1
    assert r(mp=-1) == 2 and r(mp=(1 << 24) + 1) == 2 and r(mpp=-1) == 2 and r(mpp=(1 << 24) + 1) == 2 and r(mpp=BIG) == 2
    assert r(Hq=3) == 1 and r(B=0) == 1 and r(T=-1) == 1 and r(scale=0.0) == 1
    assert r(N=2) == 1 and r(cu=FAKE, B=1) == 1 and r(cu=FAKE, B=2, N=2) == 1
    assert r(M=0) == 1 and r(M=-3) == 1 and r(M=2) == 1 and b"cu_groups" in L.gdn2_last_error()
    assert r(M=BIG, groups=FAKE) == 2
    for p in ("q", "ptab", "plens", "table", "lens", "o"):
        assert r(**{p: None}) == 1 and r(**{p: FAKE + 8}) == 1, p
    assert r(groups=FAKE + 4) == 1 and r(lse=FAKE + 4) == 1 and r(cu=FAKE + 4, B=1, N=1) == 1 and r(ws=FAKE + 8) == 1
    assert r(ws=None) == 3 and r(ws_bytes=100) == 3
    assert r(T=0) == 0 and L.gdn2_last_error() == b""


def test_workspace_bytes(L):
    f = L.gdn2_attn_paged_prefix_workspace_bytes
    n = f(2, 1, 4, 2, 64, 0, 1, 16, 5, 5)
    assert n >= 2 * 2 * 4 * 65 * 4 and n % (2 * 4 * 65 * 4) == 0  # a part of each kind at least
    assert prefix(L, ws_bytes=n - 1) == 3
    assert f(2, 1, 4, 2, 64, 0, 1, 16, 0, 0) == 2 * 2 * 4 * 65 * 4
    assert f(2, 0, 4, 2, 64, 0, 1, 16, 5, 5) == 0 and f(2, 1, 4, 2, 48, 0, 1, 16, 5, 5) == 0
    assert f(2, 1, 4, 2, 64, 0, 0, 16, 5, 5) == 0 and f(1, BIG, 4, 2, 64, 0, 1, 16, BIG, BIG) == 0
    assert L.gdn2_last_error() == b""


def test_binding_refusals():
    import gated_delta_rule_07_amd as g
    q, k = torch.zeros((2, 1, 4, 64)), torch.zeros((3, 2, 16, 64))
    t = torch.zeros((2, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        g.attn_paged_prefix(q, k, k, t[:1], t[0], t, t[:, 0])
