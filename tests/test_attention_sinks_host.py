"""Refusals and workspace sizes of the attention operators with sinks, without a GPU."""
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


def fwd(L, q=FAKE, cu=None, B=2, T=64, Hq=4, Hk=2, d=64, N=0, window=9, sinks=2, scale=0.125, dt=BF16, o=FAKE, **_):
    return L.gdn2_attn_sink_fwd(q, FAKE, FAKE, cu, B, T, Hq, Hk, d, N, window, sinks, scale, dt, o, FAKE, None)


def bwd(L, q=FAKE, cu=None, B=2, T=64, Hq=4, Hk=2, d=64, N=0, window=9, sinks=2, scale=0.125, dt=BF16, o=FAKE, ws=FAKE,
        ws_bytes=1 << 40):
    return L.gdn2_attn_sink_bwd(q, FAKE, FAKE, o, FAKE, FAKE, cu, B, T, Hq, Hk, d, N, window, sinks, scale, dt, FAKE,
                                FAKE, FAKE, ws, ws_bytes, None)


def paged(L, q=FAKE, cu=None, B=2, T=1, Hq=4, Hk=2, d=64, N=0, pages=10, page=16, mp=100, window=9, sinks=2,
          scale=0.125, dt=BF16, o=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return L.gdn2_attn_sink_paged(q, FAKE, FAKE, None, None, FAKE, FAKE, cu, B, T, Hq, Hk, d, N, pages, page, mp, window,
                                  sinks, scale, dt, dt, o, None, ws, ws_bytes, None)


@pytest.mark.parametrize("f", [fwd, bwd, paged])
def test_refusals(L, f):
    assert f(L, sinks=-1) == 1 and b"sinks" in L.gdn2_last_error()
    assert f(L, sinks=-BIG - 1) == 1 and f(L, window=-1) == 1
    T = dict(T=5000) if f is not paged else dict(mp=1000)
    assert f(L, sinks=1025, q=FAKE, **T) == 2 and b"1024" in L.gdn2_last_error()
    # where the window hides nothing any number goes: the next check answers
    assert f(L, sinks=BIG, q=None, **T) == 1 and b"null" in L.gdn2_last_error()
    assert f(L, window=BIG, sinks=BIG, q=None) == 1 and b"null" in L.gdn2_last_error()
    assert f(L, window=0, sinks=5000, q=None, **T) == 1 and b"null" in L.gdn2_last_error()
    assert f(L, sinks=1024, q=None, **T) == 1 and b"null" in L.gdn2_last_error()
    assert f(L, dt=F8) == 2 and f(L, d=32) == 2 and f(L, Hq=3) == 1 and f(L, scale=0.0) == 1
    assert f(L, o=FAKE + 8) == 1 and f(L, cu=FAKE, B=2, N=2) == 1 and f(L, N=2) == 1


def test_bwd_workspace(L):
    w, plain = L.gdn2_attn_sink_bwd_workspace_bytes, L.gdn2_attn_bwd_workspace_bytes
    assert w(2, 64, 4, 2, 64, 0, 0) == plain(2, 64, 4, 2, 64)
    need = w(2, 64, 4, 2, 64, 0, 2)
    # sums of dk and dv of 2 sinks of every sequence and kv head
    assert need == plain(2, 64, 4, 2, 64) + 2 * 2 * 2 * 2 * 64 * 4
    assert bwd(L, ws_bytes=need - 1) == 3 and bwd(L, ws=None) == 3
    # 63 of 64 tokens visible at all times: nothing behind a window of one token
    assert w(2, 64, 4, 2, 64, 0, 63) == plain(2, 64, 4, 2, 64) == w(2, 64, 4, 2, 64, 0, BIG)
    # packed: sums for every sequence
    assert w(1, 640, 4, 2, 64, 30, 2) - plain(1, 640, 4, 2, 64) == 30 * (w(1, 640, 4, 2, 64, 1, 2) - plain(1, 640, 4, 2, 64))
    # more sinks than a call takes: what a call needs whose window hides nothing
    assert w(1, 5000, 4, 2, 64, 0, 4000) == plain(1, 5000, 4, 2, 64)
    assert w(1, 64, 4, 2, 48, 0, 2) == 0 and w(0, 64, 4, 2, 64, 0, 2) == 0 and w(2, 64, 4, 2, 64, 3, 2) == 0
    assert w(BIG, BIG, 4, 2, 64, 0, 2) == 0 and w(2, 64, 4, 2, 64, 0, -1) == 0
    assert L.gdn2_last_error() == b""


def test_bwd_most_sinks(L):
    """A launch for every 32 sinks of a sequence and kv head has to fit a grid."""
    big = dict(cu=FAKE, B=1, T=1 << 22, Hq=8, Hk=8, N=1 << 16)
    assert bwd(L, sinks=1024, **big) == 2 and b"32 sinks" in L.gdn2_last_error()
    assert bwd(L, sinks=480, q=None, **big) == 1 and b"null" in L.gdn2_last_error()
    assert fwd(L, sinks=1024, q=None, **big) == 1 and b"null" in L.gdn2_last_error()
    assert L.gdn2_attn_sink_bwd_workspace_bytes(1, 1 << 22, 8, 8, 64, 1 << 16, 1024) == 0
    assert L.gdn2_attn_sink_bwd_workspace_bytes(1, 1 << 22, 8, 8, 64, 1 << 16, 480) > 0


def test_paged_workspace(L):
    w, plain = L.gdn2_attn_sink_paged_workspace_bytes, L.gdn2_attn_paged_workspace_bytes
    assert w(1, 1, 16, 4, 128, 0, 16, 1000, 0, 0) == plain(1, 1, 16, 4, 128, 0, 16, 1000, 0)
    assert w(1, 1, 16, 4, 128, 0, 16, 1000, 500, 0) == plain(1, 1, 16, 4, 128, 0, 16, 1000, 500)
    assert w(1, 1, 16, 4, 128, 0, 16, 1000, 500, 1000) > plain(1, 1, 16, 4, 128, 0, 16, 1000, 500)
    assert w(1, 1, 16, 4, 128, 0, 16, 1000, 500, 5000) == 0 and w(1, 1, 16, 4, 128, 0, 16, 1000, 500, -5) == 0


def test_binding_refusals():
    import gated_delta_rule_07_amd as g
    q, k = torch.zeros((1, 4, 4, 64)), torch.zeros((1, 4, 2, 64))
    t = torch.zeros((1, 1), dtype=torch.int32)
    for s in (-1, -2 ** 32, -2 ** 32 + 5):
        with pytest.raises(ValueError, match="sinks"):
            g.attn_fwd(q, k, k, window=2, sinks=s)
        with pytest.raises(ValueError, match="sinks"):
            g.attn_bwd(q, k, k, q, q, q, window=2, sinks=s)
        with pytest.raises(ValueError, match="sinks"):
            g.attn_paged(q, k, k, t, t[0], window=2, sinks=s)
        with pytest.raises(ValueError, match="sinks"):
            g.attn_paged_workspace_bytes(q, k, t, window=2, sinks=s)
        with pytest.raises(ValueError, match="sinks"):
            g.attn_bwd_workspace_bytes(1, 4, 4, 2, 64, sinks=s)
    with pytest.raises(TypeError):
        g.attn_fwd(q, k, k, window=2, sinks=2.5)
