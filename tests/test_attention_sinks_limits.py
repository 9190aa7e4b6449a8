"""Workspaces and parts of the attention with sinks at sizes where they grow, without a GPU."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module", params=["libgdn2.so", "libgdn2_hostcheck.so"])
def L(request):
    import gated_delta_rule_07_amd as g
    path = os.path.join(os.path.dirname(g.LIB_PATH), request.param)
    if not os.path.exists(path):
        pytest.fail(f"{request.param} is not built (run __graft_entry__.build())")
    return g.lib() if request.param == "libgdn2.so" else g.configure(ctypes.CDLL(path))


def far_parts(T, N, Hk, G, sinks):
    """Workgroups that share the rows behind the window of each 32-sink tile of a sequence and kv head:
    1024 over all tiles, at most 64, and one for every 128 rows of the call."""
    return max(1, min(64, -(-1024 // (N * Hk * -(-sinks // 32))), T * G // 128))


@pytest.mark.parametrize("T,N,Hk,d,sinks", [(32768, 512, 4, 128, 1024), (262144, 4096, 4, 128, 128), (5000, 700, 2, 64, 33),
                                            (2100, 3, 1, 64, 1000)])
def test_bwd_workspace_of_many_short_sequences(L, T, N, Hk, d, sinks):
    """Packed sequences have at most T sinks among them, however many each may have:
    the workspace holds float32 sums of dk and dv for no more in each part, beside those
    that one long sequence has more."""
    w, plain = L.gdn2_attn_sink_bwd_workspace_bytes, L.gdn2_attn_bwd_workspace_bytes
    assert N * sinks > T
    each, one = far_parts(T, N, Hk, 4, sinks), far_parts(T, 1, Hk, 4, sinks)
    far = w(1, T, 4 * Hk, Hk, d, N, sinks) - plain(1, T, 4 * Hk, Hk, d)
    assert 0 < far <= (each * T + (one - each) * sinks) * 2 * Hk * d * 4


@pytest.mark.parametrize("T,N,Hk,d,sinks", [(32550, 256, 4, 128, 4), (32512, 64, 4, 128, 4), (9973, 11, 4, 64, 33),
                                            (6000, 100, 1, 64, 40), (32768, 1, 4, 128, 4), (700, 30, 2, 64, 1)])
def test_bwd_parts_of_one_long_sequence_among_many(L, T, N, Hk, d, sinks):
    """Whatever the number of sequences, there are parts for a long one's rows as if it were alone."""
    w, plain = L.gdn2_attn_sink_bwd_workspace_bytes, L.gdn2_attn_bwd_workspace_bytes
    each, one = far_parts(T, N, Hk, 4, sinks), far_parts(T, 1, Hk, 4, sinks)
    far = w(1, T, 4 * Hk, Hk, d, N, sinks) - plain(1, T, 4 * Hk, Hk, d)
    assert N * sinks <= T and far == (each * N + one - each) * sinks * 2 * Hk * d * 4
    if N > 1:  # sequences of one length share nothing by their tokens
        B, T2 = N, 64
        fixed = w(B, T2, 4 * Hk, Hk, d, 0, sinks) - plain(B, T2, 4 * Hk, Hk, d)
        assert fixed % (B * sinks * 2 * Hk * d * 4) == 0
