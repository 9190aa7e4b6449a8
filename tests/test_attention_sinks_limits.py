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


@pytest.mark.parametrize("T,N,Hk,d,sinks", [(32768, 512, 4, 128, 1024), (262144, 4096, 4, 128, 128), (5000, 700, 2, 64, 33),
                                            (2100, 3, 1, 64, 1000)])
def test_bwd_workspace_of_many_short_sequences(L, T, N, Hk, d, sinks):
    """Packed sequences have at most T sinks among them, however many each may have:
    the workspace holds float32 sums of dk and dv for no more in each of the parts that
    share their rows (1024 workgroups over the 32-sink tiles at most, one at least)."""
    w, plain = L.gdn2_attn_sink_bwd_workspace_bytes, L.gdn2_attn_bwd_workspace_bytes
    assert N * sinks > T
    parts = max(1, min(64, -(-1024 // (N * Hk * -(-sinks // 32)))))
    far = w(1, T, 4 * Hk, Hk, d, N, sinks) - plain(1, T, 4 * Hk, Hk, d)
    assert 0 < far <= parts * 2 * T * Hk * d * 4
