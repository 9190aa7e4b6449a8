"""Limits of the attention of shared prefixes, without a GPU."""
import pytest

from test_attention_prefix_host import FAKE, L, prefix  # noqa: F401 (L: the fixture)


def test_most_rows(L):
    """The join takes four rows a workgroup of 256 work-items, of which a grid holds less than 2^32: past
    2^26 - 4 rows the call is refused before anything is launched."""
    w = L.gdn2_attn_paged_prefix_workspace_bytes
    for T in (2 ** 26 - 3, 2 ** 26 - 1):
        for kw in (dict(B=1, T=T, Hq=1, Hk=1), dict(B=1, T=T, Hq=1, Hk=1, N=1, cu=FAKE)):
            assert -(-T // 4) * 256 >= 2 ** 32
            assert prefix(L, ws_bytes=0, **kw) == 2 and b"2^26 - 4" in L.gdn2_last_error()
        assert w(1, T, 1, 1, 64, 0, 1, 16, 5, 5) == 0
    most = 2 ** 26 - 4
    assert most // 4 * 256 < 2 ** 32
    assert prefix(L, B=1, T=most, Hq=1, Hk=1, ws_bytes=0) == 3
    assert w(1, most, 1, 1, 64, 0, 1, 16, 5, 5) == 2 * most * 65 * 4
