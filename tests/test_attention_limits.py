"""Limits of the attention operators' arguments, checked without a GPU."""
import pytest
import torch


def test_windows_that_are_none():
    import gated_delta_rule_07_amd as g
    q = torch.zeros((1, 4, 4, 64))
    k = torch.zeros((1, 4, 2, 64))
    t = torch.zeros((1, 1), dtype=torch.int32)
    # (-2^32 is 0 and -2^32 + 5 is 5 in the low 32 bits)
    for w in (-1, -2 ** 32, -2 ** 32 + 5):
        with pytest.raises(ValueError, match="window"):
            g.attn_fwd(q, k, k, window=w)
        with pytest.raises(ValueError, match="window"):
            g.attn_bwd(q, k, k, q, q, q, window=w)
        with pytest.raises(ValueError, match="window"):
            g.attn_paged(q, k, k, t, t[0], window=w)
        with pytest.raises(ValueError, match="window"):
            g.attn_paged_workspace_bytes(q, k, t, window=w)
    with pytest.raises(TypeError):
        g.attn_fwd(q, k, k, window=2.5)


def test_scales_that_overflow_in_base_two():
    """The kernels take exponents in base 2: scale log2 e has to be finite in
    float32 as well (a score of 0 would become 0 times an infinity)."""
    from test_attention_host import bwd, fwd, paged
    import gated_delta_rule_07_amd as g
    L = g.lib()
    for f in (fwd, bwd, paged):
        for scale in (2.4e38, 3.4e38):
            assert f(L, scale=scale) == 1
            assert b"scale" in L.gdn2_last_error()
