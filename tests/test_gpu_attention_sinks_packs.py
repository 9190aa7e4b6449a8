"""Attention with sinks on packed batches whose sequences differ much in length, on an MI355X,
against plain float64 forms (bounds as in test_gpu_attention_sinks)."""
import pytest
import torch

from test_gpu_attention_sinks import BF16, F32, cu_of, g, randn, run  # noqa: F401 (g: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(1, 200), (60, 33), (5, 1024)])
def test_more_sinks_than_tokens(g, window, sinks, dtype):
    """Sequences that have fewer tokens among them than their sinks could be."""
    lens = [3, 0, 410, 1, 250, 40, 2, 130] + [5, 1, 0, 2] * 8
    assert len(lens) * sinks > sum(lens)
    run(g, lens, 6, 2, 64, dtype, window, sinks, seed=window, tail=11)
    run(g, lens, 4, 1, 128, dtype, window, sinks, seed=sinks)


def test_workspace_of_more_sinks_than_tokens(g):
    """The workspace asked for is all that the backward writes, and a call on it gives the bits of one on a larger one."""
    lens, Hq, Hk, d = [700, 3, 1, 300] + [4] * 60, 4, 2, 64
    T, kw = sum(lens), dict(cu_seqlens=cu_of(lens), window=20, sinks=500)
    print("workspace of more sinks than tokens", flush=True)
    q, k, v, do = (randn(70 + i, (1, T, h, d), BF16) for i, h in enumerate((Hq, Hk, Hk, Hq)))
    o, lse = g.attn_fwd(q, k, v, **kw)
    need = g.attn_bwd_workspace_bytes(1, T, Hq, Hk, d, BF16, sinks=500, num_seqs=len(lens))
    room = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    got = g.attn_bwd(q, k, v, o, lse, do, workspace=room[:need], **kw)
    assert (room[need:] == 0x5a).all()
    big = torch.full((2 * need,), 0xff, dtype=torch.uint8, device="cuda")
    again = g.attn_bwd(q, k, v, o, lse, do, workspace=big, **kw)
    assert all(torch.equal(got[n], again[n]) for n in ("dq", "dk", "dv"))
