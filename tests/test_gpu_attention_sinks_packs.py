"""Attention with sinks on packed batches whose sequences differ much in length, on an MI355X,
against plain float64 forms (bounds as in test_gpu_attention_sinks)."""
import pytest
import torch

from test_attention_sinks_limits import far_parts
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


@pytest.mark.parametrize("window", [0, 1024, 5000])
def test_sinks_where_the_window_hides_nothing(g, window):
    """Sinks have no part then, also where a window that hides would be refused for their number
    (2^23 sequence-heads times 32 sinks): the backward finds its own workspace."""
    N, T, Hk, d, sinks = 1 << 16, 2048, 8, 64, 1024
    print(f"sinks that hide nothing window={window}", flush=True)
    assert g.attn_bwd_workspace_bytes(1, T, Hk, Hk, d, BF16, sinks=sinks, num_seqs=N) == 0
    cu = torch.full((N + 1,), T, dtype=torch.int32, device="cuda")
    cu[:3] = torch.tensor([0, 1500, 1503], dtype=torch.int32, device="cuda")
    q, k, v, do = (randn(80 + i, (1, T, Hk, d), BF16) for i in range(4))
    o, lse = g.attn_fwd(q, k, v, cu, window=window, sinks=sinks)
    o0, lse0 = g.attn_fwd(q, k, v, cu)
    assert torch.equal(o, o0) and torch.equal(lse, lse0)
    got, want = g.attn_bwd(q, k, v, o, lse, do, cu, window=window, sinks=sinks), g.attn_bwd(q, k, v, o, lse, do, cu)
    assert all(torch.equal(got[n], want[n]) for n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_long_sequence_among_short_ones(g, d, dtype):
    """A long sequence's far rows go to more workgroups than its neighbours', wherever it stands."""
    short = [9, 0, 40, 1, 130, 3] * 10
    long = 2500 if dtype == BF16 else 1300
    for lens in ([long] + short, short + [long], short[:31] + [long] + short[31:], [long // 2] + short + [long // 2, 0, 5]):
        run(g, lens, 8, 2, d, dtype, 100, 4, seed=len(lens), tail=33)
    # more than 32 sinks, and more of them than tokens
    run(g, short + [long] + short, 3, 1, d, dtype, 64, 50, seed=5)
    run(g, [1] * 200 + [long] + short, 4, 2, d, dtype, 37, 40, seed=6, tail=3)


def test_long_sequence_among_short_ones_many_heads(g):
    """Heads of a group in several turns over the tokens (a tile has at most 32 of them)."""
    run(g, [5, 0, 30] * 20 + [900, 2], 96, 2, 64, BF16, 50, 7, seed=9)
    run(g, [5, 700] + [8] * 50, 66, 2, 64, BF16, 20, 3, seed=10)


def test_long_sequence_workspace_and_bits(g):
    """The workspace is all that is written, whatever it held before, and runs repeat their bits."""
    lens, Hq, Hk, d = [4] * 150 + [3000] + [7] * 50, 8, 2, 64
    T, kw = sum(lens), dict(cu_seqlens=cu_of(lens), window=128, sinks=33)
    print("long sequence's workspace", flush=True)
    q, k, v, do = (randn(90 + i, (1, T, h, d), BF16) for i, h in enumerate((Hq, Hk, Hk, Hq)))
    o, lse = g.attn_fwd(q, k, v, **kw)
    need = g.attn_bwd_workspace_bytes(1, T, Hq, Hk, d, BF16, sinks=33, num_seqs=len(lens))
    room = torch.full((need + 4096,), 0xff, dtype=torch.uint8, device="cuda")
    got = g.attn_bwd(q, k, v, o, lse, do, workspace=room[:need], **kw)
    assert (room[need:] == 0xff).all()
    for _ in range(4):
        again = g.attn_bwd(q, k, v, o, lse, do, workspace=room[:need], **kw)
        assert all(torch.equal(got[n], again[n]) for n in ("dq", "dk", "dv"))


# over 512 sequences of few tokens: each has one workgroup for a kv head's far rows, 16 tiles of
# which are left to a long one's before it has more by its tokens
MANY = ([0] * 7 + [3, 0, 1]) * 52


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_long_sequence_among_hundreds(g, d, dtype):
    """The far rows of one or two long sequences in parts that they alone have, wherever they stand."""
    long = 2500
    assert len(MANY) * 2 >= 1024 and (long - 100) * 4 // 128 > 32
    for lens in ([long] + MANY, MANY + [long], MANY[:301] + [long] + MANY[301:], [long] + MANY + [1900]):
        run(g, lens, 8, 2, d, dtype, 100, 4, seed=len(lens), tail=21)
    # more than 32 sinks, and more of them than tokens
    run(g, MANY[:200] + [long] + MANY[200:], 8, 2, d, dtype, 64, 50, seed=7)
    run(g, MANY + [long, 0, 0], 4, 1, d, dtype, 30, 130, seed=8, tail=2)


def test_long_sequence_among_hundreds_many_heads(g):
    """The same with heads of a group in several turns over the tokens."""
    run(g, MANY[:99] + [1100] + MANY, 66, 2, 64, BF16, 20, 3, seed=11)


def test_long_sequence_among_hundreds_workspace_and_bits(g):
    """The workspace is all that is written, whatever it held before; runs and replays repeat their bits."""
    lens, Hq, Hk, d = MANY[:250] + [3000] + MANY[250:], 8, 2, 64
    T, kw = sum(lens), dict(cu_seqlens=cu_of(lens), window=128, sinks=33)
    print("long sequence among hundreds, workspace", flush=True)
    q, k, v, do = (randn(95 + i, (1, T, h, d), BF16) for i, h in enumerate((Hq, Hk, Hk, Hq)))
    o, lse = g.attn_fwd(q, k, v, **kw)
    need = g.attn_bwd_workspace_bytes(1, T, Hq, Hk, d, BF16, sinks=33, num_seqs=len(lens))
    room = torch.full((need + 4096,), 0xff, dtype=torch.uint8, device="cuda")
    want = g.attn_bwd(q, k, v, o, lse, do, workspace=room[:need], **kw)
    assert (room[need:] == 0xff).all()
    # (its end holds the parts by tokens: the long sequence's are among them)
    each, one = (far_parts(T, n, Hk, Hq // Hk, 33) for n in (len(lens), 1))
    more = (one - each) * 33 * 2 * Hk * d * 4
    assert each == 1 and (room[need - more:need] != 0xff).any()
    want = {n: x.clone() for n, x in want.items()}
    gr = {n: torch.empty_like(x) for n, x in want.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.attn_bwd(q, k, v, o, lse, do, workspace=room[:need], out=gr, **kw)
    for i in range(3):
        again = g.attn_bwd(q, k, v, o, lse, do, workspace=room[:need], **kw)
        assert all(torch.equal(want[n], again[n]) for n in want)
        room.fill_(i)
        for x in gr.values():
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[n], gr[n]) for n in want), i
