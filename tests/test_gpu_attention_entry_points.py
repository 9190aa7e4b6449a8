"""The C entry points of attention without sinks, called directly on an MI355X: the same bits as the
binding's calls (which go through the entry points with sinks), every pointer in its place."""
import pytest
import torch

from test_gpu_attention_sinks import BF16, F32, Paged, cu_of, g, randn  # noqa: F401 (g: the fixture)

pytestmark = pytest.mark.gpu


def ptr(t):
    return 0 if t is None else t.data_ptr()


def code(dtype):
    return 1 if dtype == BF16 else 0


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("packed", [False, True])
def test_forward_and_backward(g, packed, dtype):
    B, T, Hq, Hk, d, window, scale = (1, 730, 6, 2, 64, 90, 0.11) if packed else (3, 250, 6, 2, 64, 90, 0.11)
    cu = cu_of([300, 0, 430]) if packed else None
    N = 3 if packed else 0
    print(f"entry points packed={packed} {dtype}", flush=True)
    L = g.lib()
    q, k, v, do = (randn(300 + i, (B, T, h, d), dtype) for i, h in enumerate((Hq, Hk, Hk, Hq)))
    want_o, want_lse = g.attn_fwd(q, k, v, cu, window=window, scale=scale)
    want = g.attn_bwd(q, k, v, want_o, want_lse, do, cu, window=window, scale=scale)
    o, lse = torch.full_like(q, 7.0), torch.full((B, T, Hq), 7.0, device="cuda")
    assert L.gdn2_attn_fwd(ptr(q), ptr(k), ptr(v), ptr(cu), B, T, Hq, Hk, d, N, window, scale, code(dtype), ptr(o),
                           ptr(lse), stream()) == 0
    assert torch.equal(o, want_o) and torch.equal(lse, want_lse)
    assert not torch.equal(o, g.attn_fwd(q, k, v, cu, scale=scale)[0])  # (the window counts)
    o2 = torch.full_like(q, 7.0)
    assert L.gdn2_attn_fwd(ptr(q), ptr(k), ptr(v), ptr(cu), B, T, Hq, Hk, d, N, window, scale, code(dtype), ptr(o2), 0,
                           stream()) == 0
    assert torch.equal(o2, want_o)
    need = L.gdn2_attn_bwd_workspace_bytes(B, T, Hq, Hk, d)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    gr = {n: torch.full_like(x, 7.0) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    assert L.gdn2_attn_bwd(ptr(q), ptr(k), ptr(v), ptr(o), ptr(lse), ptr(do), ptr(cu), B, T, Hq, Hk, d, N, window, scale,
                           code(dtype), *(ptr(gr[n]) for n in ("dq", "dk", "dv")), ptr(ws), need, stream()) == 0
    assert all(torch.equal(gr[n], want[n]) for n in gr)
    assert not torch.equal(gr["dk"], gr["dv"])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_paged(g, packed, f8, dtype):
    page, Hq, Hk, d, window, scale, T = 16, 8, 2, 64, 200, 0.13, 2
    lk = [700, 3, 0, 250]
    print(f"entry point paged packed={packed} f8={f8} {dtype}", flush=True)
    L, N = g.lib(), len(lk)
    c = Paged(g, lk, Hk, d, page, dtype, f8, seed=31)
    # (keys and values of different scales, so that one in the other's place shows)
    if f8:
        c.vs += 2
    table = c.table.cuda()
    cu = cu_of([T] * N) if packed else None
    shape = (1, N * T, Hq, d) if packed else (N, T, Hq, d)
    q = randn(311, shape, dtype)
    want_o, want_lse = g.attn_paged(q, c.k, c.v, table, c.lens, cu, window=window, scale=scale, want_lse=True, **c.scales())
    P, mp = c.k.shape[0], table.shape[1]
    B, Tq, ns = shape[0], shape[1], N if packed else 0
    need = L.gdn2_attn_paged_workspace_bytes(B, Tq, Hq, Hk, d, ns, page, mp, window)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    o, lse = torch.full_like(q, 7.0), torch.full(shape[:3], 7.0, device="cuda")
    assert L.gdn2_attn_paged(ptr(q), ptr(c.k), ptr(c.v), ptr(c.ks), ptr(c.vs), ptr(table), ptr(c.lens), ptr(cu), B, Tq, Hq,
                             Hk, d, ns, P, page, mp, window, scale, code(dtype), 2 if f8 else code(dtype), ptr(o), ptr(lse),
                             ptr(ws), need, stream()) == 0
    assert torch.equal(o, want_o) and torch.equal(lse, want_lse)
    assert not torch.equal(o, g.attn_paged(q, c.k, c.v, table, c.lens, cu, scale=scale, **c.scales())[0])
