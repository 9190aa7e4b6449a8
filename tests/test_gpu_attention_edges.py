"""Attention operators on an MI355X at the edges of what their documentation
allows: table entries outside the cache beside a page of NaN, windows past the
test_gpu_attention.py."""
import math

import pytest
import torch

import attention_ref as ref
from test_gpu_attention import CACHES, g, gen, make_cache, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,cdt", CACHES)
@pytest.mark.parametrize("T", [1, 9, 60])
def test_paged_bad_entries_beside_a_page_of_nan(g, T, dtype, cdt):
    """Entries outside the cache stand for zeros whatever the cache's pages
    hold: page 0 (no sequence's) is NaN throughout, its scales too."""
    gn = gen(71)
    Hq, Hk, page, d, n, pages = 4, 2, 16, 64, 133, 9
    kc, vc, ks, vs, kd, vd = make_cache(g, gn, pages, Hk, page, d, dtype, cdt)
    for c, s in ((kc, ks), (vc, vs)):
        if s is not None:
            s[0] = 255
            c.view(torch.uint8)[0] = 0x7f
        else:
            c[0] = math.nan
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].clone()
    kd, vd = kd.clone(), vd.clone()
    for at, e in ((0, -1), (1, pages), (4, 1 << 30), (8, -(1 << 31))):
        table[0, at] = e
        kd[at * page:(at + 1) * page] = 0
        vd[at * page:(at + 1) * page] = 0
    print(f"paged bad entries, page 0 of NaN, T={T} {dtype} {cdt}", flush=True)
    q = randn(gn, (1, T, Hq, d), dtype)
    o, lse = g.attn_paged(q, kc, vc, table, torch.tensor([n], dtype=torch.int32, device="cuda"), k_scale=ks, v_scale=vs,
                          want_lse=True)
    r = ref.attn(q[0].double(), kd[:n], vd[:n], 0, d ** -0.5)
    ref.check_attn({"o": o[0], "lse": lse[0]}, r, dtype, n, d, f"new {T}")
