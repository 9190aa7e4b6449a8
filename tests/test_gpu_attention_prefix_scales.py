"""Keys of very small and large scales in an e4m3 prefix, on an MI355X, against plain float64 forms."""
import pytest
import torch

from test_gpu_attention_prefix import BF16, F32, Call, g  # noqa: F401 (g: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("power", [-100, 60])
def test_prefix_key_scales(g, power, dtype):
    """The prefix's and the own keys' exponent bytes moved by a power of two, the queries by its inverse
    (scores of size 1), for tiles of 32 rows and of 128: the scale is applied to the prefix's codes on the
    way to shared memory, or to the scores.  Then the prefix's values' bytes as well."""
    page, Hk, d, P = 16, 1, 64, 200
    for N in (3, 70):
        print(f"prefix key scales 2^{power} N={N} {dtype}", flush=True)
        c = Call(g, [P], [0, N], [1] * N, [3] * N, 4, Hk, d, page, dtype, True, seed=41)
        o0, lse0 = c.run(g)
        c.c.ks.copy_((c.c.ks.int() + power).to(torch.uint8))
        c.q.mul_(2.0 ** -power)
        c.c.rows = [(k * 2.0 ** power, v) for k, v in c.c.rows]
        o, lse = c.run(g)
        c.check(o, lse)
        # powers of two, all of them exact: the same scores and the same bits
        assert torch.equal(o, o0) and torch.equal(lse, lse0)
        s = c.c.slots(0, P)
        c.c.vs[s // page, :, s % page] = (c.c.vs[s // page, :, s % page].int() + power // 2).to(torch.uint8)
        c.c.rows[0] = (c.c.rows[0][0], c.c.rows[0][1] * 2.0 ** (power // 2))
        c.check(*c.run(g))
