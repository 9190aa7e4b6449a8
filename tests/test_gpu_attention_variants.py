"""The attention kernels' variants on an MI355X, each at shapes that select it:
the rules that pick a variant are read from the sources, so that a changed
threshold fails here rather than leaving a variant untested.  Bounds as in
test_gpu_attention.py."""
import math
import os
import re

import pytest
import torch

import attention_ref as ref
from test_gpu_attention import BF16, CACHES, F32, g, gen, randn, run_attn, run_paged  # noqa: F401

pytestmark = pytest.mark.gpu


def source(name):
    import gated_delta_rule_07_amd as mod
    with open(os.path.join(os.path.dirname(mod.LIB_PATH), "csrc", name)) as f:
        return f.read()


def rows_128(units, tiles):
    """Whether a whole-sequence call (forward, dq) of this many 128-row tiles
    takes the 128-row kernels (few_tiles)."""
    n = re.search(r"bool few_tiles\(const order &od\) \{ return static_cast<long long>\(od\.units\) \* od\.tiles < (\d+); \}",
                  source("gdn2_attn.hpp"))
    return units * tiles >= int(n.group(1))


def fixed_128(B, T, Hq, Hk):
    return rows_128(B * Hk, -(-T * (Hq // Hk) // 128))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 2048])
def test_128_row_tiles_long(g, window, d, dtype):
    """Forward and backward over many unmasked key tiles."""
    B, T, Hq, Hk = 1, 4096, 16, 4
    assert fixed_128(B, T, Hq, Hk)
    print(f"128-row tiles, T={T} window={window} d={d} {dtype}", flush=True)
    run_attn(g, [T] * B, Hq, Hk, d, dtype, window, False, True, seed=81)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_128_row_tiles_packed(g, d, dtype):
    lens, Hq, Hk = [1300, 0, 1, 777, 2000, 129], 8, 2
    assert rows_128(Hk, sum(lens) * (Hq // Hk) // 128 + len(lens))
    for window in (0, 500):
        print(f"128-row tiles, packed window={window} d={d} {dtype}", flush=True)
        run_attn(g, lens, Hq, Hk, d, dtype, window, True, True, seed=82, tail=21)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_128_row_tiles_large_scores(g, dtype):
    """Scores of hundreds: one key takes all the weight."""
    gn = gen(83)
    B, T, Hq, Hk, d = 16, 210, 16, 4, 64
    assert fixed_128(B, T, Hq, Hk)
    print(f"128-row tiles, large scores {dtype}", flush=True)
    q, k, v = (randn(gn, (B, T, h, d), dtype) * 30 for h in (Hq, Hk, Hk))
    o, lse = g.attn_fwd(q, k, v)
    for b in range(B):
        r = ref.attn(q[b].double(), k[b].double(), v[b].double(), 0, d ** -0.5)
        ref.check_attn({"o": o[b], "lse": lse[b]}, r, dtype, T, d, f"large {b}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("window", [0, 40])
def test_128_row_tiles_nonfinite_values_reach_only_their_rows(g, window, bad, dtype):
    gn = gen(84)
    B, T, Hq, Hk, d, b, at = 16, 210, 16, 4, 128, 5, 101
    G = Hq // Hk
    assert fixed_128(B, T, Hq, Hk)
    q, k, v = (randn(gn, (B, T, h, d), dtype) for h in (Hq, Hk, Hk))
    clean, _ = g.attn_fwd(q, k, v, window=window)
    for which in ("k", "v"):
        print(f"128-row tiles, {bad} in {which} window={window} {dtype}", flush=True)
        k2, v2 = k.clone(), v.clone()
        (k2 if which == "k" else v2)[b, at, 0, 5] = bad
        o, _ = g.attn_fwd(q, k2, v2, window=window)
        see = torch.zeros((B, T, Hq), dtype=torch.bool, device="cuda")
        see[b, at:(at + window if window else T), :G] = True
        # rows that do not see the key: the same bits
        assert torch.equal(o[~see], clean[~see]), which
        if which == "v":
            x = o[see][:, 5].float()
            want = torch.full_like(x, bad)
            assert torch.equal(torch.isnan(x), torch.isnan(want))
            assert (torch.isnan(want) | (x == want)).all()
            rest = [c for c in range(d) if c != 5]
            # the same weights: the sums may differ by the order of a term
            a, c = o[see][:, rest].double(), clean[see][:, rest].double()
            assert ((a - c).abs() <= 2.0 ** -7 * c.abs() + 2.0 ** -9).all()


def whole_key_tiles(T, B, Hq, Hk, keys):
    """Whether dk and dv of a fixed-length call take the form of `keys` keys a
    workgroup, without parts: a rule on the number of its key tiles."""
    s = source("gdn2_attn_bwd.hip")
    n = re.search(r"a\.parts == 1 && static_cast<long long>\(a\.od\.units\) \* a\.od\.tiles >= (\d+)", s)
    p = re.search(r"long long p = \((\d+) \+ tiles - 1\) / \(tiles > 0 \? tiles : 1\);\s+if \(p > rows / (\d+)\)\s+p = rows / (\d+);", s)
    assert p.group(2) == p.group(3)
    tiles = B * -(-T // 64) * Hk
    parts = max(1, min((int(p.group(1)) + tiles - 1) // tiles, T * (Hq // Hk) // int(p.group(2)), 16))
    return parts == 1 and B * Hk * -(-T // keys) >= int(n.group(1))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_dkv_whole_key_tiles(g, d, dtype):
    """dk and dv where there are key tiles enough for the larger form: 128
    keys a workgroup in bfloat16, 64 in float32."""
    B, T, Hq, Hk = 64, 130, 16, 8
    assert fixed_128(B, T, Hq, Hk) and whole_key_tiles(T, B, Hq, Hk, 128 if dtype == BF16 else 64)
    for window in (0, 100):
        print(f"dk, dv of whole key tiles, window={window} d={d} {dtype}", flush=True)
        run_attn(g, [T] * B, Hq, Hk, d, dtype, window, False, True, seed=85)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [64, 128])
def test_dkv_whole_key_tiles_packed(g, d, dtype):
    """The same, packed: sequences of up to several key tiles, empty ones, and
    groups of heads that a row tile does not divide (5 of 64 rows)."""
    lens = [(97 * i * i + 13) % 401 if i % 7 else 0 for i in range(90)]
    Hq, Hk = 40, 8
    assert whole_key_tiles(sum(lens), 1, Hq, Hk, 128 if dtype == BF16 else 64)
    for window in (0, 130):
        print(f"dk, dv of whole key tiles, packed window={window} d={d} {dtype}", flush=True)
        run_attn(g, lens, Hq, Hk, d, dtype, window, True, True, seed=86, tail=3)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [1, 64, 1000])
def test_dkv_parts_under_a_window(g, window, dtype):
    """Few key tiles whose rows several workgroups share while the window
    leaves them few rows each, or none."""
    T, Hq, Hk, d = 2300, 8, 1, 128
    assert g.attn_bwd_workspace_bytes(1, T, Hq, Hk, d) > -(-T * Hq * 8 // 256) * 256  # parts
    print(f"dk, dv in parts, window={window} {dtype}", flush=True)
    run_attn(g, [T], Hq, Hk, d, dtype, window, False, True, seed=window)


def paged_rows(Ttot, N, Hq, Hk, T=None):
    """Rows of a paged call's tiles: 16 (the decode kernel, bfloat16, T tokens
    for every sequence), 32 or 128."""
    s = source("gdn2_attn_fwd.hip")
    few = int(re.search(r"z\.Ttot\) \* \(z\.Hq / z\.Hk\) <= (\d+)LL \* z\.N", s).group(1))
    dec = int(re.search(r"!z\.packed && static_cast<long long>\(z\.T\) \* \(z\.Hq / z\.Hk\) <= (\d+)", s).group(1))
    if T is not None and T * (Hq // Hk) <= dec:
        return 16
    return 32 if Ttot * (Hq // Hk) <= few * N else 128


@pytest.mark.parametrize("dtype,cdt", CACHES)
@pytest.mark.parametrize("d", [64, 128])
def test_paged_32_row_tiles(g, d, dtype, cdt):
    """17 to 32 rows for every sequence (speculative steps)."""
    for T, Hq, Hk, page, window in ((5, 8, 2, 16, 0), (8, 8, 2, 64, 50), (1, 20, 1, 32, 0), (6, 15, 3, 16, 333)):
        lk = [T, 50, 700, 1, 2049]
        assert paged_rows(T * len(lk), len(lk), Hq, Hk, T) == 32
        print(f"paged 32-row tiles T={T} Hq={Hq} Hk={Hk} page={page} W={window} d={d} {dtype} {cdt}", flush=True)
        run_paged(g, [T] * len(lk), lk, Hq, Hk, d, page, dtype, cdt, window, False, seed=T, poison=True)


@pytest.mark.parametrize("dtype,cdt", CACHES)
@pytest.mark.parametrize("d", [64, 128])
def test_paged_32_row_tiles_packed(g, d, dtype, cdt):
    """Packed batches of single tokens, and of a few tokens each."""
    for lq, lk, Hq, Hk, page, window, tail in (([1] * 9, [1, 15, 16, 17, 300, 64, 2000, 33, 128], 8, 2, 16, 0, 0),
                                               ([1] * 70, [(37 * i * i + 1) % 200 + 1 for i in range(70)], 8, 2, 32, 60, 7),
                                               ([1, 2, 0, 3, 1], [700, 420, 33, 2, 0], 8, 2, 64, 0, 13),
                                               ([1, 2, 0, 3, 1], [700, 420, 33, 2, 5], 16, 1, 256, 77, 3)):
        assert paged_rows(sum(lq) + tail, len(lq), Hq, Hk) == 32
        print(f"paged 32-row tiles packed n={len(lq)} Hq={Hq} Hk={Hk} page={page} W={window} d={d} {dtype} {cdt}", flush=True)
        run_paged(g, lq, lk, Hq, Hk, d, page, dtype, cdt, window, True, seed=page, tail=tail, poison=True)
