"""Which workgroup takes which tile of an attention call, without a GPU: every tile once,
units of one tile spread evenly over the 8 dies that consecutive workgroups go to in turn."""
import os
import subprocess

import pytest

MAIN = r"""
#include <cstdio>
#include "gdn2_attn_order.hpp"
using namespace gdn2::attn;
// lines "N T Hk packed GR BM" in; out: units, tiles, workgroups, then unit and tile of every workgroup (-1 -1: none)
int main() {
  int N, T, Hk, packed, GR, BM;
  while (std::scanf("%d %d %d %d %d %d", &N, &T, &Hk, &packed, &GR, &BM) == 6) {
    attn_sizes z = {};
    z.N = N;
    z.T = T;
    z.Hk = Hk;
    z.packed = packed != 0;
    order od;
    const unsigned n = plan_tiles(z, GR, BM, od);
    std::printf("%d %d %u", od.units, od.tiles, n);
    for (unsigned i = 0; i < n; ++i) {
      int u, t;
      const bool live = place(od, static_cast<int>(i), u, t);
      std::printf(" %d %d", live ? u : -1, live ? t : -1);
    }
    std::printf("\n");
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """plan(cases): (units, tiles, [(unit, tile) of every workgroup]) for each (N, T, Hk, packed, GR, BM)."""
    import gated_delta_rule_07_amd as g
    d = tmp_path_factory.mktemp("order")
    src, exe = d / "order.cpp", d / "order"
    src.write_text(MAIN)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", f"-I{rocm}/include",
                        "-I" + os.path.join(os.path.dirname(g.LIB_PATH), "csrc"), "-o", str(exe), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(cases):
        text = "\n".join(" ".join(str(int(x)) for x in c) for c in cases)
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout
        rows = [[int(x) for x in line.split()] for line in out.splitlines()]
        assert len(rows) == len(cases)
        return [(r[0], r[1], list(zip(r[3::2], r[4::2]))) for r in rows]

    return run


def test_every_tile_once(plan):
    cases = [(N, T, Hk, p, GR, BM) for N in (1, 2, 3, 7, 33) for T in (1, 20, 129, 1000) for Hk in (1, 2, 3, 4, 8)
             for p in (0, 1) for GR in (1, 4) for BM in (16, 32, 128)]
    for c, (units, tiles, w) in zip(cases, plan(cases)):
        live = [x for x in w if x != (-1, -1)]
        assert sorted(live) == [(u, t) for u in range(units) for t in range(tiles)], c


@pytest.mark.parametrize("parts", [1, 2, 5])
def test_units_of_one_tile_use_every_die(plan, parts):
    """Decode (T = 1): the dies' shares of the workgroups with work differ by one unit's parts at most."""
    cases = [(N, 1, Hk, 0, 4, 16) for N in list(range(1, 70)) + [85, 171, 199, 250, 1025] for Hk in (1, 2, 3, 4, 5, 8)]
    for c, (units, tiles, w) in zip(cases, plan(cases)):
        assert tiles == 1
        load = [0] * 8
        for i, x in enumerate(w):
            for s in range(parts):
                load[(i * parts + s) % 8] += x != (-1, -1)
        assert max(load) - min(load) <= parts, (c, load)


def test_a_units_tiles_stay_on_one_die(plan):
    """Units of many tiles, 8 of them or a multiple: each on one die, whose L2 holds its keys."""
    cases = [(N, 5000, Hk, 0, 4, 128) for N, Hk in ((8, 1), (2, 4), (3, 8), (6, 4))]
    for c, (units, tiles, w) in zip(cases, plan(cases)):
        assert tiles > 8
        for u in range(units):
            assert len({i % 8 for i, x in enumerate(w) if x[0] == u}) == 1, (c, u)
