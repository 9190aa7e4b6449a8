// gdn2_attn_order.hpp -- which workgroup takes which tile (host and device).
#pragma once

#include "gdn2_attn_kernels.hpp"

namespace gdn2 {
namespace attn {

// Workgroup order.  Consecutive workgroups go to the 8 dies in turn, each
// with its own L2: the tiles of one unit (a sequence's kv head, which reads
// the same keys and values) are kept on one die, or, with fewer than 8 (or
// an odd number of) units, dealt out over 8 / gcd dies.  Later tiles see more
// keys, so each die starts with its last ones.  Units of one tile (decode) share
// keys with no other workgroup and come as they are numbered, which leaves no die
// without work.  (Decode, window 2048, 4 sinks, e4m3: 85 sequences on 3 kv heads 26 us,
// as 80 take; on the one die that gcd(255, 8) gave them 148.  bfloat16: 43 and 239; 63
// sequences on 4 heads 43 and 78.)  A unit of 2 to 7 tiles, fewer than 8 / gcd, still
// leaves dies without work.
struct order {
  int units, tiles, g, tpr;  // g = gcd(units, 8) (one tile a unit: 8), tpr = ceil(tiles / (8 / g))
};
__host__ __device__ __forceinline__ bool place(const order &od, int id, int &unit, int &tile_i) {
  const int x = id & 7, idx = id >> 3, r = 8 / od.g;
  const int u = idx / od.tpr, t = (od.tpr - 1 - idx % od.tpr) * r + x / od.g;
  unit = u * od.g + x % od.g;
  tile_i = t;
  return unit < od.units && t < od.tiles;
}
// The number of workgroups of an order.
inline unsigned workgroups(const order &od) {
  return 8u * static_cast<unsigned>((od.units + od.g - 1) / od.g) * static_cast<unsigned>(od.tpr);
}
// Fills the order of tiles of BM rows (GR rows a token) and returns the
// number of workgroups.
inline unsigned plan_tiles(const attn_sizes &z, int GR, int BM, order &od) {
  const long long rows = static_cast<long long>(z.T) * GR;
  od.tiles = static_cast<int>(z.packed ? rows / BM + z.N : (rows + BM - 1) / BM);
  od.units = z.packed ? z.Hk : z.N * z.Hk;
  od.g = od.units % 8 == 0 || od.tiles == 1 ? 8 : od.units % 4 == 0 ? 4 : od.units % 2 == 0 ? 2 : 1;
  const int r = 8 / od.g;
  od.tpr = (od.tiles + r - 1) / r;
  return workgroups(od);
}

}  // namespace attn
}  // namespace gdn2
