// gdn2_attn_prefix.hip -- attention of new tokens over the paged cache where
// sequences share a prefix, for gfx950.
//
//   o_i = (2^(A_i - M) a_i + 2^(B_i - M) b_i) / (2^(A_i - M) + 2^(B_i - M)),  M = max(A_i, B_i)
// where a_i, A_i are the output and log2 of the sum of row i over its prefix's
// keys, b_i, B_i over its sequence's own.  The prefix is one set of keys for
// all rows of a group, and all of them are visible: the rows of a group are
// taken as one block of rows, whose tiles read the prefix's keys and values
// once for 128 rows, and not once a sequence.
//
// The prefix's part is bound by matrix products (many rows a key) and by the one
// tile a workgroup has under way, the own keys' by memory, so one launch has the
// workgroups of both and a CU works on one of either kind at a time.  Measured,
// 64 sequences behind 32768 keys with up to 1500 of their own, 16 heads on 4, d =
// 128, bfloat16 (17.6 GFLOP, 169 MB: 36 us at a large copy's rate), caches cold: 51 us
// and 7 for the join; the prefix alone 36, the own keys alone 29.  41 sequences in
// three groups, one of 200 new tokens, e4m3: 44 and 8, the prefixes alone 38 (in
// two launches the prefixes' took 45 us, and 62 with the codes widened behind
// shared memory).
#include "gdn2_attn_decode_body.hpp"
#include "gdn2_attn_launch.hpp"

namespace gdn2 {
namespace attn {

// The workgroups: `first` of the prefixes' (p), then those of the sequences'
// own keys (o).
template <typename P, typename O>
__global__ void __launch_bounds__(256, 2) gdn2_attn_prefix_kernel(fwd_args p, fwd_args o, int first) {
  static_assert(P::THREADS == 256 && O::THREADS == 256, "one launch for both");
  __shared__ __align__(16) char lds[P::BYTES > O::BYTES ? P::BYTES : O::BYTES];
  const int b = blockIdx.x;
  if (b < first)
    P::run(p, b, lds);
  else
    O::run(o, b - first, lds);
}

// The launch over the prefixes sees the groups as packed sequences of rows.
static attn_sizes prefix_sizes(const attn_sizes &z, const prefix_call &x) {
  attn_sizes y = z;
  y.N = x.ngroups;
  y.T = z.Ttot;
  y.packed = true;
  y.max_pages = x.max_pages;
  y.max_keys = static_cast<long long>(x.max_pages) << z.page_shift;
  return y;
}

// Parts of the keys.  The prefixes' workgroups are to fill one of the two places
// a CU has (several groups: both, since a tile is counted for every group that
// may not be there), the own keys' the other twice over; no part of the longest
// possible sequence under 128 keys, at most 128 parts.  More parts cost the
// join, fewer leave CUs without products.  Measured, us with the join, 16 heads
// on 4, d = 128, prefix of 32768 keys, up to 1500 own: 64 sequences 58 (32 parts)
// against 59, 63 and 68 with 24, 48 and 64; 256 sequences 149 (8 parts) against
// 162, 158 and 173 with 6, 12 and 16; three groups, 960 rows a kv head, 9000 keys:
// 51 with 9 and 12, 54 with 6, 57 with 19.
static int at_most(long long s, long long keys) {
  if (s > keys / 128)
    s = keys / 128;
  return s < 1 ? 1 : (s > 128 ? 128 : static_cast<int>(s));
}
void attn_prefix_splits(const attn_sizes &z, prefix_call &x) {
  const attn_sizes y = prefix_sizes(z, x);
  const int G = z.Hq / z.Hk, BM = few_rows(y) ? 32 : 128;
  const long long rows = static_cast<long long>(z.Ttot) * G;
  const long long tiles = (x.ngroups == 1 ? (rows + BM - 1) / BM : rows / BM + x.ngroups) * z.Hk;
  x.prefix_parts = at_most((x.ngroups == 1 ? 256 : 512) / tiles, y.max_keys);
  order od;
  plan_tiles(z, G, decode_rows(z) ? 16 : few_rows(z) ? 32 : 128, od);
  const long long own = static_cast<long long>(od.units) * od.tiles;
  x.own_parts = at_most((512 + own - 1) / own, z.max_keys);
}

template <typename P, typename O>
static hipError_t launch_both(const fwd_args &p, const fwd_args &o, unsigned pb, unsigned ob, hipStream_t st) {
  hipLaunchKernelGGL((gdn2_attn_prefix_kernel<P, O>), dim3(pb + ob), dim3(256), 0, st, p, o, static_cast<int>(pb));
  return hipGetLastError();
}

template <typename CT, int D, typename P>
static hipError_t launch_with(const fwd_args &p, unsigned pb, fwd_args &o, const attn_sizes &z, hipStream_t st) {
  if (decode_rows(z)) {
    const unsigned ob = plan_tiles(z, o.G, 16, o.od) * o.splits;
    return launch_both<P, decode_body<CT, D, 2, false>>(p, o, pb, ob, st);
  }
  if (few_rows(z)) {
    const unsigned ob = plan_tiles(z, o.G, 32, o.od) * o.splits;
    return launch_both<P, fwd_body<bf16_t, CT, D, 1, 4, 1, true, FWD_PLAIN>>(p, o, pb, ob, st);
  }
  const unsigned ob = plan_tiles(z, o.G, 128, o.od) * o.splits;
  return launch_both<P, fwd_body<bf16_t, CT, D, 4, 1, 2, true, FWD_PLAIN>>(p, o, pb, ob, st);
}

template <typename IO, typename CT, int D>
hipError_t launch_attn_prefix(const attn_sizes &z, const attn_ptrs &ptrs, const prefix_call &x, void *ws,
                              hipStream_t st) {
  const attn_sizes y = prefix_sizes(z, x);
  fwd_args p, o;
  fill(p, y, ptrs);
  fill_groups(p, z, x);
  p.table = x.table;
  p.seq_lens = x.lens;
  p.splits = x.prefix_parts;
  parts_at(p, z, D, ws, x.prefix_parts + x.own_parts, 0);
  fill(o, z, ptrs);
  o.splits = x.own_parts;
  o.mark = true;
  parts_at(o, z, D, ws, x.prefix_parts + x.own_parts, x.prefix_parts);
  const bool few = few_rows(y);
  if constexpr (sizeof(IO) == 2) {
    const unsigned pb = plan_tiles(y, p.G, few ? 32 : 128, p.od) * p.splits;
    return few ? launch_with<CT, D, fwd_body<IO, CT, D, 1, 4, 1, true, FWD_PREFIX>>(p, pb, o, z, st)
               : launch_with<CT, D, fwd_body<IO, CT, D, 4, 1, 2, true, FWD_PREFIX>>(p, pb, o, z, st);
  } else {
    // (float32's workgroups of the two kinds differ in size)
    constexpr int KT = sizeof(CT) <= 2 ? 2 : 1, WN = D * sizeof(IO) <= 256 ? 4 : 2;
    const hipError_t e = few ? launch_fwd<IO, CT, D, 1, WN, 1, true, FWD_PREFIX>(p, y, st)
                             : launch_fwd<IO, CT, D, 4, 1, KT, true, FWD_PREFIX>(p, y, st);
    return e == hipSuccess ? launch_paged<IO, CT, D>(o, z, st) : e;
  }
}

#define GDN2_INST_PREFIX(IO, CT, D)                                                                          \
  template hipError_t launch_attn_prefix<IO, CT, D>(const attn_sizes &, const attn_ptrs &, const prefix_call &, \
                                                    void *, hipStream_t);
GDN2_INST_PREFIX(float, float, 64)
GDN2_INST_PREFIX(float, float, 128)
GDN2_INST_PREFIX(float, f8_t, 64)
GDN2_INST_PREFIX(float, f8_t, 128)
GDN2_INST_PREFIX(bf16_t, bf16_t, 64)
GDN2_INST_PREFIX(bf16_t, bf16_t, 128)
GDN2_INST_PREFIX(bf16_t, f8_t, 64)
GDN2_INST_PREFIX(bf16_t, f8_t, 128)

}  // namespace attn
}  // namespace gdn2
