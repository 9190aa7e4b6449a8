// gdn2_attn_fwd.hpp -- what the forward attention kernels share: their
// arguments and the way a row's output leaves.
#pragma once

#include "gdn2_attn.hpp"

namespace gdn2 {
namespace attn {

struct fwd_args {
  const void *q, *k, *v;
  void *o;
  float *lse;
  const int32_t *cu;         // packed queries, or nullptr: N sequences of T tokens
  const int32_t *table;      // paged: [N, max_pages]
  const int32_t *seq_lens;   // paged: keys of each sequence
  const uint8_t *ks, *vs;    // paged e4m3: [pages, Hk, page] exponent bytes
  float *part_o, *part_lse;  // where a row leaves parts, not its output: [splits, T total, Hq(, D)]
  int N, T, Hq, Hk, G;
  int Ttot;                  // tokens of q in all
  int max_pages, num_pages, page_shift;
  int window, sinks, splits;  // sinks: 0 without a window
  float c;                   // scale log2 e
  order od;
  // Shared prefixes.  The launch over the prefixes has the groups for its
  // sequences: N, table and seq_lens are theirs, T all tokens, and group i is
  // the sequences groups[i] .. groups[i + 1] - 1 (nullptr: one group of all)
  // of tq tokens each, or packed by cu.  The launch over the sequences' own
  // keys marks rows at negative positions, and the join takes the first
  // prefix_parts parts for the groups' rows alone.
  const int32_t *groups;
  int ngroups, seqs, tq, prefix_parts;
  bool mark;
  bool wide;  // decode: WIDE_WAVES waves a workgroup and no parts, where they serve the call best
};
constexpr int WIDE_WAVES = 12;

// The first token of group i, whatever groups and cu hold.
__device__ __forceinline__ int group_start(const fwd_args &a, int i) {
  int n = a.groups ? a.groups[i] : (i > 0 ? a.seqs : 0);
  n = n < 0 ? 0 : (n > a.seqs ? a.seqs : n);
  const int t = a.cu ? a.cu[n] : n * a.tq;
  return t < 0 ? 0 : (t > a.Ttot ? a.Ttot : t);
}

// Infinities and NaN of an operand set to zero; whether there were any.
__device__ __forceinline__ bool drop_nonfinite(frag8<bf16_t> &x) {
  u32x4 w = __builtin_bit_cast(u32x4, x.v);
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool lo = (w[i] & 0x7f80u) == 0x7f80u, hi = (w[i] & 0x7f800000u) == 0x7f800000u;
    any |= lo | hi;
    w[i] &= (lo ? 0xffff0000u : 0xffffffffu) & (hi ? 0x0000ffffu : 0xffffffffu);
  }
  x.v = __builtin_bit_cast(bf16x8, w);
  return any;
}
__device__ __forceinline__ bool drop_nonfinite(frag8<float> &x) {
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool lo = !(fabsf(x.lo[i]) <= 3.4028234663852886e38f), hi = !(fabsf(x.hi[i]) <= 3.4028234663852886e38f);
    any |= lo | hi;
    x.lo[i] = lo ? 0.f : x.lo[i];
    x.hi[i] = hi ? 0.f : x.hi[i];
  }
  return any;
}

// The wave's LDS accesses before and after, by any of its lanes, keep their
// order (the hardware keeps it; this keeps the compiler to it).
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Four channels of a row: its output, or with split keys its float32 part.
template <typename IO, int D>
__device__ __forceinline__ void store_row(const fwd_args &a, f32x4 x, float l, size_t qrow, int split, bool ok, int ch) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  x *= inv;
  if (!ok)
    return;
  if (a.part_o)
    io<float>::store4(a.part_o + (static_cast<size_t>(split) * a.Ttot * a.Hq + qrow) * D + ch, x);
  else
    io<IO>::store4(static_cast<IO *>(a.o) + qrow * D + ch, x);
}
// ln of the row's sum (of a part's: in base 2).  A row at a negative position
// is marked, where asked for, by +inf, which no sum gives (a score of +inf
// makes the sum NaN).
__device__ __forceinline__ void store_lse(const fwd_args &a, float m, float l, size_t qrow, int split, int pos) {
  const float x = m + log2f(l);
  if (a.part_o)
    a.part_lse[static_cast<size_t>(split) * a.Ttot * a.Hq + qrow] = a.mark && pos < 0 ? __builtin_inff() : x;
  else if (a.lse)
    a.lse[qrow] = x * LN2;
}

// the decode kernel (a.od: a tile a sequence and kv head)
template <typename CT, int D> hipError_t launch_attn_decode(const fwd_args &a, hipStream_t st);

}  // namespace attn
}  // namespace gdn2
