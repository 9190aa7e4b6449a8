// gdn2_attn_fwd.hip -- causal attention with grouped heads, for gfx950: over
// whole packed sequences, and over a paged cache.
//
//   s_ij = scale q_i . k_j for the visible keys j (j <= pos(i), and with a
//   window W, j > pos(i) - W or, with S sinks, j < S);  o_i = sum_j softmax(s_i)_j v_j;
//   lse_i = ln sum_j exp(s_ij).  A row that sees no key gives o = 0, lse = -inf.
//
// One pass over the keys with the running maximum m and sum l of each row
// (kept in float32, in base 2: p = 2^(s c - m) with c = scale log2 e).
// Both products are formed transposed, S^T = K Q^T and O^T = V^T P^T, so that
// an accumulator's column is a query row: the row's statistics are a lane's
// own (plus one exchange between the wave's halves), rescaling O is a lane
// multiply, and P^T leaves the first product in the operand layout of the
// second.  V^T's fragments come from row-major tiles through the transposing
// LDS read.
//
// WM waves share key tiles of 32 KT keys along 32-row blocks; WN waves split
// the tile's keys (each keeps its own m, l, O, joined at the end).
//
// A wave's 32 x 64 tile at d = 128 is 32 matrix products (1024 cycles) beside
// about 240 vector operations, 32 of them exponentials.  So the operands are read
// a group of products ahead, the tiles come straight from memory into shared
// memory (no registers, no address arithmetic a chunk), and the reference of the
// exponents moves only where it has to.  The bounds left are the chip's power
// (the clock holds 2.05 GHz under it; the same call on zeros runs at 2.39 GHz in
// 3.75 ms) and the two waves a SIMD that registers allow (the products are busy
// 46 % of the cycles, 56 % with the softmax taken out, shared memory 23 %; a
// deeper read-ahead changes nothing).  Measured: one
// sequence of 32768 tokens, 16 heads on 4, d = 128, bfloat16: 4.3 to 4.5 ms,
// 975 to 1020 TFLOP/s (an 8192^3 product: 1212; without tiles straight from
// memory 4650 us, without read-ahead and with a rescale every tile 4880); 8 x
// 4096 tokens, window 2048: 480 to 500 us, with 4 sinks 500 to 510.  Paged, 1024 tokens at 12000 keys among
// 23 single tokens: 105 us with the join's 10 (341 MB: 73 us at a copy's rate).
#include "gdn2_attn_launch.hpp"

namespace gdn2 {
namespace attn {

// Joins the parts of split keys: W waves per (token, query head), wave w of a
// row takes the parts w, w + W, ..; weights 2^(lse_s - max lse); the order of
// the sums is fixed.
// With PREFIX, the first prefix_parts parts hold for the groups' rows alone, and
// a row that the others mark sees nothing.
template <typename IO, int D, int W, bool PREFIX>
__global__ void __launch_bounds__(256) gdn2_attn_join_kernel(fwd_args a) {
  __shared__ float red[W][D + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w0 = W == 1 ? 0 : wave;
  const size_t rows = static_cast<size_t>(a.Ttot) * a.Hq;
  const size_t row = W == 1 ? static_cast<size_t>(blockIdx.x) * 4 + wave : blockIdx.x;
  if (row >= rows)
    return;
  if (a.cu && row >= static_cast<size_t>(a.cu[a.N] < 0 ? 0 : a.cu[a.N]) * a.Hq)
    return;  // behind the last sequence
  int s0 = 0;
  if constexpr (PREFIX) {
    // (a wave has one row; with a branch for the second comparison the compiler
    // lost the other value of s0)
    const int tok = __builtin_amdgcn_readfirstlane(static_cast<int>(row / a.Hq));
    const int first = group_start(a, 0), end = group_start(a, a.ngroups);
    s0 = (tok >= first) & (tok < end) ? 0 : a.prefix_parts;
  }
  float M = neg_inf();
  for (int s = s0 + lane; s < a.splits; s += 64)
    M = fmaxf(M, a.part_lse[s * rows + row]);
#pragma unroll
  for (int x = 1; x < 64; x <<= 1)
    M = fmaxf(M, __shfl_xor(M, x, 64));
  constexpr int V = D / 64;
  if (PREFIX && M == __builtin_inff()) {
    if (w0 == 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        static_cast<IO *>(a.o)[row * D + V * lane + i] = io<IO>::from_f(0.f);
      if (a.lse && lane == 0)
        a.lse[row] = neg_inf();
    }
    return;
  }
  const float base = M == neg_inf() ? 0.f : M;
  float acc[V], L = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
    acc[i] = 0.f;
#pragma unroll 4
  for (int s = s0 + w0; s < a.splits; s += W) {
    // (a part without keys: weight 0 and zeros; NaN stays NaN)
    const float w = fast_exp2(a.part_lse[s * rows + row] - base);
    const float *p = a.part_o + (s * rows + row) * D + V * lane;
    L += w;
#pragma unroll
    for (int i = 0; i < V; ++i)
      acc[i] += w * p[i];
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      red[wave][V * lane + i] = acc[i];
    if (lane == 0)
      red[wave][D] = L;
    __syncthreads();
    if (wave > 0)
      return;
    L = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w)
      L += red[w][D];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      acc[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w)
        acc[i] += red[w][V * lane + i];
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  IO *o = static_cast<IO *>(a.o) + row * D + V * lane;
#pragma unroll
  for (int i = 0; i < V; ++i)
    o[i] = io<IO>::from_f(acc[i] * inv);
  if (a.lse && lane == 0)
    a.lse[row] = (base + log2f(L)) * LN2;
}

// ------------------------------------------------------------- launchers --
// The kernel's shape for a call: 32-row blocks with the keys split over 4
// waves where a sequence brings few rows (decode), else 128 rows and shared
// key tiles.
bool few_rows(const attn_sizes &z) {
  return static_cast<long long>(z.Ttot) * (z.Hq / z.Hk) <= 32LL * z.N;
}
// At most 16 rows for every sequence and kv head: the decode kernel
// (bfloat16), with 16-row products.  Packed calls have their sequences' lengths on
// the device only and take the 32-row kernel even if all are single tokens (64
// sequences of 4K to 16K keys, e4m3: 133 us with T = 1, 150 packed).
bool decode_rows(const attn_sizes &z) {
  return !z.packed && static_cast<long long>(z.T) * (z.Hq / z.Hk) <= 16;
}

// With sinks, decode's sequences are about as long as their window and sinks,
// so the parts are chosen for whole rounds over the chip: a round takes its
// tiles of 128 keys and about three more to begin and end, the join about two.
// (Window 2048, 4 sinks, 16 heads on 4, e4m3: 64 sequences 32 us with 2 or 3
// parts, 43 with 8; 200 sequences 93 with 3, 104 with one, 117 with 8; 16
// sequences 17 with 6 or 9, 25 with 2.)  In bfloat16, workgroups of 12 waves (one a
// CU, tiles of 384 keys) need no parts and no join, where one round of them is
// enough.  (Window 500, 8 to 64 sequences: 11 to 14 us, in parts 14 to 16; window
// 2048, 64 sequences 31 and 35, 32 sequences 23 and 23, 16 sequences over a bfloat16
// cache 31 and 23, 100 sequences 52 and 47.)
struct sink_plan {
  int parts;
  bool wide;
};
static sink_plan plan_sinks(const attn_sizes &z, long long blocks) {
  const bool dec = decode_rows(z);
  const long long slots = dec ? 768 : 512;
  long long keys = static_cast<long long>(z.window) + z.sinks + 30 + z.T;
  keys = keys < z.max_keys ? keys : z.max_keys;
  const long long tiles = (keys + 127) / 128;
  sink_plan p = {1, false};
  long long least = (blocks + slots - 1) / slots * (tiles + 3);
  for (long long s = 2; s <= tiles && s <= 128; ++s) {
    const long long per = (tiles + s - 1) / s;
    const long long cost = (blocks * s + slots - 1) / slots * (per + 3) + 2;
    // (a part without keys is one too many)
    if (cost < least && (s - 1) * per < tiles) {
      least = cost;
      p.parts = static_cast<int>(s);
    }
  }
  p.wide = dec && blocks <= 256 && (tiles + 2) / 3 + 3 < least;
  return p;
}
static long long paged_blocks(const attn_sizes &z) {
  order od;
  plan_tiles(z, z.Hq / z.Hk, few_rows(z) ? 32 : 128, od);
  return static_cast<long long>(od.units) * od.tiles;
}
bool attn_decode_wide(const attn_sizes &z) { return z.sinks && decode_rows(z) && plan_sinks(z, paged_blocks(z)).wide; }

// Parts along the keys of a paged call: enough workgroups that sequences of
// different lengths even out over the CUs, no part of the longest possible
// sequence under 128 keys, at most 128 parts.  (Decode of 64 sequences x 4 kv
// heads: 136 us at 2048 workgroups, 151 at 1024 and 512; one 1024-token chunk
// among 23 tokens: 113 us at 768, 125 at 1024, 137 at 2048, where its parts'
// outputs weigh more.)
int attn_paged_splits(const attn_sizes &z) {
  const bool few = few_rows(z);
  const long long blocks = paged_blocks(z);
  if (z.sinks && few)
    return plan_sinks(z, blocks).parts;
  long long keys = z.max_keys;
  if (z.window > 0 && keys > z.window + z.sinks + 128LL)
    keys = z.window + z.sinks + 128LL;
  long long s = ((few ? 2048 : 768) + blocks - 1) / blocks;
  if (s > keys / 128)
    s = keys / 128;
  return s < 1 ? 1 : (s > 128 ? 128 : static_cast<int>(s));
}

template <typename IO, typename CT, int D, int WM, int WN, int KT, bool PAGED>
static hipError_t go(fwd_args &a, const attn_sizes &z, hipStream_t st) {
  return a.sinks ? launch_fwd<IO, CT, D, WM, WN, KT, PAGED, FWD_SINK>(a, z, st)
                 : launch_fwd<IO, CT, D, WM, WN, KT, PAGED, FWD_PLAIN>(a, z, st);
}

template <typename IO, int D> hipError_t launch_attn_fwd(const attn_sizes &z, const attn_ptrs &p, hipStream_t st) {
  fwd_args a;
  fill(a, z, p);
  // (few tiles, float32: 4 waves 14 and 25 us, 2 waves 22 and 38, d = 64 and
  // 128, 1543 tokens, 4 heads, window 300)
  constexpr int KT = sizeof(IO) == 2 ? 2 : 1;
  plan_tiles(z, a.G, 128, a.od);
  return few_tiles(a.od) ? go<IO, IO, D, 1, 4, 1, false>(a, z, st) : go<IO, IO, D, 4, 1, KT, false>(a, z, st);
}

template <typename IO, typename CT, int D> hipError_t launch_paged(fwd_args &a, const attn_sizes &z, hipStream_t st) {
  constexpr int KT = sizeof(CT) <= 2 ? 2 : 1;
  if constexpr (sizeof(IO) == 2) {
    if (decode_rows(z)) {
      plan_tiles(z, a.G, 16, a.od);
      a.wide = attn_decode_wide(z);
      return launch_attn_decode<CT, D>(a, st);
    }
  }
  // (float32, d = 128: 4 waves' tiles leave one workgroup a CU; 8 sequences of
  // 2000 keys, 4 heads on 4: 36 us against 31 with 2 waves; d = 64 17 against 21)
  constexpr int WN = D * sizeof(IO) <= 256 ? 4 : 2;
  return few_rows(z) ? go<IO, CT, D, 1, WN, 1, true>(a, z, st) : go<IO, CT, D, 4, 1, KT, true>(a, z, st);
}

template <typename IO, typename CT, int D>
hipError_t launch_attn_paged(const attn_sizes &z, const attn_ptrs &p, int splits, void *ws, hipStream_t st) {
  fwd_args a;
  fill(a, z, p);
  a.splits = splits;
  if (splits > 1)
    parts_at(a, z, D, ws, splits, 0);
  return launch_paged<IO, CT, D>(a, z, st);
}

template <typename IO, int D>
hipError_t launch_attn_join(const attn_sizes &z, const attn_ptrs &p, int splits, const prefix_call *x, void *ws,
                            hipStream_t st) {
  fwd_args a;
  fill(a, z, p);
  if (x)
    fill_groups(a, z, *x);
  a.splits = splits;
  parts_at(a, z, D, ws, splits, 0);
  const size_t rows = static_cast<size_t>(z.Ttot) * z.Hq;
  // one wave a row where there are rows enough, or few parts (shared prefixes:
  // 3840 rows of 14 parts 8.0 us with one wave, 9.6 with four; 1024 of 34, 7.8 and
  // 6.3)
  const bool one = rows >= (x ? 2048 : 8192) || splits <= 4;
  const dim3 grid(static_cast<unsigned>(one ? (rows + 3) / 4 : rows));
  if (one && x)
    hipLaunchKernelGGL((gdn2_attn_join_kernel<IO, D, 1, true>), grid, dim3(256), 0, st, a);
  else if (one)
    hipLaunchKernelGGL((gdn2_attn_join_kernel<IO, D, 1, false>), grid, dim3(256), 0, st, a);
  else if (x)
    hipLaunchKernelGGL((gdn2_attn_join_kernel<IO, D, 4, true>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((gdn2_attn_join_kernel<IO, D, 4, false>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

#define GDN2_INST_PAGED(IO, CT, D)                                                                          \
  template hipError_t launch_attn_paged<IO, CT, D>(const attn_sizes &, const attn_ptrs &, int, void *,      \
                                                   hipStream_t);                                            \
  template hipError_t launch_paged<IO, CT, D>(fwd_args &, const attn_sizes &, hipStream_t);
#define GDN2_INST_ATTN(IO, D)                                                                               \
  template hipError_t launch_attn_fwd<IO, D>(const attn_sizes &, const attn_ptrs &, hipStream_t);           \
  template hipError_t launch_attn_join<IO, D>(const attn_sizes &, const attn_ptrs &, int, const prefix_call *, \
                                              void *, hipStream_t);                                         \
  GDN2_INST_PAGED(IO, IO, D)                                                                                \
  GDN2_INST_PAGED(IO, f8_t, D)
GDN2_INST_ATTN(float, 64)
GDN2_INST_ATTN(float, 128)
GDN2_INST_ATTN(bf16_t, 64)
GDN2_INST_ATTN(bf16_t, 128)

}  // namespace attn
}  // namespace gdn2
