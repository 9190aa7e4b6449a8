// gdn2_kvcache.hip -- writing keys and values into the paged cache, and
// reading them back, for gfx950.
//
// The caches are [pages, Hk, page, D]: the keys a kv head reads of a page
// are one contiguous block.  A cache of the tensors' own type takes the
// values as they are.  An e4m3 cache takes each (token, kv head) row as codes
// of x 2^-e with one exponent byte e + 127 per row,
//   e = the smallest integer with max |x| <= 448 * 2^e  (at least -126),
// so that scaling is exact in both directions: the only rounding is the
// code's own (to nearest even, 2^-4 relative at most half a step), and what
// is read back, code * 2^e, is exact in float32, and in bfloat16 for e >= -124
// (codes are multiples of 2^-9, bfloat16's smallest subnormal is 2^-133).  A row
// holding an infinity or NaN gets the byte 255 and reads back as NaN.
//
// The bound is memory: one read and one write per value.  D / 8 lanes hold a
// row, 8 values (16 bytes of bfloat16) each, so a row's maximum takes 3 or 4
// lane exchanges and every access of a wave is whole rows.  Measured, 32768
// tokens x 4 kv heads, d = 128, bfloat16 to e4m3: write 19.3 us (102 MB,
// 5.3 TB/s), read 17.6 us (5.8 TB/s); a batch of 333 tokens x 3 heads, d = 64:
// 3.5 us each, a launch's own latency.
#include "gdn2_attn.hpp"

namespace gdn2 {
namespace attn {

template <int D> __device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int s = 1; s < D / 8; s <<= 1)
    x = fmaxf(x, __shfl_xor(x, s, 64));
  return x;
}

// The exponent byte of a row with largest magnitude amax (finite).
__device__ __forceinline__ int exponent_byte(float amax) {
  if (amax == 0.f)
    return 127;
  int k;
  const float f = frexpf(amax, &k);                // amax = f 2^k, f in [0.5, 1)
  const int e = f <= 0.875f ? k - 9 : k - 8;       // 448 = 0.875 * 2^9
  return (e < -126 ? -126 : e) + 127;
}

template <typename IO, int D>
__device__ __forceinline__ void write_row(const IO *x, f8_t *codes, uint8_t *scale, int j, bool ok) {
  f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
  if (ok) {
    a = io<IO>::load4(x + 8 * j);
    b = io<IO>::load4(x + 8 * j + 4);
  }
  float m = 0.f;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    odd = odd || !(fabsf(a[i]) <= 3.4028234663852886e38f) || !(fabsf(b[i]) <= 3.4028234663852886e38f);
    m = fmaxf(m, fmaxf(fabsf(a[i]), fabsf(b[i])));
  }
  m = row_max<D>(odd ? __builtin_inff() : m);
  const bool bad = m == __builtin_inff();
  const int byte = bad ? 255 : exponent_byte(m);
  // 2^-e, a normal number: e is -126 .. 120
  const float inv = bad ? 0.f : __builtin_bit_cast(float, static_cast<uint32_t>(254 - byte) << 23);
  u32x2 w;
  int p = 0;
  p = __builtin_amdgcn_cvt_pk_fp8_f32(bad ? 0.f : a[0] * inv, bad ? 0.f : a[1] * inv, p, false);
  p = __builtin_amdgcn_cvt_pk_fp8_f32(bad ? 0.f : a[2] * inv, bad ? 0.f : a[3] * inv, p, true);
  w[0] = p;
  p = __builtin_amdgcn_cvt_pk_fp8_f32(bad ? 0.f : b[0] * inv, bad ? 0.f : b[1] * inv, p, false);
  p = __builtin_amdgcn_cvt_pk_fp8_f32(bad ? 0.f : b[2] * inv, bad ? 0.f : b[3] * inv, p, true);
  w[1] = p;
  if (ok) {
    *reinterpret_cast<u32x2 *>(codes + 8 * j) = w;
    if (j == 0)
      *scale = static_cast<uint8_t>(byte);
  }
}
template <typename IO, int D>
__device__ __forceinline__ void write_row(const IO *x, IO *y, uint8_t *, int j, bool ok) {
  if (ok) {
    io<IO>::store4(y + 8 * j, io<IO>::load4(x + 8 * j));
    io<IO>::store4(y + 8 * j + 4, io<IO>::load4(x + 8 * j + 4));
  }
}

template <typename IO, int D> __device__ __forceinline__ void read_row(const f8_t *codes, uint8_t byte, IO *y, int j) {
  const u32x2 w = *reinterpret_cast<const u32x2 *>(codes + 8 * j);
  const float sc = scale_of(byte);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[i], true);
    io<IO>::store4(y + 8 * j + 4 * i, f32x4{lo[0] * sc, lo[1] * sc, hi[0] * sc, hi[1] * sc});
  }
}
template <typename IO, int D> __device__ __forceinline__ void read_row(const IO *x, uint8_t, IO *y, int j) {
  io<IO>::store4(y + 8 * j, io<IO>::load4(x + 8 * j));
  io<IO>::store4(y + 8 * j + 4, io<IO>::load4(x + 8 * j + 4));
}

struct cache_args {
  void *k, *v, *kc, *vc;
  uint8_t *ks, *vs;
  const int64_t *slots;
  long rows;  // tokens * Hk
  int Hk, page_shift;
  long nslots;
};

// One (token, kv head) row of k and of v per D / 8 lanes.
template <typename IO, typename CT, int D, bool WRITE>
__global__ void __launch_bounds__(256) gdn2_kv_cache_kernel(cache_args A) {
  constexpr int LPR = D / 8, RPB = 256 / LPR;
  const long row = static_cast<long>(blockIdx.x) * RPB + threadIdx.x / LPR;
  const int j = threadIdx.x % LPR;
  const bool in = row < A.rows;
  const long tok = in ? row / A.Hk : 0;
  const int hk = in ? static_cast<int>(row - tok * A.Hk) : 0;
  const int64_t slot = in ? A.slots[tok] : -1;
  const bool ok = slot >= 0 && slot < A.nslots;
  size_t at = 0;
  if (ok) {
    const size_t page = static_cast<size_t>(slot) >> A.page_shift, off = slot & ((1ll << A.page_shift) - 1);
    at = ((page * A.Hk + hk) << A.page_shift) + off;
  }
  CT *kc = static_cast<CT *>(A.kc) + at * D, *vc = static_cast<CT *>(A.vc) + at * D;
  IO *k = static_cast<IO *>(A.k) + row * D, *v = static_cast<IO *>(A.v) + row * D;
  if constexpr (WRITE) {
    write_row<IO, D>(k, kc, A.ks + at, j, ok);
    write_row<IO, D>(v, vc, A.vs + at, j, ok);
  } else {
    if (!in)
      return;
    if (ok) {
      constexpr bool F8 = sizeof(CT) == 1;
      read_row<IO, D>(kc, F8 ? A.ks[at] : uint8_t(0), k, j);
      read_row<IO, D>(vc, F8 ? A.vs[at] : uint8_t(0), v, j);
    } else {
      const f32x4 z = {0.f, 0.f, 0.f, 0.f};
      io<IO>::store4(k + 8 * j, z);
      io<IO>::store4(k + 8 * j + 4, z);
      io<IO>::store4(v + 8 * j, z);
      io<IO>::store4(v + 8 * j + 4, z);
    }
  }
}

template <typename IO, typename CT, int D> hipError_t launch_kv_cache(const cache_call &z, bool write, hipStream_t st) {
  cache_args A;
  A.k = z.k;
  A.v = z.v;
  A.kc = z.kc;
  A.vc = z.vc;
  A.ks = z.ks;
  A.vs = z.vs;
  A.slots = z.slots;
  A.rows = static_cast<long>(z.tokens) * z.Hk;
  A.Hk = z.Hk;
  A.page_shift = z.page_shift;
  A.nslots = static_cast<long>(z.num_pages) << z.page_shift;
  constexpr int RPB = 256 / (D / 8);
  const unsigned blocks = static_cast<unsigned>((A.rows + RPB - 1) / RPB);
  if (write)
    hipLaunchKernelGGL((gdn2_kv_cache_kernel<IO, CT, D, true>), dim3(blocks), dim3(256), 0, st, A);
  else
    hipLaunchKernelGGL((gdn2_kv_cache_kernel<IO, CT, D, false>), dim3(blocks), dim3(256), 0, st, A);
  return hipGetLastError();
}

#define GDN2_INST_CACHE(IO, D)                                                              \
  template hipError_t launch_kv_cache<IO, IO, D>(const cache_call &, bool, hipStream_t);    \
  template hipError_t launch_kv_cache<IO, f8_t, D>(const cache_call &, bool, hipStream_t);
GDN2_INST_CACHE(float, 64)
GDN2_INST_CACHE(float, 128)
GDN2_INST_CACHE(bf16_t, 64)
GDN2_INST_CACHE(bf16_t, 128)

}  // namespace attn
}  // namespace gdn2
