// gdn2_kvrow.hpp -- one row of keys or values as the cache's e4m3 codes and
// exponent byte, and a slot's place in the cache.
#pragma once

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

// The codes of the 8 values a lane holds of a row (D / 8 lanes, all of which
// call this): w[0] of a, w[1] of b.  Returns the row's exponent byte.
template <int D> __device__ __forceinline__ uint8_t quantise_row(const f32x4 &a, const f32x4 &b, u32x2 &w) {
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
  int p = 0;
  p = __builtin_amdgcn_cvt_pk_fp8_f32(bad ? 0.f : a[0] * inv, bad ? 0.f : a[1] * inv, p, false);
  p = __builtin_amdgcn_cvt_pk_fp8_f32(bad ? 0.f : a[2] * inv, bad ? 0.f : a[3] * inv, p, true);
  w[0] = p;
  p = __builtin_amdgcn_cvt_pk_fp8_f32(bad ? 0.f : b[0] * inv, bad ? 0.f : b[1] * inv, p, false);
  p = __builtin_amdgcn_cvt_pk_fp8_f32(bad ? 0.f : b[2] * inv, bad ? 0.f : b[3] * inv, p, true);
  w[1] = p;
  return static_cast<uint8_t>(byte);
}

// Row of a slot (one of num_pages << page_shift) and kv head in the cache.
__device__ __forceinline__ size_t cache_row(int64_t slot, int Hk, int hk, int page_shift) {
  const size_t page = static_cast<size_t>(slot) >> page_shift, off = slot & ((1ll << page_shift) - 1);
  return ((page * Hk + hk) << page_shift) + off;
}

}  // namespace attn
}  // namespace gdn2
