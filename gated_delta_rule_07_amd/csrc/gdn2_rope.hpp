// gdn2_rope.hpp -- what the kernels that norm and rotate heads share: a lane's
// place in a row, the turn of its pairs, and their launch arguments.
#pragma once

#include "gdn2_attn_kernels.hpp"
#include "gdn2_device.hpp"

namespace gdn2 {
namespace attn {

struct rope_args {
  const void *q, *k;
  const float *wq, *wk;
  const double *freqs;
  const int32_t *positions;
  const void *gq, *gk;  // backward: gradients of the outputs
  void *oq, *ok;        // outputs (backward: gradients of q and k)
  float *part;          // backward: [workgroups, 2, D] partial dw
  int T, Hq, Hk, rot, parts;
  long tokens;
  float eps;
  bool norm, interleaved;
};

// What a lane holds of a row: groups a and b of 4 channels, and the turn of
// its 4 pairs.
struct lane_map {
  int a, b;
  bool turned;
};

template <int D> __device__ __forceinline__ lane_map map_lane(const rope_args &A, int j) {
  lane_map m;
  m.turned = 8 * j < A.rot;
  const bool half = m.turned && !A.interleaved;
  m.a = half ? 4 * j : 8 * j;
  m.b = half ? A.rot / 2 + 4 * j : 8 * j + 4;
  return m;
}

// cosine and sine of pos * freq, the angle reduced to a fraction of a turn in
// 64 bits
__device__ __forceinline__ void turn(double pos, double freq, float &cs, float &sn) {
  const double t = pos * freq * 0.15915494309189533577;  // turns
  const float f = static_cast<float>(t - __builtin_rint(t));
  sincospif(2.f * f, &sn, &cs);
}

__device__ __forceinline__ void turn_of(const rope_args &A, const lane_map &m, int j, long token, f32x4 &c, f32x4 &s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (!m.turned)
    return;
  const double pos = A.positions ? static_cast<double>(A.positions[token]) : static_cast<double>(token % A.T);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float sn, cs;
    turn(pos, A.freqs[4 * j + i], cs, sn);
    c[i] = cs;
    s[i] = sn;
  }
}

// (a, b) turned by the angles (sign +1) or back (sign -1)
__device__ __forceinline__ void rotate(bool interleaved, const f32x4 &c, const f32x4 &s, float sign, f32x4 &a, f32x4 &b) {
  if (interleaved) {
    const f32x4 x = a, y = b;
    a[0] = x[0] * c[0] - x[1] * (sign * s[0]);
    a[1] = x[1] * c[0] + x[0] * (sign * s[0]);
    a[2] = x[2] * c[1] - x[3] * (sign * s[1]);
    a[3] = x[3] * c[1] + x[2] * (sign * s[1]);
    b[0] = y[0] * c[2] - y[1] * (sign * s[2]);
    b[1] = y[1] * c[2] + y[0] * (sign * s[2]);
    b[2] = y[2] * c[3] - y[3] * (sign * s[3]);
    b[3] = y[3] * c[3] + y[2] * (sign * s[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[i], y = b[i], sn = sign * s[i];
      a[i] = x * c[i] - y * sn;
      b[i] = y * c[i] + x * sn;
    }
  }
}

template <int D> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int s = 1; s < D / 8; s <<= 1)
    x += __shfl_xor(x, s, 64);
  return x;
}
__device__ __forceinline__ float dot4(const f32x4 &x, const f32x4 &y) {
  return x[0] * y[0] + x[1] * y[1] + x[2] * y[2] + x[3] * y[3];
}
__device__ __forceinline__ f32x4 ones() { return f32x4{1.f, 1.f, 1.f, 1.f}; }

// Waves per token: one where there are tokens enough to fill the chip (2048
// waves), else up to one per group of heads a wave takes at once.
inline int rope_parts(long tokens, int heads, int D) {
  const int groups = (heads * (D / 8) + 63) / 64;
  long p = (2048 + tokens - 1) / tokens;
  return static_cast<int>(p > groups ? groups : p);
}
inline rope_args pack_rope(const rope_call &z) {
  rope_args A;
  A.q = z.q;
  A.k = z.k;
  A.wq = z.wq;
  A.wk = z.wk;
  A.freqs = z.freqs;
  A.positions = z.positions;
  A.gq = z.gq;
  A.gk = z.gk;
  A.oq = z.oq;
  A.ok = z.ok;
  A.part = nullptr;
  A.T = z.T;
  A.Hq = z.Hq;
  A.Hk = z.Hk;
  A.rot = z.rot;
  A.tokens = z.tokens;
  A.eps = z.eps;
  A.norm = z.norm;
  A.interleaved = z.interleaved;
  return A;
}

}  // namespace attn
}  // namespace gdn2
