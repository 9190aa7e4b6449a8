// gdn2_qkrope.hip -- the per-head norm of queries and keys with the rotation
// by position in the same pass, and its backward, for gfx950.
//
//   r = 1 / sqrt(mean(x^2) + eps);  y = R(pos) (x r (.) w)
// R turns the channel pair j of the first `rot` channels by pos * freqs[j]:
// pairs (j, j + rot / 2), or (2j, 2j + 1) in the interleaved layout; the
// other channels pass.  Backward: g = R(pos)^T dy, u = g (.) w, xh = x r,
//   dx = r (u - xh mean(u xh)),  dw = sum over rows of g (.) xh.
//
// The bound is memory: every value is read and written once (the backward
// reads two and writes one).  A head's row is held by D / 8 lanes, 8 values
// each in two groups of 4, so that both values of a rotated pair are in one
// lane, a row's sums take 3 or 4 lane exchanges, and no value passes through
// shared memory.  A wave stays on one token for all heads it takes, so the
// sines and cosines are formed once per token: the angle is reduced to a
// fraction of a turn in 64 bits (position 10^6 times a frequency of 1 keeps
// 2^-33 of a turn, where float32 would keep 2^-7), its sine and cosine are
// float32.
//
// Measured, 32768 tokens x (16 + 4) heads, d = 128, bfloat16: forward 60 to 65 us
// (336 MB, 5.2 to 5.6 TB/s), backward 109 to 123 us (503 MB) and 5 us for the sum of
// the weight gradients' parts; a large copy runs at 4.7 TB/s.  32 tokens (a
// decode step): 4 us, a launch's own latency.
#include "gdn2_rope.hpp"

namespace gdn2 {
namespace attn {

template <typename IO, int D> __global__ void __launch_bounds__(256) gdn2_rope_fwd_kernel(rope_args A) {
  constexpr int LPH = D / 8, HPW = 64 / LPH;
  const int lane = threadIdx.x & 63, j = lane % LPH, hh = lane / LPH;
  const long u = static_cast<long>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (u >= A.tokens * A.parts)
    return;
  const long token = u / A.parts;
  const int part = static_cast<int>(u % A.parts);
  const lane_map m = map_lane<D>(A, j);
  f32x4 c, s;
  turn_of(A, m, j, token, c, s);
  f32x4 wqa = ones(), wqb = ones(), wka = ones(), wkb = ones();
  if (A.wq) {
    wqa = io<float>::load4(A.wq + m.a);
    wqb = io<float>::load4(A.wq + m.b);
  }
  if (A.wk) {
    wka = io<float>::load4(A.wk + m.a);
    wkb = io<float>::load4(A.wk + m.b);
  }
  const int heads = A.Hq + A.Hk;
  // every lane stays in the loop (the sums' exchanges need whole rows)
  for (int h0 = part * HPW; h0 < heads; h0 += A.parts * HPW) {
    const int hd = h0 + hh;
    const bool ok = hd < heads, isq = hd < A.Hq;
    const size_t row = isq ? static_cast<size_t>(token) * A.Hq + hd
                           : static_cast<size_t>(token) * A.Hk + (ok ? hd - A.Hq : 0);
    const IO *x = static_cast<const IO *>(isq ? A.q : A.k) + row * D;
    f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
    if (ok) {
      a = io<IO>::load4(x + m.a);
      b = io<IO>::load4(x + m.b);
    }
    if (A.norm) {
      const float r = 1.f / sqrtf(row_sum<D>(dot4(a, a) + dot4(b, b)) * (1.f / D) + A.eps);
      a = a * r * (isq ? wqa : wka);
      b = b * r * (isq ? wqb : wkb);
    }
    if (m.turned)
      rotate(A.interleaved, c, s, 1.f, a, b);
    if (ok) {
      IO *y = static_cast<IO *>(isq ? A.oq : A.ok) + row * D;
      io<IO>::store4(y + m.a, a);
      io<IO>::store4(y + m.b, b);
    }
  }
}

template <typename IO, int D> __global__ void __launch_bounds__(256) gdn2_rope_bwd_kernel(rope_args A) {
  constexpr int LPH = D / 8, HPW = 64 / LPH;
  __shared__ __align__(16) float red[4][2][D];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, j = lane % LPH, hh = lane / LPH;
  const lane_map m = map_lane<D>(A, j);
  f32x4 wqa = ones(), wqb = ones(), wka = ones(), wkb = ones();
  if (A.wq) {
    wqa = io<float>::load4(A.wq + m.a);
    wqb = io<float>::load4(A.wq + m.b);
  }
  if (A.wk) {
    wka = io<float>::load4(A.wk + m.a);
    wkb = io<float>::load4(A.wk + m.b);
  }
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 dqa = zero, dqb = zero, dka = zero, dkb = zero;
  const int heads = A.Hq + A.Hk;
  const long units = A.tokens * A.parts;
  for (long u = static_cast<long>(blockIdx.x) * 4 + wave; u < units; u += static_cast<long>(gridDim.x) * 4) {
    const long token = u / A.parts;
    const int part = static_cast<int>(u % A.parts);
    f32x4 c, s;
    turn_of(A, m, j, token, c, s);
    for (int h0 = part * HPW; h0 < heads; h0 += A.parts * HPW) {
      const int hd = h0 + hh;
      const bool ok = hd < heads, isq = hd < A.Hq;
      const size_t row = isq ? static_cast<size_t>(token) * A.Hq + hd
                             : static_cast<size_t>(token) * A.Hk + (ok ? hd - A.Hq : 0);
      f32x4 a = zero, b = zero, ga = zero, gb = zero;
      if (ok) {
        const IO *gy = static_cast<const IO *>(isq ? A.gq : A.gk) + row * D;
        ga = io<IO>::load4(gy + m.a);
        gb = io<IO>::load4(gy + m.b);
        if (A.norm) {
          const IO *x = static_cast<const IO *>(isq ? A.q : A.k) + row * D;
          a = io<IO>::load4(x + m.a);
          b = io<IO>::load4(x + m.b);
        }
      }
      if (m.turned)
        rotate(A.interleaved, c, s, -1.f, ga, gb);
      if (A.norm) {
        const float r = 1.f / sqrtf(row_sum<D>(dot4(a, a) + dot4(b, b)) * (1.f / D) + A.eps);
        a *= r;
        b *= r;
        if (isq) {
          dqa += ga * a;
          dqb += gb * b;
        } else {
          dka += ga * a;
          dkb += gb * b;
        }
        ga *= isq ? wqa : wka;
        gb *= isq ? wqb : wkb;
        const float t = row_sum<D>(dot4(ga, a) + dot4(gb, b)) * (1.f / D);
        ga = (ga - a * t) * r;
        gb = (gb - b * t) * r;
      }
      if (ok) {
        IO *y = static_cast<IO *>(isq ? A.oq : A.ok) + row * D;
        io<IO>::store4(y + m.a, ga);
        io<IO>::store4(y + m.b, gb);
      }
    }
  }
  if (!A.part)
    return;
  // the workgroup's sum over its rows, in a fixed order
#pragma unroll
  for (int x = LPH; x < 64; x <<= 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dqa[i] += __shfl_xor(dqa[i], x, 64);
      dqb[i] += __shfl_xor(dqb[i], x, 64);
      dka[i] += __shfl_xor(dka[i], x, 64);
      dkb[i] += __shfl_xor(dkb[i], x, 64);
    }
  if (hh == 0) {
    io<float>::store4(&red[wave][0][m.a], dqa);
    io<float>::store4(&red[wave][0][m.b], dqb);
    io<float>::store4(&red[wave][1][m.a], dka);
    io<float>::store4(&red[wave][1][m.b], dkb);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += 256) {
    const float *p = &red[0][0][0] + i;
    A.part[static_cast<size_t>(blockIdx.x) * 2 * D + i] = (p[0] + p[2 * D]) + (p[4 * D] + p[6 * D]);
  }
}

// dw[i] = sum over the workgroups' parts: 16 channels a workgroup, 64 threads
// a channel with up to 16 loads under way each, joined in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024) gdn2_rope_dw_kernel(const float *part, int parts, float *dwq, float *dwk) {
  __shared__ float red[64][17];
  const int col = threadIdx.x & 15, g = threadIdx.x >> 4, i = blockIdx.x * 16 + col;
  float x[16];
#pragma unroll
  for (int p = 0; p < 16; ++p)
    x[p] = g + 64 * p < parts ? part[static_cast<size_t>(g + 64 * p) * 2 * D + i] : 0.f;
#pragma unroll
  for (int s = 8; s > 0; s >>= 1)
#pragma unroll
    for (int p = 0; p < s; ++p)
      x[p] += x[p + s];
  red[g][col] = x[0];
  __syncthreads();
  for (int s = 32; s > 0; s >>= 1) {
    if (g < s)
      red[g][col] += red[g + s][col];
    __syncthreads();
  }
  if (g == 0) {
    float *dst = i < D ? dwq : dwk;
    if (dst)
      dst[i % D] = red[0][col];
  }
}

// ------------------------------------------------------------- launchers --
int rope_bwd_groups(long tokens, int Hq, int Hk, int D) {
  const long waves = tokens * rope_parts(tokens, Hq + Hk, D);
  const long g = (waves + 3) / 4;
  return static_cast<int>(g > 1024 ? 1024 : g);  // (the join takes up to 1024 parts)
}

template <typename IO, int D> hipError_t launch_rope_fwd(const rope_call &z, hipStream_t st) {
  rope_args A = pack_rope(z);
  A.parts = rope_parts(z.tokens, z.Hq + z.Hk, D);
  const long waves = z.tokens * A.parts;
  hipLaunchKernelGGL((gdn2_rope_fwd_kernel<IO, D>), dim3(static_cast<unsigned>((waves + 3) / 4)), dim3(256), 0, st, A);
  return hipGetLastError();
}
template <typename IO, int D> hipError_t launch_rope_bwd(const rope_call &z, float *part, hipStream_t st) {
  rope_args A = pack_rope(z);
  A.parts = rope_parts(z.tokens, z.Hq + z.Hk, D);
  A.part = part;
  hipLaunchKernelGGL((gdn2_rope_bwd_kernel<IO, D>), dim3(rope_bwd_groups(z.tokens, z.Hq, z.Hk, D)), dim3(256), 0, st, A);
  return hipGetLastError();
}
template <int D> hipError_t launch_rope_dw(const float *part, int groups, float *dwq, float *dwk, hipStream_t st) {
  hipLaunchKernelGGL((gdn2_rope_dw_kernel<D>), dim3(2 * D / 16), dim3(1024), 0, st, part, groups, dwq, dwk);
  return hipGetLastError();
}

#define GDN2_INST_ROPE(IO, D)                                                    \
  template hipError_t launch_rope_fwd<IO, D>(const rope_call &, hipStream_t);    \
  template hipError_t launch_rope_bwd<IO, D>(const rope_call &, float *, hipStream_t);
GDN2_INST_ROPE(float, 64)
GDN2_INST_ROPE(float, 128)
GDN2_INST_ROPE(bf16_t, 64)
GDN2_INST_ROPE(bf16_t, 128)
template hipError_t launch_rope_dw<64>(const float *, int, float *, float *, hipStream_t);
template hipError_t launch_rope_dw<128>(const float *, int, float *, float *, hipStream_t);

}  // namespace attn
}  // namespace gdn2
