// gdn2_kvappend.hip -- new tokens into the paged cache: the norm and rotation of
// their queries and keys (gdn2_qkrope.hip) and the write of keys and values
// (gdn2_kvcache.hip) in one pass, for gfx950.
//
//   q_out = R(pos) norm(q);  row of k_cache = R(pos) norm(k);  row of v_cache = v
//
// In two calls the rotated keys pass through memory once more, rounded to the
// tensors' type on the way; here a key is formed in float32 and rounded once,
// to the cache's type.  The bound is memory (every value read and written
// once), for a decode batch a launch's latency.  A wave takes a token's heads,
// D / 8 lanes a head (q's, then k's, then v's), as in gdn2_rope_fwd_kernel, so
// that the sines and cosines are formed once a token and a row's sum and
// largest magnitude take 3 or 4 lane exchanges.  Measured, 32768 tokens x (16 + 4 +
// 4) heads, d = 128, bfloat16, three sets of inputs in turn, shuffled slots: into e4m3
// 76 to 81 us (370 MB, 4.6 to 4.9 TB/s) where the two calls it stands for take 84 to 90
// on the same cards (61 to 64 and 22 to 23), into bfloat16 78 to 80 (403 MB, 5.1 TB/s)
// and 94 to 98 (62 to 65 and 29); q, k and v as parts of one projection add 1 to 3, and
// copying them out for the two calls 83.  A large copy runs at 4.7 TB/s.  32 tokens (a
// decode step): 4.2 us, a launch's own latency.
#include "gdn2_kvrow.hpp"
#include "gdn2_rope.hpp"

namespace gdn2 {
namespace attn {

struct append_args {
  rope_args r;
  const void *v;
  long qs, ks, vs, os;  // values between two tokens of q, k, v and q's output
  void *kc, *vc;
  uint8_t *ksc, *vsc;
  const int64_t *slots;
  int page_shift;
  long nslots;
};

template <typename IO, typename CT, int D> __global__ void __launch_bounds__(256) gdn2_kv_append_kernel(append_args A) {
  constexpr int LPH = D / 8, HPW = 64 / LPH;
  constexpr bool F8 = sizeof(CT) == 1;
  const rope_args &R = A.r;
  const int lane = threadIdx.x & 63, j = lane % LPH, hh = lane / LPH;
  // (a wave is on one token: what follows from it is uniform)
  const int u = static_cast<int>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int token = u / R.parts, part = u % R.parts;
  if (token >= R.tokens)
    return;
  const int64_t slot = A.slots[token];
  const bool kept = slot >= 0 && slot < A.nslots;
  const lane_map m = map_lane<D>(R, j);
  // lane p turns pair p, and a row's lanes fetch their four
  f32x4 c = ones(), s = ones();
  if (R.rot > 0) {
    const double pos = static_cast<double>(R.positions ? R.positions[token] : token % R.T);
    const int p = lane % (D / 2);
    float cs = 1.f, sn = 0.f;
    if (2 * p < R.rot)
      turn(pos, R.freqs[p], cs, sn);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = __shfl(cs, 4 * j + i, 64);
      s[i] = __shfl(sn, 4 * j + i, 64);
    }
  }
  f32x4 wqa = ones(), wqb = ones(), wka = ones(), wkb = ones();
  if (R.wq) {
    wqa = io<float>::load4(R.wq + m.a);
    wqb = io<float>::load4(R.wq + m.b);
  }
  if (R.wk) {
    wka = io<float>::load4(R.wk + m.a);
    wkb = io<float>::load4(R.wk + m.b);
  }
  const IO *const qt = static_cast<const IO *>(R.q) + token * A.qs, *const kt = static_cast<const IO *>(R.k) + token * A.ks;
  const IO *const vt = static_cast<const IO *>(A.v) + token * A.vs;
  IO *const ot = static_cast<IO *>(R.oq) + token * A.os;
  const int heads = R.Hq + 2 * R.Hk;
  auto normed = [&](f32x4 &a, f32x4 &b, const f32x4 &wa, const f32x4 &wb) {
    const float r = 1.f / sqrtf(row_sum<D>(dot4(a, a) + dot4(b, b)) * (1.f / D) + R.eps);
    a = a * r * wa;
    b = b * r * wb;
  };
  // (heads of a token: less than 2^32 values)
  for (int h0 = part * HPW; h0 < heads; h0 += R.parts * HPW) {
    const int hd = h0 + hh;
    if (h0 + HPW <= R.Hq) {
      const unsigned at = static_cast<unsigned>(hd) * D;
      f32x4 a = io<IO>::load4(qt + at + m.a), b = io<IO>::load4(qt + at + m.b);
      if (R.norm)
        normed(a, b, wqa, wqb);
      if (m.turned)
        rotate(R.interleaved, c, s, 1.f, a, b);
      io<IO>::store4(ot + at + m.a, a);
      io<IO>::store4(ot + at + m.b, b);
      continue;
    }
    // keys and values among them; every lane stays (the rows' exchanges need
    // whole rows)
    const int hk = hd < R.Hq + R.Hk ? hd - R.Hq : hd - R.Hq - R.Hk;
    const bool ok = hd < heads, isq = hd < R.Hq, isv = hd >= R.Hq + R.Hk;
    const IO *x = (isq ? qt : isv ? vt : kt) + static_cast<unsigned>(isq ? hd : hk) * D;
    f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
    if (ok) {
      a = io<IO>::load4(x + m.a);
      b = io<IO>::load4(x + m.b);
    }
    const f32x4 va = a, vb = b;
    if (R.norm)
      normed(a, b, isq ? wqa : wka, isq ? wqb : wkb);
    if (m.turned)
      rotate(R.interleaved, c, s, 1.f, a, b);
    a = isv ? va : a;
    b = isv ? vb : b;
    u32x2 code = {0u, 0u};
    uint8_t byte = 0;
    if constexpr (F8)
      byte = quantise_row<D>(a, b, code);
    if (!ok)
      continue;
    if (isq) {
      IO *y = ot + static_cast<unsigned>(hd) * D;
      io<IO>::store4(y + m.a, a);
      io<IO>::store4(y + m.b, b);
    } else if (kept) {
      const size_t row = cache_row(slot, R.Hk, hk, A.page_shift);
      CT *y = static_cast<CT *>(isv ? A.vc : A.kc) + row * D;
      if constexpr (F8) {
        *reinterpret_cast<unsigned *>(y + m.a) = code[0];
        *reinterpret_cast<unsigned *>(y + m.b) = code[1];
        if (j == 0)
          (isv ? A.vsc : A.ksc)[row] = byte;
      } else {
        io<IO>::store4(y + m.a, a);
        io<IO>::store4(y + m.b, b);
      }
    }
  }
}

template <typename IO, typename CT, int D>
hipError_t launch_kv_append(const rope_call &z, const cache_call &c, const append_strides &t, hipStream_t st) {
  append_args A;
  A.r = pack_rope(z);
  A.r.parts = rope_parts(z.tokens, z.Hq + 2 * z.Hk, D);
  A.v = c.v;
  A.qs = t.q;
  A.ks = t.k;
  A.vs = t.v;
  A.os = t.q_out;
  A.kc = c.kc;
  A.vc = c.vc;
  A.ksc = c.ks;
  A.vsc = c.vs;
  A.slots = c.slots;
  A.page_shift = c.page_shift;
  A.nslots = static_cast<long>(c.num_pages) << c.page_shift;
  const long waves = z.tokens * A.r.parts;
  hipLaunchKernelGGL((gdn2_kv_append_kernel<IO, CT, D>), dim3(static_cast<unsigned>((waves + 3) / 4)), dim3(256), 0, st, A);
  return hipGetLastError();
}

#define GDN2_INST_APPEND(IO, D)                                                                                  \
  template hipError_t launch_kv_append<IO, IO, D>(const rope_call &, const cache_call &, const append_strides &, \
                                                  hipStream_t);                                                  \
  template hipError_t launch_kv_append<IO, f8_t, D>(const rope_call &, const cache_call &, const append_strides &, \
                                                    hipStream_t);
GDN2_INST_APPEND(float, 64)
GDN2_INST_APPEND(float, 128)
GDN2_INST_APPEND(bf16_t, 64)
GDN2_INST_APPEND(bf16_t, 128)

}  // namespace attn
}  // namespace gdn2
