// gdn2_attn_decode.hip -- attention of a few new rows a sequence over the paged
// cache (decode), bfloat16, for gfx950.
//
// The mathematics is gdn2_attn_fwd.hip's; the tiles are 16 x 16: the rows of a
// sequence and kv head ((token, head of the group) pairs, at most 16) are the
// columns of every product.  The bound is memory, the cache's keys and values
// once, so what counts is bytes under way and few instructions a byte:
//   - every wave takes its own 16 TK keys of the workgroup's tile (no
//     barrier until the end) and asks for the next as soon as their registers
//     are free;
//   - a 16-key tile never crosses a page (pages hold multiples of 16, tiles
//     start at multiples of 16), so its table entry and address are scalars,
//     fetched a tile ahead, and its rows one contiguous block;
//   - K comes in operand layout straight from memory (k of a product is
//     summed over in any order: an e4m3 lane takes 16 neighbouring channels
//     as two operands); only V, needed transposed, goes through shared memory.
// Measured, 64 sequences of 4K to 16K keys, 16 query heads on 4, d = 128, pages
// of 64: e4m3 131 us (647 MB, 4.9 TB/s; a large copy 4.7), bfloat16 5.7 TB/s;
// the general kernel's 32-row tiles took 175.  One sequence, window 2048: 7 us
// and 4 for the join, two launches' latency.
#include <type_traits>

#include "gdn2_attn_fwd.hpp"

namespace gdn2 {
namespace attn {

__device__ __forceinline__ f32x4 mma16x32(const frag8<bf16_t> &a, const frag8<bf16_t> &b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
// max over the four 16-lane groups of a wave (swaps as in half_max)
__device__ __forceinline__ float group_max(float x) {
  float y = x;
  asm("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  return half_max(fmaxf(x, y));
}

// Lane l: row (or channel, or key) c = l % 16, group g = l / 16.  An
// accumulator's register i is row 4g + i; an operand's slot (g, e) is k = 8g + e
// ("row" order) or 16 (e / 4) + 4g + e % 4 ("acc" order: two accumulators).
template <typename CT, int D, int TK>
__global__ void __launch_bounds__(256, 3) gdn2_attn_decode_kernel(fwd_args a) {
  constexpr bool F8 = sizeof(CT) == 1;
  typedef bf16_t IO;
  typedef typename std::conditional<F8, tile8<IO, D>, tile<IO, D>>::type KV;
  constexpr int WN = 4, SN = 16 * TK, BN = SN * WN;
  constexpr int ROWB = KV::ROWB, TILEB = SN * ROWB, LV = 16 * ROWB / 1024;  // loads of a 16-key tile of V
  constexpr int LK = LV, NK = D / 32;                         // of K; products along the channels
  constexpr int OLD = D + 4, JOIN = WN * 16 * (OLD * 4 + 8);
  __shared__ __align__(16) char lds[WN * TILEB > JOIN ? WN * TILEB : JOIN];
  __shared__ __align__(16) float scales[F8 ? 2 * WN * SN : 1];
  const int tid = threadIdx.x, lane = tid & 63, wn = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;

  const int id = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  int unit, slot;
  if (!place(a.od, id, unit, slot))
    return;
  const int n_seq = unit / a.Hk, hk = unit % a.Hk;
  const int rows = a.T * a.G;
  int kv_len = a.seq_lens[n_seq];
  const int cap = a.max_pages << a.page_shift;
  kv_len = kv_len < 0 ? 0 : (kv_len > cap ? cap : kv_len);
  const int shift = kv_len - a.T;  // position of the first query

  // visible keys, from a multiple of 16, and this split's part
  int k_hi = kv_len;
  int k_lo = a.window > 0 ? shift - a.window + 1 : 0;
  k_lo = k_lo < 0 ? 0 : k_lo & ~15;
  int k0 = k_lo, k1 = k_hi;
  if (a.splits > 1) {
    const int nt = k_hi > k_lo ? (k_hi - k_lo + BN - 1) / BN : 0;
    const int per = (nt + a.splits - 1) / a.splits;
    k0 = k_lo + split * per * BN;
    k1 = k0 + per * BN < k_hi ? k0 + per * BN : k_hi;
  }
  const int ntiles = k1 > k0 ? (k1 - k0 + BN - 1) / BN : 0;

  const bool row_ok = c < rows;
  const int cl_row = row_ok ? c : rows - 1;
  const int tok = cl_row / a.G, head = hk * a.G + cl_row % a.G;
  const int pos = shift + tok, pos_lo = shift, pos_hi = shift + a.T - 1;
  const size_t qrow = (static_cast<size_t>(n_seq) * a.T + tok) * a.Hq + head;

  frag8<IO> q[NK];
#pragma unroll
  for (int kk = 0; kk < NK; ++kk)
    q[kk] = load8<IO>(static_cast<const IO *>(a.q) + qrow * D +
                      (F8 ? 64 * (kk >> 1) + 16 * g + 8 * (kk & 1) : 32 * kk + 8 * g));

  // Table entries are read as scalars, an iteration ahead of the rows they
  // lead to.  Behind the last key any tile of the part stands in.
  typedef const __attribute__((address_space(4))) int32_t *table_t;
  const table_t table = (table_t)(a.table + static_cast<size_t>(n_seq) * a.max_pages);
  const int pmask = (1 << a.page_shift) - 1;
  char *const vt = lds + wn * TILEB;
  float *const ksc = scales + wn * 2 * SN, *const vsc = ksc + SN;
  int ent[TK];
  auto load_entries = [&](int wk) {
#pragma unroll
    for (int t = 0; t < TK; ++t) {
      const int j = wk + 16 * t < k1 ? wk + 16 * t : (k1 - 1) & ~15;
      ent[t] = table[j >> a.page_shift];
    }
  };
  long row[TK];  // the tiles' first rows in the cache
  int bad = 0;   // tiles whose entry is outside it: their keys and values are zeros
  auto place_tiles = [&](int wk) {
    bad = 0;
#pragma unroll
    for (int t = 0; t < TK; ++t) {
      const int j = wk + 16 * t < k1 ? wk + 16 * t : (k1 - 1) & ~15;
      const bool ok = static_cast<unsigned>(ent[t]) < static_cast<unsigned>(a.num_pages);
      bad |= ok ? 0 : 1 << t;
      row[t] = ((static_cast<long>(ok ? ent[t] : 0) * a.Hk + hk) << a.page_shift) + (j & pmask);
    }
  };
  u32x4 rk[TK][LK], rv[TK][LV];
  uint8_t bk = 127, bv = 127;
  auto load_k = [&]() {
#pragma unroll
    for (int t = 0; t < TK; ++t) {
      const char *p = static_cast<const char *>(a.k) + row[t] * ROWB;
#pragma unroll
      for (int x = 0; x < LK; ++x)
        rk[t][x] = *reinterpret_cast<const u32x4 *>(p + (c * ROWB + 16 * g + 64 * x));
    }
  };
  auto load_v = [&]() {
#pragma unroll
    for (int t = 0; t < TK; ++t) {
      const char *p = static_cast<const char *>(a.v) + row[t] * ROWB;
#pragma unroll
      for (int x = 0; x < LV; ++x)
        rv[t][x] = *reinterpret_cast<const u32x4 *>(p + (16 * lane + 1024 * x));
    }
    if constexpr (F8) {
      // lane l: the scales of key l of the wave's tile
      long at = row[0];
#pragma unroll
      for (int t = 1; t < TK; ++t)
        at = (lane >> 4) % TK == t ? row[t] : at;
      bk = a.ks[at + c];
      bv = a.vs[at + c];
    }
  };

  // V operands: a transposing read's lane j of 16 points at row j / 4 (e4m3:
  // j / 2) of its group's block
  int col_b;
  if constexpr (F8) {
    const int e = c >> 1, ra = 16 * (e >> 2) + 4 * g + (e & 3);
    col_b = ra * ROWB + (KV::f(ra) << 4) + ((c & 1) << 3);
  } else {
    const int ra = 4 * g + (c >> 2);
    col_b = ra * ROWB + ((((c & 3) >> 1) ^ KV::f(ra)) << 4) + ((c & 1) << 3);
  }
  auto v_col = [&](int base, int j32, int n) -> frag8<IO> {
    // (f has period 16 in the row)
    const char *p = vt + 32 * j32 * ROWB;
    if constexpr (F8) {
      typedef __attribute__((ext_vector_type(2))) int i32x2;
      typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
      return widen8<IO>(__builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2 *)(p + (base ^ (n << 4))))));
    } else {
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + (base ^ (n << 5))));
      const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 16 * ROWB + (base ^ (n << 5))));
      frag8<IO> f;
      f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
      return f;
    }
  };

  f32x4 o[D / 16];
#pragma unroll
  for (int n = 0; n < D / 16; ++n)
    o[n] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = neg_inf(), l = 0.f;  // l: this lane's part of the row's sum

  if (ntiles > 0) {
    load_entries(k0 + SN * wn);
    place_tiles(k0 + SN * wn);
    load_v();
    load_k();
    load_entries(k0 + SN * wn + BN);
  }
  for (int it = 0; it < ntiles; ++it) {
    const int wk = k0 + it * BN + SN * wn;  // the wave's first key
    if (bad) {
#pragma unroll
      for (int t = 0; t < TK; ++t)
        if (bad >> t & 1) {
#pragma unroll
          for (int x = 0; x < LK; ++x)
            rk[t][x] = rv[t][x] = u32x4{0u, 0u, 0u, 0u};
        }
      // (0 times the scale of whatever row was read instead need not be 0)
      if (F8 && (bad >> (lane >> 4) % TK & 1))
        bk = bv = 127;
    }
    wave_order();
#pragma unroll
    for (int t = 0; t < TK; ++t)
#pragma unroll
      for (int x = 0; x < LV; ++x) {
        const int p = lane + 64 * x, row = p / KV::CPR;  // of the 16-key tile
        *reinterpret_cast<u32x4 *>(vt + 16 * t * ROWB + KV::at(row, p % KV::CPR)) = rv[t][x];
      }
    if constexpr (F8) {
      if (lane < SN) {
        ksc[lane] = scale_of(bk);
        vsc[lane] = scale_of(bv);
      }
    }
    wave_order();
    const bool more = it + 1 < ntiles;
    if (more) {
      place_tiles(wk + BN);
      load_v();
    }
    f32x4 s[TK];
#pragma unroll
    for (int t = 0; t < TK; ++t) {
      s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        frag8<IO> k;
        if constexpr (F8)
          k = widen8<IO>(kk & 1 ? u32x2{rk[t][kk >> 1][2], rk[t][kk >> 1][3]} : u32x2{rk[t][kk >> 1][0], rk[t][kk >> 1][1]});
        else
          k.v = __builtin_bit_cast(bf16x8, rk[t][kk]);
        s[t] = mma16x32(k, q[kk], s[t]);
      }
    }
    if (more) {
      load_k();
      load_entries(wk + 2 * BN);
    }
    if (wk >= k1)
      continue;  // none of the wave's keys
    const bool masked = wk + SN - 1 > pos_lo || wk + SN > k1 || (a.window > 0 && wk <= pos_hi - a.window);
    // key of register i of tile t: wk + 16 t + 4 g + i
    const int hi_rel = (pos < k1 - 1 ? pos : k1 - 1) - wk - 4 * g;
    const int lo_rel = (a.window > 0 ? pos - a.window : -0x40000000) - wk - 4 * g;
    float mx = neg_inf();
#pragma unroll
    for (int t = 0; t < TK; ++t) {
      if constexpr (F8)
        s[t] *= *reinterpret_cast<const f32x4 *>(&ksc[16 * t + 4 * g]);
      if (masked) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[t][i] = (16 * t + i <= hi_rel && 16 * t + i > lo_rel) ? s[t][i] : neg_inf();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mx = fmaxf(mx, s[t][i]);
    }
    mx = group_max(mx) * a.c;
    const bool up = mx > m + 8.f;  // as in gdn2_attn_fwd_kernel
    if (__any(up)) {
      const float m_new = up ? mx : m;
      const float alpha = fast_exp2(m - (m_new == neg_inf() ? 0.f : m_new));
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int n = 0; n < D / 16; ++n)
        o[n] *= alpha;
    }
    const float base = m == neg_inf() ? 0.f : m;
#pragma unroll
    for (int t = 0; t < TK; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[t][i] = fast_exp2(s[t][i] * a.c - base);
      l += (s[t][0] + s[t][1]) + (s[t][2] + s[t][3]);
      if constexpr (F8) {
        const f32x4 w = *reinterpret_cast<const f32x4 *>(&vsc[16 * t + 4 * g]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s[t][i] = (!masked || (16 * t + i <= hi_rel && 16 * t + i > lo_rel)) ? s[t][i] * w[i] : 0.f;
      }
    }
    bool odd = false;
    const int cb = fresh(col_b);
#pragma unroll
    for (int j = 0; j < TK / 2; ++j) {
      // the weights as operands: bfloat16, half a step of each
      typedef __attribute__((ext_vector_type(8))) float f32x8;
      const f32x8 y = {s[2 * j][0],     s[2 * j][1],     s[2 * j][2],     s[2 * j][3],
                       s[2 * j + 1][0], s[2 * j + 1][1], s[2 * j + 1][2], s[2 * j + 1][3]};
      frag8<IO> p;
      p.v = __builtin_convertvector(y, bf16x8);
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        frag8<IO> v = v_col(cb, j, n);
        if (masked)
          odd |= drop_nonfinite(v);
        o[n] = mma16x32(v, p, o[n]);
      }
    }
    // infinities and NaN of a masked tile, for the rows that see them (as in
    // gdn2_attn_fwd_kernel)
    if (masked && __any(odd)) {
      for (int j = 0; j < SN; ++j) {
        float p = 0.f;
#pragma unroll
        for (int t = 0; t < TK; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            p = 16 * t + i == (j & ~12) ? s[t][i] : p;
        p = __shfl(p, c + 16 * ((j >> 2) & 3), 64);
        const int jr = j - 4 * g;
        const bool vis = jr <= hi_rel && jr > lo_rel;
#pragma unroll
        for (int n = 0; n < D / 16; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = KV::one(vt, j, 16 * n + 4 * g + i);
            if (vis && !(fabsf(x) <= 3.4028234663852886e38f))
              o[n][i] += p * x;
          }
      }
    }
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);

  // join the waves' parts: weights 2^(m_w - M)
  float *jo = reinterpret_cast<float *>(lds);  // [WN][16][OLD]
  float *jm = jo + WN * 16 * OLD, *jl = jm + WN * 16;
  __syncthreads();
  if (g == 0) {
    jm[wn * 16 + c] = m;
    jl[wn * 16 + c] = l;
  }
  __syncthreads();
  float M = neg_inf();
#pragma unroll
  for (int w = 0; w < WN; ++w)
    M = fmaxf(M, jm[w * 16 + c]);
  const float base = M == neg_inf() ? 0.f : M;
  float L = 0.f;
#pragma unroll
  for (int w = 0; w < WN; ++w)
    L += jl[w * 16 + c] * fast_exp2(jm[w * 16 + c] - base);
  const float f = fast_exp2(m - base);
#pragma unroll
  for (int n = 0; n < D / 16; ++n)
    *reinterpret_cast<f32x4 *>(&jo[(wn * 16 + c) * OLD + 16 * n + 4 * g]) = o[n] * f;
  __syncthreads();
  for (int n = wn; n < D / 16; n += WN) {
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < WN; ++w)
      x += *reinterpret_cast<const f32x4 *>(&jo[(w * 16 + c) * OLD + 16 * n + 4 * g]);
    store_row<IO, D>(a, x, L, qrow, split, row_ok, 16 * n + 4 * g);
  }
  if (wn == 0 && g == 0 && row_ok)
    store_lse(a, M, L, qrow, split);
}

template <typename CT, int D> hipError_t launch_attn_decode(const fwd_args &a, hipStream_t st) {
  // (32 keys a wave and tile; 64 of e4m3 leave two waves a SIMD: 166 against
  // 136 us for 64 sequences of 4K to 16K keys)
  constexpr int TK = 2;
  const unsigned blocks = 8u * static_cast<unsigned>(a.od.units / a.od.g) * static_cast<unsigned>(a.od.tpr) * a.splits;
  hipLaunchKernelGGL((gdn2_attn_decode_kernel<CT, D, TK>), dim3(blocks), dim3(256), 0, st, a);
  return hipGetLastError();
}
template hipError_t launch_attn_decode<bf16_t, 64>(const fwd_args &, hipStream_t);
template hipError_t launch_attn_decode<bf16_t, 128>(const fwd_args &, hipStream_t);
template hipError_t launch_attn_decode<f8_t, 64>(const fwd_args &, hipStream_t);
template hipError_t launch_attn_decode<f8_t, 128>(const fwd_args &, hipStream_t);

}  // namespace attn
}  // namespace gdn2
