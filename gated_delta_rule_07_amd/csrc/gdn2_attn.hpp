// gdn2_attn.hpp -- device building blocks of the attention kernels (gfx950).
//
// Every matrix product is a 32x32 tile with 16 values of k per step (for
// bfloat16 one v_mfma_f32_32x32x16_bf16, for float32 eight
// v_mfma_f32_32x32x2_f32).  Lane l has index r = l % 32 (a row of A, a column
// of B and of the accumulator) and half h = l / 32, and an operand fragment is
// 8 values per lane:
//   k slot (h, e), e = 0..7.
// Any assignment of k values to slots gives the same product as long as A and
// B agree, and two are used:
//   "row" order   (h, e) = 8h + e: 8 consecutive values of a row-major row;
//   "acc" order   (h, e) = 8 (e / 4) + 4h + e % 4: the accumulator's own row
//                 order, so that registers 8j .. 8j+7 of an accumulator are
//                 the B operand of the next product without data movement.
// Accumulator register i of lane (r, h) is row 8 (i / 4) + 4h + i % 4,
// column r.
#pragma once

#include "gdn2_attn_kernels.hpp"
#include "gdn2_attn_order.hpp"
#include "gdn2_device.hpp"

namespace gdn2 {
namespace attn {

typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) unsigned int u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned int u32x2;

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// ------------------------------------------------------------- fragments --
template <typename T> struct frag8;
template <> struct frag8<bf16_t> {
  bf16x8 v;
};
template <> struct frag8<float> {
  f32x4 lo, hi;
};

__device__ __forceinline__ void mma(f32x16 &acc, const frag8<bf16_t> &a, const frag8<bf16_t> &b) {
  acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma(f32x16 &acc, const frag8<float> &a, const frag8<float> &b) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.lo[e], b.lo[e], acc, 0, 0, 0);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.hi[e], b.hi[e], acc, 0, 0, 0);
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    z[i] = 0.f;
  return z;
}

// Registers 8j .. 8j+7 of an accumulator as an operand (acc order), rounded
// to T: the products' operands are bfloat16 for bfloat16 tensors (half a
// step, at most 2^-8 relative, per weight; the row's sum is taken before the
// rounding, and it and the accumulator stay float32).
template <typename T> __device__ __forceinline__ frag8<T> pack8(const f32x16 &x, int j);
template <> __device__ __forceinline__ frag8<bf16_t> pack8<bf16_t>(const f32x16 &x, int j) {
  typedef __attribute__((ext_vector_type(8))) float f32x8;
  f32x8 y;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    y[e] = x[8 * j + e];
  frag8<bf16_t> f;
  f.v = __builtin_convertvector(y, bf16x8);
  return f;
}
template <> __device__ __forceinline__ frag8<float> pack8<float>(const f32x16 &x, int j) {
  frag8<float> f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f.lo[e] = x[8 * j + e];
    f.hi[e] = x[8 * j + 4 + e];
  }
  return f;
}

// 8 consecutive values in memory
template <typename T> __device__ __forceinline__ frag8<T> load8(const T *p);
template <> __device__ __forceinline__ frag8<bf16_t> load8<bf16_t>(const bf16_t *p) {
  frag8<bf16_t> f;
  f.v = *reinterpret_cast<const bf16x8 *>(p);
  return f;
}
template <> __device__ __forceinline__ frag8<float> load8<float>(const float *p) {
  frag8<float> f;
  f.lo = reinterpret_cast<const f32x4 *>(p)[0];
  f.hi = reinterpret_cast<const f32x4 *>(p)[1];
  return f;
}

// ------------------------------------------------------------- LDS tiles --
// A tile of rows of D values of T, row-major, whose 16-byte chunks are
// permuted within the row (chunk c of row r is kept at c ^ f(r)), so that
// both readings of it spread over the banks: 16 rows at one chunk (row
// fragments), and 8 rows (bfloat16) or 2 rows 4 apart (float32) at 32
// neighbouring channels (column fragments).
template <typename T, int D> struct tile {
  static constexpr int ROWB = D * static_cast<int>(sizeof(T));
  static constexpr int CPR = ROWB / 16;             // 16-byte chunks per row
  static constexpr int VPC = 16 / static_cast<int>(sizeof(T));
  __device__ static __forceinline__ int f(int r) {
    if constexpr (sizeof(T) == 4)
      return (((r >> 2) & 1) << 3) | ((r & 3) << 1) | ((r >> 3) & 1);
    else if constexpr (D == 128)
      return ((r & 3) << 2) | ((r >> 2) & 3);
    else
      return (((r >> 1) & 1) << 2) | (((r >> 3) & 1) << 1) | ((r >> 2) & 1);
  }
  __device__ static __forceinline__ int at(int r, int c) { return r * ROWB + ((c ^ f(r)) << 4); }

  // at(sr + RPI i, c), b = at(sr, c)
  template <int RPI> __device__ static __forceinline__ int step(int b, int sr, int c, int i) {
    return RPI % 16 == 0 ? b + RPI * i * ROWB : at(sr + RPI * i, c);
  }

  // A fragment's place in a tile is a lane's own base, XORed with the part
  // of the chunk number that k or n gives (rows are whole multiples of the
  // permutation's span, so adding rows and XORing chunks commute): one base a
  // lane instead of an address per fragment.
  //
  // Row fragments: values 16 kk + 8h .. + 7 of row r.
  __device__ static __forceinline__ int row_base(int r, int h) {
    return r * ROWB + ((f(r) ^ (sizeof(T) == 2 ? h : 2 * h)) << 4);
  }
  __device__ static __forceinline__ frag8<T> row(const char *t, int base, int kk) {
    frag8<T> x;
    if constexpr (sizeof(T) == 2) {
      x.v = *reinterpret_cast<const bf16x8 *>(t + (base ^ (kk << 5)));
    } else {
      x.lo = *reinterpret_cast<const f32x4 *>(t + (base ^ (kk << 6)));
      x.hi = *reinterpret_cast<const f32x4 *>(t + (base ^ (kk << 6) ^ 16));
    }
    return x;
  }
  // Column fragments, of the transposed tile: channel 32 n + lane % 32, tile
  // rows r0 + 8 (e / 4) + 4h + e % 4 (acc order), r0 a multiple of 16.
  __device__ static __forceinline__ int col_base(int lane) {
    const int h = lane >> 5;
    if constexpr (sizeof(T) == 2) {
      // a transposing read hands lane i of 16 the values of column i of a
      // 4 x 16 block whose row j / 4, values 4 (j % 4) .. + 3 lane j points at
      const int j = lane & 15, ch = (lane >> 4) & 1, ra = 4 * h + (j >> 2);
      return ra * ROWB + (((2 * ch + ((j & 3) >> 1)) ^ f(ra)) << 4) + ((j & 1) << 3);
    } else {
      return 4 * h * ROWB + ((((lane & 31) >> 2) ^ f(4 * h)) << 4) + ((lane & 3) << 2);
    }
  }
  __device__ static __forceinline__ frag8<T> col(const char *t, int base, int r0, int n) {
    frag8<T> x;
    if constexpr (sizeof(T) == 2) {
      // f(r + 8) = f(r) ^ 2
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const char *p = t + r0 * ROWB;
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + (base ^ (n << 6))));
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 8 * ROWB + (base ^ (n << 6) ^ 32)));
      x.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      // f(4h + e) = f(4h) ^ 2e, f(r + 8) = f(r) ^ 1
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const char *p = t + (r0 + e) * ROWB;
        x.lo[e] = *reinterpret_cast<const float *>(p + (base ^ (n << 7) ^ (e << 5)));
        x.hi[e] = *reinterpret_cast<const float *>(p + 8 * ROWB + (base ^ (n << 7) ^ (e << 5) ^ 16));
      }
    }
    return x;
  }
  // one value
  __device__ static __forceinline__ float one(const char *t, int r, int ch) {
    return io<T>::to_f(*reinterpret_cast<const T *>(t + at(r, ch / VPC) + (ch % VPC) * sizeof(T)));
  }
};

// Between groups of products: LDS reads and products keep their groups, so
// that a group's operands are read while the group before is multiplied.
__device__ __forceinline__ void group_fence() {
  __builtin_amdgcn_sched_barrier(0x6);  // vector and scalar ALU may move across
}

// Hides a value's origin, so that what depends on it is formed where it is
// used and not kept in registers across a loop.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// max over the two halves of a wave (lanes l and l ^ 32).  The swap puts the
// lower halves of both registers into the first and the upper halves into the
// second; the no-op covers the two wait states it needs behind the write of
// its operands.  (The builtin's two results were taken for equal and the max
// dropped.)
__device__ __forceinline__ float half_max(float x) {
  float y = x;
  asm("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  return fmaxf(x, y);
}

// 16 bytes a lane from global memory straight into shared memory, lane i's at
// lds + 16 i (lds: one address for the wave); there after dma_wait() and a
// barrier.
__device__ __forceinline__ void dma16(const void *src, char *lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                   (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}
__device__ __forceinline__ void dma_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// 8 e4m3 codes as an operand: the values they stand for (the row's scale is
// applied to the scores and weights, in float32), which both formats hold
// exactly.
template <typename T> __device__ __forceinline__ frag8<T> widen8(u32x2 x);
// (times a power of two)
__device__ __forceinline__ frag8<bf16_t> widen8_by(u32x2 x, float scale) {
  u32x4 y;
  y[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[0], scale, false));
  y[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[0], scale, true));
  y[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[1], scale, false));
  y[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[1], scale, true));
  frag8<bf16_t> f;
  f.v = __builtin_bit_cast(bf16x8, y);
  return f;
}
template <> __device__ __forceinline__ frag8<bf16_t> widen8<bf16_t>(u32x2 x) { return widen8_by(x, 1.0f); }
template <> __device__ __forceinline__ frag8<float> widen8<float>(u32x2 x) {
  const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(x[0], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(x[0], true);
  const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8(x[1], false), d = __builtin_amdgcn_cvt_pk_f32_fp8(x[1], true);
  frag8<float> f;
  f.lo = f32x4{a[0], a[1], b[0], b[1]};
  f.hi = f32x4{c[0], c[1], d[0], d[1]};
  return f;
}

// A tile of rows of D e4m3 codes, read as operands of T; laid out and read
// like the tile above (chunks of 16 codes).
template <typename T, int D> struct tile8 {
  static constexpr int ROWB = D, CPR = D / 16, VPC = 16;
  __device__ static __forceinline__ int f(int r) { return D == 128 ? (r >> 1) & 7 : (r >> 2) & 3; }
  __device__ static __forceinline__ int at(int r, int c) { return r * ROWB + ((c ^ f(r)) << 4); }
  __device__ static __forceinline__ int row_base(int r, int h) { return r * ROWB + (f(r) << 4) + 8 * h; }
  __device__ static __forceinline__ frag8<T> row(const char *t, int base, int kk) {
    return widen8<T>(*reinterpret_cast<const u32x2 *>(t + (base ^ (kk << 4))));
  }
  // a transposing read hands lane i of 16 the codes of column i of an 8 x 16
  // block whose row j / 2, codes 8 (j % 2) .. + 7 lane j points at; the
  // block's rows are the tile's in acc order
  __device__ static __forceinline__ int col_base(int lane) {
    const int h = lane >> 5, j = lane & 15, ch = (lane >> 4) & 1, e = j >> 1, ra = 8 * (e >> 2) + 4 * h + (e & 3);
    return ra * ROWB + ((ch ^ f(ra)) << 4) + ((j & 1) << 3);
  }
  __device__ static __forceinline__ frag8<T> col(const char *t, int base, int r0, int n) {
    // (f has period 16 in the row: r0 is a multiple of 16)
    typedef __attribute__((ext_vector_type(2))) int i32x2;
    typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
    return widen8<T>(__builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_i32x2 *)(t + r0 * ROWB + (base ^ (n << 5))))));
  }
  __device__ static __forceinline__ float one(const char *t, int r, int ch) {
    const unsigned code = *reinterpret_cast<const uint8_t *>(t + at(r, ch >> 4) + (ch & 15));
    return __builtin_amdgcn_cvt_f32_fp8(code, 0);
  }
};

// 2^(byte - 127); the byte 255 stands for NaN
__device__ __forceinline__ float scale_of(uint8_t byte) {
  if (byte == 255)
    return __builtin_nanf("");
  return byte ? __builtin_bit_cast(float, static_cast<uint32_t>(byte) << 23) : 5.877471754111438e-39f;
}

// ----------------------------------------------- sequences and row tiles --
// The rows a workgroup works on: (token, query head of the group) pairs of
// one sequence and one kv head, token-major, so that the G query heads that
// share a kv head share its tiles and their gradients' sum is one product.
struct span {
  int n;       // sequence
  int start;   // its first token in the packed tensors
  int len;     // its tokens
};

// Tile slots of packed sequences: sequence n owns the slots from
// floor(cu[n] G / BM) + n up; ceil(len G / BM) never exceeds the distance to
// the next sequence's first slot, so no table is needed.  One wave finds the
// last n whose first slot is <= s, 64 candidates a step.  Every wave of the
// workgroup calls this with the same arguments.
// holds(i): true for the numbers up to one, and false behind it; the last one of
// 0 .. N - 1 (0 if there is none).
template <typename P> __device__ __forceinline__ int find_last(P holds, int N, int lane) {
  int lo = 0, cnt = N;  // the answer lies in [lo, lo + cnt)
  while (cnt > 1) {
    const int step = (cnt + 63) / 64;
    const int i = lo + lane * step;
    const bool le = i < lo + cnt && holds(i);
    const unsigned long long m = __ballot(le);
    const int last = m ? 63 - __builtin_clzll(m) : 0;
    const int end = lo + cnt;
    lo += last * step;
    cnt = step < end - lo ? step : end - lo;
  }
  return lo;
}
// first(i): cu[i].
template <typename F> __device__ __forceinline__ int find_seq_by(F first, int N, int G, int BM, long s, int lane) {
  return find_last([=](int i) { return static_cast<long>(first(i)) * G / BM + i <= s; }, N, lane);
}

__device__ __forceinline__ int find_seq(const int32_t *cu, int N, int G, int BM, long s, int lane) {
  return find_seq_by([cu](int i) { return cu[i]; }, N, G, BM, s, lane);
}

// Sequence n's tokens (a to b - 1) in the tensors of T tokens a call may touch,
// whatever cu holds.
__device__ __forceinline__ span clamped_span(int n, int a, int b, int T) {
  span x;
  x.n = n;
  a = a < 0 ? 0 : (a > T ? T : a);
  b = b > T ? T : b;
  x.start = a;
  x.len = b > a ? b - a : 0;
  return x;
}
__device__ __forceinline__ span packed_span(const int32_t *cu, int n, int T) {
  return clamped_span(n, cu[n], cu[n + 1], T);
}

// Fewer 128-row tiles than CUs: such calls take 32-row tiles whose keys the
// waves split.  (float32, 5 sequences, 1543 tokens, 4 heads: 54 tiles, forward
// and backward 118 us with 128 rows, 69 with 32; bfloat16, 11 sequences, 9973
// tokens, 12 heads on 4: 980 tiles, forward 66 us with 128 rows, 78 with 32,
// dq 70 and 88.)
inline bool few_tiles(const order &od) { return static_cast<long long>(od.units) * od.tiles < 256; }

}  // namespace attn
}  // namespace gdn2
