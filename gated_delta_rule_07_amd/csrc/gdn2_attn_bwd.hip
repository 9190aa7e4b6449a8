// gdn2_attn_bwd.hip -- backward of the whole-sequence attention, for gfx950.
//
//   delta_i = do_i . o_i;  p_ij = exp(s_ij - lse_i);
//   ds_ij = p_ij (do_i . v_j - delta_i);
//   dv_j = sum_i p_ij do_i;  dk_j = scale sum_i ds_ij q_i;
//   dq_i = scale sum_j ds_ij k_j.
//
// Two kernels recompute p from the forward's lse: one owns key rows (dk, dv)
// and walks the queries, one owns query rows (dq) and walks the keys.  That
// is seven products where one kernel with atomic additions into dq would do
// five, and in exchange every sum has a fixed order (the same bits every run)
// and no float32 copy of dq passes through memory.  The query rows are the
// (token, head of the group) pairs of a kv head, so the sum over the heads
// that share a key row is part of the same product.
#include "gdn2_attn.hpp"

namespace gdn2 {
namespace attn {

struct bwd_args {
  const void *q, *k, *v, *o, *dout;
  const float *lse;
  void *dq, *dk, *dv;
  f32x2 *stat;  // [Hk, Ttot, G]: lse log2 e, delta
  const int32_t *cu;
  int N, T, Ttot, Hq, Hk, G, window;
  float c, scale;
  order od;
};

// delta and the base-2 lse of every row, in row-tile order.  A wave takes
// one row at a time, D / 64 channels a lane.
template <typename IO, int D> __global__ void __launch_bounds__(256) gdn2_attn_stat_kernel(bwd_args a) {
  const int lane = threadIdx.x & 63;
  const size_t rows = static_cast<size_t>(a.Ttot) * a.Hq;
  const size_t row = static_cast<size_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= rows)
    return;
  const size_t tok = row / a.Hq;
  const int head = static_cast<int>(row % a.Hq), hk = head / a.G, g = head % a.G;
  if (a.cu && static_cast<long>(tok) >= a.cu[a.N])
    return;  // behind the last sequence
  constexpr int V = D / 64;
  const IO *o = static_cast<const IO *>(a.o) + row * D + V * lane;
  const IO *d = static_cast<const IO *>(a.dout) + row * D + V * lane;
  float x = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
    x += io<IO>::to_f(o[i]) * io<IO>::to_f(d[i]);
#pragma unroll
  for (int s = 1; s < 64; s <<= 1)
    x += __shfl_xor(x, s, 64);
  if (lane == 0)
    a.stat[(static_cast<size_t>(hk) * a.Ttot + tok) * a.G + g] = f32x2{a.lse[row] * LOG2E, x};
}

// The sequence of a workgroup's tile and the tile's first row in it (rows:
// GR per token).
__device__ __forceinline__ bool locate(const bwd_args &a, int unit, int slot, int GR, int BM, int lane, span &sq, int &hk,
                                       int &first) {
  if (a.cu) {
    hk = unit;
    const int n = find_seq(a.cu, a.N, GR, BM, slot, lane);
    sq = packed_span(a.cu, n, a.T);
    first = static_cast<int>((slot - (static_cast<long>(a.cu[n]) * GR / BM + n)) * BM);
  } else {
    sq.n = unit / a.Hk;
    hk = unit % a.Hk;
    sq.start = sq.n * a.T;
    sq.len = a.T;
    first = slot * BM;
  }
  return first >= 0 && first < sq.len * GR;
}

// ------------------------------------------------------------------- dq --
template <typename IO, int D, int KT>
__global__ void __launch_bounds__(256, (D * sizeof(IO) <= 256 ? 2 : 1)) gdn2_attn_dq_kernel(bwd_args a) {
  typedef tile<IO, D> TL;
  constexpr int BM = 128, BN = 32 * KT, CPR = TL::CPR, CH = BN * CPR / 256, RPI = 256 / CPR;
  constexpr int TILEB = BN * TL::ROWB;
  static_assert(BN * CPR % 256 == 0, "staging split");
  __shared__ __align__(16) char lds[4 * TILEB];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 31, h = lane >> 5;
  int unit, slot, hk, row0;
  span sq;
  if (!place(a.od, blockIdx.x, unit, slot) || !locate(a, unit, slot, a.G, BM, lane, sq, hk, row0))
    return;
  const int rows = sq.len * a.G;
  const int last_row = row0 + BM - 1 < rows - 1 ? row0 + BM - 1 : rows - 1;
  const int k1 = last_row / a.G + 1;
  int k0 = 0;
  if (a.window > 0) {
    k0 = row0 / a.G - a.window + 1;
    k0 = k0 < 0 ? 0 : k0;
  }
  const int ntiles = (k1 - k0 + BN - 1) / BN;
  const int my_row = row0 + 32 * wave + r;
  const bool row_ok = my_row < rows;
  const int cl_row = row_ok ? my_row : rows - 1;
  const int pos = cl_row / a.G, g = cl_row % a.G;
  const size_t qrow = static_cast<size_t>(sq.start + pos) * a.Hq + hk * a.G + g;
  const int wr0 = row0 + 32 * wave < rows ? row0 + 32 * wave : rows - 1;
  const int wr1 = row0 + 32 * wave + 31 < rows ? row0 + 32 * wave + 31 : rows - 1;
  const int pos_lo = wr0 / a.G, pos_hi = wr1 / a.G;
  const f32x2 st = a.stat[(static_cast<size_t>(hk) * a.Ttot + sq.start) * a.G + cl_row];

  frag8<IO> q[D / 16], d[D / 16];
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    q[kk] = load8<IO>(static_cast<const IO *>(a.q) + qrow * D + 16 * kk + 8 * h);
    d[kk] = load8<IO>(static_cast<const IO *>(a.dout) + qrow * D + 16 * kk + 8 * h);
  }
  const int sc = tid % CPR, sr0 = tid / CPR;
  u32x4 rk[CH], rv[CH];
  auto load_tile = [&](int kb) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      int j = kb + sr0 + RPI * i;
      j = j < k1 ? j : k1 - 1;
      const size_t off = (static_cast<size_t>(sq.start + j) * a.Hk + hk) * D + sc * TL::VPC;
      rk[i] = *reinterpret_cast<const u32x4 *>(static_cast<const IO *>(a.k) + off);
      rv[i] = *reinterpret_cast<const u32x4 *>(static_cast<const IO *>(a.v) + off);
    }
  };
  f32x16 dq[D / 32];
#pragma unroll
  for (int n = 0; n < D / 32; ++n)
    dq[n] = zero16();
  load_tile(k0);
  for (int it = 0; it < ntiles; ++it) {
    const int kb = k0 + it * BN;
    char *kt = lds + (it & 1) * 2 * TILEB, *vt = kt + TILEB;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int at = TL::at(sr0 + RPI * i, sc);
      *reinterpret_cast<u32x4 *>(kt + at) = rk[i];
      *reinterpret_cast<u32x4 *>(vt + at) = rv[i];
    }
    __syncthreads();
    if (it + 1 < ntiles)
      load_tile(kb + BN);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int wk = kb + 32 * t;
      if (wk > pos_hi || (a.window > 0 && wk + 31 <= pos_lo - a.window))
        continue;  // nothing visible to the wave
      const bool masked = wk + 31 > pos_lo || (a.window > 0 && wk <= pos_hi - a.window);
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        mma(s, TL::row(kt, 32 * t + r, kk, h), q[kk]);
        mma(dp, TL::row(vt, 32 * t + r, kk, h), d[kk]);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        s[i] = fast_exp2(s[i] * a.c - st[0]) * (dp[i] - st[1]);
      if (masked) {
        const int hi_rel = pos - wk - 4 * h, lo_rel = (a.window > 0 ? pos - a.window : -0x40000000) - wk - 4 * h;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = 8 * (i >> 2) + (i & 3);
          s[i] = (j <= hi_rel && j > lo_rel) ? s[i] : 0.f;
        }
      }
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        const frag8<IO> x = pack8<IO>(s, jj);
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
          mma(dq[n], TL::col(kt, 32 * t + 16 * jj, n, lane), x);
      }
    }
  }
  if (!row_ok)
    return;
#pragma unroll
  for (int n = 0; n < D / 32; ++n)
#pragma unroll
    for (int gg = 0; gg < 4; ++gg) {
      f32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = dq[n][4 * gg + i] * a.scale;
      io<IO>::store4(static_cast<IO *>(a.dq) + qrow * D + 32 * n + 8 * gg + 4 * h, x);
    }
}

// --------------------------------------------------------------- dk, dv --
// A workgroup owns 32 keys per wave (K and V in registers) and walks the
// rows that see any of them, 32 at a time through shared memory.
template <typename IO, int D, int W>
__global__ void __launch_bounds__(64 * W, 1) gdn2_attn_dkv_kernel(bwd_args a) {
  typedef tile<IO, D> TL;
  constexpr int NT = 64 * W, BK = 32 * W, BQ = 32, CPR = TL::CPR, CH = BQ * CPR / NT, RPI = NT / CPR;
  constexpr int TILEB = BQ * TL::ROWB;
  static_assert(BQ * CPR % NT == 0, "staging split");
  __shared__ __align__(16) char lds[4 * TILEB];
  __shared__ __align__(16) float s_lse[2][BQ], s_delta[2][BQ];
  __shared__ __align__(16) int s_pos[2][BQ];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 31, h = lane >> 5;
  int unit, slot, hk, key0;
  span sq;
  if (!place(a.od, blockIdx.x, unit, slot) || !locate(a, unit, a.od.tiles - 1 - slot, 1, BK, lane, sq, hk, key0))
    return;
  const int key_end = key0 + BK < sq.len ? key0 + BK : sq.len;
  // rows (token, head of the group) that see a key of the workgroup
  const int row0 = key0 * a.G;
  int tok_end = sq.len;
  if (a.window > 0 && key_end - 1 + static_cast<long>(a.window) < tok_end)
    tok_end = key_end - 1 + a.window;
  const int row1 = tok_end * a.G;
  const int wk = key0 + 32 * wave;        // the wave's first key
  const int key = wk + r;                 // the lane's
  const bool key_ok = key < sq.len;
  const size_t krow = static_cast<size_t>(sq.start + (key_ok ? key : sq.len - 1)) * a.Hk + hk;
  const int wk_hi = wk + 31 < sq.len - 1 ? wk + 31 : sq.len - 1;

  frag8<IO> k[D / 16], v[D / 16];
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    k[kk] = load8<IO>(static_cast<const IO *>(a.k) + krow * D + 16 * kk + 8 * h);
    v[kk] = load8<IO>(static_cast<const IO *>(a.v) + krow * D + 16 * kk + 8 * h);
  }
  const int sc = tid % CPR, sr0 = tid / CPR;
  u32x4 rq[CH], rd[CH];
  f32x2 rs = {0.f, 0.f};
  int rp = 0;
  auto load_tile = [&](int rb) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int row = rb + sr0 + RPI * i;
      if (row < row1) {
        const int tok = row / a.G;
        const size_t off =
            (static_cast<size_t>(sq.start + tok) * a.Hq + hk * a.G + (row - tok * a.G)) * D + sc * TL::VPC;
        rq[i] = *reinterpret_cast<const u32x4 *>(static_cast<const IO *>(a.q) + off);
        rd[i] = *reinterpret_cast<const u32x4 *>(static_cast<const IO *>(a.dout) + off);
      } else {
        rq[i] = rd[i] = u32x4{0u, 0u, 0u, 0u};
      }
    }
    if (tid < BQ) {
      const int row = rb + tid;
      // a row behind the last: weight 2^(0 - inf) = 0
      rs = f32x2{__builtin_inff(), 0.f};
      rp = 0x3fffffff;
      if (row < row1) {
        rs = a.stat[(static_cast<size_t>(hk) * a.Ttot + sq.start) * a.G + row];
        rp = row / a.G;
      }
    }
  };
  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int n = 0; n < D / 32; ++n)
    dk[n] = dv[n] = zero16();
  const int ntiles = (row1 - row0 + BQ - 1) / BQ;
  load_tile(row0);
  for (int it = 0; it < ntiles; ++it) {
    const int rb = row0 + it * BQ, buf = it & 1;
    char *qt = lds + buf * 2 * TILEB, *dt = qt + TILEB;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int at = TL::at(sr0 + RPI * i, sc);
      *reinterpret_cast<u32x4 *>(qt + at) = rq[i];
      *reinterpret_cast<u32x4 *>(dt + at) = rd[i];
    }
    if (tid < BQ) {
      s_lse[buf][tid] = rs[0];
      s_delta[buf][tid] = rs[1];
      s_pos[buf][tid] = rp;
    }
    __syncthreads();
    if (it + 1 < ntiles)
      load_tile(rb + BQ);
    const int lr = rb + BQ - 1 < row1 - 1 ? rb + BQ - 1 : row1 - 1;
    const int p_lo = rb / a.G, p_hi = lr / a.G;
    if (wk > p_hi || wk >= sq.len || (a.window > 0 && wk_hi <= p_lo - a.window))
      continue;  // no row sees a key of the wave
    const bool masked = wk_hi > p_lo || (a.window > 0 && wk <= p_hi - a.window);
    f32x16 s = zero16(), dp = zero16();
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      mma(s, TL::row(qt, r, kk, h), k[kk]);
      mma(dp, TL::row(dt, r, kk, h), v[kk]);
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x4 ls = *reinterpret_cast<const f32x4 *>(&s_lse[buf][8 * g + 4 * h]);
      const f32x4 de = *reinterpret_cast<const f32x4 *>(&s_delta[buf][8 * g + 4 * h]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = fast_exp2(s[4 * g + i] * a.c - ls[i]);
        s[4 * g + i] = p;
        dp[4 * g + i] = p * (dp[4 * g + i] - de[i]);
      }
    }
    if (masked) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        typedef __attribute__((ext_vector_type(4))) int i32x4;
        const i32x4 ps = *reinterpret_cast<const i32x4 *>(&s_pos[buf][8 * g + 4 * h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool vis = key <= ps[i] && (a.window <= 0 || key > ps[i] - a.window);
          s[4 * g + i] = vis ? s[4 * g + i] : 0.f;
          dp[4 * g + i] = vis ? dp[4 * g + i] : 0.f;
        }
      }
    }
#pragma unroll
    for (int jj = 0; jj < 2; ++jj) {
      const frag8<IO> p = pack8<IO>(s, jj), ds = pack8<IO>(dp, jj);
#pragma unroll
      for (int n = 0; n < D / 32; ++n) {
        mma(dv[n], TL::col(dt, 16 * jj, n, lane), p);
        mma(dk[n], TL::col(qt, 16 * jj, n, lane), ds);
      }
    }
  }
  if (!key_ok)
    return;
#pragma unroll
  for (int n = 0; n < D / 32; ++n)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      f32x4 x, y;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = dk[n][4 * g + i] * a.scale;
        y[i] = dv[n][4 * g + i];
      }
      io<IO>::store4(static_cast<IO *>(a.dk) + krow * D + 32 * n + 8 * g + 4 * h, x);
      io<IO>::store4(static_cast<IO *>(a.dv) + krow * D + 32 * n + 8 * g + 4 * h, y);
    }
}

// ------------------------------------------------------------- launchers --
static void fill(bwd_args &a, const attn_sizes &z, const attn_ptrs &p, void *ws) {
  a.q = p.q;
  a.k = p.k;
  a.v = p.v;
  a.o = p.o;
  a.dout = p.dout;
  a.lse = p.lse;
  a.dq = p.dq;
  a.dk = p.dk;
  a.dv = p.dv;
  a.stat = static_cast<f32x2 *>(ws);
  a.cu = p.cu;
  a.N = z.N;
  a.T = z.T;
  a.Ttot = z.Ttot;
  a.Hq = z.Hq;
  a.Hk = z.Hk;
  a.G = z.Hq / z.Hk;
  a.window = z.window;
  a.c = z.scale * LOG2E;
  a.scale = z.scale;
}

template <typename IO, int D>
hipError_t launch_attn_bwd_stat(const attn_sizes &z, const attn_ptrs &p, void *ws, hipStream_t st) {
  bwd_args a;
  fill(a, z, p, ws);
  const size_t rows = static_cast<size_t>(z.Ttot) * z.Hq;
  hipLaunchKernelGGL((gdn2_attn_stat_kernel<IO, D>), dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(256), 0, st, a);
  return hipGetLastError();
}
template <typename IO, int D>
hipError_t launch_attn_bwd_dq(const attn_sizes &z, const attn_ptrs &p, void *ws, hipStream_t st) {
  bwd_args a;
  fill(a, z, p, ws);
  const unsigned blocks = plan_tiles(z, z.Hq / z.Hk, 128, a.od);
  constexpr int KT = sizeof(IO) == 2 ? 2 : 1;
  hipLaunchKernelGGL((gdn2_attn_dq_kernel<IO, D, KT>), dim3(blocks), dim3(256), 0, st, a);
  return hipGetLastError();
}
template <typename IO, int D>
hipError_t launch_attn_bwd_dkv(const attn_sizes &z, const attn_ptrs &p, void *ws, hipStream_t st) {
  bwd_args a;
  fill(a, z, p, ws);
  constexpr int W = 4;
  const unsigned blocks = plan_tiles(z, 1, 32 * W, a.od);
  hipLaunchKernelGGL((gdn2_attn_dkv_kernel<IO, D, W>), dim3(blocks), dim3(64 * W), 0, st, a);
  return hipGetLastError();
}

#define GDN2_INST_ATTN_BWD(IO, D)                                                                           \
  template hipError_t launch_attn_bwd_stat<IO, D>(const attn_sizes &, const attn_ptrs &, void *, hipStream_t); \
  template hipError_t launch_attn_bwd_dq<IO, D>(const attn_sizes &, const attn_ptrs &, void *, hipStream_t);   \
  template hipError_t launch_attn_bwd_dkv<IO, D>(const attn_sizes &, const attn_ptrs &, void *, hipStream_t);
GDN2_INST_ATTN_BWD(float, 64)
GDN2_INST_ATTN_BWD(float, 128)
GDN2_INST_ATTN_BWD(bf16_t, 64)
GDN2_INST_ATTN_BWD(bf16_t, 128)

}  // namespace attn
}  // namespace gdn2
