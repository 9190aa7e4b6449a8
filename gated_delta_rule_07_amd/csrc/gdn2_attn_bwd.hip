// gdn2_attn_bwd.hip -- backward of the whole-sequence attention, for gfx950.
//
//   delta_i = do_i . o_i;  p_ij = exp(s_ij - lse_i);
//   ds_ij = p_ij (do_i . v_j - delta_i);
//   dv_j = sum_i p_ij do_i;  dk_j = scale sum_i ds_ij q_i;
//   dq_i = scale sum_j ds_ij k_j.
//
// Two kernels recompute p from the forward's lse: one owns query rows (dq) and
// walks the keys, one owns key rows (dk, dv) and walks the queries; the first
// also forms delta, from the rows of dO it holds, and leaves the rows'
// statistics for the second (a pass of its own: 2170 us against 2146 for a step
// at the sizes below, 54.5 against 52.3 for 1543 float32 tokens).  That
// is seven products where one kernel with atomic additions into dq would do
// five, and in exchange every sum has a fixed order (the same bits every run)
// and no float32 copy of dq passes through memory.  The query rows are the
// (token, head of the group) pairs of a kv head, so the sum over the heads
// that share a key row is part of the same product.
//
// Measured, 8 x 4096 tokens, 16 heads on 4, d = 128, window 2048, bfloat16 (206
// GFLOP a product; an 8192^3 product runs at 1212 TFLOP/s): dq 590 to 610 us
// (1010 to 1050 TFLOP/s), dk and dv 940 to 990 us (830 to 877 TFLOP/s).
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
  int gs;            // heads of a row tile of the dk, dv kernel
  int parts;         // workgroups that share a key tile's rows (dk, dv kernel)
  float *part_sums;  // parts > 1: [parts, 2, Ttot, Hk, D], sums of dk / scale and dv
  order od;
};

// the sum of products of 8 values, in float32
__device__ __forceinline__ float dot8(const frag8<bf16_t> &x, const frag8<bf16_t> &y) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    s += static_cast<float>(x.v[i]) * static_cast<float>(y.v[i]);
  return s;
}
__device__ __forceinline__ float dot8(const frag8<float> &x, const frag8<float> &y) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    s += x.lo[i] * y.lo[i] + x.hi[i] * y.hi[i];
  return s;
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
// WM waves of 32 rows each share key tiles; WN waves split a tile's keys and
// join their sums at the end.  Wave (wm, wn) multiplies 32 KT keys of a tile.
// q and dO stay in registers (64 at d = 128 beside dq's 64: two waves a SIMD),
// K and V come straight from memory into shared memory, a tile ahead (621 us
// through registers, 575 so).
template <typename IO, int D, int WM, int WN, int KT>
__global__ void __launch_bounds__(64 * WM * WN, (D * sizeof(IO) <= 256 ? 2 : 1)) gdn2_attn_dq_kernel(bwd_args a) {
  typedef tile<IO, D> TL;
  constexpr int NT = 64 * WM * WN, BM = 32 * WM, BN = 32 * KT * WN, CPR = TL::CPR, CH = BN * CPR / NT, RPI = NT / CPR;
  constexpr int TILEB = BN * TL::ROWB;
  static_assert(BN * CPR % NT == 0, "staging split");
  static_assert(WN == 1 || WN * 32 * D * 4 <= 4 * TILEB, "join space");
  __shared__ __align__(16) char lds[4 * TILEB];  // K and V tiles, double-buffered
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 31, h = lane >> 5;
  const int wm = WN == 1 ? wave : 0, wn = WN == 1 ? 0 : wave;
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
  const int my_row = row0 + 32 * wm + r;
  const bool row_ok = my_row < rows;
  const int cl_row = row_ok ? my_row : rows - 1;
  const int pos = cl_row / a.G, g = cl_row % a.G;
  const size_t qrow = static_cast<size_t>(sq.start + pos) * a.Hq + hk * a.G + g;
  const int wr0 = row0 + 32 * wm < rows ? row0 + 32 * wm : rows - 1;
  const int wr1 = row0 + 32 * wm + 31 < rows ? row0 + 32 * wm + 31 : rows - 1;
  const int pos_lo = wr0 / a.G, pos_hi = wr1 / a.G;
  frag8<IO> q[D / 16], d[D / 16];
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    q[kk] = load8<IO>(static_cast<const IO *>(a.q) + qrow * D + 16 * kk + 8 * h);
    d[kk] = load8<IO>(static_cast<const IO *>(a.dout) + qrow * D + 16 * kk + 8 * h);
  }
  // the row's statistics, left for the dk, dv kernel too
  f32x2 st = {a.lse[qrow] * LOG2E, 0.f};
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    st[1] += dot8(load8<IO>(static_cast<const IO *>(a.o) + qrow * D + 16 * kk + 8 * h), d[kk]);
  st[1] += __shfl_xor(st[1], 32, 64);
  if (h == 0 && wn == 0 && row_ok)
    a.stat[(static_cast<size_t>(hk) * a.Ttot + sq.start) * a.G + cl_row] = st;
  // Tiles come straight from memory: position p of one is chunk (p % CPR) ^ f
  // of row p / CPR.
  const int sc = tid % CPR, sr0 = tid / CPR, wv = __builtin_amdgcn_readfirstlane(wave);
  const int row_b = TL::row_base(r, h), col_b = TL::col_base(lane);
  const unsigned kstep = static_cast<unsigned>(a.Hk) * D;  // values of a token
  char *const kt = lds, *const vt = lds + TILEB;
  auto load_tile = [&](int kb, int buf) {
    const size_t base = (static_cast<size_t>(sq.start + kb) * a.Hk + hk) * D;
    const IO *const kp = static_cast<const IO *>(a.k) + base, *const vp = static_cast<const IO *>(a.v) + base;
    const int left = k1 - 1 - kb;  // (a key behind the last: any, its score is masked)
    char *const to = lds + buf * 2 * TILEB + 1024 * wv;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int x = sr0 + RPI * i;
      const unsigned off = (x < left ? x : left) * kstep + (sc ^ TL::f(x)) * TL::VPC;
      dma16(kp + off, to + 16 * NT * i);
      dma16(vp + off, to + TILEB + 16 * NT * i);
    }
  };
  f32x16 dq[D / 32];
#pragma unroll
  for (int n = 0; n < D / 32; ++n)
    dq[n] = zero16();
  load_tile(k0, 0);
  for (int it = 0; it < ntiles; ++it) {
    const int kb = k0 + it * BN, bo = (it & 1) * 2 * TILEB;
    dma_wait();
    __syncthreads();
    if (it + 1 < ntiles)
      load_tile(kb + BN, (it + 1) & 1);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const int wk = kb + 32 * (KT * wn + t);
      if (wk > pos_hi || (a.window > 0 && wk + 31 <= pos_lo - a.window))
        continue;  // nothing visible to the wave
      const bool masked = wk + 31 > pos_lo || (a.window > 0 && wk <= pos_hi - a.window);
      const int rb = row_b + bo + 32 * KT * wn * TL::ROWB, cb = col_b + bo + 32 * KT * wn * TL::ROWB;
      f32x16 s = zero16(), dp = zero16();
      {
        // operands read a group of products ahead
        constexpr int GR = 2, NK = D / 16, NG = 2 * NK / GR;
        frag8<IO> fa[2][GR];
        auto fetch = [&](int x0) {
#pragma unroll
          for (int x = 0; x < GR; ++x) {
            const int y = x0 * GR + x;
            fa[x0 & 1][x] = TL::row((y < NK ? kt : vt) + 32 * t * TL::ROWB, rb, y % NK);
          }
        };
        fetch(0);
#pragma unroll
        for (int x0 = 0; x0 < NG; ++x0) {
          if (x0 + 1 < NG)
            fetch(x0 + 1);
          group_fence();
#pragma unroll
          for (int x = 0; x < GR; ++x) {
            const int y = x0 * GR + x;
            mma(y < NK ? s : dp, fa[x0 & 1][x], y < NK ? q[y % NK] : d[y % NK]);
          }
          group_fence();
        }
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
          mma(dq[n], TL::col(kt, cb, 32 * t + 16 * jj, n), x);
      }
    }
  }
  IO *const out = static_cast<IO *>(a.dq) + qrow * D + 4 * h;
  if constexpr (WN > 1) {
    // wave w sums the waves' parts of channel blocks w, w + WN, ..
    float *const j = reinterpret_cast<float *>(lds) + 4 * lane;  // [wave][n, gg][lane]
    __syncthreads();
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
      for (int gg = 0; gg < 4; ++gg)
        *reinterpret_cast<f32x4 *>(j + (wn * (D / 8) + 4 * n + gg) * 256) =
            f32x4{dq[n][4 * gg], dq[n][4 * gg + 1], dq[n][4 * gg + 2], dq[n][4 * gg + 3]};
    __syncthreads();
    if (!row_ok)
      return;
    for (int n = wn; n < D / 32; n += WN)
#pragma unroll
      for (int gg = 0; gg < 4; ++gg) {
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < WN; ++w)
          x += *reinterpret_cast<const f32x4 *>(j + (w * (D / 8) + 4 * n + gg) * 256);
        io<IO>::store4(out + 32 * n + 8 * gg, x * a.scale);
      }
    return;
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
      io<IO>::store4(out + 32 * n + 8 * gg, x);
    }
}

// --------------------------------------------------------------- dk, dv --
// A workgroup owns 32 WK keys and walks the rows that see any of them, 32 WR
// at a time: wave (wk, wr) takes keys 32 wk .. + 31 and of every tile the rows
// 32 wr .. + 31; the row parts' sums are joined at the end.  K, V and the
// tile of Q and dO are read from shared memory: K and V in registers would
// leave one wave a SIMD (their 64 registers beside the 128 of the sums): 1584 us
// at the sizes above, and 940 as it is.  Now the products are busy 36 % of the
// cycles, shared memory a third, and a wave waits 40 % of its life, for operands
// and at the barrier, in step with the other wave of its SIMD.  Two groups of
// waves half a tile apart (1190), operands four or five products ahead (1005 to
// 1025) and the statistics and first operands of the second half read early
// (990), all beside 1005 on that card, do not change that; at d = 64 K and V in
// registers gain 3 %, not enough for a second form.
template <typename IO, int D, int WK, int WR>
__global__ void __launch_bounds__(64 * WK * WR, (D * sizeof(IO) <= 256 ? 2 : 1)) gdn2_attn_dkv_kernel(bwd_args a) {
  typedef tile<IO, D> TL;
  constexpr int NT = 64 * WK * WR, BK = 32 * WK, BQ = 32 * WR, CPR = TL::CPR, CH = BQ * CPR / NT, RPI = NT / CPR;
  constexpr int TILEB = BQ * TL::ROWB, KTB = BK * TL::ROWB, KCH = BK * CPR / NT;
  // A second buffer for the tile where it fits and does not cost a workgroup a
  // CU (8 waves of over 128 registers are alone on one anyway).
  constexpr int ONE = 2 * KTB + 2 * TILEB, TWO = ONE + 2 * TILEB;
  constexpr int NB = TWO <= 80000 || (TWO <= 150000 && (ONE > 80000 || NT == 512)) ? 2 : 1;
  static_assert(BQ * CPR % NT == 0 && BK * CPR % NT == 0, "staging split");
  // K, V, Q and dO; in the end the room in which the sums are joined
  constexpr int TILES = 2 * KTB + NB * 2 * TILEB, JOIN = WK * WR * 32 * D * 4;
  __shared__ __align__(16) char lds[TILES > JOIN ? TILES : JOIN];
  __shared__ __align__(16) float s_lse[NB][BQ], s_delta[NB][BQ];
  __shared__ __align__(16) int s_pos[NB][BQ];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 31, h = lane >> 5;
  const int wkey = wave % WK, wrow = wave / WK;
  int unit, slot, hk, key0;
  span sq;
  const int part = blockIdx.x % a.parts;
  if (!place(a.od, blockIdx.x / a.parts, unit, slot) ||
      !locate(a, unit, a.od.tiles - 1 - slot, 1, BK, lane, sq, hk, key0))
    return;
  const int key_end = key0 + BK < sq.len ? key0 + BK : sq.len;
  // Tokens whose rows see a key of the workgroup.  A tile is TB whole tokens
  // of GS heads (GS: the largest divisor of G up to 32; its TB GS rows come
  // first, the rest of the tile's are no rows), so that a thread's rows keep
  // their places in it and only the tile's base moves; G / GS turns over the
  // tokens take all heads.
  int tok_end = sq.len;
  if (a.window > 0 && key_end - 1 + static_cast<long>(a.window) < tok_end)
    tok_end = key_end - 1 + a.window;
  const int GS = a.gs, TB = BQ / GS, nrows = TB * GS;
  const int wk = key0 + 32 * wkey;  // the wave's first key
  const int key = wk + r;           // the lane's
  const int wk_hi = wk + 31 < sq.len - 1 ? wk + 31 : sq.len - 1;

  const int sc = tid % CPR, sr0 = tid / CPR;
  const int row_b = TL::row_base(r, h), col_b = TL::col_base(lane), st_b = TL::at(sr0, sc);
  char *const kt = lds, *const vt = lds + KTB, *const qt = lds + 2 * KTB, *const dt = qt + TILEB;
#pragma unroll
  for (int i = 0; i < KCH; ++i) {
    // (a key behind the last: any row, it is not stored)
    const int x = sr0 + RPI * i, j = key0 + x < sq.len ? key0 + x : sq.len - 1;
    const size_t off = (static_cast<size_t>(sq.start + j) * a.Hk + hk) * D + sc * TL::VPC;
    *reinterpret_cast<u32x4 *>(lds + TL::at(x, sc)) =
        *reinterpret_cast<const u32x4 *>(static_cast<const IO *>(a.k) + off);
    *reinterpret_cast<u32x4 *>(lds + KTB + TL::at(x, sc)) =
        *reinterpret_cast<const u32x4 *>(static_cast<const IO *>(a.v) + off);
  }
  // With two buffers a tile comes straight from memory: position p of it is
  // chunk (p % CPR) ^ f of row p / CPR.  With one it passes through registers.
  const int wv = __builtin_amdgcn_readfirstlane(wave);
  u32x4 rq[NB == 2 ? 1 : CH], rd[NB == 2 ? 1 : CH];
  f32x2 rs = {0.f, 0.f};
  int rp = 0;
  int tok_of[CH];  // token of a thread's row in the tile, and its values' place
  unsigned at_of[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    int x = sr0 + RPI * i;
    x = x < nrows ? x : nrows - 1;
    tok_of[i] = x / GS;
    at_of[i] = static_cast<unsigned>(x % GS * D + (NB == 2 ? sc ^ TL::f(sr0 + RPI * i) : sc) * TL::VPC);
  }
  const int my_x = tid < nrows ? tid : nrows - 1, my_tok = my_x / GS, my_g = my_x % GS;
  const bool my_ok = tid < nrows;
  const unsigned tstep = static_cast<unsigned>(a.Hq) * D;  // values of a token
  const int ntok = (tok_end - key0 + TB - 1) / TB, ntiles = ntok * (a.G / GS);
  // Order of the tiles: a sequence's workgroups run side by side on one die,
  // whose L2 holds a part of its rows, so they walk the tokens in step: without
  // a window from the end down, where all have rows; with one from the first
  // tile whose index is a multiple of the window's tiles.
  int turn = 0;
  if (a.window > 0) {
    const int period = static_cast<int>((static_cast<long>(a.window) + BK - 1) / TB) + 1;
    turn = (period - key0 / TB % period) % period;
    turn = turn < ntok ? turn : 0;
  }
  auto load_tile = [&](int it) {
    const int sub = it / ntok;
    int x = it - sub * ntok;
    x = a.window > 0 ? (x + turn < ntok ? x + turn : x + turn - ntok) : ntok - 1 - x;
    const int t0 = key0 + x * TB;
    const size_t base = (static_cast<size_t>(sq.start + t0) * a.Hq + hk * a.G + sub * GS) * D;
    const IO *const qb = static_cast<const IO *>(a.q) + base, *const db = static_cast<const IO *>(a.dout) + base;
    const int left = tok_end - 1 - t0;  // (a token behind the last: any, its weight is 0)
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const unsigned off = (tok_of[i] < left ? tok_of[i] : left) * tstep + at_of[i];
      if constexpr (NB == 2) {
        char *const to = qt + (it & 1) * 2 * TILEB + 1024 * wv + 16 * NT * i;
        dma16(qb + off, to);
        dma16(db + off, to + TILEB);
      } else {
        rq[i] = *reinterpret_cast<const u32x4 *>(qb + off);
        rd[i] = *reinterpret_cast<const u32x4 *>(db + off);
      }
    }
    if (tid < BQ) {
      const bool ok = my_ok && my_tok <= left;
      const f32x2 x = a.stat[(static_cast<size_t>(hk) * a.Ttot + sq.start + t0 + (ok ? my_tok : 0)) * a.G + sub * GS + my_g];
      // no row: weight 2^(0 - inf) = 0
      rs = f32x2{ok ? x[0] : __builtin_inff(), ok ? x[1] : 0.f};
      rp = t0 + my_tok;
    }
  };
  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int n = 0; n < D / 32; ++n)
    dk[n] = dv[n] = zero16();
  // this workgroup's share of the tiles
  const int per = (ntiles + a.parts - 1) / a.parts, it0 = part * per, it1 = it0 + per < ntiles ? it0 + per : ntiles;
  if (it0 < it1)
    load_tile(it0);
  for (int it = it0; it < it1; ++it) {
    const int buf = NB == 2 ? it & 1 : 0;
    const int bo = buf * 2 * TILEB;
    if (NB == 1 && it > it0)
      __syncthreads();  // the tile before is read
    if constexpr (NB == 2) {
      dma_wait();
    } else {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int at = TL::template step<RPI>(st_b, sr0, sc, i);
        *reinterpret_cast<u32x4 *>(qt + at) = rq[i];
        *reinterpret_cast<u32x4 *>(dt + at) = rd[i];
      }
    }
    if (tid < BQ) {
      s_lse[buf][tid] = rs[0];
      s_delta[buf][tid] = rs[1];
      s_pos[buf][tid] = rp;
    }
    __syncthreads();
    if (it + 1 < it1)
      load_tile(it + 1);
    const int u0 = 32 * wrow;
    if (u0 >= nrows)
      continue;
    const int p_lo = __builtin_amdgcn_readfirstlane(s_pos[buf][u0]);
    const int p_hi = __builtin_amdgcn_readfirstlane(s_pos[buf][u0 + 31]);
    if (p_lo >= tok_end || wk > p_hi || wk >= sq.len || (a.window > 0 && wk_hi <= p_lo - a.window))
      continue;  // no row sees a key of the wave
    const bool masked = wk_hi > p_lo || (a.window > 0 && wk <= p_hi - a.window);
    const int rb = row_b + bo + u0 * TL::ROWB, cb = col_b + bo + u0 * TL::ROWB;
    const int kb = fresh(row_b + 32 * wkey * TL::ROWB);
    f32x16 s = zero16(), dp = zero16();
    {
      // operands read a group of products ahead
      constexpr int GR = 2, NK = D / 16, NG = 2 * NK / GR;
      frag8<IO> fa[2][GR], fb[2][GR];
      auto fetch = [&](int g) {
#pragma unroll
        for (int x = 0; x < GR; ++x) {
          const int y = g * GR + x;
          fa[g & 1][x] = TL::row(y < NK ? qt : dt, rb, y % NK);
          fb[g & 1][x] = TL::row(y < NK ? kt : vt, kb, y % NK);
        }
      };
      fetch(0);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (g + 1 < NG)
          fetch(g + 1);
        group_fence();
#pragma unroll
        for (int x = 0; x < GR; ++x)
          mma(g * GR + x < NK ? s : dp, fa[g & 1][x], fb[g & 1][x]);
        group_fence();
      }
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x4 ls = *reinterpret_cast<const f32x4 *>(&s_lse[buf][u0 + 8 * g + 4 * h]);
      const f32x4 de = *reinterpret_cast<const f32x4 *>(&s_delta[buf][u0 + 8 * g + 4 * h]);
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
        const i32x4 ps = *reinterpret_cast<const i32x4 *>(&s_pos[buf][u0 + 8 * g + 4 * h]);
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
        mma(dv[n], TL::col(dt, cb, 16 * jj, n), p);
        mma(dk[n], TL::col(qt, cb, 16 * jj, n), ds);
      }
    }
  }
  // The row parts joined: halves until two are left; of those, wave (wk, 1)
  // leaves dk and takes dv, wave (wk, 0) the other way round.
  constexpr int PART = 32 * D;  // floats
  auto slot_of = [&](int x) { return reinterpret_cast<float *>(lds) + (x * WK + wkey) * PART + 4 * lane; };
  auto leave = [&](const f32x16(&x)[D / 32], float *to) {
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4 *>(to + (4 * n + g) * 256) =
            f32x4{x[n][4 * g], x[n][4 * g + 1], x[n][4 * g + 2], x[n][4 * g + 3]};
  };
  auto take = [&](f32x16(&x)[D / 32], const float *from) {
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 y = *reinterpret_cast<const f32x4 *>(from + (4 * n + g) * 256);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[n][4 * g + i] += y[i];
      }
  };
  auto store = [&](const f32x16(&x)[D / 32], float scale, IO *out) {
    if (key >= sq.len)
      return;
    const size_t at = (static_cast<size_t>(sq.start + key) * a.Hk + hk) * D + 4 * h;
    if (a.parts > 1) {
      float *const sums = a.part_sums + (2 * part + (wrow == 0 ? 0 : 1)) * (static_cast<size_t>(a.Ttot) * a.Hk * D) + at;
#pragma unroll
      for (int n = 0; n < D / 32; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          io<float>::store4(sums + 32 * n + 8 * g,
                            f32x4{x[n][4 * g], x[n][4 * g + 1], x[n][4 * g + 2], x[n][4 * g + 3]});
      return;
    }
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4 z;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          z[i] = x[n][4 * g + i] * scale;
        io<IO>::store4(out + at + 32 * n + 8 * g, z);
      }
  };
#pragma unroll
  for (int half = WR / 2; half > 1; half /= 2) {
    __syncthreads();
    if (wrow >= half && wrow < 2 * half) {
      leave(dk, slot_of(wrow - half));
      leave(dv, slot_of(wrow));
    }
    __syncthreads();
    if (wrow < half) {
      take(dk, slot_of(wrow));
      take(dv, slot_of(wrow + half));
    }
  }
  __syncthreads();
  if (wrow == 0)
    leave(dv, slot_of(0));
  else if (wrow == 1)
    leave(dk, slot_of(1));
  __syncthreads();
  if (wrow == 0) {
    take(dk, slot_of(1));
    store(dk, a.scale, static_cast<IO *>(a.dk));
  } else if (wrow == 1) {
    take(dv, slot_of(0));
    store(dv, 1.f, static_cast<IO *>(a.dv));
  }
}

// The parts' sums, in order, to dk and dv: four channels a thread, dk's then
// dv's.
template <typename IO, int D> __global__ void __launch_bounds__(256) gdn2_attn_dkv_join_kernel(bwd_args a) {
  const size_t rows = static_cast<size_t>(a.Ttot) * a.Hk * D;
  const size_t at = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (at >= 2 * rows)
    return;
  const bool is_v = at >= rows;
  const size_t e = is_v ? at - rows : at;
  if (a.cu && static_cast<long>(e / (static_cast<size_t>(a.Hk) * D)) >= a.cu[a.N])
    return;  // behind the last sequence
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int p = 0; p < a.parts; ++p)
    x += io<float>::load4(a.part_sums + 2 * p * rows + at);
  io<IO>::store4(static_cast<IO *>(is_v ? a.dv : a.dk) + e, x * (is_v ? 1.f : a.scale));
}

// ------------------------------------------------------------- launchers --
// Workgroups that share a 64-key tile's rows: where a call has few key tiles
// (few tokens, or one kv head for many query heads), enough for 1024 of them,
// at most 16 and at most one for every 1024 rows of the call, whether or not a
// window or a sequence's end hides rows from a tile.  (4096 tokens, 16 query heads on one
// kv head, d = 128: dk and dv 1867 us with one, 320 with 16; 11 packed
// sequences, 9973 tokens, 12 heads on 4, d = 64: 166 with one, 130 with two;
// 1543 float32 tokens, 4 heads on 4: 22 with one, 34 with three.)  The rule sees
// the sizes the workspace is asked for: tokens and heads, no sequence lengths
// and no window.  Counting only the rows a window leaves a tile gains where
// the parts' sums outweigh the call and loses where few tiles need the parts:
// 4096 tokens, d = 128, 4 heads on 4, window 100: 42 us as it is, 20 counted so;
// 16 heads on one, window 64: 49 and 72, window 512: 79 and 98; 16 on 2, d = 64,
// window 256: 49 and 30.
int attn_bwd_parts(const attn_sizes &z) {
  const long long seqs = z.packed ? 1 : z.N;
  const long long tiles = seqs * ((z.T + 63) / 64) * z.Hk, rows = static_cast<long long>(z.T) * (z.Hq / z.Hk);
  long long p = (1024 + tiles - 1) / (tiles > 0 ? tiles : 1);
  if (p > rows / 1024)
    p = rows / 1024;
  return p < 1 ? 1 : (p > 16 ? 16 : static_cast<int>(p));
}

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
  a.parts = attn_bwd_parts(z);
  a.part_sums = a.parts > 1 ? reinterpret_cast<float *>(static_cast<char *>(ws) + attn_bwd_stat_bytes(z)) : nullptr;
  a.gs = a.G < 32 ? a.G : 32;
  while (a.G % a.gs)
    --a.gs;
}

template <typename IO, int D>
hipError_t launch_attn_bwd_dq(const attn_sizes &z, const attn_ptrs &p, void *ws, hipStream_t st) {
  bwd_args a;
  fill(a, z, p, ws);
  // (few tiles: 4 waves where their tiles fit shared memory; float32, d = 64,
  // 1543 tokens, 4 heads, window 300: 17 us, 25 with 2)
  constexpr int KT = sizeof(IO) == 2 ? 2 : 1, WN = D * sizeof(IO) <= 256 ? 4 : 2;
  const unsigned blocks = plan_tiles(z, z.Hq / z.Hk, 128, a.od);
  if (few_tiles(a.od)) {
    const unsigned few = plan_tiles(z, z.Hq / z.Hk, 32, a.od);
    hipLaunchKernelGGL((gdn2_attn_dq_kernel<IO, D, 1, WN, 1>), dim3(few), dim3(64 * WN), 0, st, a);
  } else {
    hipLaunchKernelGGL((gdn2_attn_dq_kernel<IO, D, 4, 1, KT>), dim3(blocks), dim3(256), 0, st, a);
  }
  return hipGetLastError();
}
template <typename IO, int D>
hipError_t launch_attn_bwd_dkv(const attn_sizes &z, const attn_ptrs &p, void *ws, hipStream_t st) {
  bwd_args a;
  fill(a, z, p, ws);
  // Where the tiles do not give every CU two, the longest sequence's first
  // keys, which every row sees, take as long as the call: d = 64 then takes
  // half as many keys and twice the row parts a workgroup.  (bfloat16, 11 packed
  // sequences of up to 3167 tokens x 4 kv heads: 356 tiles, 157 against 200 us;
  // d = 128 has no registers for it, 8 waves of 64 keys would go through
  // scratch.)
  constexpr int WK = sizeof(IO) == 2 ? 4 : 2;
  constexpr bool HALF = D * sizeof(IO) <= 128 || sizeof(IO) == 4;
  constexpr int WKH = HALF ? WK / 2 : WK, WRH = D == 64 ? 4 : 2;
  unsigned blocks = plan_tiles(z, 1, 32 * WK, a.od);
  if (!HALF || (a.parts == 1 && static_cast<long long>(a.od.units) * a.od.tiles >= 512)) {
    hipLaunchKernelGGL((gdn2_attn_dkv_kernel<IO, D, WK, 2>), dim3(blocks * a.parts), dim3(128 * WK), 0, st, a);
  } else {
    blocks = plan_tiles(z, 1, 32 * WKH, a.od);
    hipLaunchKernelGGL((gdn2_attn_dkv_kernel<IO, D, WKH, WRH>), dim3(blocks * a.parts), dim3(64 * WKH * WRH), 0, st, a);
  }
  if (a.parts > 1) {
    const size_t n = static_cast<size_t>(z.Ttot) * z.Hk * D / 2;  // threads
    hipLaunchKernelGGL((gdn2_attn_dkv_join_kernel<IO, D>), dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

#define GDN2_INST_ATTN_BWD(IO, D)                                                                         \
  template hipError_t launch_attn_bwd_dq<IO, D>(const attn_sizes &, const attn_ptrs &, void *, hipStream_t); \
  template hipError_t launch_attn_bwd_dkv<IO, D>(const attn_sizes &, const attn_ptrs &, void *, hipStream_t);
GDN2_INST_ATTN_BWD(float, 64)
GDN2_INST_ATTN_BWD(float, 128)
GDN2_INST_ATTN_BWD(bf16_t, 64)
GDN2_INST_ATTN_BWD(bf16_t, 128)

}  // namespace attn
}  // namespace gdn2
