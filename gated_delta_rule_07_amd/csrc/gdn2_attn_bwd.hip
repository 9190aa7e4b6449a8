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
// that share a key row is part of the same product.  delta is formed from the
// stored o, for bfloat16 rounded (half a step a value): a float32 o would have to be
// kept from the forward, twice o's bytes.  p and ds are rounded as operands (pack8).
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
  int sinks;         // first keys visible behind the window (0: none, or no window)
  int far_parts;     // workgroups that share the rows which see a sink from behind the window, a sequence
  int far_extra;     // packed: so many more, one for every far_step tokens
  int far_step;
  float *far_sums;   // sinks > 0: [far_parts, 2, far_rows, Hk, D], their sums of dk / scale and dv, then
                     // [far_extra, 2, sinks, Hk, D]
  size_t far_rows;   // a row for every sink of every sequence, or (far_by_token) for every token
  bool far_by_token;
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
// SINK: keys and positions are numbered without the gap between the sinks and
// the window, as in the forward.
template <typename IO, int D, int WM, int WN, int KT, bool SINK>
__global__ void __launch_bounds__(64 * WM * WN, (D * sizeof(IO) <= 256 ? 2 : 1)) gdn2_attn_dq_kernel(bwd_args a) {
  typedef tile<IO, D> TL;
  constexpr int NT = 64 * WM * WN, BM = 32 * WM, BN = 32 * KT * WN, CPR = TL::CPR, CH = BN * CPR / NT, RPI = NT / CPR;
  constexpr int TILEB = BN * TL::ROWB;
  static_assert(BN * CPR % NT == 0, "staging split");
  static_assert(WN == 1 || WN * 32 * D * 4 <= 4 * TILEB, "join space");
  __shared__ __align__(16) char lds[4 * TILEB];  // K and V tiles, double-buffered
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // (uniform: so is what follows from it)
  const int wm = WN == 1 ? wave : 0, wn = WN == 1 ? 0 : wave;
  int unit, slot, hk, row0;
  span sq;
  if (!place(a.od, blockIdx.x, unit, slot) || !locate(a, unit, slot, a.G, BM, lane, sq, hk, row0))
    return;
  const int rows = sq.len * a.G;
  const int last_row = row0 + BM - 1 < rows - 1 ? row0 + BM - 1 : rows - 1;
  int k1 = last_row / a.G + 1;
  int k0 = 0;
  if (a.window > 0) {
    k0 = row0 / a.G - a.window + 1;
    k0 = k0 < 0 ? 0 : k0;
  }
  int gap = 0;
  if constexpr (SINK) {
    gap = k0 > a.sinks ? k0 - a.sinks : 0;
    k0 = 0;
    k1 -= gap;
  }
  const int ntiles = (k1 - k0 + BN - 1) / BN;
  const int my_row = row0 + 32 * wm + r;
  const bool row_ok = my_row < rows;
  const int cl_row = row_ok ? my_row : rows - 1;
  const int tok = cl_row / a.G, pos = tok - gap, g = cl_row % a.G;
  const size_t qrow = static_cast<size_t>(sq.start + tok) * a.Hq + hk * a.G + g;
  const int wr0 = row0 + 32 * wm < rows ? row0 + 32 * wm : rows - 1;
  const int wr1 = row0 + 32 * wm + 31 < rows ? row0 + 32 * wm + 31 : rows - 1;
  const int pos_lo = wr0 / a.G - gap, pos_hi = wr1 / a.G - gap;
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
  const int sc = tid % CPR, sr0 = tid / CPR;
  const int row_b = TL::row_base(r, h), col_b = TL::col_base(lane);
  const unsigned kstep = static_cast<unsigned>(a.Hk) * D;  // values of a token
  char *const kt = lds, *const vt = lds + TILEB;
  auto load_tile = [&](int kb, int buf) {
    // (a tile with sinks takes its keys one by one, from the sequence's first)
    const bool mixed = SINK && kb < a.sinks;
    const size_t base = (static_cast<size_t>(sq.start + (mixed ? 0 : kb + gap)) * a.Hk + hk) * D;
    const IO *const kp = static_cast<const IO *>(a.k) + base, *const vp = static_cast<const IO *>(a.v) + base;
    const int left = k1 - 1 - kb;  // (a key behind the last: any, its score is masked)
    char *const to = lds + buf * 2 * TILEB + 1024 * wave;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int x = sr0 + RPI * i;
      auto bring = [&](auto off) {
        off += (sc ^ TL::f(x)) * TL::VPC;
        dma16(kp + off, to + 16 * NT * i);
        dma16(vp + off, to + TILEB + 16 * NT * i);
      };
      if (mixed) {
        const int j = kb + (x < left ? x : left);
        bring(static_cast<size_t>(j < a.sinks ? j : j + gap) * kstep);
      } else {
        bring((x < left ? x : left) * kstep);
      }
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
      if (wk > pos_hi || (a.window > 0 && wk + 31 <= pos_lo - a.window && !(SINK && wk < a.sinks)))
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
        const int sink_rel = SINK ? a.sinks - wk - 4 * h : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = 8 * (i >> 2) + (i & 3);
          s[i] = (j <= hi_rel && (j > lo_rel || (SINK && j < sink_rel))) ? s[i] : 0.f;
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
//
// Sinks.  The rows that see a sink from behind the window (all later ones) are
// many for few keys: a launch of its own (DKV_FAR) shares them among far_parts
// workgroups a 32-key tile and leaves float32 sums, and the workgroup that owns
// the keys (DKV_SINK) begins with them.  Every sum has a fixed order.
enum dkv_mode { DKV_PLAIN, DKV_SINK, DKV_FAR };
// Tile of the DKV_FAR launch: 128 rows where two of them fit shared memory
// beside the keys (64 would pass through registers and spill).
constexpr int FAR_KEYS = 32;
constexpr int FAR_TILES = 16;  // of a workgroup beyond a sequence's far_parts
template <typename IO, int D> constexpr int FAR_ROWS = D * sizeof(IO) <= 256 ? 128 : 64;
// Tiles of TB tokens of the rows of a sequence of len tokens that see a key
// from key0 on from behind the window, and how many of them a part takes.
__device__ __forceinline__ int far_tiles(const bwd_args &a, int len, int key0, int TB) {
  const long n = static_cast<long>(len) - key0 - a.window;
  return n > 0 ? static_cast<int>((n + TB - 1) / TB) * (a.G / a.gs) : 0;
}
// The workgroups that share the n far tiles of a sequence's keys: far_parts, and
// number e of the far_extra where token far_step (e + 1) - 1 of the call is the
// sequence's, so that a long one among short ones has nearly all of them; but those
// only while a workgroup has FAR_TILES, since the keys' owner adds the parts one by one.
__device__ __forceinline__ int far_share(const bwd_args &a, const span &sq, int n) {
  int share = a.far_parts;
  if (a.far_extra) {
    const int more = share + (sq.start + sq.len) / a.far_step - sq.start / a.far_step, most = (n + FAR_TILES - 1) / FAR_TILES;
    const int x = more < most ? more : most;
    share = x > share ? x : share;
  }
  return share;
}
// Parts that hold sums for a sink (their workgroups had rows).
template <typename IO, int D> __device__ __forceinline__ int far_parts_of(const bwd_args &a, const span &sq, int key) {
  const int n = far_tiles(a, sq.len, key - key % FAR_KEYS, FAR_ROWS<IO, D> / a.gs), share = far_share(a, sq, n);
  const int per = (n + share - 1) / share;
  return n ? (n + per - 1) / per : 0;
}
template <int D>
__device__ __forceinline__ float *far_sum(const bwd_args &a, int part, bool is_v, const span &sq, int key, int hk) {
  const int v = is_v ? 1 : 0;
  size_t row;
  if (part < a.far_parts) {
    row = (2 * part + v) * a.far_rows + (a.far_by_token ? sq.start : static_cast<size_t>(sq.n) * a.sinks) + key;
  } else {
    const int e = sq.start / a.far_step + part - a.far_parts;
    row = 2 * a.far_parts * a.far_rows + static_cast<size_t>(2 * e + v) * a.sinks + key;
  }
  return a.far_sums + (row * a.Hk + hk) * D;
}
template <typename IO, int D, int WK, int WR, dkv_mode M>
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
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // (uniform: so is what follows from it)
  const int wkey = wave % WK, wrow = wave / WK;
  int unit, slot, hk, key0;
  span sq;
  int parts = a.parts, part = blockIdx.x % parts;
  if constexpr (M == DKV_FAR) {
    // a unit a sequence and kv head, a tile for every 32 sinks; behind all sequences'
    // parts, those that long sequences have in addition
    const int tiles = (a.sinks + BK - 1) / BK, block = blockIdx.x, first = a.N * a.Hk * tiles * a.far_parts;
    if (block < first) {
      const int id = block / a.far_parts;
      part = block % a.far_parts;
      unit = id / tiles;
      sq.n = unit / a.Hk;
      hk = unit % a.Hk;
      key0 = id % tiles * BK;
      if (a.cu) {
        sq = packed_span(a.cu, sq.n, a.T);
      } else {
        sq.start = sq.n * a.T;
        sq.len = a.T;
      }
    } else {
      const int id = (block - first) / a.far_extra, e = (block - first) % a.far_extra;
      hk = id / tiles;
      key0 = id % tiles * BK;
      const int last = e * a.far_step + a.far_step - 1;
      sq = packed_span(a.cu, find_last([&](int i) { return a.cu[i] <= last; }, a.N, lane), a.T);
      part = a.far_parts + e - sq.start / a.far_step;
      if (part < a.far_parts)
        return;
    }
    if (key0 >= sq.len)
      return;
    parts = far_share(a, sq, far_tiles(a, sq.len, key0, BQ / a.gs));
    if (part >= parts)
      return;
  } else {
    if (!place(a.od, blockIdx.x / parts, unit, slot) ||
        !locate(a, unit, a.od.tiles - 1 - slot, 1, BK, lane, sq, hk, key0))
      return;
  }
  // keys of the workgroup: all of the sequence's, or its sinks
  const int last_key = M == DKV_FAR && a.sinks < sq.len ? a.sinks : sq.len;
  const int key_end = key0 + BK < last_key ? key0 + BK : last_key;
  // Tokens whose rows see a key of the workgroup.  A tile is TB whole tokens
  // of GS heads (GS: the largest divisor of G up to 32; its TB GS rows come
  // first, the rest of the tile's are no rows), so that a thread's rows keep
  // their places in it and only the tile's base moves; G / GS turns over the
  // tokens take all heads.
  const int tok_0 = M == DKV_FAR ? key0 + a.window : key0;  // (less than len where there are tiles)
  int tok_end = sq.len;
  if (M != DKV_FAR && a.window > 0 && key_end - 1 + static_cast<long>(a.window) < tok_end)
    tok_end = key_end - 1 + a.window;
  const int GS = a.gs, TB = BQ / GS, nrows = TB * GS;
  const int wk = key0 + 32 * wkey;  // the wave's first key
  const int key = wk + r;           // the lane's
  const int wk_hi = wk + 31 < last_key - 1 ? wk + 31 : last_key - 1;

  const int sc = tid % CPR, sr0 = tid / CPR;
  const int row_b = TL::row_base(r, h), col_b = TL::col_base(lane), st_b = TL::at(sr0, sc);
  char *const kt = lds, *const vt = lds + KTB, *const qt = lds + 2 * KTB, *const dt = qt + TILEB;
#pragma unroll
  for (int i = 0; i < KCH; ++i) {
    // (a key behind the last: any row, it is not stored)
    const int x = sr0 + RPI * i, j = key0 + x < last_key ? key0 + x : last_key - 1;
    const size_t off = (static_cast<size_t>(sq.start + j) * a.Hk + hk) * D + sc * TL::VPC;
    *reinterpret_cast<u32x4 *>(lds + TL::at(x, sc)) =
        *reinterpret_cast<const u32x4 *>(static_cast<const IO *>(a.k) + off);
    *reinterpret_cast<u32x4 *>(lds + KTB + TL::at(x, sc)) =
        *reinterpret_cast<const u32x4 *>(static_cast<const IO *>(a.v) + off);
  }
  // With two buffers a tile comes straight from memory: position p of it is
  // chunk (p % CPR) ^ f of row p / CPR.  With one it passes through registers.
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
  const int ntiles = M == DKV_FAR ? far_tiles(a, sq.len, key0, TB) : (tok_end - key0 + TB - 1) / TB * (a.G / GS);
  const int ntok = ntiles / (a.G / GS);
  // Order of the tiles: a sequence's workgroups run side by side on one die,
  // whose L2 holds a part of its rows, so they walk the tokens in step: without
  // a window from the end down, where all have rows; with one from the first
  // tile whose index is a multiple of the window's tiles.
  int turn = 0;
  if (M != DKV_FAR && a.window > 0) {
    const int period = static_cast<int>((static_cast<long>(a.window) + BK - 1) / TB) + 1;
    turn = (period - key0 / TB % period) % period;
    turn = turn < ntok ? turn : 0;
  }
  auto load_tile = [&](int it) {
    const int sub = it / ntok;
    int x = it - sub * ntok;
    x = a.window > 0 ? (x + turn < ntok ? x + turn : x + turn - ntok) : ntok - 1 - x;
    const int t0 = tok_0 + x * TB;
    const size_t base = (static_cast<size_t>(sq.start + t0) * a.Hq + hk * a.G + sub * GS) * D;
    const IO *const qb = static_cast<const IO *>(a.q) + base, *const db = static_cast<const IO *>(a.dout) + base;
    const int left = tok_end - 1 - t0;  // (a token behind the last: any, its weight is 0)
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const unsigned off = (tok_of[i] < left ? tok_of[i] : left) * tstep + at_of[i];
      if constexpr (NB == 2) {
        char *const to = qt + (it & 1) * 2 * TILEB + 1024 * wave + 16 * NT * i;
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
  const int per = (ntiles + parts - 1) / parts, it0 = part * per, it1 = it0 + per < ntiles ? it0 + per : ntiles;
  if (M == DKV_FAR && it0 >= it1)
    return;  // (no sums: far_parts_of does not count the part)
  if (it0 < it1)
    load_tile(it0);
  if constexpr (M == DKV_SINK) {
    // a sink's sums over the far rows: part 0's row parts begin with them
    if (part == 0 && key < a.sinks && key < last_key) {
      const int np = far_parts_of<IO, D>(a, sq, key);
      for (int p = wrow; p < np; p += WR) {
        const float *const sk = far_sum<D>(a, p, false, sq, key, hk) + 4 * h;
        const float *const sv = far_sum<D>(a, p, true, sq, key, hk) + 4 * h;
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x4 x = io<float>::load4(sk + 32 * n + 8 * g), y = io<float>::load4(sv + 32 * n + 8 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              dk[n][4 * g + i] += x[i];
              dv[n][4 * g + i] += y[i];
            }
          }
      }
    }
  }
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
    if (p_lo >= tok_end || wk >= last_key ||
        (M == DKV_FAR ? wk > p_hi - a.window : wk > p_hi || (a.window > 0 && wk_hi <= p_lo - a.window)))
      continue;  // no row sees a key of the wave
    // (keys behind the last are not stored)
    const bool masked = M == DKV_FAR ? wk_hi > p_lo - a.window : wk_hi > p_lo || (a.window > 0 && wk <= p_hi - a.window);
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
          const bool vis = M == DKV_FAR ? key <= ps[i] - a.window : key <= ps[i] && (a.window <= 0 || key > ps[i] - a.window);
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
    if (key >= last_key)
      return;
    const size_t at = (static_cast<size_t>(sq.start + key) * a.Hk + hk) * D + 4 * h;
    const bool is_v = wrow != 0;
    if constexpr (M == DKV_FAR) {
      float *const sums = far_sum<D>(a, part, is_v, sq, key, hk) + 4 * h;
#pragma unroll
      for (int n = 0; n < D / 32; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          io<float>::store4(sums + 32 * n + 8 * g,
                            f32x4{x[n][4 * g], x[n][4 * g + 1], x[n][4 * g + 2], x[n][4 * g + 3]});
      return;
    }
    if (a.parts > 1) {
      float *const sums = a.part_sums + (2 * part + (is_v ? 1 : 0)) * (static_cast<size_t>(a.Ttot) * a.Hk * D) + at;
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

// Workgroups that share the rows behind the window of a 32-sink tile of a
// sequence and kv head: one a CU, or where sequences are packed, whose lengths
// differ, four; at most 64 and at most one for every 128 rows of the call.  (8 x
// 4096 tokens, window 2048, 4 sinks, 16 heads on 4, d = 128: 33 us for 256
// workgroups, 40 and 48 for 512 and 1024, 134 MB read; 32768 tokens: 57, 252 MB;
// 11 packed sequences, 9973 tokens, window 500, 33 sinks, d = 64: 35 for 256, 22
// and 19 for 512 and 1024; 1543 float32 tokens, 7 sinks: 10.3, and 15.1 for 512
// rows a workgroup.)
//
// Packed sequences may be one long one and many short ones, which leave their parts
// without rows: what one sequence alone would have in addition (far_extra) is
// dealt out by the tokens.  (16 heads on 4, d = 128, window 2048, 4 sinks: one of 30000
// tokens before 255 of 10: 82 to 87 us, behind them 60 to 63, alone 54, and 2030 with the same parts for
// all; one of 16384 before 63 of 256: 49 to 53, alone 29, and 279.  All of them whatever the rows: 6
// sequences of up to 2833 tokens, 163 sinks, 2 heads on one, d = 64: dk and dv 50, not 30.)
static int far_parts_for(const attn_sizes &z, int N) {
  const long long units = static_cast<long long>(N) * z.Hk * ((z.sinks + FAR_KEYS - 1) / FAR_KEYS);
  const long long rows = static_cast<long long>(z.T) * (z.Hq / z.Hk);
  long long p = ((z.packed ? 1024 : 256) + units - 1) / units;
  if (p > rows / 128)
    p = rows / 128;
  return p < 1 ? 1 : (p > 64 ? 64 : static_cast<int>(p));
}
int attn_bwd_far_parts(const attn_sizes &z) { return far_parts_for(z, z.N); }
int attn_bwd_far_extra(const attn_sizes &z) { return z.packed ? far_parts_for(z, 1) - far_parts_for(z, z.N) : 0; }

static void fill(bwd_args &a, const attn_sizes &z, const attn_ptrs &p, void *ws, int d, int far_tile) {
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
  if (z.sinks) {
    // Here a window counts (the workspace has room for more): about 2048 rows
    // of 64 channels, or 1024 of 128, a part.  (4 sinks, windows of 100, 500, 2000:
    // 4096 tokens, 4 heads on 4, d = 128: 33, 44, 58 us with 1, 1, 2 parts, 57, 62, 72
    // with 4; 16 heads on 2: 69, 95, 176 with 2, 5, 8, and 103, 195, 541 with one;
    // 9973 packed tokens, 12 heads on 4, d = 64, window 500: 72 with one, 90 with 2.)
    const long long keys = z.T < z.window + 128LL ? z.T : z.window + 128LL, rows = keys * a.G;
    const long long most = (rows * d + 65536) / 131072;
    a.parts = most < 1 ? 1 : (most < a.parts ? static_cast<int>(most) : a.parts);
  }
  a.part_sums = a.parts > 1 ? reinterpret_cast<float *>(static_cast<char *>(ws) + attn_bwd_stat_bytes(z)) : nullptr;
  a.sinks = z.sinks;
  a.far_parts = z.sinks ? attn_bwd_far_parts(z) : 0;
  a.far_extra = z.sinks ? attn_bwd_far_extra(z) : 0;
  a.far_rows = attn_bwd_far_rows(z);
  a.far_by_token = attn_bwd_far_by_token(z);
  a.far_sums = z.sinks ? reinterpret_cast<float *>(static_cast<char *>(ws) + attn_bwd_bytes(z, d)) : nullptr;
  a.gs = a.G < 32 ? a.G : 32;
  while (a.G % a.gs)
    --a.gs;
  // (none where even one sequence of all tokens would leave far_parts less than 2
  // FAR_TILES each: workgroups that find nothing to do cost 1 us of the packed d = 64 case)
  const int tb = far_tile / a.gs;
  if ((z.T - z.window + tb - 1) / tb * (a.G / a.gs) <= 2 * FAR_TILES * a.far_parts)
    a.far_extra = 0;
  a.far_step = a.far_extra ? (z.T + a.far_extra - 1) / a.far_extra : 1;
}

template <typename IO, int D>
hipError_t launch_attn_bwd_dq(const attn_sizes &z, const attn_ptrs &p, void *ws, hipStream_t st) {
  bwd_args a;
  fill(a, z, p, ws, D, FAR_ROWS<IO, D>);
  // (few tiles: 4 waves where their tiles fit shared memory; float32, d = 64,
  // 1543 tokens, 4 heads, window 300: 17 us, 25 with 2)
  constexpr int KT = sizeof(IO) == 2 ? 2 : 1, WN = D * sizeof(IO) <= 256 ? 4 : 2;
  const unsigned blocks = plan_tiles(z, z.Hq / z.Hk, 128, a.od);
  if (few_tiles(a.od)) {
    const unsigned few = plan_tiles(z, z.Hq / z.Hk, 32, a.od);
    if (a.sinks)
      hipLaunchKernelGGL((gdn2_attn_dq_kernel<IO, D, 1, WN, 1, true>), dim3(few), dim3(64 * WN), 0, st, a);
    else
      hipLaunchKernelGGL((gdn2_attn_dq_kernel<IO, D, 1, WN, 1, false>), dim3(few), dim3(64 * WN), 0, st, a);
  } else if (a.sinks) {
    hipLaunchKernelGGL((gdn2_attn_dq_kernel<IO, D, 4, 1, KT, true>), dim3(blocks), dim3(256), 0, st, a);
  } else {
    hipLaunchKernelGGL((gdn2_attn_dq_kernel<IO, D, 4, 1, KT, false>), dim3(blocks), dim3(256), 0, st, a);
  }
  return hipGetLastError();
}
template <typename IO, int D>
hipError_t launch_attn_bwd_far(const attn_sizes &z, const attn_ptrs &p, void *ws, hipStream_t st) {
  bwd_args a;
  fill(a, z, p, ws, D, FAR_ROWS<IO, D>);
  const unsigned tiles = static_cast<unsigned>(z.Hk) * ((z.sinks + FAR_KEYS - 1) / FAR_KEYS);
  const unsigned blocks = tiles * (static_cast<unsigned>(z.N) * a.far_parts + a.far_extra);
  hipLaunchKernelGGL((gdn2_attn_dkv_kernel<IO, D, FAR_KEYS / 32, FAR_ROWS<IO, D> / 32, DKV_FAR>), dim3(blocks),
                     dim3(2 * FAR_ROWS<IO, D>), 0, st, a);
  return hipGetLastError();
}
template <typename IO, int D, int WK, int WR>
static void launch_dkv(const bwd_args &a, unsigned blocks, hipStream_t st) {
  if (a.sinks)
    hipLaunchKernelGGL((gdn2_attn_dkv_kernel<IO, D, WK, WR, DKV_SINK>), dim3(blocks), dim3(64 * WK * WR), 0, st, a);
  else
    hipLaunchKernelGGL((gdn2_attn_dkv_kernel<IO, D, WK, WR, DKV_PLAIN>), dim3(blocks), dim3(64 * WK * WR), 0, st, a);
}
template <typename IO, int D>
hipError_t launch_attn_bwd_dkv(const attn_sizes &z, const attn_ptrs &p, void *ws, hipStream_t st) {
  bwd_args a;
  fill(a, z, p, ws, D, FAR_ROWS<IO, D>);
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
    launch_dkv<IO, D, WK, 2>(a, blocks * a.parts, st);
  } else {
    blocks = plan_tiles(z, 1, 32 * WKH, a.od);
    launch_dkv<IO, D, WKH, WRH>(a, blocks * a.parts, st);
  }
  if (a.parts > 1) {
    const size_t n = static_cast<size_t>(z.Ttot) * z.Hk * D / 2;  // threads
    hipLaunchKernelGGL((gdn2_attn_dkv_join_kernel<IO, D>), dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

#define GDN2_INST_ATTN_BWD(IO, D)                                                                         \
  template hipError_t launch_attn_bwd_dq<IO, D>(const attn_sizes &, const attn_ptrs &, void *, hipStream_t); \
  template hipError_t launch_attn_bwd_far<IO, D>(const attn_sizes &, const attn_ptrs &, void *, hipStream_t); \
  template hipError_t launch_attn_bwd_dkv<IO, D>(const attn_sizes &, const attn_ptrs &, void *, hipStream_t);
GDN2_INST_ATTN_BWD(float, 64)
GDN2_INST_ATTN_BWD(float, 128)
GDN2_INST_ATTN_BWD(bf16_t, 64)
GDN2_INST_ATTN_BWD(bf16_t, 128)

}  // namespace attn
}  // namespace gdn2
