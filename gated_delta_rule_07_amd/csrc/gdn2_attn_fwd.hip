// gdn2_attn_fwd.hip -- causal attention with grouped heads, for gfx950: over
// whole packed sequences, and over a paged cache.
//
//   s_ij = scale q_i . k_j for the visible keys j (j <= pos(i), and with a
//   window W, j > pos(i) - W);  o_i = sum_j softmax(s_i)_j v_j;
//   lse_i = ln sum_j exp(s_ij).  A row that sees no key gives o = 0, lse = -inf.
//
// One pass over the keys with the running maximum m and sum l of each row
// (kept in float32, in base 2: p = 2^(s c - m) with c = scale log2 e).
// Both products are formed transposed, S^T = K Q^T and O^T = V^T P^T, so that
// an accumulator's column is a query row: the row's statistics are a lane's
// own (plus one exchange between the wave's halves), rescaling O is a lane
// multiply, and P^T leaves the first product in the operand layout of the
// second.  V^T's fragments come from row-major tiles through the transposing
// LDS read.
//
// WM waves share key tiles of 32 KT keys along 32-row blocks; WN waves split
// the tile's keys (each keeps its own m, l, O, joined at the end).
//
// A wave's 32 x 64 tile at d = 128 is 32 matrix products (1024 cycles) beside
// about 240 vector operations, 32 of them exponentials.  So the operands are read
// a group of products ahead, the tiles come straight from memory into shared
// memory (no registers, no address arithmetic a chunk), and the reference of the
// exponents moves only where it has to.  The bounds left are the chip's power
// (the clock holds 2.05 GHz under it; the same call on zeros runs at 2.39 GHz in
// 3.75 ms) and the two waves a SIMD that registers allow (the products are busy
// 46 % of the cycles, 56 % with the softmax taken out, shared memory 23 %; a
// deeper read-ahead changes nothing).  Measured: one
// sequence of 32768 tokens, 16 heads on 4, d = 128, bfloat16: 4.3 to 4.5 ms,
// 975 to 1020 TFLOP/s (an 8192^3 product: 1212; without tiles straight from
// memory 4650 us, without read-ahead and with a rescale every tile 4880); 8 x
// 4096 tokens, window 2048: 480 to 500 us.  Paged, 1024 tokens at 12000 keys among
// 23 single tokens: 105 us with the join's 10 (341 MB: 73 us at a copy's rate).
#include "gdn2_attn_fwd.hpp"
#include <type_traits>

namespace gdn2 {
namespace attn {

template <typename IO, typename CT, int D, int WM, int WN, int KT, bool PAGED>
__global__ void __launch_bounds__(64 * WM * WN, (D * sizeof(IO) <= 256 ? 2 : 1))
    gdn2_attn_fwd_kernel(fwd_args a) {
  typedef tile<IO, D> TL;
  typedef typename std::conditional<sizeof(CT) == 1, tile8<IO, D>, TL>::type KV;  // a tile of the cache's own type
  // SHARED: the workgroup's waves share a tile, double-buffered, with one
  // barrier a tile.  Else every wave stages the keys it alone reads (single
  // buffer, no barrier: a wave's LDS accesses stay in order).
  constexpr bool SHARED = WN == 1;
  constexpr int NT = SHARED ? 64 * WM : 64, BM = 32 * WM, BN = 32 * KT * WN, SN = 32 * KT, NB = SHARED ? 2 : 1;
  constexpr int CPR = KV::CPR, CH = SN * CPR / NT;  // 16-byte chunks a thread stages of K (and of V)
  constexpr int TILEB = SN * KV::ROWB;
  constexpr bool F8 = sizeof(CT) == 1;
  // Whole sequences' tiles come straight from memory: position p of a tile is
  // chunk (p % CPR) ^ f of row p / CPR.
  constexpr bool DMA = SHARED && !PAGED;
  static_assert(SN * CPR % NT == 0 && NT % CPR == 0, "staging split");
  constexpr int ROWS_PER_I = NT / CPR;
  // K and V tiles; with split keys also the room in which the waves join
  // (a part of JC channels at a time)
  constexpr int JC = 64, JOIN = SHARED ? 0 : WN * 32 * ((JC + 4) * 4 + 8);
  constexpr int LDSB = 2 * NB * WN * TILEB > JOIN ? 2 * NB * WN * TILEB : JOIN;
  __shared__ __align__(16) char lds[LDSB];
  // waves of their own keep the queries, the same for all of them, here
  // rather than in 32 registers
  __shared__ __align__(16) char lq[SHARED ? 16 : 32 * TL::ROWB];
  __shared__ __align__(16) float scales[F8 ? 2 * NB * WN * SN : 1];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 31, h = lane >> 5;
  const int wm = WN == 1 ? wave : 0, wn = WN == 1 ? 0 : wave;

  // ---- which rows
  const int id = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  int unit, slot;
  if (!place(a.od, id, unit, slot))
    return;
  span sq;
  int hk, row0;
  if (a.cu) {
    hk = unit;
    const int n = find_seq(a.cu, a.N, a.G, BM, slot, lane);
    sq = packed_span(a.cu, n, a.T);
    row0 = static_cast<int>((slot - (static_cast<long>(a.cu[n]) * a.G / BM + n)) * BM);
  } else {
    sq.n = unit / a.Hk;
    hk = unit % a.Hk;
    sq.start = sq.n * a.T;
    sq.len = a.T;
    row0 = slot * BM;
  }
  const int rows = sq.len * a.G;
  if (row0 < 0 || row0 >= rows)
    return;
  int kv_len = sq.len;
  if constexpr (PAGED) {
    kv_len = a.seq_lens[sq.n];
    const int cap = a.max_pages << a.page_shift;
    kv_len = kv_len < 0 ? 0 : (kv_len > cap ? cap : kv_len);
  }
  const int shift = kv_len - sq.len;  // position of the sequence's first query

  // ---- visible keys of the workgroup, and this split's part
  const int t_lo = row0 / a.G;
  const int last_row = row0 + BM - 1 < rows - 1 ? row0 + BM - 1 : rows - 1;
  const int t_hi = last_row / a.G;
  int k_hi = shift + t_hi + 1;
  k_hi = k_hi < 0 ? 0 : k_hi;
  int k_lo = 0;
  if (a.window > 0) {
    k_lo = shift + t_lo - a.window + 1;
    k_lo = k_lo < 0 ? 0 : k_lo;
  }
  int k0 = k_lo, k1 = k_hi;
  if (a.splits > 1) {
    const int nt = k_hi > k_lo ? (k_hi - k_lo + BN - 1) / BN : 0;
    const int per = (nt + a.splits - 1) / a.splits;
    k0 = k_lo + split * per * BN;
    k1 = k0 + per * BN < k_hi ? k0 + per * BN : k_hi;
  }
  const int ntiles = k1 > k0 ? (k1 - k0 + BN - 1) / BN : 0;

  // ---- this lane's row
  const int my_row = row0 + 32 * wm + r;
  const bool row_ok = my_row < rows;
  const int cl_row = row_ok ? my_row : rows - 1;
  const int tok = cl_row / a.G, head = hk * a.G + cl_row % a.G;
  const int pos = shift + tok;
  const size_t qrow = static_cast<size_t>(sq.start + tok) * a.Hq + head;
  // positions of the wave's first and last row
  const int wr0 = row0 + 32 * wm < rows ? row0 + 32 * wm : rows - 1;
  const int wr1 = row0 + 32 * wm + 31 < rows ? row0 + 32 * wm + 31 : rows - 1;
  const int pos_lo = shift + wr0 / a.G, pos_hi = shift + wr1 / a.G;

  frag8<IO> q[SHARED ? D / 16 : 1];
  const IO *const qp = static_cast<const IO *>(a.q) + qrow * D;
  if constexpr (SHARED) {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      q[kk] = load8<IO>(qp + 16 * kk + 8 * h);
  } else {
    // every wave has the same rows: wave w brings every WN-th chunk pair
    for (int c = 2 * wn + h; c < TL::CPR; c += 2 * WN)
      *reinterpret_cast<u32x4 *>(lq + TL::at(r, c)) = *reinterpret_cast<const u32x4 *>(qp + c * TL::VPC);
    __syncthreads();
  }

  // ---- staging: thread's chunk c of rows sr0 + ROWS_PER_I i
  const int st = SHARED ? tid : lane;
  const int sc = st % CPR, sr0 = st / CPR + (SHARED ? 0 : SN * wn);
  const int wave_b = wn * 2 * TILEB;  // the wave's tiles
  const int row_b = KV::row_base(r, h) + wave_b, col_b = KV::col_base(lane) + wave_b;
  char *const kt = lds, *const vt = lds + TILEB;
  float *const kscale = scales + wn * 2 * SN, *const vscale = kscale + SN;
  const int wv = __builtin_amdgcn_readfirstlane(wave);
  u32x4 rk[DMA ? 1 : CH], rv[DMA ? 1 : CH];
  int ent[CH], bad = 0;
  uint8_t bk = 127, bv = 127;
  int ent_b = 0;
  const int32_t *table = PAGED ? a.table + static_cast<size_t>(sq.n) * a.max_pages : nullptr;
  const int pmask = (1 << a.page_shift) - 1;
  // Rows of the tile at key kb; one behind the last key stands for that key's
  // row (its score is masked).  Paged: the table's entries are fetched a tile
  // ahead of the rows they lead to.
  auto load_entries = [&](int kb) {
    if constexpr (PAGED) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int j = kb + sr0 + ROWS_PER_I * i;
        ent[i] = table[(j < k1 ? j : k1 - 1) >> a.page_shift];
      }
      if constexpr (F8) {
        const int j = kb + SN * wn + st % SN;
        ent_b = table[(j < k1 ? j : k1 - 1) >> a.page_shift];
      }
    }
  };
  const unsigned kstep = static_cast<unsigned>(a.Hk) * D;  // values of a token
  auto load_tile = [&](int kb, int buf) {
    const size_t base = PAGED ? 0 : (static_cast<size_t>(sq.start + kb) * a.Hk + hk) * D;
    const CT *const kp = static_cast<const CT *>(a.k) + base, *const vp = static_cast<const CT *>(a.v) + base;
    if constexpr (PAGED)
      bad = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      int j = kb + sr0 + ROWS_PER_I * i;
      j = j < k1 ? j : k1 - 1;
      if constexpr (PAGED) {
        // (an entry outside the cache stands for zeros, see store_tile)
        const bool ok = static_cast<unsigned>(ent[i]) < static_cast<unsigned>(a.num_pages);
        bad |= ok ? 0 : 1 << i;
        const size_t off = (((static_cast<size_t>(ok ? ent[i] : 0) * a.Hk + hk) << a.page_shift) + (j & pmask)) * D +
                           sc * KV::VPC;
        rk[i] = *reinterpret_cast<const u32x4 *>(kp + off);
        rv[i] = *reinterpret_cast<const u32x4 *>(vp + off);
      } else {
        if constexpr (DMA) {
          const unsigned off = static_cast<unsigned>(j - kb) * kstep + (sc ^ KV::f(sr0 + ROWS_PER_I * i)) * KV::VPC;
          char *const to = lds + (buf * 2 * TILEB + 1024 * wv + 16 * NT * i);
          dma16(kp + off, to);
          dma16(vp + off, to + TILEB);
        } else {
          const unsigned off = static_cast<unsigned>(j - kb) * kstep + sc * KV::VPC;
          rk[i] = *reinterpret_cast<const u32x4 *>(kp + off);
          rv[i] = *reinterpret_cast<const u32x4 *>(vp + off);
        }
      }
    }
    if constexpr (F8) {
      int j = kb + SN * wn + st % SN;
      j = j < k1 ? j : k1 - 1;
      const bool ok = static_cast<unsigned>(ent_b) < static_cast<unsigned>(a.num_pages);
      bad |= ok ? 0 : 1 << CH;
      const size_t off = ((static_cast<size_t>(ok ? ent_b : 0) * a.Hk + hk) << a.page_shift) + (j & pmask);
      bk = a.ks[off];
      bv = a.vs[off];
    }
  };
  auto store_tile = [&](int buf) {
    if constexpr (DMA)
      return;
    if constexpr (PAGED) {
      if (__any(bad)) {
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (bad >> i & 1)
            rk[i] = rv[i] = u32x4{0u, 0u, 0u, 0u};
        // (0 times the scale of whatever row was read instead need not be 0)
        if (F8 && (bad >> CH & 1))
          bk = bv = 127;
      }
    }
#pragma unroll
    for (int i = 0; i < (DMA ? 1 : CH); ++i) {
      const int at = wave_b + buf * 2 * TILEB + KV::at(st / CPR + ROWS_PER_I * i, sc);
      *reinterpret_cast<u32x4 *>(kt + at) = rk[i];
      *reinterpret_cast<u32x4 *>(vt + at) = rv[i];
    }
    if constexpr (F8) {
      if (st < SN) {
        kscale[buf * 2 * SN + st] = scale_of(bk);
        vscale[buf * 2 * SN + st] = scale_of(bv);
      }
    }
  };

  f32x16 o[D / 32];
#pragma unroll
  for (int n = 0; n < D / 32; ++n)
    o[n] = zero16();
  float m = neg_inf(), l = 0.f;  // l: this half's part of the sum

  if (ntiles > 0) {
    load_entries(k0);
    load_tile(k0, 0);
    load_entries(k0 + BN);
  }
  for (int it = 0; it < ntiles; ++it) {
    const int kb = k0 + it * BN, buf = SHARED ? it & 1 : 0;
    if constexpr (DMA) {
      dma_wait();
      __syncthreads();
    } else if constexpr (SHARED) {
      store_tile(buf);
      __syncthreads();
    } else {
      // the lanes' reads of the tile before come first, their writes before
      // the reads below
      wave_order();
      store_tile(buf);
      wave_order();
    }
    if (it + 1 < ntiles) {
      load_tile(kb + BN, buf ^ 1);
      load_entries(kb + 2 * BN);
    }
    const int rb = row_b + buf * 2 * TILEB, cb = col_b + buf * 2 * TILEB;
    const float *const ksc = kscale + buf * 2 * SN, *const vsc = vscale + buf * 2 * SN;
    const int wk = kb + SN * wn;  // the wave's first key
    // no rows, or nothing of the tile is visible to the wave
    if (row0 + 32 * wm >= rows || wk > pos_hi || wk >= k1 || (a.window > 0 && wk + 32 * KT - 1 <= pos_lo - a.window))
      continue;
    const bool masked = wk + 32 * KT - 1 > pos_lo || wk + 32 * KT > k1 ||
                        (a.window > 0 && wk <= pos_hi - a.window);

    // S^T, and further down O^T, in groups of GR products whose operands are
    // read a group ahead
    constexpr int GR = sizeof(IO) == 2 && !PAGED ? 4 : 2, NS = KT * (D / 16);
    const int qb = fresh(TL::row_base(r, h));
    f32x16 s[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t)
      s[t] = zero16();
    {
      frag8<IO> kf[2][GR], qf[2][SHARED ? 1 : GR];
      auto fetch = [&](int g) {
#pragma unroll
        for (int x = 0; x < GR; ++x) {
          const int y = g * GR + x;
          if constexpr (!SHARED)
            qf[g & 1][x] = TL::row(lq, qb, y % (D / 16));
          kf[g & 1][x] = KV::row(kt + 32 * (y / (D / 16)) * KV::ROWB, rb, y % (D / 16));
        }
      };
      fetch(0);
#pragma unroll
      for (int g = 0; g < NS / GR; ++g) {
        if (g + 1 < NS / GR)
          fetch(g + 1);
        group_fence();
#pragma unroll
        for (int x = 0; x < GR; ++x) {
          const int y = g * GR + x;
          mma(s[y / (D / 16)], kf[g & 1][x], SHARED ? q[SHARED ? y % (D / 16) : 0] : qf[g & 1][SHARED ? 0 : x]);
        }
        group_fence();
      }
    }
    if constexpr (F8) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 sc4 = *reinterpret_cast<const f32x4 *>(&ksc[32 * t + 8 * g + 4 * h]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s[t][4 * g + i] *= sc4[i];
        }
    }
    // key of register i: wk + 32 t + 8 (i / 4) + 4 h + i % 4; visible when
    // j <= pos, j > pos - W and j < k1
    const int hi_rel = (pos < k1 - 1 ? pos : k1 - 1) - wk - 4 * h;
    const int lo_rel = (a.window > 0 ? pos - a.window : -0x40000000) - wk - 4 * h;
    if (masked) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = 32 * t + 8 * (i >> 2) + (i & 3);
          s[t][i] = (j <= hi_rel && j > lo_rel) ? s[t][i] : neg_inf();
        }
    }
    float mx = s[0][0];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        mx = fmaxf(mx, s[t][i]);
    mx = half_max(mx) * a.c;
    // The reference of a row's exponents stays while its maximum is not more
    // than 8 above it (weights up to 2^8: no loss, they are floating point),
    // so that most tiles rescale nothing.  (A published refinement of the running
    // maximum: the rescale is conditional on how far it rose.)
    const bool up = mx > m + 8.f;
    if (__any(up)) {
      const float m_new = up ? mx : m;
      const float alpha = fast_exp2(m - (m_new == neg_inf() ? 0.f : m_new));
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int n = 0; n < D / 32; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          o[n][i] *= alpha;
    }
    const float base = m == neg_inf() ? 0.f : m;  // a row without keys yet
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float p = fast_exp2(s[t][i] * a.c - base);
        s[t][i] = p;
        sum[i & 3] += p;
      }
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
    if constexpr (F8) {
      // the values' scales go to the weights (a masked weight stays 0
      // whatever its row's scale holds)
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4 sc4 = *reinterpret_cast<const f32x4 *>(&vsc[32 * t + 8 * g + 4 * h]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = 32 * t + 8 * g + i;
            s[t][4 * g + i] = (!masked || (j <= hi_rel && j > lo_rel)) ? s[t][4 * g + i] * sc4[i] : 0.f;
          }
        }
    }
    bool odd = false;  // infinities or NaN among the values of a masked tile
    {
      constexpr int NN = D / 32, GV = NN < GR ? NN : GR, PER = NN / GV;
      frag8<IO> vf[2][GV];
      auto fetch = [&](int g) {
#pragma unroll
        for (int x = 0; x < GV; ++x)
          vf[g & 1][x] = KV::col(vt, cb, 16 * (g / PER), g % PER * GV + x);
      };
      fetch(0);
#pragma unroll
      for (int g = 0; g < 2 * KT * PER; ++g) {
        if (g + 1 < 2 * KT * PER)
          fetch(g + 1);
        group_fence();
        const frag8<IO> p = pack8<IO>(s[g / PER / 2], g / PER & 1);
#pragma unroll
        for (int x = 0; x < GV; ++x) {
          if (masked)
            odd |= drop_nonfinite(vf[g & 1][x]);
          mma(o[g % PER * GV + x], vf[g & 1][x], p);
        }
        group_fence();
      }
    }
    // 0 times an infinity would reach rows that do not see its key: in a
    // masked tile such values are left out of the product above and added
    // here for the rows that do see them.
    if (masked && __any(odd)) {
      for (int j = 0; j < 32 * KT; ++j) {
        float p = 0.f;  // weight of key j, kept by half (j / 4) % 2
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            p = (32 * t + 8 * (i >> 2) + (i & 3)) == j - 4 * ((j >> 2) & 1) ? s[t][i] : p;
        p = __shfl(p, r + 32 * ((j >> 2) & 1), 64);
        const int jr = j - 4 * h;
        const bool vis = jr <= hi_rel && jr > lo_rel;
#pragma unroll
        for (int n = 0; n < D / 32; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = KV::one(vt + wave_b + buf * 2 * TILEB, j, 32 * n + 8 * (i >> 2) + 4 * h + (i & 3));
            if (vis && !(fabsf(x) <= 3.4028234663852886e38f))
              o[n][i] += p * x;
          }
      }
    }
  }

  l += __shfl_xor(l, 32, 64);

  if constexpr (WN > 1) {
    // join the waves' parts: weights 2^(m_w - M)
    static_assert(WM == 1, "one row block");
    constexpr int OLD = JC + 4;
    float *jo = reinterpret_cast<float *>(lds);  // [WN][32][OLD]
    float *jm = jo + WN * 32 * OLD, *jl = jm + WN * 32;
    __syncthreads();
    if (h == 0) {
      jm[wn * 32 + r] = m;
      jl[wn * 32 + r] = l;
    }
    __syncthreads();
    float M = neg_inf();
#pragma unroll
    for (int w = 0; w < WN; ++w)
      M = fmaxf(M, jm[w * 32 + r]);
    const float base = M == neg_inf() ? 0.f : M;
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < WN; ++w)
      L += jl[w * 32 + r] * fast_exp2(jm[w * 32 + r] - base);
    const float f = fast_exp2(m - base);
#pragma unroll
    for (int n0 = 0; n0 < D / 32; n0 += JC / 32) {
      if (n0 > 0)
        __syncthreads();
#pragma unroll
      for (int n = 0; n < JC / 32; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          f32x4 x;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = o[n0 + n][4 * g + i] * f;
          *reinterpret_cast<f32x4 *>(&jo[(wn * 32 + r) * OLD + 32 * n + 8 * g + 4 * h]) = x;
        }
      __syncthreads();
      // the waves take the part's groups of 8 channels of every row in turn
      for (int y = wn; y < JC / 8; y += WN) {
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < WN; ++w)
          x += *reinterpret_cast<const f32x4 *>(&jo[(w * 32 + r) * OLD + 8 * y + 4 * h]);
        store_row<IO, D>(a, x, L, qrow, split, row_ok, 32 * n0 + 8 * y + 4 * h);
      }
    }
    if (wn == 0 && h == 0 && row_ok)
      store_lse(a, M, L, qrow, split);
  } else {
#pragma unroll
    for (int n = 0; n < D / 32; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        f32x4 x;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = o[n][4 * g + i];
        store_row<IO, D>(a, x, l, qrow, split, row_ok, 32 * n + 8 * g + 4 * h);
      }
    if (h == 0 && row_ok)
      store_lse(a, m, l, qrow, split);
  }
}

// Joins the parts of split keys: W waves per (token, query head), wave w of a
// row takes the parts w, w + W, ..; weights 2^(lse_s - max lse); the order of
// the sums is fixed.
template <typename IO, int D, int W> __global__ void __launch_bounds__(256) gdn2_attn_join_kernel(fwd_args a) {
  __shared__ float red[W][D + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w0 = W == 1 ? 0 : wave;
  const size_t rows = static_cast<size_t>(a.Ttot) * a.Hq;
  const size_t row = W == 1 ? static_cast<size_t>(blockIdx.x) * 4 + wave : blockIdx.x;
  if (row >= rows)
    return;
  if (a.cu && row >= static_cast<size_t>(a.cu[a.N] < 0 ? 0 : a.cu[a.N]) * a.Hq)
    return;  // behind the last sequence
  float M = neg_inf();
  for (int s = lane; s < a.splits; s += 64)
    M = fmaxf(M, a.part_lse[s * rows + row]);
#pragma unroll
  for (int x = 1; x < 64; x <<= 1)
    M = fmaxf(M, __shfl_xor(M, x, 64));
  const float base = M == neg_inf() ? 0.f : M;
  constexpr int V = D / 64;
  float acc[V], L = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
    acc[i] = 0.f;
#pragma unroll 4
  for (int s = w0; s < a.splits; s += W) {
    // (a part without keys: weight 0 and zeros; NaN stays NaN)
    const float w = fast_exp2(a.part_lse[s * rows + row] - base);
    const float *p = a.part_o + (s * rows + row) * D + V * lane;
    L += w;
#pragma unroll
    for (int i = 0; i < V; ++i)
      acc[i] += w * p[i];
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      red[wave][V * lane + i] = acc[i];
    if (lane == 0)
      red[wave][D] = L;
    __syncthreads();
    if (wave > 0)
      return;
    L = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w)
      L += red[w][D];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      acc[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w)
        acc[i] += red[w][V * lane + i];
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  IO *o = static_cast<IO *>(a.o) + row * D + V * lane;
#pragma unroll
  for (int i = 0; i < V; ++i)
    o[i] = io<IO>::from_f(acc[i] * inv);
  if (a.lse && lane == 0)
    a.lse[row] = (base + log2f(L)) * LN2;
}

// ------------------------------------------------------------- launchers --
// The kernel's shape for a call: 32-row blocks with the keys split over 4
// waves where a sequence brings few rows (decode), else 128 rows and shared
// key tiles.
static bool few_rows(const attn_sizes &z) {
  return static_cast<long long>(z.Ttot) * (z.Hq / z.Hk) <= 32LL * z.N;
}
// At most 16 rows for every sequence and kv head: the decode kernel
// (bfloat16), with 16-row products.  Packed calls have their sequences' lengths on
// the device only and take the 32-row kernel even if all are single tokens (64
// sequences of 4K to 16K keys, e4m3: 133 us with T = 1, 150 packed).
static bool decode_rows(const attn_sizes &z) {
  return !z.packed && static_cast<long long>(z.T) * (z.Hq / z.Hk) <= 16;
}

// Parts along the keys of a paged call: enough workgroups that sequences of
// different lengths even out over the CUs, no part of the longest possible
// sequence under 128 keys, at most 128 parts.  (Decode of 64 sequences x 4 kv
// heads: 136 us at 2048 workgroups, 151 at 1024 and 512; one 1024-token chunk
// among 23 tokens: 113 us at 768, 125 at 1024, 137 at 2048, where its parts'
// outputs weigh more.)
int attn_paged_splits(const attn_sizes &z) {
  order od;
  const bool few = few_rows(z);
  plan_tiles(z, z.Hq / z.Hk, few ? 32 : 128, od);
  const long long blocks = static_cast<long long>(od.units) * od.tiles;
  long long keys = z.max_keys;
  if (z.window > 0 && keys > z.window + 128LL)
    keys = z.window + 128LL;
  long long s = ((few ? 2048 : 768) + blocks - 1) / blocks;
  if (s > keys / 128)
    s = keys / 128;
  return s < 1 ? 1 : (s > 128 ? 128 : static_cast<int>(s));
}

template <typename IO, typename CT, int D, int WM, int WN, int KT, bool PAGED>
static hipError_t go(fwd_args &a, const attn_sizes &z, hipStream_t st) {
  const unsigned blocks = plan_tiles(z, a.G, 32 * WM, a.od) * a.splits;
  hipLaunchKernelGGL((gdn2_attn_fwd_kernel<IO, CT, D, WM, WN, KT, PAGED>), dim3(blocks), dim3(64 * WM * WN), 0, st, a);
  return hipGetLastError();
}

static void fill(fwd_args &a, const attn_sizes &z, const attn_ptrs &p) {
  a.q = p.q;
  a.k = p.k;
  a.v = p.v;
  a.o = p.o;
  a.lse = p.lse;
  a.cu = p.cu;
  a.table = p.table;
  a.seq_lens = p.seq_lens;
  a.ks = p.ks;
  a.vs = p.vs;
  a.part_o = a.part_lse = nullptr;
  a.N = z.N;
  a.T = z.T;
  a.Ttot = z.Ttot;
  a.Hq = z.Hq;
  a.Hk = z.Hk;
  a.G = z.Hq / z.Hk;
  a.max_pages = z.max_pages;
  a.num_pages = z.num_pages;
  a.page_shift = z.page_shift;
  a.window = z.window;
  a.splits = 1;
  a.c = z.scale * LOG2E;
}

template <typename IO, int D> hipError_t launch_attn_fwd(const attn_sizes &z, const attn_ptrs &p, hipStream_t st) {
  fwd_args a;
  fill(a, z, p);
  // (few tiles, float32: 4 waves 14 and 25 us, 2 waves 22 and 38, d = 64 and
  // 128, 1543 tokens, 4 heads, window 300)
  constexpr int KT = sizeof(IO) == 2 ? 2 : 1;
  plan_tiles(z, a.G, 128, a.od);
  return few_tiles(a.od) ? go<IO, IO, D, 1, 4, 1, false>(a, z, st) : go<IO, IO, D, 4, 1, KT, false>(a, z, st);
}

template <typename IO, typename CT, int D>
hipError_t launch_attn_paged(const attn_sizes &z, const attn_ptrs &p, int splits, void *ws, hipStream_t st) {
  fwd_args a;
  fill(a, z, p);
  a.splits = splits;
  constexpr int KT = sizeof(CT) <= 2 ? 2 : 1;
  if (splits > 1) {
    const size_t rows = static_cast<size_t>(z.Ttot) * z.Hq;
    a.part_o = static_cast<float *>(ws);
    a.part_lse = a.part_o + rows * D * splits;
  }
  if constexpr (sizeof(IO) == 2) {
    if (decode_rows(z)) {
      plan_tiles(z, a.G, 16, a.od);
      return launch_attn_decode<CT, D>(a, st);
    }
  }
  // (float32, d = 128: 4 waves' tiles leave one workgroup a CU; 8 sequences of
  // 2000 keys, 4 heads on 4: 36 us against 31 with 2 waves; d = 64 17 against 21)
  constexpr int WN = D * sizeof(IO) <= 256 ? 4 : 2;
  return few_rows(z) ? go<IO, CT, D, 1, WN, 1, true>(a, z, st) : go<IO, CT, D, 4, 1, KT, true>(a, z, st);
}

template <typename IO, int D>
hipError_t launch_attn_join(const attn_sizes &z, const attn_ptrs &p, int splits, void *ws, hipStream_t st) {
  fwd_args a;
  fill(a, z, p);
  a.splits = splits;
  const size_t rows = static_cast<size_t>(z.Ttot) * z.Hq;
  a.part_o = static_cast<float *>(ws);
  a.part_lse = a.part_o + rows * D * splits;
  // one wave a row where there are rows enough, or few parts
  if (rows >= 8192 || splits <= 4)
    hipLaunchKernelGGL((gdn2_attn_join_kernel<IO, D, 1>), dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((gdn2_attn_join_kernel<IO, D, 4>), dim3(static_cast<unsigned>(rows)), dim3(256), 0, st, a);
  return hipGetLastError();
}

#define GDN2_INST_ATTN(IO, D)                                                                              \
  template hipError_t launch_attn_fwd<IO, D>(const attn_sizes &, const attn_ptrs &, hipStream_t);          \
  template hipError_t launch_attn_paged<IO, IO, D>(const attn_sizes &, const attn_ptrs &, int, void *,     \
                                                   hipStream_t);                                           \
  template hipError_t launch_attn_paged<IO, f8_t, D>(const attn_sizes &, const attn_ptrs &, int, void *,   \
                                                     hipStream_t);                                         \
  template hipError_t launch_attn_join<IO, D>(const attn_sizes &, const attn_ptrs &, int, void *, hipStream_t);
GDN2_INST_ATTN(float, 64)
GDN2_INST_ATTN(float, 128)
GDN2_INST_ATTN(bf16_t, 64)
GDN2_INST_ATTN(bf16_t, 128)

}  // namespace attn
}  // namespace gdn2
