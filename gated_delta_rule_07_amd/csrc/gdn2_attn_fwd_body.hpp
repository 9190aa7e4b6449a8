// gdn2_attn_fwd_body.hpp -- one workgroup of the forward attention: over whole
// sequences, over a paged cache, and over prefixes that sequences share.  (The
// mathematics and what bounds it: gdn2_attn_fwd.hip.)
#pragma once

#include <type_traits>

#include "gdn2_attn_fwd.hpp"

namespace gdn2 {
namespace attn {

// FWD_SINK: the first `sinks` keys of the sequence stay visible behind the window.
// The workgroup numbers the keys it visits without the gap between the two:
// the sinks, then the keys from its first row's window on, so that few sinks
// cost no tile of their own; positions are numbered with them.
//
// FWD_PREFIX: the rows are a group's, all of whose sequences share the keys of one
// table; every row sees every key.
enum fwd_mode { FWD_PLAIN, FWD_SINK, FWD_PREFIX };
template <typename IO, typename CT, int D, int WM, int WN, int KT, bool PAGED, fwd_mode MODE> struct fwd_body {
  static constexpr bool SINK = MODE == FWD_SINK, PREFIX = MODE == FWD_PREFIX;
  typedef tile<IO, D> TL;
  // SHARED: the workgroup's waves share a tile, double-buffered, with one
  // barrier a tile.  Else every wave stages the keys it alone reads (single
  // buffer, no barrier: a wave's LDS accesses stay in order).
  static constexpr bool SHARED = WN == 1, F8 = sizeof(CT) == 1;
  // A prefix's e4m3 codes, which several waves read, become bfloat16 on the way
  // to shared memory, scaled: a power of two changes no bit of a value but those
  // below 2^-126 (which float32 scores would keep), and costs nothing there.
  // Elsewhere the codes are operands and the scales (SCALED) go to the scores
  // and weights.
  static constexpr bool WIDEN = F8 && SHARED && PREFIX && sizeof(IO) == 2, SCALED = F8 && !WIDEN;
  typedef typename std::conditional<F8 && !WIDEN, tile8<IO, D>, TL>::type KV;  // a tile in shared memory
  static constexpr int NT = SHARED ? 64 * WM : 64, BM = 32 * WM, BN = 32 * KT * WN, SN = 32 * KT, NB = SHARED ? 2 : 1;
  // 16-byte chunks of a row in memory, the values of one, and how many a thread
  // stages of K (and of V)
  static constexpr int CPR = D * static_cast<int>(sizeof(CT)) / 16, VPC = 16 / static_cast<int>(sizeof(CT));
  static constexpr int CH = SN * CPR / NT, TILEB = SN * KV::ROWB;
  // Tiles whose values pass unchanged come straight from memory where the
  // waves share them (not through a cache's pages for single tokens' or a
  // chunk's own keys, where that measured slower): position p of a tile is
  // chunk (p % CPR) ^ f of row p / CPR.
  static constexpr bool DMA = SHARED && !F8 && (!PAGED || PREFIX);
  static_assert(SN * CPR % NT == 0 && NT % CPR == 0, "staging split");
  static constexpr int ROWS_PER_I = NT / CPR;
  // K and V tiles; with split keys also the room in which the waves join
  // (a part of JC channels at a time)
  static constexpr int JC = 64, JOIN = SHARED ? 0 : WN * 32 * ((JC + 4) * 4 + 8);
  static constexpr int LDSB = 2 * NB * WN * TILEB > JOIN ? 2 * NB * WN * TILEB : JOIN;
  // waves of their own keep the queries, the same for all of them, behind that
  // rather than in 32 registers; then the scales
  static constexpr int LQB = SHARED ? 0 : 32 * TL::ROWB, SCALESB = SCALED ? 2 * NB * WN * SN * 4 : 0;
  static constexpr int THREADS = 64 * WM * WN, BYTES = LDSB + LQB + SCALESB;

  // One workgroup's part of a call; lds: BYTES of its shared memory.
  static __device__ __forceinline__ void run(const fwd_args &a, int block, char *const lds) {
    char *const lq = lds + LDSB;
    float *const scales = reinterpret_cast<float *>(lds + LDSB + LQB);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int r = lane & 31, h = lane >> 5;
    const int wm = WN == 1 ? wave : 0, wn = WN == 1 ? 0 : wave;

    // ---- which rows
    const int id = block / a.splits, split = block % a.splits;
    int unit, slot;
    if (!place(a.od, id, unit, slot))
      return;
    span sq;
    int hk, row0;
    if constexpr (PREFIX) {
      hk = unit;
      auto first = [&](int i) { return group_start(a, i); };
      const int n = find_seq_by(first, a.N, a.G, BM, slot, lane);
      sq = clamped_span(n, first(n), first(n + 1), a.T);
      row0 = static_cast<int>((slot - (static_cast<long>(first(n)) * a.G / BM + n)) * BM);
    } else if (a.cu) {
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
    int k_hi = PREFIX ? kv_len : shift + t_hi + 1;
    k_hi = k_hi < 0 ? 0 : k_hi;
    int k_lo = 0;
    if (a.window > 0) {
      k_lo = shift + t_lo - a.window + 1;
      k_lo = k_lo < 0 ? 0 : k_lo;
    }
    // keys behind the sinks are numbered `gap` less than they are
    int gap = 0;
    if constexpr (SINK) {
      gap = k_lo > a.sinks ? k_lo - a.sinks : 0;
      k_lo = 0;
      k_hi -= gap;
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
    const int pos = PREFIX ? kv_len - 1 : shift - gap + tok;
    const size_t qrow = static_cast<size_t>(sq.start + tok) * a.Hq + head;
    // positions of the wave's first and last row
    const int wr0 = row0 + 32 * wm < rows ? row0 + 32 * wm : rows - 1;
    const int wr1 = row0 + 32 * wm + 31 < rows ? row0 + 32 * wm + 31 : rows - 1;
    const int pos_lo = PREFIX ? pos : shift - gap + wr0 / a.G, pos_hi = PREFIX ? pos : shift - gap + wr1 / a.G;

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
    uint8_t bk = 127, bv = 127, wk8[WIDEN ? CH : 1], wv8[WIDEN ? CH : 1];
    int ent_b = 0;
    const int32_t *table = PAGED ? a.table + static_cast<size_t>(sq.n) * a.max_pages : nullptr;
    const int pmask = (1 << a.page_shift) - 1;
    auto key_of = [&](int j) { return SINK && j >= a.sinks ? j + gap : j; };  // of a numbered key
    // Rows of the tile at key kb; one behind the last key stands for that key's
    // row (its score is masked).  Paged: the table's entries are fetched a tile
    // ahead of the rows they lead to.
    auto load_entries = [&](int kb) {
      if constexpr (PAGED) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int j = kb + sr0 + ROWS_PER_I * i;
          ent[i] = table[key_of(j < k1 ? j : k1 - 1) >> a.page_shift];
        }
        if constexpr (SCALED) {
          const int j = kb + SN * wn + st % SN;
          ent_b = table[key_of(j < k1 ? j : k1 - 1) >> a.page_shift];
        }
      }
    };
    const unsigned kstep = static_cast<unsigned>(a.Hk) * D;  // values of a token
    auto load_tile = [&](int kb, int buf) {
      // (a tile with sinks takes its keys one by one, from the sequence's first)
      const bool mixed = SINK && kb < a.sinks;
      const size_t base = PAGED ? 0 : (static_cast<size_t>(sq.start + (mixed ? 0 : kb + gap)) * a.Hk + hk) * D;
      const CT *const kp = static_cast<const CT *>(a.k) + base, *const vp = static_cast<const CT *>(a.v) + base;
      if constexpr (PAGED)
        bad = 0;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        int j = kb + sr0 + ROWS_PER_I * i;
        const bool in = j < k1;
        j = in ? j : k1 - 1;
        if constexpr (PAGED) {
          j = key_of(j);
          // (an entry outside the cache stands for zeros, see store_tile; so do a
          // prefix's rows behind the last key, whose weights are 0 for every row)
          const bool ok = static_cast<unsigned>(ent[i]) < static_cast<unsigned>(a.num_pages);
          bad |= ok && (in || !PREFIX) ? 0 : 1 << i;
          const size_t off = (((static_cast<size_t>(ok ? ent[i] : 0) * a.Hk + hk) << a.page_shift) + (j & pmask)) * D +
                             sc * VPC;
          if constexpr (DMA) {
            const int x = ((sc ^ KV::f(sr0 + ROWS_PER_I * i)) - sc) * VPC;
            char *const to = lds + (buf * 2 * TILEB + 1024 * wv + 16 * NT * i);
            dma16(kp + off + x, to);
            dma16(vp + off + x, to + TILEB);
          } else {
            rk[i] = *reinterpret_cast<const u32x4 *>(kp + off);
            rv[i] = *reinterpret_cast<const u32x4 *>(vp + off);
          }
          if constexpr (WIDEN) {
            wk8[i] = a.ks[off / D];
            wv8[i] = a.vs[off / D];
          }
        } else {
          auto bring = [&](auto off) {
            if constexpr (DMA) {
              off += (sc ^ KV::f(sr0 + ROWS_PER_I * i)) * VPC;
              char *const to = lds + (buf * 2 * TILEB + 1024 * wv + 16 * NT * i);
              dma16(kp + off, to);
              dma16(vp + off, to + TILEB);
            } else {
              off += sc * VPC;
              rk[i] = *reinterpret_cast<const u32x4 *>(kp + off);
              rv[i] = *reinterpret_cast<const u32x4 *>(vp + off);
            }
          };
          if (mixed)
            bring(static_cast<size_t>(key_of(j)) * kstep);
          else
            bring(static_cast<unsigned>(j - kb) * kstep);
        }
      }
      if constexpr (SCALED) {
        int j = kb + SN * wn + st % SN;
        j = key_of(j < k1 ? j : k1 - 1);
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
          if (SCALED && (bad >> CH & 1))
            bk = bv = 127;
        }
      }
#pragma unroll
      for (int i = 0; i < (DMA ? 1 : CH); ++i) {
        const int row = st / CPR + ROWS_PER_I * i, to = wave_b + buf * 2 * TILEB;
        if constexpr (WIDEN) {
          // (the byte 255 stands for NaN; zeros stay zeros under any scale)
          constexpr unsigned NAN8 = 0x7f7f7f7fu;
          const bool zero = PAGED && (bad >> i & 1);
          const bool nk = wk8[i] == 255 && !zero, nv = wv8[i] == 255 && !zero;
          const float ks = scale_of(wk8[i] == 255 ? 127 : wk8[i]), vs = scale_of(wv8[i] == 255 ? 127 : wv8[i]);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int at = to + KV::at(row, 2 * sc + y);
            const u32x2 k = nk ? u32x2{NAN8, NAN8} : u32x2{rk[i][2 * y], rk[i][2 * y + 1]};
            const u32x2 v = nv ? u32x2{NAN8, NAN8} : u32x2{rv[i][2 * y], rv[i][2 * y + 1]};
            *reinterpret_cast<bf16x8 *>(kt + at) = widen8_by(k, ks).v;
            *reinterpret_cast<bf16x8 *>(vt + at) = widen8_by(v, vs).v;
          }
        } else {
          const int at = to + KV::at(row, sc);
          *reinterpret_cast<u32x4 *>(kt + at) = rk[i];
          *reinterpret_cast<u32x4 *>(vt + at) = rv[i];
        }
      }
      if constexpr (SCALED) {
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
        if constexpr (PAGED) {
          // (an entry outside the cache stands for zeros)
          if (__any(bad)) {
#pragma unroll
            for (int i = 0; i < CH; ++i)
              if (bad >> i & 1) {
                char *const to = lds + (buf * 2 * TILEB + 16 * tid + 16 * NT * i);
                *reinterpret_cast<u32x4 *>(to) = u32x4{0u, 0u, 0u, 0u};
                *reinterpret_cast<u32x4 *>(to + TILEB) = u32x4{0u, 0u, 0u, 0u};
              }
          }
        }
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
      if (row0 + 32 * wm >= rows || wk > pos_hi || wk >= k1 ||
          (a.window > 0 && wk + 32 * KT - 1 <= pos_lo - a.window && !(SINK && wk < a.sinks)))
        continue;
      const bool masked = wk + 32 * KT - 1 > pos_lo || wk + 32 * KT > k1 ||
                          (a.window > 0 && wk <= pos_hi - a.window);

      // S^T, and further down O^T, in groups of GR products whose operands are
      // read a group ahead
      constexpr int GR = sizeof(IO) == 2 && (!PAGED || DMA) ? 4 : 2, NS = KT * (D / 16);
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
      if constexpr (SCALED) {
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
      // j <= pos, j > pos - W (or a sink) and j < k1
      const int hi_rel = (pos < k1 - 1 ? pos : k1 - 1) - wk - 4 * h;
      const int lo_rel = (a.window > 0 ? pos - a.window : -0x40000000) - wk - 4 * h;
      const int sink_rel = SINK ? a.sinks - wk - 4 * h : 0;
      auto visible = [&](int j) { return j <= hi_rel && (j > lo_rel || (SINK && j < sink_rel)); };
      if (masked) {
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = 32 * t + 8 * (i >> 2) + (i & 3);
            s[t][i] = visible(j) ? s[t][i] : neg_inf();
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
      if constexpr (SCALED) {
        // the values' scales go to the weights (a masked weight stays 0
        // whatever its row's scale holds)
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x4 sc4 = *reinterpret_cast<const f32x4 *>(&vsc[32 * t + 8 * g + 4 * h]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              s[t][4 * g + i] *= sc4[i];
          }
        if (masked) {
#pragma unroll
          for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              s[t][i] = visible(32 * t + 8 * (i >> 2) + (i & 3)) ? s[t][i] : 0.f;
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
            if (!PREFIX && masked)
              odd |= drop_nonfinite(vf[g & 1][x]);
            mma(o[g % PER * GV + x], vf[g & 1][x], p);
          }
          group_fence();
        }
      }
      // 0 times an infinity would reach rows that do not see its key: in a
      // masked tile such values are left out of the product above and added
      // here for the rows that do see them.  (A prefix's keys are seen by all rows.)
      if (!PREFIX && masked && __any(odd)) {
        for (int j = 0; j < 32 * KT; ++j) {
          float p = 0.f;  // weight of key j, kept by half (j / 4) % 2
#pragma unroll
          for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              p = (32 * t + 8 * (i >> 2) + (i & 3)) == j - 4 * ((j >> 2) & 1) ? s[t][i] : p;
          p = __shfl(p, r + 32 * ((j >> 2) & 1), 64);
          const int jr = j - 4 * h;
          const bool vis = visible(jr);
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
        store_lse(a, M, L, qrow, split, pos);
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
        store_lse(a, m, l, qrow, split, pos);
    }
  }
};

}  // namespace attn
}  // namespace gdn2
