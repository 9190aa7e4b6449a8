// gdn2_attn_api.cpp -- the C ABI of the attention operators (include/gdn2.h,
// "Attention layers of a hybrid stack"): argument checks, kernel selection
// and launches on the caller's stream.  No memory is allocated and the stream
// is never synchronised.
#include "../../include/gdn2.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "gdn2_attn_kernels.hpp"
#include "gdn2_host.hpp"

using namespace gdn2::host;
using gdn2::attn::attn_ptrs;
using gdn2::attn::attn_sizes;
using gdn2::attn::cache_call;
using gdn2::attn::prefix_call;
using gdn2::attn::rope_call;

namespace {

constexpr long long MAX_ROWS = (1LL << 26) - 1;   // query rows (token, head): a wave each, work-items in 32 bits
constexpr long long MAX_UNITS = (1LL << 20) - 1;  // sequence x kv head
constexpr int MAX_SINKS = 1024;

bool attn_dim(int d) { return d == 64 || d == 128; }
bool known(gdn2_dtype_t dt) { return dt == GDN2_F32 || dt == GDN2_BF16; }
int page_shift(int page) {
  switch (page) {
  case 16:
    return 4;
  case 32:
    return 5;
  case 64:
    return 6;
  case 128:
    return 7;
  case 256:
    return 8;
  default:
    return -1;
  }
}

// Calls F<IO, D>::run(args...) for a dtype and head width checked before.
#define GDN2_ATTN_DISPATCH(e, dt, d, FN, ...)                                          \
  do {                                                                                 \
    if ((dt) == GDN2_F32)                                                              \
      e = (d) == 64 ? gdn2::attn::FN<float, 64>(__VA_ARGS__)                           \
                    : gdn2::attn::FN<float, 128>(__VA_ARGS__);                         \
    else                                                                               \
      e = (d) == 64 ? gdn2::attn::FN<gdn2::bf16_t, 64>(__VA_ARGS__)                    \
                    : gdn2::attn::FN<gdn2::bf16_t, 128>(__VA_ARGS__);                  \
  } while (0)
// the same with the cache's element type: the tensors' own, or e4m3
#define GDN2_CACHE_DISPATCH(e, dt, f8, d, FN, ...)                                                     \
  do {                                                                                                 \
    if ((dt) == GDN2_F32)                                                                              \
      e = (f8) ? ((d) == 64 ? gdn2::attn::FN<float, gdn2::f8_t, 64>(__VA_ARGS__)                       \
                            : gdn2::attn::FN<float, gdn2::f8_t, 128>(__VA_ARGS__))                     \
               : ((d) == 64 ? gdn2::attn::FN<float, float, 64>(__VA_ARGS__)                            \
                            : gdn2::attn::FN<float, float, 128>(__VA_ARGS__));                         \
    else                                                                                               \
      e = (f8) ? ((d) == 64 ? gdn2::attn::FN<gdn2::bf16_t, gdn2::f8_t, 64>(__VA_ARGS__)                \
                            : gdn2::attn::FN<gdn2::bf16_t, gdn2::f8_t, 128>(__VA_ARGS__))              \
               : ((d) == 64 ? gdn2::attn::FN<gdn2::bf16_t, gdn2::bf16_t, 64>(__VA_ARGS__)              \
                            : gdn2::attn::FN<gdn2::bf16_t, gdn2::bf16_t, 128>(__VA_ARGS__));           \
  } while (0)

gdn2_status_t launched(const char *fn, hipError_t e) {
  if (e != hipSuccess)
    return fail(GDN2_ERR_HIP, "%s: launch failed: %s", fn, hipGetErrorString(e));
  return ok();
}

gdn2_status_t check_heads(const char *fn, int Hq, int Hk, int d, gdn2_dtype_t dt) {
  if (!known(dt))
    return fail(GDN2_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, static_cast<int>(dt));
  if (Hq <= 0 || Hk <= 0)
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: bad head counts Hq=%d Hk=%d", fn, Hq, Hk);
  if (!attn_dim(d))
    return fail(GDN2_ERR_UNSUPPORTED, "%s: unsupported head dim d=%d (need 64 or 128)", fn, d);
  return GDN2_OK;
}

// The window and its sinks of a call whose sequences have at most `keys` keys:
// none of either where they hide nothing.
gdn2_status_t check_window(const char *fn, int window, int sinks, long long keys, attn_sizes &z) {
  if (window < 0 || sinks < 0)
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: negative %s %d", fn, window < 0 ? "window" : "number of sinks",
                window < 0 ? window : sinks);
  const bool hides = window > 0 && static_cast<long long>(window) + sinks < keys;
  if (hides && sinks > MAX_SINKS)
    return fail(GDN2_ERR_UNSUPPORTED, "%s: %d sinks (at most %d)", fn, sinks, MAX_SINKS);
  z.window = hides ? window : 0;
  z.sinks = hides ? sinks : 0;
  return GDN2_OK;
}

// Sizes of a call on B sequences of T tokens (num_seqs == 0) or num_seqs
// packed sequences of T tokens in all.
gdn2_status_t check_attn(const char *fn, int B, int T, int Hq, int Hk, int d, int num_seqs, bool packed, int window,
                         int sinks, float scale, gdn2_dtype_t dt, attn_sizes &z) {
  const gdn2_status_t st = check_heads(fn, Hq, Hk, d, dt);
  if (st != GDN2_OK)
    return st;
  if (Hq % Hk != 0)
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: Hq=%d is not a multiple of Hk=%d", fn, Hq, Hk);
  if (B <= 0 || T < 0 || num_seqs < 0)
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: bad sizes B=%d T=%d num_seqs=%d", fn, B, T, num_seqs);
  if (packed && (B != 1 || num_seqs == 0))
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: packed sequences need B == 1 and num_seqs > 0", fn);
  if (!packed && num_seqs != 0)
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: num_seqs without cu_seqlens", fn);
  const gdn2_status_t sw = check_window(fn, window, sinks, T, z);
  if (sw != GDN2_OK)
    return sw;
  // (the kernels' exponents are in base 2, scale log2 e: finite too)
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f))
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: scale must be positive and at most 2.3e38", fn);
  const long long tot = static_cast<long long>(B) * T, N = packed ? num_seqs : B;
  // (a row tile's offsets within 128 tokens are 32-bit: 2^15 heads of 128)
  if (Hq > (1 << 15) || tot > MAX_ROWS || tot * Hq > MAX_ROWS || N * Hk > MAX_UNITS)
    return fail(GDN2_ERR_UNSUPPORTED,
                "%s: too large (at most 2^15 query heads, 2^26 - 1 query rows, 2^20 - 1 sequence-heads)", fn);
  z.N = static_cast<int>(N);
  z.T = T;
  z.Ttot = static_cast<int>(tot);
  z.Hq = Hq;
  z.Hk = Hk;
  z.packed = packed;
  z.scale = scale;
  z.max_pages = z.num_pages = z.page_shift = 0;
  z.max_keys = T;
  return GDN2_OK;
}

// The backward with sinks has a launch of a workgroup at least for every 32
// sinks of a sequence and kv head, of 256 threads each.
gdn2_status_t check_far(const char *fn, const attn_sizes &z) {
  if (static_cast<long long>(z.N) * z.Hk * ((z.sinks + 31) / 32) >= (1LL << 23))
    return fail(GDN2_ERR_UNSUPPORTED, "%s: too large (at most 2^23 - 1 sequence-heads times 32 sinks)", fn);
  return GDN2_OK;
}

gdn2_status_t check_ptrs(const char *fn, std::initializer_list<const void *> need,
                         std::initializer_list<const void *> optional = {}) {
  for (const void *p : need)
    if (!p)
      return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: null pointer", fn);
  for (const void *p : need)
    if (!aligned16(p))
      return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: pointers must be 16-byte aligned", fn);
  for (const void *p : optional)
    if (p && !aligned16(p))
      return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: pointers must be 16-byte aligned", fn);
  return GDN2_OK;
}

gdn2_status_t check_rope(const char *fn, int B, int T, int Hq, int Hk, int d, int rot, const double *freqs, float eps,
                         gdn2_dtype_t dt, uint32_t flags, const float *wq, const float *wk) {
  const gdn2_status_t st = check_heads(fn, Hq, Hk, d, dt);
  if (st != GDN2_OK)
    return st;
  if (B <= 0 || T < 0)
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: bad sizes B=%d T=%d", fn, B, T);
  if (flags & ~(GDN2_ROPE_INTERLEAVED | GDN2_ROPE_NO_NORM))
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: unknown flags 0x%x", fn, flags);
  if (rot < 0 || rot > d || rot % 8 != 0)
    return fail(GDN2_ERR_UNSUPPORTED, "%s: rotary_dim=%d must be a multiple of 8 up to d=%d", fn, rot, d);
  if ((rot > 0) != (freqs != nullptr))
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: freqs goes with rotary_dim > 0", fn);
  if ((flags & GDN2_ROPE_NO_NORM) && (wq || wk))
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: weights without the norm", fn);
  if (!(flags & GDN2_ROPE_NO_NORM) && !(eps >= 0.f))
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: eps must not be negative", fn);
  const long long tot = static_cast<long long>(B) * T;
  if (tot > MAX_ROWS || tot * (static_cast<long long>(Hq) + Hk) > MAX_ROWS)
    return fail(GDN2_ERR_UNSUPPORTED, "%s: too large (at most 2^26 - 1 query and key rows)", fn);
  return GDN2_OK;
}

gdn2_status_t check_cache(const char *fn, int num_pages, int page_size, gdn2_dtype_t dt, gdn2_dtype_t cache_dt,
                          const void *ks, const void *vs) {
  if (page_shift(page_size) < 0)
    return fail(GDN2_ERR_UNSUPPORTED, "%s: unsupported page size %d (need 16, 32, 64, 128 or 256)", fn, page_size);
  if (num_pages <= 0 || static_cast<long long>(num_pages) * page_size > 0x7fffffffLL)
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: bad page count %d (1 .. 2^31 / page size)", fn, num_pages);
  if (cache_dt != dt && cache_dt != GDN2_F8E4M3)
    return fail(GDN2_ERR_UNSUPPORTED, "%s: cache dtype %d (the tensors' own or e4m3)", fn, static_cast<int>(cache_dt));
  if ((cache_dt == GDN2_F8E4M3) != (ks != nullptr) || (ks != nullptr) != (vs != nullptr))
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: an e4m3 cache goes with k_scale and v_scale", fn);
  return GDN2_OK;
}

rope_call rope_of(const void *q, const void *k, const float *wq, const float *wk, const double *freqs,
                  const int32_t *positions, int B, int T, int Hq, int Hk, int rot, float eps, uint32_t flags, void *oq,
                  void *ok_) {
  rope_call z;
  z.q = q;
  z.k = k;
  z.wq = wq;
  z.wk = wk;
  z.freqs = freqs;
  z.positions = positions;
  z.gq = z.gk = nullptr;
  z.oq = oq;
  z.ok = ok_;
  z.T = T;
  z.Hq = Hq;
  z.Hk = Hk;
  z.rot = rot;
  z.tokens = static_cast<long>(B) * T;
  z.eps = eps;
  z.norm = !(flags & GDN2_ROPE_NO_NORM);
  z.interleaved = (flags & GDN2_ROPE_INTERLEAVED) != 0;
  return z;
}

gdn2_status_t kv_cache_io(const char *fn, const void *k, const void *v, const int64_t *slots, int n, int Hk, int d,
                          int num_pages, int page_size, gdn2_dtype_t dt, gdn2_dtype_t cache_dt, const void *k_cache,
                          const void *v_cache, const uint8_t *k_scale, const uint8_t *v_scale, bool write, void *stream) {
  gdn2_status_t st = check_heads(fn, 1, Hk, d, dt);
  if (st != GDN2_OK)
    return st;
  st = check_cache(fn, num_pages, page_size, dt, cache_dt, k_scale, v_scale);
  if (st != GDN2_OK)
    return st;
  if (n < 0)
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: bad token count %d", fn, n);
  if (static_cast<long long>(n) * Hk > MAX_ROWS)
    return fail(GDN2_ERR_UNSUPPORTED, "%s: too large (at most 2^26 - 1 rows)", fn);
  if (n == 0)
    return ok();
  st = check_ptrs(fn, {k, v, k_cache, v_cache});
  if (st != GDN2_OK)
    return st;
  if (!slots || (reinterpret_cast<uintptr_t>(slots) & 7u))
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: slots must be an aligned pointer", fn);
  cache_call z;
  z.k = const_cast<void *>(k);
  z.v = const_cast<void *>(v);
  z.kc = const_cast<void *>(k_cache);
  z.vc = const_cast<void *>(v_cache);
  z.ks = const_cast<uint8_t *>(k_scale);
  z.vs = const_cast<uint8_t *>(v_scale);
  z.slots = slots;
  z.tokens = n;
  z.Hk = Hk;
  z.num_pages = num_pages;
  z.page_shift = page_shift(page_size);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  prof_scope p(write ? "kv_cache_write" : "kv_cache_read", s);
  GDN2_CACHE_DISPATCH(e, dt, cache_dt == GDN2_F8E4M3, d, launch_kv_cache, z, write, s);
  return launched(fn, e);
}

// Sizes of a paged call, without its pointers.
gdn2_status_t check_paged(const char *fn, int B, int T, int Hq, int Hk, int d, int num_seqs, int page_size,
                          int max_pages, int window, int sinks, float scale, gdn2_dtype_t dt, attn_sizes &z) {
  gdn2_status_t st = check_attn(fn, B, T, Hq, Hk, d, num_seqs, num_seqs > 0, window < 0 ? window : 0,
                                sinks < 0 ? sinks : 0, scale, dt, z);
  if (st != GDN2_OK)
    return st;
  const int sh = page_shift(page_size);
  if (sh < 0)
    return fail(GDN2_ERR_UNSUPPORTED, "%s: unsupported page size %d (need 16, 32, 64, 128 or 256)", fn, page_size);
  if (max_pages < 0 || static_cast<long long>(max_pages) * page_size > (1LL << 28))
    return fail(GDN2_ERR_UNSUPPORTED, "%s: at most 2^28 keys a sequence (max_pages=%d)", fn, max_pages);
  z.page_shift = sh;
  z.max_pages = max_pages;
  z.max_keys = static_cast<long long>(max_pages) * page_size;
  // a query sees at most max_keys + T positions
  return check_window(fn, window, sinks, z.max_keys + T, z);
}

// Sizes of a shared-prefix call, without its pointers; x gets its parts.
gdn2_status_t check_prefix(const char *fn, int B, int T, int Hq, int Hk, int d, int num_seqs, int num_groups,
                           int page_size, int max_prefix_pages, int max_pages, float scale, gdn2_dtype_t dt,
                           attn_sizes &z, prefix_call &x) {
  gdn2_status_t st = check_paged(fn, B, T, Hq, Hk, d, num_seqs, page_size, max_pages, 0, 0, scale, dt, z);
  if (st != GDN2_OK)
    return st;
  if (num_groups <= 0)
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: bad number of groups %d", fn, num_groups);
  if (max_prefix_pages < 0 || static_cast<long long>(max_prefix_pages) * page_size > (1LL << 28))
    return fail(GDN2_ERR_UNSUPPORTED, "%s: at most 2^28 keys a prefix (max_prefix_pages=%d)", fn, max_prefix_pages);
  if (static_cast<long long>(num_groups) * Hk > MAX_UNITS)
    return fail(GDN2_ERR_UNSUPPORTED, "%s: too large (at most 2^20 - 1 group-heads)", fn);
  // (the join always runs, four rows a workgroup of 256 work-items, in 32 bits with the last one filled up)
  if (static_cast<long long>(z.Ttot) * Hq > MAX_ROWS - 3)
    return fail(GDN2_ERR_UNSUPPORTED, "%s: too large (at most 2^26 - 4 query rows)", fn);
  x = {};
  x.ngroups = num_groups;
  x.max_pages = max_prefix_pages;
  if (T > 0)
    gdn2::attn::attn_prefix_splits(z, x);
  return GDN2_OK;
}
size_t prefix_bytes(const attn_sizes &z, const prefix_call &x, int d) {
  return static_cast<size_t>(x.prefix_parts + x.own_parts) * z.Ttot * z.Hq * (d + 1) * sizeof(float);
}

size_t paged_bytes(const attn_sizes &z, int d) {
  const int s = gdn2::attn::attn_paged_splits(z);
  return s <= 1 ? 0 : static_cast<size_t>(s) * z.Ttot * z.Hq * (d + 1) * sizeof(float);
}

gdn2_status_t attn_fwd(const char *fn, const void *q, const void *k, const void *v, const int32_t *cu_seqlens, int B,
                       int T, int Hq, int Hk, int d, int num_seqs, int window, int sinks, float scale, gdn2_dtype_t dt,
                       void *o, float *lse, void *stream) {
  attn_sizes z;
  gdn2_status_t st = check_attn(fn, B, T, Hq, Hk, d, num_seqs, cu_seqlens != nullptr, window, sinks, scale, dt, z);
  if (st != GDN2_OK)
    return st;
  if (T == 0)
    return ok();
  st = check_ptrs(fn, {q, k, v, o}, {cu_seqlens, lse});
  if (st != GDN2_OK)
    return st;
  attn_ptrs p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.cu = cu_seqlens;
  p.o = o;
  p.lse = lse;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  prof_scope ps("attn_fwd", s);
  GDN2_ATTN_DISPATCH(e, dt, d, launch_attn_fwd, z, p, s);
  return launched(fn, e);
}

gdn2_status_t attn_bwd(const char *fn, const void *q, const void *k, const void *v, const void *o, const float *lse,
                       const void *dout, const int32_t *cu_seqlens, int B, int T, int Hq, int Hk, int d, int num_seqs,
                       int window, int sinks, float scale, gdn2_dtype_t dt, void *dq, void *dk, void *dv,
                       void *workspace, size_t workspace_bytes, void *stream) {
  attn_sizes z;
  gdn2_status_t st = check_attn(fn, B, T, Hq, Hk, d, num_seqs, cu_seqlens != nullptr, window, sinks, scale, dt, z);
  if (st != GDN2_OK)
    return st;
  if (T == 0)
    return ok();
  st = check_far(fn, z);
  if (st != GDN2_OK)
    return st;
  st = check_ptrs(fn, {q, k, v, o, lse, dout, dq, dk, dv}, {cu_seqlens, workspace});
  if (st != GDN2_OK)
    return st;
  const size_t need = gdn2::attn::attn_bwd_bytes(z, d) + gdn2::attn::attn_bwd_far_bytes(z, d);
  if (!workspace || workspace_bytes < need)
    return fail(GDN2_ERR_WORKSPACE_TOO_SMALL, "%s: workspace holds %zu bytes, %zu are needed", fn, workspace_bytes,
                need);
  attn_ptrs p = {};
  p.q = q;
  p.k = k;
  p.v = v;
  p.cu = cu_seqlens;
  p.o = const_cast<void *>(o);
  p.lse = const_cast<float *>(lse);
  p.dout = dout;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  {
    prof_scope ps("attn_bwd_dq", s);
    GDN2_ATTN_DISPATCH(e, dt, d, launch_attn_bwd_dq, z, p, workspace, s);
  }
  if (e == hipSuccess && z.sinks) {
    prof_scope ps("attn_bwd_far", s);
    GDN2_ATTN_DISPATCH(e, dt, d, launch_attn_bwd_far, z, p, workspace, s);
  }
  if (e == hipSuccess) {
    prof_scope ps("attn_bwd_dkv", s);
    GDN2_ATTN_DISPATCH(e, dt, d, launch_attn_bwd_dkv, z, p, workspace, s);
  }
  return launched(fn, e);
}

gdn2_status_t attn_paged(const char *fn, const void *q, const void *k_cache, const void *v_cache,
                         const uint8_t *k_scale, const uint8_t *v_scale, const int32_t *block_table,
                         const int32_t *seq_lens, const int32_t *cu_seqlens, int B, int T, int Hq, int Hk, int d,
                         int num_seqs, int num_pages, int page_size, int max_pages, int window, int sinks, float scale,
                         gdn2_dtype_t dt, gdn2_dtype_t cache_dt, void *o, float *lse, void *workspace,
                         size_t workspace_bytes, void *stream) {
  attn_sizes z;
  if ((cu_seqlens != nullptr) != (num_seqs > 0))
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: cu_seqlens goes with num_seqs > 0", fn);
  gdn2_status_t st = check_paged(fn, B, T, Hq, Hk, d, num_seqs, page_size, max_pages, window, sinks, scale, dt, z);
  if (st != GDN2_OK)
    return st;
  st = check_cache(fn, num_pages, page_size, dt, cache_dt, k_scale, v_scale);
  if (st != GDN2_OK)
    return st;
  if (T == 0)
    return ok();
  // (a table of no pages has no entries: nothing reads it)
  st = check_ptrs(fn, {q, k_cache, v_cache, max_pages ? block_table : seq_lens, seq_lens, o},
                  {cu_seqlens, lse, workspace, block_table});
  if (st != GDN2_OK)
    return st;
  const int splits = dt == GDN2_BF16 && gdn2::attn::attn_decode_wide(z) ? 1 : gdn2::attn::attn_paged_splits(z);
  const size_t need = splits > 1 ? paged_bytes(z, d) : 0;
  if (need && (!workspace || workspace_bytes < need))
    return fail(GDN2_ERR_WORKSPACE_TOO_SMALL, "%s: workspace holds %zu bytes, %zu are needed", fn, workspace_bytes,
                need);
  z.num_pages = num_pages;
  attn_ptrs p = {};
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.ks = k_scale;
  p.vs = v_scale;
  p.table = block_table;
  p.seq_lens = seq_lens;
  p.cu = cu_seqlens;
  p.o = o;
  p.lse = lse;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  {
    prof_scope ps("attn_paged", s);
    GDN2_CACHE_DISPATCH(e, dt, cache_dt == GDN2_F8E4M3, d, launch_attn_paged, z, p, splits, workspace, s);
  }
  if (e == hipSuccess && splits > 1) {
    prof_scope ps("attn_paged_join", s);
    GDN2_ATTN_DISPATCH(e, dt, d, launch_attn_join, z, p, splits, nullptr, workspace, s);
  }
  return launched(fn, e);
}

}  // namespace

extern "C" {

gdn2_status_t gdn2_qk_norm_rope_fwd(const void *q, const void *k, const float *wq, const float *wk,
                                    const double *freqs, const int32_t *positions, int B, int T, int Hq, int Hk, int d,
                                    int rotary_dim, float eps, gdn2_dtype_t dt, uint32_t flags, void *q_out,
                                    void *k_out, void *stream) {
  const char *fn = "gdn2_qk_norm_rope_fwd";
  gdn2_status_t st = check_rope(fn, B, T, Hq, Hk, d, rotary_dim, freqs, eps, dt, flags, wq, wk);
  if (st != GDN2_OK)
    return st;
  if (T == 0)
    return ok();
  st = check_ptrs(fn, {q, k, q_out, k_out}, {wq, wk, freqs, positions});
  if (st != GDN2_OK)
    return st;
  const rope_call z = rope_of(q, k, wq, wk, freqs, positions, B, T, Hq, Hk, rotary_dim, eps, flags, q_out, k_out);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  prof_scope p("qk_norm_rope_fwd", s);
  GDN2_ATTN_DISPATCH(e, dt, d, launch_rope_fwd, z, s);
  return launched(fn, e);
}

size_t gdn2_qk_norm_rope_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int d) {
  if (B <= 0 || T <= 0 || Hq <= 0 || Hk <= 0 || !attn_dim(d) ||
      static_cast<long long>(B) * T > MAX_ROWS ||
      static_cast<long long>(B) * T * (static_cast<long long>(Hq) + Hk) > MAX_ROWS)
    return 0;
  return static_cast<size_t>(gdn2::attn::rope_bwd_groups(static_cast<long>(B) * T, Hq, Hk, d)) * 2 * d * sizeof(float);
}

gdn2_status_t gdn2_qk_norm_rope_bwd(const void *q, const void *k, const float *wq, const float *wk,
                                    const double *freqs, const int32_t *positions, const void *dq_out,
                                    const void *dk_out, int B, int T, int Hq, int Hk, int d, int rotary_dim, float eps,
                                    gdn2_dtype_t dt, uint32_t flags, void *dq, void *dk, float *dwq, float *dwk,
                                    void *workspace, size_t workspace_bytes, void *stream) {
  const char *fn = "gdn2_qk_norm_rope_bwd";
  gdn2_status_t st = check_rope(fn, B, T, Hq, Hk, d, rotary_dim, freqs, eps, dt, flags, wq, wk);
  if (st != GDN2_OK)
    return st;
  const bool norm = !(flags & GDN2_ROPE_NO_NORM), want_dw = dwq || dwk;
  if (!norm && want_dw)
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: weight gradients without the norm", fn);
  if (T > 0) {
    st = norm ? check_ptrs(fn, {q, k, dq_out, dk_out, dq, dk}, {wq, wk, freqs, positions, dwq, dwk, workspace})
              : check_ptrs(fn, {dq_out, dk_out, dq, dk}, {freqs, positions});
    if (st != GDN2_OK)
      return st;
    const size_t need = want_dw ? gdn2_qk_norm_rope_bwd_workspace_bytes(B, T, Hq, Hk, d) : 0;
    if (workspace_bytes < need || (need && !workspace))
      return fail(GDN2_ERR_WORKSPACE_TOO_SMALL, "%s: workspace holds %zu bytes, %zu are needed", fn, workspace_bytes,
                  need);
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  int groups = 0;
  if (T > 0) {
    rope_call z = rope_of(q, k, wq, wk, freqs, positions, B, T, Hq, Hk, rotary_dim, eps, flags, dq, dk);
    z.gq = dq_out;
    z.gk = dk_out;
    groups = gdn2::attn::rope_bwd_groups(z.tokens, Hq, Hk, d);
    prof_scope p("qk_norm_rope_bwd", s);
    GDN2_ATTN_DISPATCH(e, dt, d, launch_rope_bwd, z, want_dw ? static_cast<float *>(workspace) : nullptr, s);
  }
  if (e == hipSuccess && want_dw) {
    prof_scope p("qk_norm_rope_dw", s);
    e = d == 64 ? gdn2::attn::launch_rope_dw<64>(static_cast<const float *>(workspace), groups, dwq, dwk, s)
                : gdn2::attn::launch_rope_dw<128>(static_cast<const float *>(workspace), groups, dwq, dwk, s);
  }
  return launched(fn, e);
}

gdn2_status_t gdn2_attn_fwd(const void *q, const void *k, const void *v, const int32_t *cu_seqlens, int B, int T,
                            int Hq, int Hk, int d, int num_seqs, int window, float scale, gdn2_dtype_t dt, void *o,
                            float *lse, void *stream) {
  return attn_fwd("gdn2_attn_fwd", q, k, v, cu_seqlens, B, T, Hq, Hk, d, num_seqs, window, 0, scale, dt, o, lse, stream);
}

gdn2_status_t gdn2_attn_sink_fwd(const void *q, const void *k, const void *v, const int32_t *cu_seqlens, int B, int T,
                                 int Hq, int Hk, int d, int num_seqs, int window, int sinks, float scale,
                                 gdn2_dtype_t dt, void *o, float *lse, void *stream) {
  return attn_fwd("gdn2_attn_sink_fwd", q, k, v, cu_seqlens, B, T, Hq, Hk, d, num_seqs, window, sinks, scale, dt, o, lse,
                  stream);
}

size_t gdn2_attn_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int d) {
  attn_sizes z;
  if (check_attn("gdn2_attn_bwd_workspace_bytes", B, T, Hq, Hk, d, 0, false, 0, 0, 1.f, GDN2_F32, z) != GDN2_OK) {
    (void)ok();
    return 0;
  }
  return T == 0 ? 0 : gdn2::attn::attn_bwd_bytes(z, d);
}

size_t gdn2_attn_sink_bwd_workspace_bytes(int B, int T, int Hq, int Hk, int d, int num_seqs, int sinks) {
  attn_sizes z;
  // (no window hides more than one token's; a call that takes more sinks has none that hides anything)
  if (check_attn("gdn2_attn_sink_bwd_workspace_bytes", B, T, Hq, Hk, d, num_seqs, num_seqs > 0, 1,
                 sinks > MAX_SINKS ? 0 : sinks, 1.f, GDN2_F32, z) != GDN2_OK ||
      check_far("gdn2_attn_sink_bwd_workspace_bytes", z) != GDN2_OK) {
    (void)ok();
    return 0;
  }
  return T == 0 ? 0 : gdn2::attn::attn_bwd_bytes(z, d) + gdn2::attn::attn_bwd_far_bytes(z, d);
}

gdn2_status_t gdn2_attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                            const void *dout, const int32_t *cu_seqlens, int B, int T, int Hq, int Hk, int d,
                            int num_seqs, int window, float scale, gdn2_dtype_t dt, void *dq, void *dk, void *dv,
                            void *workspace, size_t workspace_bytes, void *stream) {
  return attn_bwd("gdn2_attn_bwd", q, k, v, o, lse, dout, cu_seqlens, B, T, Hq, Hk, d, num_seqs, window, 0, scale, dt,
                  dq, dk, dv, workspace, workspace_bytes, stream);
}

gdn2_status_t gdn2_attn_sink_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                                 const void *dout, const int32_t *cu_seqlens, int B, int T, int Hq, int Hk, int d,
                                 int num_seqs, int window, int sinks, float scale, gdn2_dtype_t dt, void *dq, void *dk,
                                 void *dv, void *workspace, size_t workspace_bytes, void *stream) {
  return attn_bwd("gdn2_attn_sink_bwd", q, k, v, o, lse, dout, cu_seqlens, B, T, Hq, Hk, d, num_seqs, window, sinks,
                  scale, dt, dq, dk, dv, workspace, workspace_bytes, stream);
}

size_t gdn2_attn_paged_workspace_bytes(int B, int T, int Hq, int Hk, int d, int num_seqs, int page_size, int max_pages,
                                       int window) {
  return gdn2_attn_sink_paged_workspace_bytes(B, T, Hq, Hk, d, num_seqs, page_size, max_pages, window, 0);
}

size_t gdn2_attn_sink_paged_workspace_bytes(int B, int T, int Hq, int Hk, int d, int num_seqs, int page_size,
                                            int max_pages, int window, int sinks) {
  attn_sizes z;
  if (check_paged("gdn2_attn_sink_paged_workspace_bytes", B, T, Hq, Hk, d, num_seqs, page_size, max_pages, window, sinks,
                  1.f, GDN2_F32, z) != GDN2_OK) {
    (void)ok();
    return 0;
  }
  return T == 0 ? 0 : paged_bytes(z, d);
}

gdn2_status_t gdn2_attn_paged(const void *q, const void *k_cache, const void *v_cache, const uint8_t *k_scale,
                              const uint8_t *v_scale, const int32_t *block_table, const int32_t *seq_lens,
                              const int32_t *cu_seqlens, int B, int T, int Hq, int Hk, int d, int num_seqs,
                              int num_pages, int page_size, int max_pages, int window, float scale, gdn2_dtype_t dt,
                              gdn2_dtype_t cache_dt, void *o, float *lse, void *workspace, size_t workspace_bytes,
                              void *stream) {
  return attn_paged("gdn2_attn_paged", q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens, B, T,
                    Hq, Hk, d, num_seqs, num_pages, page_size, max_pages, window, 0, scale, dt, cache_dt, o, lse,
                    workspace, workspace_bytes, stream);
}

gdn2_status_t gdn2_attn_sink_paged(const void *q, const void *k_cache, const void *v_cache, const uint8_t *k_scale,
                                   const uint8_t *v_scale, const int32_t *block_table, const int32_t *seq_lens,
                                   const int32_t *cu_seqlens, int B, int T, int Hq, int Hk, int d, int num_seqs,
                                   int num_pages, int page_size, int max_pages, int window, int sinks, float scale,
                                   gdn2_dtype_t dt, gdn2_dtype_t cache_dt, void *o, float *lse, void *workspace,
                                   size_t workspace_bytes, void *stream) {
  return attn_paged("gdn2_attn_sink_paged", q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, cu_seqlens, B,
                    T, Hq, Hk, d, num_seqs, num_pages, page_size, max_pages, window, sinks, scale, dt, cache_dt, o, lse,
                    workspace, workspace_bytes, stream);
}

size_t gdn2_attn_paged_prefix_workspace_bytes(int B, int T, int Hq, int Hk, int d, int num_seqs, int num_groups,
                                              int page_size, int max_prefix_pages, int max_pages) {
  attn_sizes z;
  prefix_call x;
  if (check_prefix("gdn2_attn_paged_prefix_workspace_bytes", B, T, Hq, Hk, d, num_seqs, num_groups, page_size,
                   max_prefix_pages, max_pages, 1.f, GDN2_F32, z, x) != GDN2_OK) {
    (void)ok();
    return 0;
  }
  return prefix_bytes(z, x, d);
}

gdn2_status_t gdn2_attn_paged_prefix(const void *q, const void *k_cache, const void *v_cache, const uint8_t *k_scale,
                                     const uint8_t *v_scale, const int32_t *prefix_table, const int32_t *prefix_lens,
                                     const int32_t *cu_groups, const int32_t *block_table, const int32_t *seq_lens,
                                     const int32_t *cu_seqlens, int B, int T, int Hq, int Hk, int d, int num_seqs,
                                     int num_groups, int num_pages, int page_size, int max_prefix_pages, int max_pages,
                                     float scale, gdn2_dtype_t dt, gdn2_dtype_t cache_dt, void *o, float *lse,
                                     void *workspace, size_t workspace_bytes, void *stream) {
  const char *fn = "gdn2_attn_paged_prefix";
  attn_sizes z;
  prefix_call x;
  if ((cu_seqlens != nullptr) != (num_seqs > 0))
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: cu_seqlens goes with num_seqs > 0", fn);
  gdn2_status_t st = check_prefix(fn, B, T, Hq, Hk, d, num_seqs, num_groups, page_size, max_prefix_pages, max_pages,
                                  scale, dt, z, x);
  if (st != GDN2_OK)
    return st;
  if (!cu_groups && num_groups != 1)
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: %d groups without cu_groups", fn, num_groups);
  st = check_cache(fn, num_pages, page_size, dt, cache_dt, k_scale, v_scale);
  if (st != GDN2_OK)
    return st;
  if (T == 0)
    return ok();
  // (a table of no pages has no entries: nothing reads it)
  st = check_ptrs(fn, {q, k_cache, v_cache, max_pages ? block_table : seq_lens, max_prefix_pages ? prefix_table : seq_lens,
                       prefix_lens, seq_lens, o},
                  {cu_groups, cu_seqlens, lse, workspace, block_table, prefix_table});
  if (st != GDN2_OK)
    return st;
  const size_t need = prefix_bytes(z, x, d);
  if (!workspace || workspace_bytes < need)
    return fail(GDN2_ERR_WORKSPACE_TOO_SMALL, "%s: workspace holds %zu bytes, %zu are needed", fn, workspace_bytes,
                need);
  z.num_pages = num_pages;
  x.table = prefix_table;
  x.lens = prefix_lens;
  x.groups = cu_groups;
  attn_ptrs p = {};
  p.q = q;
  p.k = k_cache;
  p.v = v_cache;
  p.ks = k_scale;
  p.vs = v_scale;
  p.table = block_table;
  p.seq_lens = seq_lens;
  p.cu = cu_seqlens;
  p.o = o;
  p.lse = lse;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const bool f8 = cache_dt == GDN2_F8E4M3;
  hipError_t e;
  {
    prof_scope ps("attn_prefix", s);
    GDN2_CACHE_DISPATCH(e, dt, f8, d, launch_attn_prefix, z, p, x, workspace, s);
  }
  if (e == hipSuccess) {
    prof_scope ps("attn_prefix_join", s);
    GDN2_ATTN_DISPATCH(e, dt, d, launch_attn_join, z, p, x.prefix_parts + x.own_parts, &x, workspace, s);
  }
  return launched(fn, e);
}

gdn2_status_t gdn2_kv_cache_write(const void *k, const void *v, const int64_t *slots, int n, int Hk, int d,
                                  int num_pages, int page_size, gdn2_dtype_t dt, gdn2_dtype_t cache_dt, void *k_cache,
                                  void *v_cache, uint8_t *k_scale, uint8_t *v_scale, void *stream) {
  return kv_cache_io("gdn2_kv_cache_write", k, v, slots, n, Hk, d, num_pages, page_size, dt, cache_dt, k_cache, v_cache,
                     k_scale, v_scale, true, stream);
}

gdn2_status_t gdn2_kv_cache_read(const int64_t *slots, int n, int Hk, int d, int num_pages, int page_size,
                                 gdn2_dtype_t dt, gdn2_dtype_t cache_dt, const void *k_cache, const void *v_cache,
                                 const uint8_t *k_scale, const uint8_t *v_scale, void *k, void *v, void *stream) {
  return kv_cache_io("gdn2_kv_cache_read", k, v, slots, n, Hk, d, num_pages, page_size, dt, cache_dt, k_cache, v_cache,
                     k_scale, v_scale, false, stream);
}

gdn2_status_t gdn2_kv_cache_append(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
                                   int64_t v_stride, const float *wq, const float *wk, const double *freqs,
                                   const int32_t *positions, const int64_t *slots, int B, int T, int Hq, int Hk, int d,
                                   int rotary_dim, float eps, int num_pages, int page_size, gdn2_dtype_t dt,
                                   gdn2_dtype_t cache_dt, uint32_t flags, void *q_out, int64_t q_out_stride,
                                   void *k_cache, void *v_cache, uint8_t *k_scale, uint8_t *v_scale, void *stream) {
  const char *fn = "gdn2_kv_cache_append";
  gdn2_status_t st = check_rope(fn, B, T, Hq, Hk, d, rotary_dim, freqs, eps, dt, flags, wq, wk);
  if (st != GDN2_OK)
    return st;
  st = check_cache(fn, num_pages, page_size, dt, cache_dt, k_scale, v_scale);
  if (st != GDN2_OK)
    return st;
  if (static_cast<long long>(B) * T * (static_cast<long long>(Hq) + 2LL * Hk) > MAX_ROWS)
    return fail(GDN2_ERR_UNSUPPORTED, "%s: too large (at most 2^26 - 1 query, key and value rows)", fn);
  const int per16 = dt == GDN2_F32 ? 4 : 8;
  const struct {
    const char *name;
    int64_t stride;
    int heads;
  } strides[] = {{"q", q_stride, Hq}, {"k", k_stride, Hk}, {"v", v_stride, Hk}, {"q_out", q_out_stride, Hq}};
  for (const auto &x : strides)
    if (x.stride < static_cast<int64_t>(x.heads) * d || x.stride > 0xffffffffLL || x.stride % per16 != 0)
      return fail(GDN2_ERR_INVALID_ARGUMENT,
                  "%s: token stride %lld of %s (at least %lld values, less than 2^32, a multiple of 16 bytes)", fn,
                  static_cast<long long>(x.stride), x.name, static_cast<long long>(x.heads) * d);
  if (T == 0)
    return ok();
  st = check_ptrs(fn, {q, k, v, q_out, k_cache, v_cache}, {wq, wk, freqs, positions});
  if (st != GDN2_OK)
    return st;
  if (!slots || (reinterpret_cast<uintptr_t>(slots) & 7u))
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: slots must be an aligned pointer", fn);
  if (q_out == q && q_out_stride != q_stride)
    return fail(GDN2_ERR_INVALID_ARGUMENT, "%s: q_out in place of q needs q's stride", fn);
  const rope_call z = rope_of(q, k, wq, wk, freqs, positions, B, T, Hq, Hk, rotary_dim, eps, flags, q_out, nullptr);
  cache_call c = {};
  c.v = const_cast<void *>(v);
  c.kc = k_cache;
  c.vc = v_cache;
  c.ks = k_scale;
  c.vs = v_scale;
  c.slots = slots;
  c.tokens = static_cast<int>(z.tokens);
  c.Hk = Hk;
  c.num_pages = num_pages;
  c.page_shift = page_shift(page_size);
  const gdn2::attn::append_strides t = {static_cast<long>(q_stride), static_cast<long>(k_stride),
                                        static_cast<long>(v_stride), static_cast<long>(q_out_stride)};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  prof_scope p("kv_cache_append", s);
  GDN2_CACHE_DISPATCH(e, dt, cache_dt == GDN2_F8E4M3, d, launch_kv_append, z, c, t, s);
  return launched(fn, e);
}

}  // extern "C"
