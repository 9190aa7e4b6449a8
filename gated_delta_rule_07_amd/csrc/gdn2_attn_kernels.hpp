// gdn2_attn_kernels.hpp -- host-side declarations of the attention operators'
// kernel launchers.  (Apart from gdn2_kernels.hpp: the recurrence's counter
// records hold for that file's text.)
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn2_kernels.hpp"

namespace gdn2 {

struct f8_t {  // one e4m3 code
  uint8_t bits;
};

namespace attn {

// Sizes of an attention call.  T: tokens per sequence, or in all when packed;
// Ttot: tokens of q in all.  Paged calls: max_keys = max_pages * page size.
struct attn_sizes {
  int N, T, Ttot, Hq, Hk;
  bool packed;
  int window;
  float scale;
  int max_pages, num_pages, page_shift;
  long long max_keys;
};
struct attn_ptrs {
  const void *q, *k, *v;
  void *o;
  float *lse;
  const int32_t *cu, *table, *seq_lens;
  const uint8_t *ks, *vs;
  // backward: k, v as above
  const void *dout;
  void *dq, *dk, *dv;
};

template <typename IO, int D> hipError_t launch_attn_fwd(const attn_sizes &z, const attn_ptrs &p, hipStream_t st);
// keys in `splits` parts (attn_paged_splits); more than one: the parts go to
// ws, [splits, Ttot, Hq, D] and [splits, Ttot, Hq] float32, and the join
// writes o and lse
int attn_paged_splits(const attn_sizes &z);
template <typename IO, typename CT, int D>
hipError_t launch_attn_paged(const attn_sizes &z, const attn_ptrs &p, int splits, void *ws, hipStream_t st);
template <typename IO, int D>
hipError_t launch_attn_join(const attn_sizes &z, const attn_ptrs &p, int splits, void *ws, hipStream_t st);
// Backward: dq, which leaves the rows' statistics in ws, then dk and dv, which
// read them.  ws holds the statistics and, where attn_bwd_parts workgroups share a key tile's rows,
// their sums.
int attn_bwd_parts(const attn_sizes &z);
inline size_t attn_bwd_stat_bytes(const attn_sizes &z) {
  return (static_cast<size_t>(z.Ttot) * z.Hq * 8 + 255) & ~static_cast<size_t>(255);
}
inline size_t attn_bwd_bytes(const attn_sizes &z, int d) {
  const size_t parts = static_cast<size_t>(attn_bwd_parts(z));
  return attn_bwd_stat_bytes(z) + (parts > 1 ? parts * 2 * z.Ttot * z.Hk * d * 4 : 0);
}
template <typename IO, int D>
hipError_t launch_attn_bwd_dq(const attn_sizes &z, const attn_ptrs &p, void *ws, hipStream_t st);
template <typename IO, int D>
hipError_t launch_attn_bwd_dkv(const attn_sizes &z, const attn_ptrs &p, void *ws, hipStream_t st);

// Query/key norm and rotation.  Backward: gq, gk the outputs' gradients, oq,
// ok the inputs'.
struct rope_call {
  const void *q, *k;
  const float *wq, *wk;
  const double *freqs;
  const int32_t *positions;
  const void *gq, *gk;
  void *oq, *ok;
  int T, Hq, Hk, rot;
  long tokens;
  float eps;
  bool norm, interleaved;
};
template <typename IO, int D> hipError_t launch_rope_fwd(const rope_call &z, hipStream_t st);
// part: [rope_bwd_groups, 2, D] float32, or nullptr (no weight gradients)
int rope_bwd_groups(long tokens, int Hq, int Hk, int D);
template <typename IO, int D> hipError_t launch_rope_bwd(const rope_call &z, float *part, hipStream_t st);
template <int D> hipError_t launch_rope_dw(const float *part, int groups, float *dwq, float *dwk, hipStream_t st);

// Paged cache: write k, v into (or read them from) the slots.
struct cache_call {
  void *k, *v, *kc, *vc;
  uint8_t *ks, *vs;
  const int64_t *slots;
  int tokens, Hk, num_pages, page_shift;
};
template <typename IO, typename CT, int D> hipError_t launch_kv_cache(const cache_call &z, bool write, hipStream_t st);

}  // namespace attn

}  // namespace gdn2
