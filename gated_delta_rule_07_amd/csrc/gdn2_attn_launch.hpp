// gdn2_attn_launch.hpp -- how the forward attention's launchers choose a kernel's
// shape and fill its arguments.
#pragma once

#include "gdn2_attn_fwd_body.hpp"

namespace gdn2 {
namespace attn {

template <typename IO, typename CT, int D, int WM, int WN, int KT, bool PAGED, fwd_mode MODE>
__global__ void __launch_bounds__(64 * WM * WN, (D * sizeof(IO) <= 256 ? 2 : 1)) gdn2_attn_fwd_kernel(fwd_args a) {
  typedef fwd_body<IO, CT, D, WM, WN, KT, PAGED, MODE> F;
  __shared__ __align__(16) char lds[F::BYTES];
  F::run(a, blockIdx.x, lds);
}

template <typename IO, typename CT, int D, int WM, int WN, int KT, bool PAGED, fwd_mode MODE>
hipError_t launch_fwd(fwd_args &a, const attn_sizes &z, hipStream_t st) {
  const unsigned blocks = plan_tiles(z, a.G, 32 * WM, a.od) * a.splits;
  hipLaunchKernelGGL((gdn2_attn_fwd_kernel<IO, CT, D, WM, WN, KT, PAGED, MODE>), dim3(blocks), dim3(64 * WM * WN), 0, st,
                     a);
  return hipGetLastError();
}
// A call's rows a sequence and kv head: at most 32 on average (32-row tiles,
// else 128), and at most 16 (the decode kernel)
bool few_rows(const attn_sizes &z);
bool decode_rows(const attn_sizes &z);

inline void fill(fwd_args &a, const attn_sizes &z, const attn_ptrs &p) {
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
  a.sinks = z.sinks;
  a.splits = 1;
  a.c = z.scale * LOG2E;
  a.groups = nullptr;
  a.ngroups = a.seqs = a.tq = a.prefix_parts = 0;
  a.mark = a.wide = false;
}

// Where part s of a call's parts lies in ws: [parts, Ttot, Hq, D] outputs, then
// [parts, Ttot, Hq] sums.
inline void parts_at(fwd_args &a, const attn_sizes &z, int D, void *ws, int parts, int s) {
  const size_t rows = static_cast<size_t>(z.Ttot) * z.Hq;
  a.part_o = static_cast<float *>(ws) + s * rows * D;
  a.part_lse = static_cast<float *>(ws) + parts * rows * D + s * rows;
}

inline void fill_groups(fwd_args &a, const attn_sizes &z, const prefix_call &x) {
  a.groups = x.groups;
  a.ngroups = x.ngroups;
  a.seqs = z.N;
  a.tq = z.packed ? 0 : z.T;
  a.prefix_parts = x.prefix_parts;
}

// a's launch over the keys a paged call holds for its sequences
template <typename IO, typename CT, int D> hipError_t launch_paged(fwd_args &a, const attn_sizes &z, hipStream_t st);

}  // namespace attn
}  // namespace gdn2
