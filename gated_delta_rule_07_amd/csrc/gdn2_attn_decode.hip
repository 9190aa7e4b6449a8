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
#include "gdn2_attn_decode_body.hpp"

namespace gdn2 {
namespace attn {

template <typename CT, int D, int TK, bool SINK, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, 3) gdn2_attn_decode_kernel(fwd_args a) {
  typedef decode_body<CT, D, TK, SINK, WAVES> F;
  __shared__ __align__(16) char lds[F::BYTES];
  F::run(a, blockIdx.x, lds);
}

template <typename CT, int D> hipError_t launch_attn_decode(const fwd_args &a, hipStream_t st) {
  // (32 keys a wave and tile; 64 of e4m3 leave two waves a SIMD: 166 against
  // 136 us for 64 sequences of 4K to 16K keys)
  constexpr int TK = 2;
  const unsigned blocks = workgroups(a.od) * a.splits;
  if (a.sinks && a.wide)
    hipLaunchKernelGGL((gdn2_attn_decode_kernel<CT, D, TK, true, WIDE_WAVES>), dim3(blocks), dim3(64 * WIDE_WAVES), 0,
                       st, a);
  else if (a.sinks)
    hipLaunchKernelGGL((gdn2_attn_decode_kernel<CT, D, TK, true, 4>), dim3(blocks), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((gdn2_attn_decode_kernel<CT, D, TK, false, 4>), dim3(blocks), dim3(256), 0, st, a);
  return hipGetLastError();
}
template hipError_t launch_attn_decode<bf16_t, 64>(const fwd_args &, hipStream_t);
template hipError_t launch_attn_decode<bf16_t, 128>(const fwd_args &, hipStream_t);
template hipError_t launch_attn_decode<f8_t, 64>(const fwd_args &, hipStream_t);
template hipError_t launch_attn_decode<f8_t, 128>(const fwd_args &, hipStream_t);

}  // namespace attn
}  // namespace gdn2
