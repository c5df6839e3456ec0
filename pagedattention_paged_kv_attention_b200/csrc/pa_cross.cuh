// pa_cross.cuh -- the join of cross attention whose keys were split over several CTAs (paged_prefill_kernel,
// mode kCross).
//
// Split p of a query row holds its own softmax: m_p = max z, l_p = sum 2^(z - m_p) and the normalised row o_p.
//     out = sum_p w_p o_p / sum_p w_p,   w_p = l_p 2^(m_p - max_q m_q).
#pragma once

#include <math.h>

#include "pa_prefill.cuh"

namespace pa {
namespace pf {

constexpr int kMergeWarps = 8;

// grid (rows / kMergeWarps, sequences): one warp per (chunk token, head).
template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
cross_merge_kernel(const PrefillArgs a) {
  constexpr int kPer = D / 32;
  const int s = blockIdx.y, lane = threadIdx.x & 31;
  const long long idx = static_cast<long long>(blockIdx.x) * kMergeWarps + (threadIdx.x >> 5);
  const int q0 = a.q_start[s], n = a.q_start[s + 1] - q0, ctx = a.context_lens[s];
  const int tok = static_cast<int>(idx / a.num_heads), h = static_cast<int>(idx % a.num_heads);
  if (tok >= n || chunk_too_long(a, n) || q0 < 0 || q0 + n > a.num_q_tokens || ctx < 0 || ctx > a.max_context_len ||
      static_cast<long long>(ctx) > static_cast<long long>(a.max_blocks_per_seq) * a.block_size ||
      ctx <= a.split_tiles * kKvTile)
    return;
  const int parts = (ctx - 1) / (a.split_tiles * kKvTile) + 1;
  const size_t rowi = static_cast<size_t>(q0 + tok) * a.num_heads + h, base = rowi * a.splits;
  float M = -INFINITY;
  for (int p = 0; p < parts; ++p) M = fmaxf(M, a.part_m[base + p]);
  float wsum = 0.f, acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  for (int p = 0; p < parts; ++p) {
    const float w = a.part_l[base + p] * ex2(a.part_m[base + p] - M);
    const float* o = a.part_o + (base + p) * D + lane * kPer;
    wsum += w;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] += w * o[k];
  }
  const float inv = 1.f / wsum;
  T* dst = static_cast<T*>(a.out) + rowi * D + lane * kPer;
#pragma unroll
  for (int k = 0; k < kPer; k += 2)
    *reinterpret_cast<uint32_t*>(dst + k) = pack_pair<T>(acc[k] * inv, acc[k + 1] * inv);
}

}  // namespace pf
}  // namespace pa
