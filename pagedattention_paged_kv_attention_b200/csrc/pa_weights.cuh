// pa_weights.cuh -- attention weights added to the cached tokens' scores.
//
// A token's score is the sum of the softmax weights that queries have given it, per kv head:
//   scores[s][kvh][t] += sum_g 2^(z_gt - lse_g),   lse_g = m_g + log2 sum_t 2^(z_gt - m_g),
// over the query heads g of the kv head; z is the scaled score in log2 units. One decode step's z (every
// token of every head) and the softmax statistics of each context partition come from
// paged_attention_main's W instantiations; this kernel joins the partitions' statistics and sums the
// heads' weights. A thread owns its tokens' scores and adds the heads in order, so results do not depend
// on timing.
#pragma once

#include <math.h>

#include "pa_attention.cuh"

namespace pa {

constexpr int kWeightThreads = 256;
constexpr int kWeightTokens = 1024;    // tokens of one CTA
constexpr int kWeightHeads = 64;       // query heads whose statistics are joined at a time

// grid (token chunks, kv heads, sequences)
__global__ void __launch_bounds__(kWeightThreads)
attention_weights_kernel(const AttnArgs a, float* __restrict__ scores, long long score_stride) {
  __shared__ float lse[kWeightHeads];
  grid_dependency_wait();
  grid_dependents_launch();
  const int s = blockIdx.z, kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = a.context_lens[s];
  const long long t0 = static_cast<long long>(blockIdx.x) * kWeightTokens;
  if (L <= 0 || context_len_invalid(L, a) || t0 >= L) return;
  const int n_parts = (L - 1) / a.partition_size + 1;
  constexpr int kPer = kWeightTokens / kWeightThreads;
  float acc[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
  for (int g0 = 0; g0 < a.group; g0 += kWeightHeads) {
    const int heads = min(kWeightHeads, a.group - g0);
    const size_t row0 = static_cast<size_t>(s) * a.num_heads + static_cast<size_t>(kvh) * a.group + g0;
    if (g0 > 0) __syncthreads();
    for (int g = warp; g < heads; g += kWeightThreads / 32) {
      const float2* st = a.stats + (row0 + g) * a.num_partitions;
      float M = -INFINITY;
      for (int p = lane; p < n_parts; p += 32) M = fmaxf(M, st[p].x);
#pragma unroll
      for (int b = 16; b > 0; b >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, b));
      float sum = 0.f;
      for (int p = lane; p < n_parts; p += 32) sum += st[p].y * fast_exp2(st[p].x - M);
#pragma unroll
      for (int b = 16; b > 0; b >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, b);
      if (lane == 0) lse[g] = M + log2f(sum);
    }
    __syncthreads();
    const float* z = a.logits + row0 * a.logit_stride + t0 + threadIdx.x;
    for (int g = 0; g < heads; ++g, z += a.logit_stride) {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (t0 + threadIdx.x + k * kWeightThreads < L) acc[k] += fast_exp2(z[k * kWeightThreads] - lse[g]);
    }
  }
  float* out = scores + (static_cast<size_t>(s) * a.num_kv_heads + kvh) * score_stride + t0 + threadIdx.x;
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (t0 + threadIdx.x + k * kWeightThreads < L) out[k * kWeightThreads] += acc[k];
}

}  // namespace pa
