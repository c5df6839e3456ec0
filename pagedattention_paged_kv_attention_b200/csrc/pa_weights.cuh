// pa_weights.cuh -- attention weights added to the cached tokens' scores.
//
// A token's score is the sum of the softmax weights that queries have given it, per kv head:
//   scores[s][kvh][t] += sum_g 2^(z_gt - lse_g),   lse_g = m_g + log2 sum_t 2^(z_gt - m_g),
// over the query heads g of the kv head; z is the scaled score in log2 units. One decode step's z (every
// token of every head) and the softmax statistics of each context partition come from paged_attention_main's
// kDecodeWeights instantiations; the finish kernel joins the partitions' statistics and sums the heads' weights.
// A thread owns its tokens' scores and adds the heads in order, so results do not depend on timing. Bound by the
// scores' bytes, 4 written and 4 read per token and query head: profiled alone, 64 sequences of up to 1996 tokens,
// 32/32 heads, 14 us beside a main kernel of 210; 128 of up to 4092, 64/8 heads, 29 beside 206.
#pragma once

#include <math.h>

#include "pa_attention.cuh"

namespace pa {

constexpr int kWeightThreads = 128;
constexpr int kWeightRound = 4 * kWeightThreads;   // tokens of a CTA's round, 4 consecutive ones a thread
constexpr int kWeightTokens = 4 * kWeightRound;    // tokens of one CTA
constexpr int kWeightHeads = 64;                   // query heads whose statistics are joined at a time

// U: heads whose scores a thread has in flight. The first ones' scores and sums are fetched beside the statistics,
// so a CTA's first round costs one chain of loads.
template <int U>
__device__ __forceinline__ void weight_tokens(const AttnArgs& a, float* __restrict__ scores, long long score_stride,
                                              unsigned int chunk, int kvh, int s) {
  __shared__ float lse[kWeightHeads];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = a.context_lens[s];
  const long long t0 = static_cast<long long>(chunk) * kWeightTokens;
  if (L <= 0 || context_len_invalid(L, a) || t0 >= L) return;
  const int left = static_cast<int>(min(static_cast<long long>(kWeightTokens), L - t0));
  const int n_parts = (L - 1) / a.partition_size + 1;
  const size_t row0 = static_cast<size_t>(s) * a.num_heads + static_cast<size_t>(kvh) * a.group;
  // Rows of scores are padded to a multiple of 64, so the 16-byte reads past L stay inside them.
  const float* z = a.logits + row0 * a.logit_stride + t0;
  float* out = scores + (static_cast<size_t>(s) * a.num_kv_heads + kvh) * score_stride + t0;
  float4 zv[U];
  float old[4];
  auto fetch = [&](int g, int t) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t < left && g + u < a.group) zv[u] = *reinterpret_cast<const float4*>(z + (g + u) * a.logit_stride + t);
  };
  auto fetch_old = [&](int t) {
#pragma unroll
    for (int k = 0; k < 4; ++k) old[k] = t + k < left ? out[t + k] : 0.f;
  };
  int t = 4 * static_cast<int>(threadIdx.x);
  fetch(0, t);
  fetch_old(t);
  for (int g0 = 0; g0 < a.group; g0 += kWeightHeads) {
    const int heads = min(kWeightHeads, a.group - g0);
    if (g0 > 0) __syncthreads();
    for (int g = warp; g < heads; g += kWeightThreads / 32) {
      const float2* st = a.stats + (row0 + g0 + g) * a.num_partitions;
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
    for (t = 4 * static_cast<int>(threadIdx.x); t < left; t += kWeightRound) {
      const bool first = g0 == 0 && t < kWeightRound;
      if (!first) fetch_old(t);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int g = 0; g < heads; g += U) {
        if (!first || g > 0) fetch(g0 + g, t);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (g + u < heads) {
            const float e = lse[g + u];
            acc[0] += fast_exp2(zv[u].x - e);
            acc[1] += fast_exp2(zv[u].y - e);
            acc[2] += fast_exp2(zv[u].z - e);
            acc[3] += fast_exp2(zv[u].w - e);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (t + k < left) out[t + k] = old[k] + acc[k];
    }
  }
}

// What is left after the main kernel: the merge of the partitions (its first reduce_blocks CTAs; none with one
// partition) and the weights, side by side as neither needs the other.
template <typename QT, int D, bool SPLIT, int MAXP, int U>
__global__ void __launch_bounds__(kWeightThreads)
attention_finish_kernel(const AttnArgs a, float* scores, long long score_stride, unsigned int chunks,
                        unsigned int reduce_blocks) {
  static_assert(kWeightThreads == kReduceWarps * 32, "one block shape for both");
  grid_dependency_wait();
  grid_dependents_launch();
  if (blockIdx.x < reduce_blocks) {
    reduce_rows<QT, D, SPLIT, MAXP, false>(a, blockIdx.x);
    return;
  }
  unsigned int i = blockIdx.x - reduce_blocks;
  const unsigned int chunk = i % chunks;
  i /= chunks;
  weight_tokens<U>(a, scores, score_stride, chunk, static_cast<int>(i % a.num_kv_heads),
                   static_cast<int>(i / a.num_kv_heads));
}

}  // namespace pa
