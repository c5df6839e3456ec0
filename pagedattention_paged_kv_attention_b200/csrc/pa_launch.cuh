// pa_launch.cuh -- host-side launch of the attention kernels for one (query dtype, cache dtype) pair.
// Included by the per-dtype translation units so that their template instantiations compile in
// parallel.
#pragma once

#include <cuda_runtime.h>

#include "pa_attention.cuh"
#include "pa_host_util.h"

namespace pa {

// The split-K merge of a launch with more than one partition.
template <typename QT, int D, bool ROWS = false>
cudaError_t launch_reduce(const AttnArgs& a, cudaStream_t stream) {
  const long rows = static_cast<long>(a.num_heads) * a.num_seqs;
  if (a.num_partitions > kReduceSplitAbove)
    return pa_host::launch_overlapped(paged_attention_reduce<QT, D, true, kReduceSplitAbove, ROWS>,
                                      dim3(static_cast<unsigned>(rows)), dim3(kReduceWarps * 32), 0, stream, a);
  const dim3 grid(static_cast<unsigned>((rows + kReduceWarps - 1) / kReduceWarps));
  if (a.num_partitions <= 4)
    return pa_host::launch_overlapped(paged_attention_reduce<QT, D, false, 4, ROWS>, grid, dim3(kReduceWarps * 32), 0,
                                      stream, a);
  if (a.num_partitions <= 8)
    return pa_host::launch_overlapped(paged_attention_reduce<QT, D, false, 8, ROWS>, grid, dim3(kReduceWarps * 32), 0,
                                      stream, a);
  return pa_host::launch_overlapped(paged_attention_reduce<QT, D, false, 16, ROWS>, grid, dim3(kReduceWarps * 32), 0,
                                    stream, a);
}

// kDecodeWeights: the caller launches the kernel that merges and forms the weights.
template <typename QT, typename KVT, int D, int G, bool BS = false, int MODE = kDecode>
cudaError_t launch_attention_one(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, int grid,
                                 cudaStream_t stream) {
  constexpr int EB = Elem<KVT>::kBytes;
  constexpr size_t smem = Layout<QT, D, G, EB>::kAllocBytes;
  auto kernel = paged_attention_main<QT, KVT, D, G, BS, MODE>;
  // The attribute is per device; setting it on every call costs a few microseconds of host time at
  // most and keeps multi-device processes correct.
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  e = pa_host::launch_overlapped(kernel, dim3(grid), dim3(kThreads), smem, stream, tk, tv, a);
  if (e != cudaSuccess) return e;
  if constexpr (MODE != kDecodeWeights) {
    if (a.num_partitions > 1) e = launch_reduce<QT, D, MODE == kDecodeRows>(a, stream);
  }
  return e;
}

template <typename QT, typename KVT, int MODE = kDecode>
cudaError_t launch_attention(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, int D, int G,
                             int grid, cudaStream_t stream) {
  if constexpr (sizeof(KVT) == 1) {
    if (D == 128 && a.scale_block_stride != 0) {  // per-block scales
      switch (G) {
        case 1: return launch_attention_one<QT, KVT, 128, 1, true, MODE>(tk, tv, a, grid, stream);
        case 2: return launch_attention_one<QT, KVT, 128, 2, true, MODE>(tk, tv, a, grid, stream);
        case 4: return launch_attention_one<QT, KVT, 128, 4, true, MODE>(tk, tv, a, grid, stream);
        case 8: return launch_attention_one<QT, KVT, 128, 8, true, MODE>(tk, tv, a, grid, stream);
      }
    } else if (D == 128) {
      switch (G) {
        case 1: return launch_attention_one<QT, KVT, 128, 1, false, MODE>(tk, tv, a, grid, stream);
        case 2: return launch_attention_one<QT, KVT, 128, 2, false, MODE>(tk, tv, a, grid, stream);
        case 4: return launch_attention_one<QT, KVT, 128, 4, false, MODE>(tk, tv, a, grid, stream);
        case 8: return launch_attention_one<QT, KVT, 128, 8, false, MODE>(tk, tv, a, grid, stream);
      }
    }
  } else {
    if (D == 128) {
      switch (G) {
        case 1: return launch_attention_one<QT, KVT, 128, 1, false, MODE>(tk, tv, a, grid, stream);
        case 2: return launch_attention_one<QT, KVT, 128, 2, false, MODE>(tk, tv, a, grid, stream);
        case 4: return launch_attention_one<QT, KVT, 128, 4, false, MODE>(tk, tv, a, grid, stream);
        case 8: return launch_attention_one<QT, KVT, 128, 8, false, MODE>(tk, tv, a, grid, stream);
      }
    } else if (D == 64) {
      switch (G) {
        case 1: return launch_attention_one<QT, KVT, 64, 1, false, MODE>(tk, tv, a, grid, stream);
        case 2: return launch_attention_one<QT, KVT, 64, 2, false, MODE>(tk, tv, a, grid, stream);
        case 4: return launch_attention_one<QT, KVT, 64, 4, false, MODE>(tk, tv, a, grid, stream);
        case 8: return launch_attention_one<QT, KVT, 64, 8, false, MODE>(tk, tv, a, grid, stream);
      }
    }
  }
  return cudaErrorInvalidValue;
}

// Per-dtype entry points (defined in pa_attention_<dtype>.cu).
cudaError_t launch_attention_bf16(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, bool fp8_cache,
                                  int D, int G, int grid, cudaStream_t stream);
cudaError_t launch_attention_f16(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, bool fp8_cache,
                                 int D, int G, int grid, cudaStream_t stream);

// The launches of the other modes (pa_rows_<dtype>.cu, pa_accumulate_<dtype>.cu), and the kernel that follows the
// weight-scoring one: the merge and the weights.
cudaError_t launch_finish_bf16(const AttnArgs& a, int D, float* scores, long long score_stride, int max_context_len,
                               cudaStream_t stream);
cudaError_t launch_finish_f16(const AttnArgs& a, int D, float* scores, long long score_stride, int max_context_len,
                              cudaStream_t stream);
cudaError_t launch_rows_bf16(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, bool fp8_cache, int D,
                             int G, int grid, cudaStream_t stream);
cudaError_t launch_rows_f16(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, bool fp8_cache, int D,
                            int G, int grid, cudaStream_t stream);
cudaError_t launch_accumulate_bf16(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, bool fp8_cache,
                                   int D, int G, int grid, cudaStream_t stream);
cudaError_t launch_accumulate_f16(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, bool fp8_cache,
                                  int D, int G, int grid, cudaStream_t stream);

}  // namespace pa
