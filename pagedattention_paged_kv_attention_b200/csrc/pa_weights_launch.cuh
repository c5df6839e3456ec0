// pa_weights_launch.cuh -- host-side launch of the kernel that ends a weight-scoring step, included by
// pa_accumulate_<dtype>.cu so that the query dtypes build in parallel.
#pragma once

#include "pa_launch.cuh"
#include "pa_weights.cuh"

namespace pa {

template <typename QT, int D, bool SPLIT, int MAXP, int U>
cudaError_t launch_finish_one(const AttnArgs& a, float* scores, long long score_stride, unsigned chunks,
                              unsigned reduce_blocks, unsigned blocks, cudaStream_t stream) {
  return pa_host::launch_overlapped(attention_finish_kernel<QT, D, SPLIT, MAXP, U>, dim3(blocks), dim3(kWeightThreads),
                                    0, stream, a, scores, score_stride, chunks, reduce_blocks);
}

template <typename QT, int D, int U>
cudaError_t launch_finish_heads(const AttnArgs& a, float* scores, long long score_stride, unsigned chunks,
                                unsigned weight_blocks, cudaStream_t stream) {
  const unsigned rows = static_cast<unsigned>(a.num_heads) * static_cast<unsigned>(a.num_seqs);
  const unsigned merges = a.num_partitions == 1 ? 0 : (rows + kReduceWarps - 1) / kReduceWarps;
  if (a.num_partitions > kReduceSplitAbove)
    return launch_finish_one<QT, D, true, kReduceSplitAbove, U>(a, scores, score_stride, chunks, rows,
                                                                weight_blocks + rows, stream);
  if (a.num_partitions <= 4)
    return launch_finish_one<QT, D, false, 4, U>(a, scores, score_stride, chunks, merges, weight_blocks + merges, stream);
  if (a.num_partitions <= 8)
    return launch_finish_one<QT, D, false, 8, U>(a, scores, score_stride, chunks, merges, weight_blocks + merges, stream);
  return launch_finish_one<QT, D, false, 16, U>(a, scores, score_stride, chunks, merges, weight_blocks + merges, stream);
}

// max_context_len > 0; the caller has checked that the blocks fit a grid.
template <typename QT, int D>
cudaError_t launch_finish(const AttnArgs& a, float* scores, long long score_stride, int max_context_len,
                          cudaStream_t stream) {
  const unsigned chunks = static_cast<unsigned>(pa_host::ceil_div(max_context_len, kWeightTokens));
  const unsigned blocks = chunks * static_cast<unsigned>(a.num_kv_heads) * static_cast<unsigned>(a.num_seqs);
  if (a.group == 1) return launch_finish_heads<QT, D, 1>(a, scores, score_stride, chunks, blocks, stream);
  if (a.group == 2) return launch_finish_heads<QT, D, 2>(a, scores, score_stride, chunks, blocks, stream);
  if (a.group <= 4) return launch_finish_heads<QT, D, 4>(a, scores, score_stride, chunks, blocks, stream);
  return launch_finish_heads<QT, D, 8>(a, scores, score_stride, chunks, blocks, stream);
}

}  // namespace pa
