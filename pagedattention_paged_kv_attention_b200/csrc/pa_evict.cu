// pa_evict.cu -- C ABI of the eviction by accumulated attention weight (include/pagedattn.h): validation
// before any CUDA call, then pa::evict_kernel (pa_evict.cuh).
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_evict.cuh"
#include "pa_host_util.h"
#include "pagedattn.h"

using pa_host::aligned;

extern "C" pa_status pa_evict_tokens(int32_t* kept, int32_t* new_lens, float* scores_out, const float* scores,
                                     int score_stride, void* key_cache, void* value_cache, pa_dtype kv_dtype,
                                     const int32_t* block_tables, int max_blocks_per_seq,
                                     const int32_t* dst_block_tables, int max_dst_blocks_per_seq,
                                     const int32_t* context_lens, int num_seqs, int num_kv_heads, int head_size,
                                     int block_size, int num_blocks, int max_context_len, int budget, int num_sink,
                                     int num_recent, void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  if (num_seqs < 0 || num_kv_heads <= 0 || head_size <= 0 || block_size <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0 || max_dst_blocks_per_seq <= 0 || max_context_len < 0 || budget <= 0 || num_sink < 0 ||
      num_recent < 0 || static_cast<int64_t>(num_sink) + num_recent > budget || score_stride <= 0 ||
      score_stride < max_context_len || !pa_host::is_dtype(kv_dtype))
    return PA_ERR_INVALID_ARGUMENT;
  // The kept tokens have to fit their destination table.
  if (std::min(budget, max_context_len) > static_cast<int64_t>(max_dst_blocks_per_seq) * block_size)
    return PA_ERR_INVALID_ARGUMENT;
  if (num_seqs == 0) return PA_OK;
  if (!kept || !new_lens || !scores_out || !scores || !key_cache || !value_cache || !block_tables ||
      !dst_block_tables || !context_lens || !workspace)
    return PA_ERR_INVALID_ARGUMENT;
  if (!aligned(kept, 4) || !aligned(new_lens, 4) || !aligned(scores_out, 4) || !aligned(scores, 4) ||
      !aligned(key_cache, 16) || !aligned(value_cache, 16) || !aligned(block_tables, 4) ||
      !aligned(dst_block_tables, 4) || !aligned(context_lens, 4) || !aligned(workspace, 16))
    return PA_ERR_INVALID_ARGUMENT;
  if (new_lens == context_lens) return PA_ERR_INVALID_ARGUMENT;  // other CTAs still read the old lengths
  if (workspace_bytes < PA_WORKSPACE_HEADER_BYTES) return PA_ERR_WORKSPACE_TOO_SMALL;
  // A token that moves to another block would need its codes scaled anew.
  if (kv_dtype == PA_FP8_E4M3_BLOCK) return PA_ERR_UNSUPPORTED;
  const int64_t row_bytes = static_cast<int64_t>(head_size) * pa_host::elem_bytes(kv_dtype);
  if (row_bytes % 16 != 0 || row_bytes > 1024 || num_seqs > 65535 || num_kv_heads > 65535 || score_stride > (1 << 30) ||
      budget > (1 << 30) || static_cast<int64_t>(num_blocks) * block_size >= pa::kNoMove)
    return PA_ERR_UNSUPPORTED;

  pa::EvictArgs a{};
  a.kept = kept;
  a.new_lens = new_lens;
  a.scores_out = scores_out;
  a.scores = scores;
  a.key_cache = static_cast<uint8_t*>(key_cache);
  a.value_cache = static_cast<uint8_t*>(value_cache);
  a.block_tables = block_tables;
  a.dst_tables = dst_block_tables;
  a.context_lens = context_lens;
  a.error_word = static_cast<unsigned int*>(workspace);
  a.score_stride = score_stride;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_dst_blocks_per_seq = max_dst_blocks_per_seq;
  a.num_kv_heads = num_kv_heads;
  a.row_bytes = static_cast<int>(row_bytes);
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.max_context_len = max_context_len;
  a.budget = budget;
  a.num_sink = num_sink;
  a.num_recent = num_recent;
  a.log_block = -1;
  for (int i = 0; i < 31; ++i)
    if (block_size == 1 << i) a.log_block = i;
  // A row's strip is as wide as the row up to 256 bytes: whole 128-byte lines a request.
  a.log_lanes = pa::kMoveMinLogLanes;
  while (a.log_lanes < 4 && (16 << a.log_lanes) < row_bytes) ++a.log_lanes;
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms <= 0)
    return PA_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const unsigned heads = static_cast<unsigned>(num_kv_heads), seqs = static_cast<unsigned>(num_seqs);
  // As many CTAs a row as the GPU holds at once, so that no row waits for another's CTAs (16 rows of 16384 tokens
  // x 8 heads, cut to 2048, into other blocks and in place: 4 CTAs 69 and 68 us, 2 CTAs 78 and 91, 8 CTAs, two waves,
  // 79 and 82), but none without a share.
  const int64_t fit = static_cast<int64_t>(sms) * pa::kEvictPerSm / (static_cast<int64_t>(heads) * seqs);
  const int64_t share = pa_host::ceil_div(max_context_len, pa::kEvictShare);
  const unsigned cluster = static_cast<unsigned>(
      std::max<int64_t>(1, std::min<int64_t>(pa::kEvictCluster, std::min(fit, share))));
  const cudaError_t e = pa_host::launch_overlapped_clusters(cluster, pa::evict_kernel, dim3(cluster, heads, seqs),
                                                            dim3(pa::kEvictThreads), 0, st, a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
