// pa_prefill.cu -- C ABI of the causal paged prefill attention (include/pagedattn.h): validation before
// any CUDA call, TMA descriptors for the query and the two caches, and the launch of
// pa::pf::paged_prefill_kernel (pa_prefill.cuh, pa_prefill_launch.cuh).
#include "pa_prefill_launch.cuh"

extern "C" pa_status pa_paged_prefill(void* out, const void* query, pa_dtype q_dtype, const void* key_cache,
                                      const void* value_cache, pa_dtype kv_dtype, const float* k_scale,
                                      const float* v_scale, const int32_t* block_tables,
                                      int max_blocks_per_seq, const int32_t* context_lens, const int32_t* q_start,
                                      int num_seqs, int num_q_tokens, int num_heads, int num_kv_heads,
                                      int head_size, int block_size, int num_blocks, int max_q_len, float scale,
                                      void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  bool empty;
  const pa_status st = pa_host::check_prefill(
      out, query, q_dtype, key_cache, value_cache, kv_dtype, k_scale, v_scale, block_tables, max_blocks_per_seq,
      context_lens, q_start, num_seqs, num_q_tokens, num_heads, num_kv_heads, head_size, block_size, num_blocks,
      max_q_len, scale, workspace, workspace_bytes, PA_WORKSPACE_HEADER_BYTES, &empty);
  if (st != PA_OK || empty) return st;
  pa_host::PrefillLaunch l;
  const pa_status built = pa_host::build_prefill(
      &l, out, query, key_cache, value_cache, kv_dtype, k_scale, v_scale, block_tables, max_blocks_per_seq,
      context_lens, q_start, num_seqs, num_q_tokens, num_heads, num_kv_heads, head_size, block_size, num_blocks,
      max_q_len, scale, workspace);
  if (built != PA_OK) return built;
  const cudaError_t e = pa_host::launch_prefill<pa::pf::kCausal>(l, q_dtype, kv_dtype, head_size,
                                                                 reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
