// pa_prefill_accumulate.cu -- C ABI of the causal prefill that adds its attention weights to the cached tokens'
// scores (include/pagedattn.h): paged_prefill_kernel with row statistics, then prefill_weights_kernel.
#include "pa_prefill_launch.cuh"
#include "pa_prefill_weights.cuh"

namespace {

size_t layout_bytes(int num_q_tokens, int num_heads) {
  return PA_WORKSPACE_HEADER_BYTES +
         pa_host::round_up(static_cast<size_t>(num_q_tokens) * num_heads * sizeof(float), 256);
}

template <typename T, int D, int KVB>
cudaError_t launch_weights_one(const pa_host::PrefillLaunch& l, const pa::pf::WeightArgs& wa, dim3 grid,
                               cudaStream_t st) {
  auto kernel = pa::pf::prefill_weights_kernel<T, D, KVB>;
  const int smem = static_cast<int>(pa::pf::WLayout<D>::kBytes);
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return pa_host::launch_plain(kernel, grid, dim3(pa::pf::kWThreads), static_cast<size_t>(smem), st, l.tq, l.tk, l.a,
                               wa);
}

template <typename T>
cudaError_t launch_weights(const pa_host::PrefillLaunch& l, const pa::pf::WeightArgs& wa, dim3 grid, pa_dtype kv_dtype,
                           int head_size, cudaStream_t st) {
  if (pa_host::is_fp8(kv_dtype)) return launch_weights_one<T, 128, 1>(l, wa, grid, st);
  return head_size == 128 ? launch_weights_one<T, 128, 2>(l, wa, grid, st)
                          : launch_weights_one<T, 64, 2>(l, wa, grid, st);
}

}  // namespace

extern "C" {

size_t pa_paged_prefill_accumulate_workspace_size(int num_q_tokens, int num_heads) {
  return num_q_tokens < 0 || num_heads <= 0 ? 0 : layout_bytes(num_q_tokens, num_heads);
}

pa_status pa_paged_prefill_accumulate(void* out, float* scores, int score_stride, const void* query, pa_dtype q_dtype,
                                      const void* key_cache, const void* value_cache, pa_dtype kv_dtype,
                                      const float* k_scale, const float* v_scale, const int32_t* block_tables,
                                      int max_blocks_per_seq, const int32_t* context_lens, const int32_t* q_start,
                                      int num_seqs, int num_q_tokens, int num_heads, int num_kv_heads, int head_size,
                                      int block_size, int num_blocks, int max_q_len, int max_context_len, int window,
                                      float scale, void* workspace, size_t workspace_bytes, pa_stream_t stream) {
  if (max_context_len < 0 || window < 0 || score_stride <= 0 || score_stride < max_context_len)
    return PA_ERR_INVALID_ARGUMENT;
  bool empty;
  const pa_status checked = pa_host::check_prefill(
      out, query, q_dtype, key_cache, value_cache, kv_dtype, k_scale, v_scale, block_tables, max_blocks_per_seq,
      context_lens, q_start, num_seqs, num_q_tokens, num_heads, num_kv_heads, head_size, block_size, num_blocks,
      max_q_len, scale, workspace, workspace_bytes, layout_bytes(std::max(0, num_q_tokens), std::max(1, num_heads)),
      &empty);
  if (checked != PA_OK || empty) return checked;
  if (!scores || !pa_host::aligned(scores, 4)) return PA_ERR_INVALID_ARGUMENT;
  const int key_tiles = pa_host::ceil_div(max_context_len, pa::pf::kKvTile);
  const int64_t items = static_cast<int64_t>(key_tiles) * num_seqs * num_kv_heads;
  if (items > 0x3fffffff) return PA_ERR_UNSUPPORTED;
  pa_host::PrefillLaunch l;
  const pa_status built = pa_host::build_prefill(
      &l, out, query, key_cache, value_cache, kv_dtype, k_scale, v_scale, block_tables, max_blocks_per_seq,
      context_lens, q_start, num_seqs, num_q_tokens, num_heads, num_kv_heads, head_size, block_size, num_blocks,
      max_q_len, scale, workspace);
  if (built != PA_OK) return built;
  l.a.lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + PA_WORKSPACE_HEADER_BYTES);
  l.a.max_context_len = max_context_len;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = pa_host::launch_prefill<pa::pf::kCausalStats>(l, q_dtype, kv_dtype, head_size, st);
  if (e == cudaSuccess && key_tiles > 0) {
    pa::pf::WeightArgs wa{};
    wa.scores = scores;
    wa.score_stride = score_stride;
    wa.lse = l.a.lse;
    wa.window = window;
    wa.num_items = static_cast<unsigned>(items);
    const int counted = window > 0 ? std::min(window, max_q_len) : max_q_len;
    wa.draw = pa_host::ceil_div(counted, l.a.tile_tokens) > pa::pf::kDealTiles;
    int device = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms <= 0)
      return PA_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(sms, items)));
    e = q_dtype == PA_BF16 ? launch_weights<__nv_bfloat16>(l, wa, grid, kv_dtype, head_size, st)
                           : launch_weights<__half>(l, wa, grid, kv_dtype, head_size, st);
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
