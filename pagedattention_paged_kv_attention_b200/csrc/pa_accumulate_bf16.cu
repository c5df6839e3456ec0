// Weight-accumulating attention kernels instantiated for bfloat16 queries (bfloat16 or FP8-E4M3 caches).
#include "pa_weights_launch.cuh"

namespace pa {
cudaError_t launch_accumulate_bf16(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, bool fp8_cache,
                                  int D, int G, int grid, cudaStream_t stream) {
  if (fp8_cache) return launch_attention<__nv_bfloat16, __nv_fp8_e4m3, kDecodeWeights>(tk, tv, a, D, G, grid, stream);
  return launch_attention<__nv_bfloat16, __nv_bfloat16, kDecodeWeights>(tk, tv, a, D, G, grid, stream);
}
cudaError_t launch_finish_bf16(const AttnArgs& a, int D, float* scores, long long score_stride, int max_context_len,
                              cudaStream_t stream) {
  return D == 128 ? launch_finish<__nv_bfloat16, 128>(a, scores, score_stride, max_context_len, stream)
                  : launch_finish<__nv_bfloat16, 64>(a, scores, score_stride, max_context_len, stream);
}
}  // namespace pa
