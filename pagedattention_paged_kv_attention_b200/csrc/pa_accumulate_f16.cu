// Weight-accumulating attention kernels instantiated for float16 queries (float16 or FP8-E4M3 caches).
#include "pa_weights_launch.cuh"

namespace pa {
cudaError_t launch_accumulate_f16(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, bool fp8_cache,
                                  int D, int G, int grid, cudaStream_t stream) {
  if (fp8_cache) return launch_attention<__half, __nv_fp8_e4m3, kDecodeWeights>(tk, tv, a, D, G, grid, stream);
  return launch_attention<__half, __half, kDecodeWeights>(tk, tv, a, D, G, grid, stream);
}
cudaError_t launch_finish_f16(const AttnArgs& a, int D, float* scores, long long score_stride, int max_context_len,
                              cudaStream_t stream) {
  return D == 128 ? launch_finish<__half, 128>(a, scores, score_stride, max_context_len, stream)
                  : launch_finish<__half, 64>(a, scores, score_stride, max_context_len, stream);
}
}  // namespace pa
