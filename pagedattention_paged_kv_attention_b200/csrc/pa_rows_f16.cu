// Decode attention over rows found by q_start (cross attention of single tokens), for float16 queries.
#include "pa_launch.cuh"

namespace pa {
cudaError_t launch_rows_f16(const CUtensorMap& tk, const CUtensorMap& tv, const AttnArgs& a, bool fp8_cache, int D,
                         int G, int grid, cudaStream_t stream) {
  if (fp8_cache) return launch_attention<__half, __nv_fp8_e4m3, kDecodeRows>(tk, tv, a, D, G, grid, stream);
  return launch_attention<__half, __half, kDecodeRows>(tk, tv, a, D, G, grid, stream);
}
}  // namespace pa
