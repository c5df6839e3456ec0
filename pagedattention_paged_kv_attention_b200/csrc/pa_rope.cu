// pa_rope.cu -- C ABI of the rotary cache write (include/pagedattn.h): validation before any CUDA call
// and the launch of pa::rope_reshape_and_cache_kernel (pa_rope.cuh).
#include <cuda_runtime.h>

#include <algorithm>

#include "pa_host_util.h"
#include "pa_rope.cuh"
#include "pagedattn.h"

namespace {

using pa_host::aligned;
using pa_host::is_16bit;
using pa_host::is_dtype;

constexpr int64_t kMaxRowElems = int64_t(1) << 24;  // elements of one token's row that are indexed with int

template <typename T, typename KVT>
cudaError_t launch_rope(const pa::RopeArgs& a, bool interleaved, cudaStream_t st) {
  const unsigned tokens = static_cast<unsigned>(a.num_tokens);
  const int64_t units = static_cast<int64_t>(a.num_heads + a.num_kv_heads) * a.units +
                        static_cast<int64_t>(a.num_kv_heads) * a.head_size / 8;
  const unsigned threads = static_cast<unsigned>(std::min<int64_t>(pa::kRopeThreads, (units + 31) / 32 * 32));
  if (interleaved)
    return pa_host::launch_overlapped(pa::rope_reshape_and_cache_kernel<T, KVT, true>, dim3(tokens),
                                      dim3(threads), 0, st, a);
  return pa_host::launch_overlapped(pa::rope_reshape_and_cache_kernel<T, KVT, false>, dim3(tokens),
                                    dim3(threads), 0, st, a);
}

}  // namespace

extern "C" pa_status pa_rope_reshape_and_cache(
    void* query_out, int64_t query_out_stride, const void* query, int64_t query_stride, const void* key,
    int64_t key_stride, const void* value, int64_t value_stride, pa_dtype in_dtype, void* key_cache, void* value_cache,
    pa_dtype kv_dtype, const float* k_scale, const float* v_scale, const int64_t* slot_mapping,
    const int32_t* positions, int num_axes, const float* inv_freq, const int32_t* freq_axis, int rotary_size,
    int interleaved, int num_tokens, int num_heads, int num_kv_heads, int head_size, int block_size, int num_blocks,
    pa_stream_t stream) {
  if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_size <= 0 || block_size <= 0 || num_blocks <= 0 ||
      num_axes <= 0 || rotary_size <= 0 || rotary_size > head_size || rotary_size % 2 != 0 ||
      (interleaved != 0 && interleaved != 1))
    return PA_ERR_INVALID_ARGUMENT;
  if (!is_dtype(in_dtype) || !is_dtype(kv_dtype) || !is_16bit(in_dtype)) return PA_ERR_INVALID_ARGUMENT;
  if (num_tokens == 0) return PA_OK;  // empty batch: nothing is read, pointers may be null
  if (!query_out || !query || !key || !value || !key_cache || !value_cache || !slot_mapping || !positions ||
      !inv_freq || !freq_axis)
    return PA_ERR_INVALID_ARGUMENT;
  if (!aligned(query_out, 16) || !aligned(query, 16) || !aligned(key, 16) || !aligned(value, 16) ||
      !aligned(key_cache, 16) || !aligned(value_cache, 16) || !aligned(slot_mapping, 8) || !aligned(positions, 4) ||
      !aligned(inv_freq, 4) || !aligned(freq_axis, 4))
    return PA_ERR_INVALID_ARGUMENT;
  const int64_t q_row = static_cast<int64_t>(num_heads) * head_size;
  const int64_t kv_row = static_cast<int64_t>(num_kv_heads) * head_size;
  // Rows may lie further apart than their own width (slices of one fused projection), in 16-byte steps.
  if (query_out_stride < q_row || query_stride < q_row || key_stride < kv_row || value_stride < kv_row)
    return PA_ERR_INVALID_ARGUMENT;
  if (query_out == query && query_out_stride != query_stride) return PA_ERR_INVALID_ARGUMENT;
  const bool fp8 = pa_host::is_fp8(kv_dtype);
  if (fp8 && (!k_scale || !v_scale || !aligned(k_scale, 4) || !aligned(v_scale, 4))) return PA_ERR_INVALID_ARGUMENT;
  if (!fp8 && kv_dtype != in_dtype) return PA_ERR_UNSUPPORTED;
  if (head_size % 8 != 0 || rotary_size % 16 != 0 || rotary_size > pa::kRopeMaxRotary ||
      head_size > pa::kRopeMaxHead || q_row > kMaxRowElems || kv_row > kMaxRowElems)
    return PA_ERR_UNSUPPORTED;
  if (query_out_stride % 8 != 0 || query_stride % 8 != 0 || key_stride % 8 != 0 || value_stride % 8 != 0)
    return PA_ERR_UNSUPPORTED;

  pa::RopeArgs a{};
  a.query_out = query_out;
  a.query = query;
  a.key = key;
  a.value = value;
  a.key_cache = key_cache;
  a.value_cache = value_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.slot_mapping = slot_mapping;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.freq_axis = freq_axis;
  a.query_out_stride = query_out_stride;
  a.query_stride = query_stride;
  a.key_stride = key_stride;
  a.value_stride = value_stride;
  a.num_tokens = num_tokens;
  a.num_axes = num_axes;
  a.num_heads = num_heads;
  a.num_kv_heads = num_kv_heads;
  a.head_size = head_size;
  a.rotary = rotary_size;
  a.units = rotary_size / (interleaved ? 8 : 16) + (head_size - rotary_size) / 8;
  auto reciprocal = [](int n) { return static_cast<unsigned>(((uint64_t(1) << 32) + n - 1) / n); };
  a.inv_units = reciprocal(a.units);
  a.inv_plain = reciprocal(head_size / 8);
  a.block_size = block_size;
  a.num_blocks = num_blocks;
  a.scale_stride = pa_host::scale_block_stride(kv_dtype, num_kv_heads);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (in_dtype == PA_BF16)
    e = fp8 ? launch_rope<__nv_bfloat16, __nv_fp8_e4m3>(a, interleaved != 0, st)
            : launch_rope<__nv_bfloat16, __nv_bfloat16>(a, interleaved != 0, st);
  else
    e = fp8 ? launch_rope<__half, __nv_fp8_e4m3>(a, interleaved != 0, st)
            : launch_rope<__half, __half>(a, interleaved != 0, st);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
