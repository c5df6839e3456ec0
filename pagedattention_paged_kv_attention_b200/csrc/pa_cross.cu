// pa_cross.cu -- C ABI of cross attention over an encoder's cached states (include/pagedattn.h): validation
// before any CUDA call, paged_prefill_kernel in its kCross mode, and the join of split keys (pa_cross.cuh).
#include "pa_cross.cuh"
#include "pa_prefill_launch.cuh"

namespace {

// How a call's keys are split. Enough CTAs for every SM twice over when the batch has few query tiles, at
// least four key tiles each.
struct CrossPlan {
  int splits, split_tiles;
  size_t part_m, part_l, part_o, total;
};

CrossPlan plan_cross(int num_seqs, int num_q_tokens, int num_heads, int num_kv_heads, int head_size, int max_q_len,
                     int max_context_len) {
  CrossPlan p{};
  const int tile_tokens = std::max(1, pa::pf::kRows / (num_heads / num_kv_heads));
  const long long ctas = static_cast<long long>(pa_host::ceil_div(max_q_len, tile_tokens * pa::pf::kTiles)) *
                         num_kv_heads * num_seqs;
  const int tiles = std::max(1, pa_host::ceil_div(max_context_len, pa::pf::kKvTile));
  const long long want = ctas > 0 ? (2 * pa_host::kPlanSMs + ctas - 1) / ctas : 1;
  const int splits = static_cast<int>(std::max<long long>(1, std::min<long long>(want, tiles / 4)));
  p.split_tiles = pa_host::ceil_div(tiles, splits);
  p.splits = pa_host::ceil_div(tiles, p.split_tiles);
  p.part_m = PA_WORKSPACE_HEADER_BYTES;
  const size_t rows = p.splits > 1 ? static_cast<size_t>(num_q_tokens) * num_heads * p.splits : 0;
  p.part_l = p.part_m + pa_host::round_up(rows * sizeof(float), 256);
  p.part_o = p.part_l + pa_host::round_up(rows * sizeof(float), 256);
  p.total = p.part_o + rows * head_size * sizeof(float);
  return p;
}

template <typename T>
cudaError_t launch_merge(const pa::pf::PrefillArgs& a, int head_size, cudaStream_t st) {
  // Every chunk that the tiles cover.
  const long long rows = static_cast<long long>(a.num_pairs) * pa::pf::kTiles * a.tile_tokens * a.num_heads;
  const dim3 grid(static_cast<unsigned>((rows + pa::pf::kMergeWarps - 1) / pa::pf::kMergeWarps),
                  static_cast<unsigned>(a.num_seqs));
  const dim3 block(pa::pf::kMergeWarps * 32);
  return head_size == 128 ? pa_host::launch_plain(pa::pf::cross_merge_kernel<T, 128>, grid, block, 0, st, a)
                          : pa_host::launch_plain(pa::pf::cross_merge_kernel<T, 64>, grid, block, 0, st, a);
}

}  // namespace

extern "C" {

size_t pa_paged_cross_attention_workspace_size(int num_seqs, int num_q_tokens, int num_heads, int num_kv_heads,
                                               int head_size, int max_q_len, int max_context_len) {
  if (num_seqs < 0 || num_q_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
      head_size <= 0 || max_q_len < 0 || max_context_len < 0)
    return 0;
  const size_t tiles =
      plan_cross(num_seqs, num_q_tokens, num_heads, num_kv_heads, head_size, max_q_len, max_context_len).total;
  if (max_q_len > 1) return tiles;
  return std::max(tiles,
                  pa_host::decode_rows_workspace(num_seqs, num_heads, num_kv_heads, head_size, max_context_len));
}

pa_status pa_paged_cross_attention(void* out, const void* query, pa_dtype q_dtype, const void* key_cache,
                                   const void* value_cache, pa_dtype kv_dtype, const float* k_scale,
                                   const float* v_scale, const int32_t* block_tables, int max_blocks_per_seq,
                                   const int32_t* context_lens, const int32_t* q_start, int num_seqs, int num_q_tokens,
                                   int num_heads, int num_kv_heads, int head_size, int block_size, int num_blocks,
                                   int max_q_len, int max_context_len, float scale, void* workspace,
                                   size_t workspace_bytes, pa_stream_t stream) {
  if (max_context_len < 0) return PA_ERR_INVALID_ARGUMENT;
  const size_t need = pa_paged_cross_attention_workspace_size(num_seqs, num_q_tokens, num_heads, num_kv_heads,
                                                              head_size, max_q_len, max_context_len);
  bool empty;
  const pa_status checked = pa_host::check_prefill(
      out, query, q_dtype, key_cache, value_cache, kv_dtype, k_scale, v_scale, block_tables, max_blocks_per_seq,
      context_lens, q_start, num_seqs, num_q_tokens, num_heads, num_kv_heads, head_size, block_size, num_blocks,
      max_q_len, scale, workspace, workspace_bytes, need, &empty);
  if (checked != PA_OK || empty) return checked;
  // Single tokens are bound by the states' bytes: the decode kernel reads them at 82% of the copy bandwidth, a
  // tile of 128 query rows with few of them used at half (32 sequences, 8 kv heads, up to 6404 states: 87 and
  // 135 us).
  if (max_q_len == 1 && pa_host::decode_rows_supported(block_size, num_blocks))
    return pa_host::decode_rows(out, query, q_dtype, key_cache, value_cache, kv_dtype, k_scale, v_scale, block_tables,
                                max_blocks_per_seq, context_lens, q_start, num_seqs, num_q_tokens, num_heads,
                                num_kv_heads, head_size, block_size, num_blocks, max_context_len, scale, workspace,
                                stream);
  pa_host::PrefillLaunch l;
  const pa_status built = pa_host::build_prefill(
      &l, out, query, key_cache, value_cache, kv_dtype, k_scale, v_scale, block_tables, max_blocks_per_seq,
      context_lens, q_start, num_seqs, num_q_tokens, num_heads, num_kv_heads, head_size, block_size, num_blocks,
      max_q_len, scale, workspace);
  if (built != PA_OK) return built;
  const CrossPlan p =
      plan_cross(num_seqs, num_q_tokens, num_heads, num_kv_heads, head_size, max_q_len, max_context_len);
  uint8_t* wsb = static_cast<uint8_t*>(workspace);
  l.a.splits = p.splits;
  l.a.split_tiles = p.split_tiles;
  l.a.max_context_len = max_context_len;
  l.a.part_m = reinterpret_cast<float*>(wsb + p.part_m);
  l.a.part_l = reinterpret_cast<float*>(wsb + p.part_l);
  l.a.part_o = reinterpret_cast<float*>(wsb + p.part_o);
  if (static_cast<long long>(l.grid.x) * p.splits > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
  l.grid.x *= static_cast<unsigned>(p.splits);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = pa_host::launch_prefill<pa::pf::kCross>(l, q_dtype, kv_dtype, head_size, st);
  if (e == cudaSuccess && p.splits > 1)
    e = q_dtype == PA_BF16 ? launch_merge<__nv_bfloat16>(l.a, head_size, st)
                           : launch_merge<__half>(l.a, head_size, st);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // extern "C"
