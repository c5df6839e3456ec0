// pa_evict.cuh -- eviction of cached tokens by their accumulated attention weight.
//
// Per sequence s and kv head h, of the L cached tokens with scores w[t] at most `budget` stay: the first
// num_sink, the last num_recent, and of those in between the ones with the largest scores (equal scores:
// the lower index first; a NaN counts as -inf). The kept tokens move together in their order:
// token kept[j] becomes token j, in the destination table's blocks. Each head keeps tokens of its own;
// attention does not depend on which slot a key sits in, so heads need only agree on their number.
//
// evict_select_kernel finds the kept tokens: a radix selection of the q-th largest score on a monotone
// 32-bit image of the fp32 values, three digits of 11, 11 and 10 bits, then one ordered compaction.
// evict_move_kernel moves the rows. A kept token never moves up (kept[j] >= j), so a warp that walks j
// upwards, reading a group of rows before it writes them, may write over the very blocks it reads:
// a slot it writes is a source only of rows it has read already.
#pragma once

#include <math.h>

#include "pa_device.cuh"

namespace pa {

constexpr int kSelectThreads = 1024;
constexpr int kSelectBins = 2048;
constexpr int kMoveWarps = 8;
constexpr int kMoveRows = 8;          // rows of a warp's load: 4 lanes x 16 bytes each
constexpr int kMoveUnroll = 8;        // loads in flight per lane

struct EvictArgs {
  int32_t* kept;                // [S][Hkv][budget]
  int32_t* new_lens;            // [S]
  float* scores_out;            // [S][Hkv][score_stride]
  const float* scores;
  uint8_t* key_cache;
  uint8_t* value_cache;
  const int32_t* block_tables;  // [S][max_blocks_per_seq]
  const int32_t* dst_tables;    // [S][max_dst_blocks_per_seq]
  const int32_t* context_lens;  // [S]
  unsigned int* error_word;
  int score_stride, max_blocks_per_seq, max_dst_blocks_per_seq, num_kv_heads, row_bytes, block_size, num_blocks,
      max_context_len, budget, num_sink, num_recent;
};

__device__ __forceinline__ bool evict_len_invalid(int L, const EvictArgs& a) {
  return L < 0 || L > a.max_context_len ||
         static_cast<long long>(L) > static_cast<long long>(a.max_blocks_per_seq) * a.block_size;
}

// Larger float <=> larger unsigned key; -0 equals +0, NaN equals -inf.
__device__ __forceinline__ uint32_t score_key(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// One CTA per (kv head, sequence).
__global__ void __launch_bounds__(kSelectThreads)
evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[kSelectBins];
  __shared__ int warp_gt[kSelectThreads / 32], warp_eq[kSelectThreads / 32];
  __shared__ uint32_t sh_prefix;
  __shared__ int sh_need;
  grid_dependency_wait();
  grid_dependents_launch();
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const size_t rowi = static_cast<size_t>(s) * a.num_kv_heads + h;
  int32_t* kept = a.kept + rowi * a.budget;
  const float* w = a.scores + rowi * a.score_stride;
  float* wo = a.scores_out + rowi * a.score_stride;
  const int L = a.context_lens[s];
  if (evict_len_invalid(L, a)) {
    if (tid == 0) {
      atomicOr(a.error_word, PA_DEVERR_CONTEXT_LEN);
      if (h == 0) a.new_lens[s] = 0;
    }
    for (int j = tid; j < a.budget; j += kSelectThreads) kept[j] = -1;
    return;
  }
  const int n = min(L, a.budget);
  if (h == 0 && tid == 0) a.new_lens[s] = n;
  for (int j = n + tid; j < a.budget; j += kSelectThreads) kept[j] = -1;
  if (L <= a.budget) {
    for (int j = tid; j < n; j += kSelectThreads) kept[j] = j;
  } else {
    const int c0 = a.num_sink, c1 = L - a.num_recent;  // candidates; c1 - c0 > need as L > budget
    int need = a.budget - a.num_sink - a.num_recent;
    uint32_t prefix = 0;                               // leading digits of the need-th largest key
    int shift = 32;
    if (need > 0) {
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass < 2 ? 11 : 10, high = shift;
        shift -= bits;
        for (int i = tid; i < kSelectBins; i += kSelectThreads) hist[i] = 0;
        __syncthreads();
        for (int t = c0 + tid; t < c1; t += kSelectThreads) {
          const uint32_t k = score_key(w[t]);
          if (pass == 0 || (k >> high) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1);
        }
        __syncthreads();
        if (warp == 0) {  // the digit whose suffix count reaches `need`
          const int per = (1 << bits) / 32, top = (1 << bits) - 1;
          int sum = 0;
          for (int i = 0; i < per; ++i) sum += hist[top - (lane * per + i)];
          int incl = sum;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
          }
          int run = incl - sum;
          if (run < need && incl >= need) {
            int i = 0;
            while (run + hist[top - (lane * per + i)] < need) run += hist[top - (lane * per + i++)];
            sh_prefix = (prefix << bits) | static_cast<uint32_t>(top - (lane * per + i));
            sh_need = need - run;
          }
        }
        __syncthreads();
        prefix = sh_prefix;
        need = sh_need;
      }
    }
    // Kept: the ends, keys above the threshold `prefix`, and the first `need` equal to it (need == 0: no
    // candidate at all). Each warp takes a contiguous segment; counts first, then places.
    const bool any = a.budget > a.num_sink + a.num_recent;
    const int seg = (L + kSelectThreads - 1) / kSelectThreads * 32;
    const int t0 = min(L, warp * seg), t1 = min(L, t0 + seg);
    int gt = 0, eq = 0;
    for (int t = t0 + lane; t < t1; t += 32) {
      const bool end = t < c0 || t >= c1;
      const uint32_t k = score_key(w[t]);
      gt += end || (any && k > prefix);
      eq += !end && any && k == prefix;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
      warp_gt[warp] = gt;
      warp_eq[warp] = eq;
    }
    __syncthreads();
    int eq_before = lane < warp ? warp_eq[lane] : 0, gt_before = lane < warp ? warp_gt[lane] : 0;
    eq_before = __reduce_add_sync(0xffffffffu, eq_before);
    gt_before = __reduce_add_sync(0xffffffffu, gt_before);
    int place = gt_before + min(eq_before, need);
    const unsigned lt = (1u << lane) - 1u;
    for (int b = t0; b < t1; b += 32) {
      const int t = b + lane;
      const bool in = t < t1;
      const bool end = in && (t < c0 || t >= c1);
      const uint32_t k = in ? score_key(w[t]) : 0u;
      const bool is_eq = in && !end && any && k == prefix;
      const unsigned eqs = __ballot_sync(0xffffffffu, is_eq);
      const bool take = end || (in && any && k > prefix) || (is_eq && eq_before + __popc(eqs & lt) < need);
      const unsigned takes = __ballot_sync(0xffffffffu, take);
      if (take) kept[place + __popc(takes & lt)] = t;
      place += __popc(takes);
      eq_before += __popc(eqs);
    }
  }
  __syncthreads();
  // The scores move with their tokens, a group read before it is written (scores_out may be scores); the
  // rest of the row starts from zero.
  for (int b = 0; b < n; b += kSelectThreads) {
    const int j = b + tid;
    const float x = j < n ? w[kept[j]] : 0.f;
    __syncthreads();
    if (j < n) wo[j] = x;
  }
  __syncthreads();
  for (int j = n + tid; j < a.score_stride; j += kSelectThreads) wo[j] = 0.f;
}

// grid (kv heads, sequences, groups of kMoveWarps strips); each warp moves one 64-byte strip of the head's key or
// value rows.
__global__ void __launch_bounds__(kMoveWarps * 32)
evict_move_kernel(const EvictArgs a) {
  grid_dependency_wait();
  grid_dependents_launch();
  const int h = blockIdx.x, s = blockIdx.y, lane = threadIdx.x & 31;
  const int warp = blockIdx.z * kMoveWarps + (threadIdx.x >> 5);
  const int L = a.context_lens[s];
  const int strips = (a.row_bytes + 63) / 64;
  if (evict_len_invalid(L, a) || warp >= 2 * strips) return;
  const int n = min(L, a.budget);
  uint8_t* cache = warp < strips ? a.key_cache : a.value_cache;
  const int col = (warp % strips) * 64 + (lane & 3) * 16;
  if (col >= a.row_bytes) cache = nullptr;  // ragged last strip: these lanes only keep the warp together
  const int32_t* kept = a.kept + (static_cast<size_t>(s) * a.num_kv_heads + h) * a.budget;
  const int32_t* src = a.block_tables + static_cast<size_t>(s) * a.max_blocks_per_seq;
  const int32_t* dst = a.dst_tables + static_cast<size_t>(s) * a.max_dst_blocks_per_seq;
  const size_t token_bytes = static_cast<size_t>(a.num_kv_heads) * a.row_bytes;
  const size_t head_off = static_cast<size_t>(h) * a.row_bytes + col;
  const int bs = a.block_size;
  for (int base = 0; base < n; base += kMoveRows * kMoveUnroll) {
    uint4 x[kMoveUnroll];
    uint8_t* to[kMoveUnroll];
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i) {
      const int j = base + i * kMoveRows + (lane >> 2);
      to[i] = nullptr;
      if (j < n && cache) {
        const int t = kept[j];
        const int sb = src[t / bs], db = dst[j / bs];
        if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks) {
          atomicOr(a.error_word, PA_DEVERR_BLOCK_ID);
        } else if (sb != db || t % bs != j % bs) {
          const uint8_t* from = cache + (static_cast<size_t>(sb) * bs + t % bs) * token_bytes + head_off;
          to[i] = cache + (static_cast<size_t>(db) * bs + j % bs) * token_bytes + head_off;
          x[i] = *reinterpret_cast<const uint4*>(from);
        }
      }
    }
    __syncwarp();  // every lane has read its rows before any lane writes
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i)
      if (to[i]) *reinterpret_cast<uint4*>(to[i]) = x[i];
  }
}

}  // namespace pa
