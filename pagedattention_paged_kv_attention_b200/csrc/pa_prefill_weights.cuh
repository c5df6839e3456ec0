// pa_prefill_weights.cuh -- the attention weights of a causal prefill, added to the cached tokens' scores.
//
// With lse[row] = log2 sum_t 2^(z[row][t]) of every query row from paged_prefill_kernel (kCausalStats), z the
// scaled score in log2 units, this kernel forms for every kv head and cached token t
//     scores[s][kvh][t] += sum over the counted rows (tokens j of the chunk that see t, x the G heads of the
//                          kv head) of 2^(z[row][t] - lse[row]).
// The weights cannot be summed while the attention runs: a row's sum is known only after its last key.
//
// The score tile is formed transposed, S^T = K Q^T (M = 128 keys, N = 128 query rows): a key is one TMEM
// lane, so the thread that owns the lane sums its key's weights over the columns in registers and nothing
// is reduced across threads. An item is a 128-key tile of a kv head and sequence, with the query tiles that see it;
// persistent CTAs walk the items, the key tiles that the most rows see first, alternating the direction
// from round to round so that the CTAs' sums of work come out alike. The roles run ahead over item borders:
//   warp 0        TMA: an item's K boxes (straight from the cache blocks) into one of two slots, and its query
//                 tiles into a 4-deep ring;
//   warp 1        one thread issues S^T of each tile into one of four 128-column TMEM buffers;
//   warps 2-3     widen E4M3 keys to T in place (exact: every E4M3 value is a T value);
//   warps 4..7    take the even tiles, warps 8..11 the odd ones: each thread reads its lane's 128 scores,
//                 frees the buffer and adds 2^(z - lse) (lse of the tile's rows broadcast from shared memory); at
//                 an item's end the first adds the second's sum and its own to the score.
// Every (s, kvh, t) is added to by one thread in a fixed order: results do not depend on timing.
// Bound by the exponentials (one per visible pair and head, 16 per SM and cycle), as the attention itself.
#pragma once

#include "pa_prefill.cuh"

namespace pa {
namespace pf {

constexpr int kWStages = 4;            // query ring depth = TMEM buffers

struct WeightArgs {
  float* scores;                       // [S][Hkv][score_stride]
  long long score_stride;
  const float* lse;                    // [T][H], log2 units
  int window;                          // rows counted: the last `window` of each chunk (0: all)
  unsigned int num_items;              // key tiles x sequences x kv heads
};

template <int D>
struct WLayout {
  static constexpr int kChunks = D / 64;
  static constexpr uint32_t kTile = kChunks * 128 * 128;      // 128 rows of d 16-bit elements
  static constexpr uint32_t kK = 0;                           // two slots
  static constexpr uint32_t kQ = 2 * kTile;
  static constexpr uint32_t kBars = kQ + kWStages * kTile;
  static constexpr uint32_t kLse = kBars + 256;               // [2 warpgroups][2][128] floats
  static constexpr uint32_t kSums = kLse + 4 * 128 * 4;       // [2][128] floats
  static constexpr uint32_t kEnd = kSums + 2 * 128 * 4 + 1024;
  static constexpr uint32_t kBytes = kEnd > 120u * 1024 ? kEnd : 120u * 1024;  // one CTA holds all TMEM columns
};

struct WBars {
  uint64_t k_load[2], k_full[2], k_empty[2], q_full[kWStages], q_empty[kWStages], s_full[kWStages],
      s_empty[kWStages], mma_done;
  uint32_t tmem_base;
  int abort;
};

// One item: the tile's first key, the chunk, and the query tiles [j0 + i * tile_tokens, n) that see the key tile.
struct WItem {
  int kvh, s, t0, q0, n, ctx, j0, tiles;
};

__device__ __forceinline__ WItem weight_item(const PrefillArgs& a, int window, unsigned int idx) {
  WItem w;
  w.kvh = static_cast<int>(idx % a.num_kv_heads);
  idx /= a.num_kv_heads;
  w.s = static_cast<int>(idx % a.num_seqs);
  w.t0 = static_cast<int>(idx / a.num_seqs) * kKvTile;
  w.q0 = __ldg(a.q_start + w.s);
  w.n = __ldg(a.q_start + w.s + 1) - w.q0;
  w.ctx = __ldg(a.context_lens + w.s);
  w.j0 = w.tiles = 0;
  if (w.n <= 0 || w.q0 < 0 || w.n > w.ctx || w.ctx > a.max_context_len || w.q0 + w.n > a.num_q_tokens ||
      static_cast<long long>(w.ctx) > static_cast<long long>(a.max_blocks_per_seq) * a.block_size || w.t0 >= w.ctx)
    return w;  // nothing to add; the attention has flagged what is invalid
  const int first_counted = window > 0 ? max(0, w.n - window) : 0;
  w.j0 = max(first_counted, w.t0 - (w.ctx - w.n));  // first chunk token that counts and sees key t0
  w.tiles = (w.n - w.j0 + a.tile_tokens - 1) / a.tile_tokens;  // j0 < n, as t0 < ctx
  return w;
}

// The CTA's item of a round, alternating the direction; past the last one when there is none.
__device__ __forceinline__ unsigned int weight_index(unsigned int round) {
  return round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

__device__ __forceinline__ bool w_wait(WBars* b, uint64_t* bar, uint32_t parity, unsigned int* err) {
  bool ok = false;
  if (*reinterpret_cast<volatile int*>(&b->abort) == 0) {
    ok = mbar_wait(bar, parity, err);
    if (!ok) *reinterpret_cast<volatile int*>(&b->abort) = 1;
  }
  return __all_sync(0xffffffffu, ok);
}

// Row r of an E4M3 key tile staged in the second chunk becomes T.
template <typename T>
__device__ __forceinline__ void widen_key_row(uint8_t* tile, int r) {
  if constexpr (std::is_same<T, __half>::value) {
    widen_row(tile, tile + kKvTile * 128, r, __float2half2_rn(1.f), false);
  } else {
    uint4 q[8];
    const uint8_t* staged = tile + kKvTile * 128 + r * 128;
#pragma unroll
    for (int u = 0; u < 8; ++u) q[u] = *reinterpret_cast<const uint4*>(staged + ((u ^ (r & 7)) << 4));
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
      uint32_t h[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = e4m3x2_to_float2(static_cast<uint16_t>(w[k] & 0xffffu));
        const float2 c = e4m3x2_to_float2(static_cast<uint16_t>(w[k] >> 16));
        h[2 * k] = pack2<T>(a.x, a.y);
        h[2 * k + 1] = pack2<T>(c.x, c.y);
      }
      uint8_t* row = tile + (u >> 2) * (kKvTile * 128) + r * 128;
      *reinterpret_cast<uint4*>(row + (((2 * (u & 3)) ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(row + (((2 * (u & 3) + 1) ^ (r & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
    }
  }
}

template <typename T, int D, int KVB>
__global__ void __launch_bounds__(kThreads, 1)
prefill_weights_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const PrefillArgs a, const WeightArgs wa) {
  using L = WLayout<D>;
  constexpr bool kFp8 = KVB == 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  WBars* b = reinterpret_cast<WBars*>(sm + L::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.group;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b->k_load[i], 1);
      mbar_init(&b->k_full[i], kFp8 ? 64 : 1);   // FP8: the 64 widening threads arrive
      mbar_init(&b->k_empty[i], 1);
    }
    for (int i = 0; i < kWStages; ++i) {
      mbar_init(&b->q_full[i], 1);
      mbar_init(&b->q_empty[i], 1);
      mbar_init(&b->s_full[i], 1);
      mbar_init(&b->s_empty[i], 128);
    }
    mbar_init(&b->mma_done, 1);
    b->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
  }
  if (warp == 1) {
    tmem_alloc(&b->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = b->tmem_base;
  unsigned int* err = a.error_word;

  if (warp == 0) {
    // ================================ TMA producer ================================
    const int bs = a.block_size;
    int items = 0, tile = 0;  // items and query tiles loaded so far
    bool go = true;
    for (unsigned int round = 0, idx; go && (idx = weight_index(round)) < wa.num_items; ++round) {
      const WItem w = weight_item(a, wa.window, idx);
      if (w.tiles == 0) continue;
      const int slot = items & 1;
      const int nblk = (min(kKvTile, w.ctx - w.t0) + bs - 1) / bs;
      int blk = 0;
      bool ok = false;
      if (lane < nblk) {
        blk = __ldg(a.block_tables + static_cast<size_t>(w.s) * a.max_blocks_per_seq + w.t0 / bs + lane);
        ok = blk >= 0 && blk < a.num_blocks;  // flagged by the attention; rows that see it have a NaN lse
      }
      const unsigned okmask = __ballot_sync(0xffffffffu, ok);
      if (items >= 2 && !w_wait(b, &b->k_empty[slot], ((items >> 1) - 1) & 1, err)) break;
      uint64_t* k_bar = kFp8 ? &b->k_load[slot] : &b->k_full[slot];
      uint8_t* ks = sm + L::kK + slot * L::kTile;
      if (lane == 0) mbar_arrive_expect_tx(k_bar, __popc(okmask) * bs * 128 * (kFp8 ? 1 : L::kChunks));
      __syncwarp();
      if (ok) {
        if constexpr (kFp8) {
          tma_load_4d(ks + kKvTile * 128 + lane * bs * 128, &tk, k_bar, 0, 0, w.kvh, blk);
        } else {
          for (int c = 0; c < L::kChunks; ++c)
            tma_load_4d(ks + c * (kKvTile * 128) + lane * bs * 128, &tk, k_bar, c * 64, 0, w.kvh, blk);
        }
      }
      ++items;
      for (int i = 0; i < w.tiles; ++i, ++tile) {
        const int st = tile % kWStages;
        if (tile >= kWStages && !(go = w_wait(b, &b->q_empty[st], ((tile / kWStages) - 1) & 1, err))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&b->q_full[st], L::kTile);
          for (int c = 0; c < L::kChunks; ++c)
            tma_load_3d(sm + L::kQ + st * L::kTile + c * (kRows * 128), &tq, &b->q_full[st], c * 64, w.kvh * G,
                        w.q0 + w.j0 + i * a.tile_tokens);
        }
        __syncwarp();
      }
    }
    // Wind-down: every load issued has landed (immediate unless the CTA aborted).
    for (int i = max(0, items - 2); i < items; ++i)
      mbar_wait(kFp8 ? &b->k_load[i & 1] : &b->k_full[i & 1], (i >> 1) & 1, err);
    for (int i = max(0, tile - kWStages); i < tile; ++i)
      mbar_wait(&b->q_full[i % kWStages], (i / kWStages) & 1, err);
  } else if (kFp8 && (warp == 2 || warp == 3)) {
    // ================================ E4M3 widening (FP8 caches) ================================
    int items = 0;
    for (unsigned int round = 0, idx; (idx = weight_index(round)) < wa.num_items; ++round) {
      if (weight_item(a, wa.window, idx).tiles == 0) continue;
      const int slot = items & 1;
      if (!w_wait(b, &b->k_load[slot], (items >> 1) & 1, err)) break;
      for (int h = 0; h < 2; ++h) widen_key_row<T>(sm + L::kK + slot * L::kTile, threadIdx.x - 64 + 64 * h);
      fence_proxy_async_smem();
      mbar_arrive(&b->k_full[slot]);
      ++items;
    }
  } else if (warp == 1) {
    // ================================ MMA issuer ================================
    constexpr uint32_t idesc = mma_idesc_f16<T>(kKvTile, kRows, false);
    int items = 0, tile = 0;
    bool ok = true;
    for (unsigned int round = 0, idx; ok && (idx = weight_index(round)) < wa.num_items; ++round) {
      const int tiles = weight_item(a, wa.window, idx).tiles;
      if (tiles == 0) continue;
      const int slot = items & 1;
      if (!(ok = w_wait(b, &b->k_full[slot], (items >> 1) & 1, err))) break;
      for (int i = 0; i < tiles; ++i, ++tile) {
        const int st = tile % kWStages;
        if (!(ok = w_wait(b, &b->q_full[st], (tile / kWStages) & 1, err))) break;
        if (tile >= kWStages && !(ok = w_wait(b, &b->s_empty[st], ((tile / kWStages) - 1) & 1, err))) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t k_addr = smem_u32(sm + L::kK + slot * L::kTile);
          const uint32_t q_addr = smem_u32(sm + L::kQ + st * L::kTile);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t o = (k >> 2) * (128 * 128) + (k & 3) * 32;
            mma_f16_ss(tmem + st * kRows, smem_desc_sw128(k_addr + o, 16, 1024), smem_desc_sw128(q_addr + o, 16, 1024),
                       idesc, k > 0);
          }
          mma_commit(&b->s_full[st]);
          mma_commit(&b->q_empty[st]);
          if (i == tiles - 1) mma_commit(&b->k_empty[slot]);
        }
        __syncwarp();
      }
      ++items;
    }
    if (lane == 0) {
      mma_commit(&b->mma_done);
      mbar_wait(&b->mma_done, 0, err);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ================================ weights ================================
    const int wg = (warp - 4) >> 2;
    const int r = threadIdx.x - 128 - wg * 128;   // key of the tile == TMEM lane; also the row whose lse it fetches
    const int r_tok = r / G, r_head = r % G;
    float* lse_sm = reinterpret_cast<float*>(sm + L::kLse) + wg * 256;
    float* sums = reinterpret_cast<float*>(sm + L::kSums);
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(r & ~31) << 16);
    bool ok = true;
    int items = 0, tile = 0, par = 0;
    for (unsigned int round = 0, idx; (idx = weight_index(round)) < wa.num_items; ++round) {
      const WItem w = weight_item(a, wa.window, idx);
      if (w.tiles == 0) continue;
      const int t = w.t0 + r;
      float* dst = wa.scores + (static_cast<size_t>(w.s) * a.num_kv_heads + w.kvh) * wa.score_stride + t;
      const bool owner = wg == 0 && t < w.ctx;
      const float old = owner ? *dst : 0.f;
      float sl2 = a.scale_log2;
      if (kFp8 && t < w.ctx) {
        // K's scale is an exact fp32 factor of the key's scores.
        const int blk = a.scale_block_stride
                            ? __ldg(a.block_tables + static_cast<size_t>(w.s) * a.max_blocks_per_seq + t / a.block_size)
                            : 0;
        if (blk >= 0 && blk < a.num_blocks)
          sl2 *= __ldg(a.k_scale + static_cast<size_t>(blk) * a.scale_block_stride + w.kvh);
      }
      auto fetch = [&](int i) {  // -lse of this thread's row of tile i; rows past the chunk are masked below
        const int tok = w.j0 + i * a.tile_tokens + r_tok;
        return tok < w.n ? -__ldg(wa.lse + static_cast<size_t>(w.q0 + tok) * a.num_heads + w.kvh * G + r_head) : 0.f;
      };
      float2 acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.f, 0.f);
      const float2 sl2x2 = make_float2(sl2, sl2);
      const int own = (wg ^ tile) & 1;  // this warpgroup's first tile of the item
      float cur = own < w.tiles ? fetch(own) : 0.f;
      for (int i = own; i < w.tiles; i += 2, par ^= 1) {
        const int g = tile + i, st = g % kWStages;
        lse_sm[par * 128 + r] = cur;
        named_barrier(1 + wg, 128);
        if (i + 2 < w.tiles) cur = fetch(i + 2);
        // After a wait that gave up, the remaining rounds keep only the barriers.
        if (ok) ok = w_wait(b, &b->s_full[st], (g / kWStages) & 1, err);
        if (!ok) continue;
        tc_fence_after();
        const int tok0 = w.j0 + i * a.tile_tokens;
        // Columns [lo, hi) are rows that see this key and lie in the chunk.
        const int lo = max(0, t - (w.ctx - w.n) - tok0) * G, hi = min(kRows, (w.n - tok0) * G);
        const bool full = w.t0 + kKvTile - 1 - (w.ctx - w.n) <= tok0 && tok0 + a.tile_tokens <= w.n;  // for every key
        const float4* nl = reinterpret_cast<const float4*>(lse_sm + par * 128);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t v[2][32];
#pragma unroll
          for (int c = 0; c < 2; ++c) tmem_ld32(t_lane + st * kRows + 64 * half + 32 * c, v[c]);
#pragma unroll
          for (int c = 0; c < 2; ++c) tmem_wait_ld(v[c]);
          if (half == 1) {
            tc_fence_before();
            mbar_arrive(&b->s_empty[st]);
          }
          if (full) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float4 l4 = nl[half * 16 + c * 8 + k];
                const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[c][4 * k]), __uint_as_float(v[c][4 * k + 1])),
                                            sl2x2, make_float2(l4.x, l4.y));
                const float2 y = __ffma2_rn(
                    make_float2(__uint_as_float(v[c][4 * k + 2]), __uint_as_float(v[c][4 * k + 3])), sl2x2,
                    make_float2(l4.z, l4.w));
                acc[(2 * k) & 3] = __fadd2_rn(acc[(2 * k) & 3], make_float2(ex2(x.x), ex2(x.y)));
                acc[(2 * k + 1) & 3] = __fadd2_rn(acc[(2 * k + 1) & 3], make_float2(ex2(y.x), ex2(y.y)));
              }
          } else {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const int col = 64 * half + 32 * c + 2 * k;
                const float2 l2 = reinterpret_cast<const float2*>(nl)[half * 32 + c * 16 + k];
                const float2 x =
                    __ffma2_rn(make_float2(__uint_as_float(v[c][2 * k]), __uint_as_float(v[c][2 * k + 1])), sl2x2, l2);
                acc[k & 3] = __fadd2_rn(acc[k & 3], make_float2(col >= lo && col < hi ? ex2(x.x) : 0.f,
                                                                col + 1 >= lo && col + 1 < hi ? ex2(x.y) : 0.f));
              }
          }
        }
      }
      const float2 s2 = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
      const float sum = s2.x + s2.y;
      // The second warpgroup's sum goes through shared memory; two buffers, so one barrier an item is enough.
      float* other = sums + (items & 1) * 128 + r;
      if (wg == 1) *other = ok ? sum : __int_as_float(0x7fc00000);
      named_barrier(3, 256);
      if (owner && ok) *dst = old + (sum + *other);
      tile += w.tiles;
      ++items;
    }
  }

  // ---- teardown: every role has finished with TMEM ----
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace pf
}  // namespace pa
