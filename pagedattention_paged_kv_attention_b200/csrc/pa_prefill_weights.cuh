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
// persistent CTAs take items, the key tiles that the most rows see first. The roles run ahead over item borders:
//   warp 0        finds the items (a ring of four) and issues the TMA loads: an item's K boxes (straight from the
//                 cache blocks) into one of two slots, and its query tiles into a 4-deep ring;
//   warps 4..7    copy an item's K into one of two TMEM slots, widening E4M3 on the way (exact: every E4M3 value
//                 is a T value). With both operands in shared memory the MMA reads 128 bytes a cycle and takes
//                 1000 cycles a tile; with A in TMEM, half of both;
//   warp 1        one thread issues S^T of each tile into one of three 128-column TMEM buffers;
//   warps 8..19   three warpgroups, one to a buffer: each thread reads its lane's 128 scores, frees the buffer and
//                 adds 2^(z - lse) (lse of the tile's rows broadcast from shared memory).
//   warps 2-3     add an item's sums to the scores, so that no warpgroup waits for another's tile.
// Tile i of an item adds to sum i % 3, and the three are added in that order, whichever warpgroup had them:
// results depend neither on timing nor on which CTA had the item.
// Bound by the exponentials (one per visible pair and head, 16 per SM and cycle), as the attention itself, and by a
// warpgroup's chain of score load and exponentials: 8 prompts of 300 to 2048 tokens, 32/8 heads, 96 us, the
// exponential unit 58% busy on four of them; with one CTA per item and two warpgroups it was 144 us.
#pragma once

#include "pa_prefill.cuh"

namespace pa {
namespace pf {

constexpr int kWStages = 4;            // query ring depth
constexpr int kWBufs = 3;              // score buffers in TMEM = warpgroups that read them
constexpr int kWItems = 4;             // item ring depth
// Items of at most this many tiles are dealt, not drawn. The whole call, 16 chunks over contexts of 1024 to 4096, 32/8
// heads, dealt and drawn: 1 tile 114 and 130 us, 4 tiles 200 and 206, 6 tiles 267 and 263, 8 tiles 326 and 317.
constexpr int kDealTiles = 6;
constexpr int kWLoaders = 4;           // first of the warps that copy K
constexpr int kWReaders = 8;           // first of the warps that read scores
constexpr int kWThreads = 32 * (kWReaders + 4 * kWBufs);
constexpr uint32_t kWTmemK = 0, kWTmemS = 128;  // columns: two slots of K (64 each), the score buffers
constexpr int kWsWork = 1, kWsDone = 2;  // workspace header words after the error word: items drawn, CTAs done

struct WeightArgs {
  float* scores;                       // [S][Hkv][score_stride]
  long long score_stride;
  const float* lse;                    // [T][H], log2 units
  int window;                          // rows counted: the last `window` of each chunk (0: all)
  unsigned int num_items;              // key tiles x sequences x kv heads
  int draw;                            // items are drawn as CTAs come free (1), or dealt in turn (0)
};

template <int D>
struct WLayout {
  static constexpr int kChunks = D / 64;
  static constexpr uint32_t kTile = kChunks * 128 * 128;      // 128 rows of d 16-bit elements
  static constexpr uint32_t kK = 0;                           // two slots
  static constexpr uint32_t kQ = 2 * kTile;
  static constexpr uint32_t kBars = kQ + kWStages * kTile;
  static constexpr uint32_t kLse = kBars + 512;               // [warps that read scores][128] floats
  static constexpr uint32_t kSums = kLse + kWBufs * 4 * 128 * 4;  // [kWItems][kWBufs][128] floats
  static constexpr uint32_t kEnd = kSums + kWItems * kWBufs * 128 * 4 + 1024;
  static constexpr uint32_t kBytes = kEnd > 120u * 1024 ? kEnd : 120u * 1024;  // one CTA holds all TMEM columns
};

// One item: the tile's first key, the chunk, and the query tiles [j0 + i * tile_tokens, n) that see the key tile.
struct WItem {
  int kvh, s, t0, q0, n, ctx, j0, tiles;  // tiles 0: there is no such item
};

struct WBars {
  uint64_t k_full[2], k_empty[2], kt_full[2], kt_empty[2], q_full[kWStages], q_empty[kWStages], s_full[kWBufs],
      s_empty[kWBufs], i_full[kWItems], i_empty[kWItems], sum_full[kWItems], mma_done;
  WItem item[kWItems];
  uint32_t tmem_base;
  int abort;
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
  if (w.n <= 0 || w.q0 < 0 || w.n > w.ctx || chunk_too_long(a, w.n) || w.ctx > a.max_context_len ||
      w.q0 + w.n > a.num_q_tokens ||
      static_cast<long long>(w.ctx) > static_cast<long long>(a.max_blocks_per_seq) * a.block_size || w.t0 >= w.ctx)
    return w;  // nothing to add; the attention has flagged what is invalid
  const int first_counted = window > 0 ? max(0, w.n - window) : 0;
  w.j0 = max(first_counted, w.t0 - (w.ctx - w.n));  // first chunk token that counts and sees key t0
  w.tiles = (w.n - w.j0 + a.tile_tokens - 1) / a.tile_tokens;  // j0 < n, as t0 < ctx
  return w;
}

__device__ __forceinline__ bool w_wait(WBars* b, uint64_t* bar, uint32_t parity, unsigned int* err) {
  bool ok = false;
  if (*reinterpret_cast<volatile int*>(&b->abort) == 0) {
    ok = mbar_wait(bar, parity, err);
    if (!ok) *reinterpret_cast<volatile int*>(&b->abort) = 1;
  }
  return __all_sync(0xffffffffu, ok);
}

// The same by one thread.
__device__ __forceinline__ bool w_wait_one(WBars* b, uint64_t* bar, uint32_t parity, unsigned int* err) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*reinterpret_cast<volatile int*>(&b->abort) != 0) return false;
  if (mbar_wait(bar, parity, err)) return true;
  *reinterpret_cast<volatile int*>(&b->abort) = 1;
  return false;
}

// The CTA's item number i, read by a whole warp; no tiles after the last one or when a wait gave up.
__device__ __forceinline__ WItem w_item(WBars* b, int i, unsigned int* err) {
  if (!w_wait(b, &b->i_full[i % kWItems], (i / kWItems) & 1, err)) return WItem{};
  const WItem w = b->item[i % kWItems];
  __syncwarp();
  return w;
}

// Row r of the key tile at `tile` (128-byte rows, 128-byte swizzled) into this thread's TMEM lane as 16-bit pairs.
template <typename T, int D, bool kFp8>
__device__ __forceinline__ void key_row_to_tmem(const uint8_t* tile, int r, uint32_t t_k) {
  if constexpr (kFp8) {
#pragma unroll
    for (int u = 0; u < 8; u += 2) {
      uint32_t w[16];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 q = *reinterpret_cast<const uint4*>(tile + r * 128 + (((u + h) ^ (r & 7)) << 4));
        const uint32_t c[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (std::is_same<T, __half>::value) {
            w[8 * h + 2 * k] = e4m3x2_to_f16x2(static_cast<uint16_t>(c[k] & 0xffffu));
            w[8 * h + 2 * k + 1] = e4m3x2_to_f16x2(static_cast<uint16_t>(c[k] >> 16));
          } else {
            const float2 lo = e4m3x2_to_float2(static_cast<uint16_t>(c[k] & 0xffffu));
            const float2 hi = e4m3x2_to_float2(static_cast<uint16_t>(c[k] >> 16));
            w[8 * h + 2 * k] = pack2<T>(lo.x, lo.y);
            w[8 * h + 2 * k + 1] = pack2<T>(hi.x, hi.y);
          }
        }
      }
      tmem_st16(t_k + 8 * u, w);
    }
  } else {
#pragma unroll
    for (int u = 0; u < D / 8; u += 4) {
      uint32_t w[16];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const uint4 q = *reinterpret_cast<const uint4*>(tile + ((u + h) >> 3) * (kKvTile * 128) + r * 128 +
                                                        ((((u + h) & 7) ^ (r & 7)) << 4));
        w[4 * h] = q.x;
        w[4 * h + 1] = q.y;
        w[4 * h + 2] = q.z;
        w[4 * h + 3] = q.w;
      }
      tmem_st16(t_k + 4 * u, w);
    }
  }
}

template <typename T, int D, int KVB>
__global__ void __launch_bounds__(kWThreads, 1)
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
      mbar_init(&b->k_full[i], 1);
      mbar_init(&b->k_empty[i], 128);
      mbar_init(&b->kt_full[i], 128);
      mbar_init(&b->kt_empty[i], 1);
    }
    for (int i = 0; i < kWStages; ++i) {
      mbar_init(&b->q_full[i], 1);
      mbar_init(&b->q_empty[i], 1);
    }
    for (int i = 0; i < kWBufs; ++i) {
      mbar_init(&b->s_full[i], 1);
      mbar_init(&b->s_empty[i], 128);
    }
    for (int i = 0; i < kWItems; ++i) {
      mbar_init(&b->i_full[i], 1);
      mbar_init(&b->i_empty[i], 1 + 4 + 2);  // warps 1 to 7; the sums of warps 8 to 19 come before the adders'
      mbar_init(&b->sum_full[i], kWBufs * 4);
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
    // The next item, no tiles after the last one. Large items are drawn when the one before has been issued whole:
    // they come first, and a CTA that held one more would finish late. Items of a few tiles are dealt in turn (a
    // draw would take as long as they do), and looked up 32 at a time, one a lane.
    unsigned int at = 0;      // items of this CTA looked up so far
    unsigned int left = 0;    // lanes whose item is still to come
    WItem held{};
    auto next_item = [&]() {
      WItem w{};
      if (wa.draw) {
        while (w.tiles == 0) {
          unsigned int idx = 0;
          if (lane == 0) idx = atomicAdd(err + kWsWork, 1u);
          idx = __shfl_sync(0xffffffffu, idx, 0);
          if (idx >= wa.num_items) break;
          w = weight_item(a, wa.window, idx);
        }
        return w;
      }
      while (left == 0) {
        if (at * gridDim.x + blockIdx.x >= wa.num_items) return w;
        const unsigned int idx = (at + lane) * gridDim.x + blockIdx.x;
        held = idx < wa.num_items ? weight_item(a, wa.window, idx) : WItem{};
        left = __ballot_sync(0xffffffffu, held.tiles > 0);
        at += 32;
      }
      const int from = __ffs(left) - 1;
      left &= left - 1;
      w.kvh = __shfl_sync(0xffffffffu, held.kvh, from);
      w.s = __shfl_sync(0xffffffffu, held.s, from);
      w.t0 = __shfl_sync(0xffffffffu, held.t0, from);
      w.q0 = __shfl_sync(0xffffffffu, held.q0, from);
      w.n = __shfl_sync(0xffffffffu, held.n, from);
      w.ctx = __shfl_sync(0xffffffffu, held.ctx, from);
      w.j0 = __shfl_sync(0xffffffffu, held.j0, from);
      w.tiles = __shfl_sync(0xffffffffu, held.tiles, from);
      return w;
    };
    auto blocks_of = [&](const WItem& w) { return (min(kKvTile, w.ctx - w.t0) + bs - 1) / bs; };
    auto block_id = [&](const WItem& w) {  // of this lane's box
      return w.tiles > 0 && lane < blocks_of(w)
                 ? __ldg(a.block_tables + static_cast<size_t>(w.s) * a.max_blocks_per_seq + w.t0 / bs + lane)
                 : -1;
    };
    WItem following = next_item();
    int following_blk = block_id(following);
    for (;;) {
      const WItem w = following;
      const int blk = following_blk;
      if (!wa.draw) {
        following = next_item();
        following_blk = block_id(following);
      }
      const int islot = items % kWItems;
      if (items >= kWItems && !w_wait(b, &b->i_empty[islot], ((items / kWItems) - 1) & 1, err)) break;
      if (lane == 0) {
        b->item[islot] = w;
        mbar_arrive(&b->i_full[islot]);
      }
      __syncwarp();
      if (w.tiles == 0) break;
      const int slot = items & 1;
      // A block outside the pool is flagged by the attention; rows that see it have a NaN lse.
      const bool ok = blk >= 0 && blk < a.num_blocks;
      const unsigned okmask = __ballot_sync(0xffffffffu, ok);
      if (items >= 2 && !w_wait(b, &b->k_empty[slot], ((items >> 1) - 1) & 1, err)) break;
      uint64_t* k_bar = &b->k_full[slot];
      uint8_t* ks = sm + L::kK + slot * L::kTile;
      if (lane == 0) mbar_arrive_expect_tx(k_bar, __popc(okmask) * bs * 128 * (kFp8 ? 1 : L::kChunks));
      __syncwarp();
      if (ok) {
        if constexpr (kFp8) {
          tma_load_4d(ks + lane * bs * 128, &tk, k_bar, 0, 0, w.kvh, blk);
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
      if (!go) break;
      if (wa.draw) {
        following = next_item();
        following_blk = block_id(following);
      }
    }
    // Wind-down: every load issued has landed (immediate unless the CTA aborted).
    for (int i = max(0, items - 2); i < items; ++i)
      mbar_wait(&b->k_full[i & 1], (i >> 1) & 1, err);
    for (int i = max(0, tile - kWStages); i < tile; ++i)
      mbar_wait(&b->q_full[i % kWStages], (i / kWStages) & 1, err);
  } else if (warp >= kWLoaders && warp < kWLoaders + 4) {
    // ================================ K to TMEM ================================
    const int r = threadIdx.x - 32 * kWLoaders;   // key of the tile == TMEM lane
    for (int items = 0; w_item(b, items, err).tiles > 0; ++items) {
      if (lane == 0) mbar_arrive(&b->i_empty[items % kWItems]);
      const int slot = items & 1;
      if (!w_wait(b, &b->k_full[slot], (items >> 1) & 1, err)) break;
      if (items >= 2 && !w_wait(b, &b->kt_empty[slot], ((items >> 1) - 1) & 1, err)) break;
      tc_fence_after();
      key_row_to_tmem<T, D, kFp8>(sm + L::kK + slot * L::kTile, r,
                                  tmem + kWTmemK + 64 * slot + (static_cast<uint32_t>(r & ~31) << 16));
      mbar_arrive(&b->k_empty[slot]);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&b->kt_full[slot]);
    }
  } else if (warp == 1) {
    // ================================ MMA issuer ================================
    constexpr uint32_t idesc = mma_idesc_f16<T>(kKvTile, kRows, false);
    if (lane == 0) {
      int items = 0, tile = 0;
      bool ok = true;
      while (ok && w_wait_one(b, &b->i_full[items % kWItems], (items / kWItems) & 1, err)) {
        const int tiles = b->item[items % kWItems].tiles;
        if (tiles == 0) break;
        mbar_arrive(&b->i_empty[items % kWItems]);
        const int slot = items & 1;
        if (!w_wait_one(b, &b->kt_full[slot], (items >> 1) & 1, err)) break;
        for (int i = 0; i < tiles; ++i, ++tile) {
          const int st = tile % kWStages, buf = tile % kWBufs;
          if (!(ok = w_wait_one(b, &b->q_full[st], (tile / kWStages) & 1, err))) break;
          if (tile >= kWBufs && !(ok = w_wait_one(b, &b->s_empty[buf], ((tile / kWBufs) - 1) & 1, err))) break;
          tc_fence_after();
          const uint32_t q_addr = smem_u32(sm + L::kQ + st * L::kTile);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t o = (k >> 2) * (128 * 128) + (k & 3) * 32;
            mma_f16_ts(tmem + kWTmemS + buf * kRows, tmem + kWTmemK + 64 * slot + 8 * k,
                       smem_desc_sw128(q_addr + o, 16, 1024), idesc, k > 0);
          }
          mma_commit(&b->s_full[buf]);
          mma_commit(&b->q_empty[st]);
          if (i == tiles - 1) mma_commit(&b->kt_empty[slot]);
        }
        ++items;
      }
      mma_commit(&b->mma_done);
      mbar_wait(&b->mma_done, 0, err);
    }
    __syncwarp();
  } else if (warp == 2 || warp == 3) {
    // ================================ scores ================================
    const int r = threadIdx.x - 64;               // keys r and r + 64 of the tile
    for (int items = 0;; ++items) {
      const WItem w = w_item(b, items, err);
      if (w.tiles == 0) break;
      const int slot = items % kWItems;
      float* dst = wa.scores + (static_cast<size_t>(w.s) * a.num_kv_heads + w.kvh) * wa.score_stride + w.t0 + r;
      float x[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) x[h] = w.t0 + r + 64 * h < w.ctx ? dst[64 * h] : 0.f;
      if (!w_wait(b, &b->sum_full[slot], (items / kWItems) & 1, err)) break;
      const float* sums = reinterpret_cast<const float*>(sm + L::kSums) + slot * kWBufs * 128 + r;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = sums[64 * h];
#pragma unroll
        for (int c = 1; c < kWBufs; ++c)
          if (c < w.tiles) sum += sums[c * 128 + 64 * h];
        if (w.t0 + r + 64 * h < w.ctx) dst[64 * h] = x[h] + sum;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->i_empty[slot]);
    }
  } else if (warp >= kWReaders) {
    // ================================ weights ================================
    const int wg = (warp - kWReaders) >> 2;
    const int r = threadIdx.x - 32 * kWReaders - wg * 128;  // key of the tile == TMEM lane
    const int log_g = __ffs(G) - 1;               // G divides 128
    float* lse_sm = reinterpret_cast<float*>(sm + L::kLse) + (warp - kWReaders) * 128;
    const uint32_t t_s = tmem + kWTmemS + wg * kRows + (static_cast<uint32_t>(r & ~31) << 16);
    int tile = 0, turn = 0;                       // tiles before the item, and that modulo kWBufs
    bool ok = true;
    for (int items = 0; ok; ++items) {
      const int slot = items % kWItems;
      const WItem w = w_item(b, items, err);
      if (w.tiles == 0) break;
      const int t = w.t0 + r;
      // This warpgroup's first tile of the item, and which sum it adds to.
      const int first = wg >= turn ? wg - turn : wg - turn + kWBufs;
      float sl2 = a.scale_log2;
      if (kFp8 && first < w.tiles && t < w.ctx) {
        // K's scale is an exact fp32 factor of the key's scores.
        const int blk = a.scale_block_stride
                            ? __ldg(a.block_tables + static_cast<size_t>(w.s) * a.max_blocks_per_seq + t / a.block_size)
                            : 0;
        if (blk >= 0 && blk < a.num_blocks)
          sl2 *= __ldg(a.k_scale + static_cast<size_t>(blk) * a.scale_block_stride + w.kvh);
      }
      float2 acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.f, 0.f);
      const float2 sl2x2 = make_float2(sl2, sl2);
      float nl[4];                                // -lse of rows lane + 32 k of the next tile; masked past the chunk
      auto fetch = [&](int i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = lane + 32 * k, tok = w.j0 + i * a.tile_tokens + (row >> log_g);
          nl[k] = i < w.tiles && tok < w.n
                      ? -__ldg(wa.lse + static_cast<size_t>(w.q0 + tok) * a.num_heads + w.kvh * G + (row & (G - 1)))
                      : 0.f;
        }
      };
      fetch(first);
      for (int i = first; i < w.tiles; i += kWBufs) {
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) lse_sm[lane + 32 * k] = nl[k];
        __syncwarp();
        fetch(i + kWBufs);
        if (!(ok = w_wait(b, &b->s_full[wg], ((tile + i) / kWBufs) & 1, err))) break;
        tc_fence_after();
        const int tok0 = w.j0 + i * a.tile_tokens;
        // Columns [lo, hi) are rows that see this key and lie in the chunk; a warp skips 32 columns that none of
        // its keys has a part in, and masks those that only some have.
        const int lo = max(0, t - (w.ctx - w.n) - tok0) << log_g, hi = min(kRows, (w.n - tok0) << log_g);
        const int lo_min = __shfl_sync(0xffffffffu, lo, 0), lo_max = __shfl_sync(0xffffffffu, lo, 31);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bool some = 32 * c + 31 >= lo_min && 32 * c < hi;
          uint32_t v[32];
          if (some) {
            tmem_ld32(t_s + 32 * c, v);
            tmem_wait_ld(v);
          }
          if (c == 3) {
            tc_fence_before();
            mbar_arrive(&b->s_empty[wg]);
          }
          if (!some) continue;
          const float4* nl4 = reinterpret_cast<const float4*>(lse_sm) + c * 8;
          if (32 * c >= lo_max && 32 * c + 32 <= hi) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 l4 = nl4[k];
              const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1])), sl2x2,
                                          make_float2(l4.x, l4.y));
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3])),
                                          sl2x2, make_float2(l4.z, l4.w));
              acc[(2 * k) & 3] = __fadd2_rn(acc[(2 * k) & 3], make_float2(ex2(x.x), ex2(x.y)));
              acc[(2 * k + 1) & 3] = __fadd2_rn(acc[(2 * k + 1) & 3], make_float2(ex2(y.x), ex2(y.y)));
            }
          } else {
            const unsigned span = static_cast<unsigned>(hi - lo);  // hi > lo, or no column is below it
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int col = 32 * c + 2 * k;
              const float2 l2 = reinterpret_cast<const float2*>(nl4)[k];
              const float2 x =
                  __ffma2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), sl2x2, l2);
              acc[k & 3] = __fadd2_rn(
                  acc[k & 3], make_float2(hi > lo && static_cast<unsigned>(col - lo) < span ? ex2(x.x) : 0.f,
                                          hi > lo && static_cast<unsigned>(col + 1 - lo) < span ? ex2(x.y) : 0.f));
            }
          }
        }
      }
      if (!ok) break;
      const float2 s2 = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
      // The slot is free: its item before this one has been added.
      if (first < w.tiles) reinterpret_cast<float*>(sm + L::kSums)[(slot * kWBufs + first) * 128 + r] = s2.x + s2.y;
      __syncwarp();
      if (lane == 0) mbar_arrive(&b->sum_full[slot]);
      tile += w.tiles;
      turn = tile % kWBufs;
    }
  }

  // ---- teardown: every role has finished with TMEM ----
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // The last CTA to finish resets the draw for the next launch on this workspace.
  if (wa.draw && threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(err + kWsDone, 1u) == gridDim.x - 1) {
      atomicExch(err + kWsWork, 0u);
      atomicExch(err + kWsDone, 0u);
    }
  }
}

}  // namespace pf
}  // namespace pa
