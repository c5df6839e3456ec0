// pa_evict.cuh -- eviction of cached tokens by their accumulated attention weight.
//
// Per sequence s and kv head h, of the L cached tokens with scores w[t] at most `budget` stay: the first
// num_sink, the last num_recent, and of those in between the ones with the largest scores (equal scores:
// the lower index first; a NaN counts as -inf). The kept tokens move together in their order:
// token kept[j] becomes token j, in the destination table's blocks. Each head keeps tokens of its own;
// attention does not depend on which slot a key sits in, so heads need only agree on their number.
//
// One cluster of CTAs per (sequence, kv head) does both steps, so that one cluster's selection runs while
// another's rows move, and the scores cross the chip once.
// Selection: a radix selection of the q-th largest score on a monotone 32-bit image of the fp32 values, up
// to four digits of 8 bits (few candidates left after a digit are ranked directly, usually after the second),
// then one ordered compaction. The keys of up to kEvictPer tokens a thread stay in registers. A digit is
// counted in 16 copies of the histogram, one per two lanes, since scores crowd into few exponents and one copy
// would serialise a warp's atomics; the CTAs' counts are added through distributed shared memory.
// Move: bound by HBM, every kept row is read and written once. A kept token never moves up (kept[j] >= j), so
// walking j upwards, a round of rows read before any of them is written, may write over the very blocks that
// are read: a slot is written after the rows that come from it were read. Where a destination block is one of
// the sequence's own, the cluster's barrier orders each round's reads before its writes (release and acquire: a
// barrier without them does not wait for loads in flight); rows that go to other blocks need no order.
// 16 rows of 4096 to 16384 tokens x 8 heads of 128 (16-bit), cut to 2048: 68.6 us into other blocks, 4.12 TB/s, 67.9
// in place; one of 16384 tokens 19.2 and 22.2. Selection and move in kernels of their own took 79 us.
#pragma once

#include <math.h>
#include <stddef.h>

#include "pa_device.cuh"

namespace pa {

constexpr int kEvictThreads = 256;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictPerSm = 4;        // CTAs that an SM holds
constexpr int kEvictCluster = 8;      // most CTAs of a cluster
constexpr int kEvictShare = 1024;     // fewest tokens worth a CTA of their own
constexpr int kEvictPer = 16;         // tokens of a tile per thread
constexpr int kEvictTile = kEvictPer * kEvictThreads;
constexpr int kHistCopies = 16;
constexpr int kEvictFew = 32;         // keys that are ranked among themselves
constexpr int kMoveUnroll = 4;        // 16-byte loads per lane and step; two steps are in flight
constexpr int kMoveLogLoads = 5;      // log2 of a CTA's warps x loads
static_assert(kEvictWarps * kMoveUnroll == 1 << kMoveLogLoads, "a round is a power of two");
constexpr int kMoveMinLogLanes = 2;
constexpr int kMoveStage = 2048;      // rows of a CTA whose slots are resolved at a time, whole rounds of them
constexpr uint32_t kNoMove = 0xffffffffu;

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
      max_context_len, budget, num_sink, num_recent, log_lanes,
      log_block;  // log2(block_size), or -1
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

// Place of key i of a tile in shared memory: each thread's kEvictPer consecutive keys, 16 bytes apart from the
// next thread's, so that 16-byte reads of a warp do not meet in a bank.
__device__ __forceinline__ int key_slot(int i) { return i + i / kEvictPer * 4; }

struct alignas(16) EvictShared {
  union {
    struct {
      int hist[256 * kHistCopies];                // [digit][lane % kHistCopies]
      uint32_t keys[kEvictTile / kEvictPer * (kEvictPer + 4)];
    };
    struct {
      uint32_t slots[2 * kMoveStage];             // of a stage's rows: from (kNoMove: the row stays), then to
      float score[kMoveStage];
    };
  };
  int bins[2][256];                    // read by the cluster's other CTAs, as the next three
  uint32_t few[kEvictFew];
  int num_few, cta_sum[2];
  uint32_t all_few[kEvictFew];
  int warp_sum[kEvictWarps];           // of two counts, 16 bits each, in a scan
  uint32_t prefix;
  int need, count;
};
static_assert(alignof(EvictShared) % 16 == 0 && offsetof(EvictShared, keys) % 16 == 0 && (kEvictPer + 4) % 4 == 0,
              "keys are read 16 bytes at a time");

// Keys of tokens that are not ranked: past the row, or kept whatever their score.
constexpr uint32_t kKeyOut = 0u, kKeyEnd = 0xffffffffu;  // no score's key is either

__device__ __forceinline__ void evict_sync(int ctas) {
  if (ctas > 1)
    cluster_barrier();
  else
    __syncthreads();
}

// Exclusive scan of (x, y) over the CTA's threads, 0 <= x, y <= kEvictPer; *total receives the sums.
__device__ __forceinline__ int2 evict_scan(EvictShared& sh, int x, int y, int2* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int v = x | (y << 16);               // at most kEvictTile = 2^12 each
  const int own = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();                     // the last scan's sums have been read
  if (lane == 31) sh.warp_sum[warp] = v;
  __syncthreads();
  int all = 0, before = v - own;
#pragma unroll
  for (int i = 0; i < kEvictWarps; ++i) {
    const int c = sh.warp_sum[i];
    before += i < warp ? c : 0;
    all += c;
  }
  *total = make_int2(all & 0xffff, all >> 16);
  return make_int2(before & 0xffff, before >> 16);
}

// Selects among L > budget tokens and writes kept. The cluster's CTAs take contiguous chunks, a chunk goes in
// tiles of kEvictTile tokens, and a thread takes kEvictPer consecutive tokens of a tile.
__device__ __forceinline__ void evict_select(EvictShared& sh, const EvictArgs& a, int L, int rank, int ctas,
                                             const float* w, int32_t* kept) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunk = (L + ctas - 1) / ctas;
  const int t0 = min(L, rank * chunk), t1 = min(L, t0 + chunk);
  const int c0 = a.num_sink, c1 = L - a.num_recent;  // candidates; more than are needed, as L > budget
  int need = a.budget - a.num_sink - a.num_recent;
  uint32_t k[kEvictPer];
  auto load_tile = [&](int tile) {     // read in lines, handed out by threads
    __syncthreads();
    uint32_t v[kEvictPer];
#pragma unroll
    for (int i = 0; i < kEvictPer; ++i) {
      const int t = tile + i * kEvictThreads + tid;
      v[i] = t < t1 ? __float_as_uint(w[t]) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kEvictPer; ++i) {
      const int t = tile + i * kEvictThreads + tid;
      sh.keys[key_slot(i * kEvictThreads + tid)] =
          t >= t1 ? kKeyOut : t < c0 || t >= c1 ? kKeyEnd : score_key(__uint_as_float(v[i]));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEvictPer; i += 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(&sh.keys[key_slot(tid * kEvictPer) + i]);
      k[i] = q.x;
      k[i + 1] = q.y;
      k[i + 2] = q.z;
      k[i + 3] = q.w;
    }
  };
  const bool one_tile = t1 - t0 <= kEvictTile;
  if (one_tile) load_tile(t0);
  // f() with each tile's keys in k; the keys of a single tile stay there.
  auto each_tile = [&](auto f) {
    if (one_tile) {
      f(t0);
    } else {
      for (int tile = t0; tile < t1; tile += kEvictTile) {
        load_tile(tile);
        f(tile);
      }
    }
  };
  auto ranked = [](uint32_t key) { return key - 1u < kKeyEnd - 1u; };
  uint32_t threshold = kKeyEnd;        // the need-th largest key; `need` of its equals stay
  if (need > 0) {
    uint32_t prefix = 0;
    for (int i = tid; i < 256 * kHistCopies; i += kEvictThreads) sh.hist[i] = 0;
    if (tid == 0) sh.num_few = 0;
    __syncthreads();
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      each_tile([&](int) {
#pragma unroll
        for (int i = 0; i < kEvictPer; ++i)
          if (ranked(k[i]) && (shift == 24 || (k[i] >> (shift + 8)) == prefix))
            atomicAdd(&sh.hist[((k[i] >> shift) & 255u) * kHistCopies + lane % kHistCopies], 1);
      });
      __syncthreads();
      // Thread i adds up digit 255 - i, here and then over the cluster; a scan finds the digit, from the top,
      // at which the count reaches `need`.
      const int digit = 255 - tid;
      int* bins = sh.bins[(shift >> 3) & 1];
      int sum = 0;
#pragma unroll 8
      for (int i = 0; i < kHistCopies; ++i) {
        int* c = &sh.hist[digit * kHistCopies + (i + tid / 2) % kHistCopies];
        sum += *c;
        *c = 0;
      }
      if (ctas > 1) {
        bins[digit] = sum;
        cluster_barrier();
        sum = 0;
        for (int r = 0; r < ctas; ++r) sum += cluster_load(&bins[digit], r);
      }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) sh.warp_sum[warp] = incl;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kEvictWarps; ++i) incl += i < warp ? sh.warp_sum[i] : 0;
      if (incl - sum < need && incl >= need) {
        sh.prefix = (prefix << 8) | static_cast<uint32_t>(digit);
        sh.need = need - (incl - sum);
        sh.count = sum;
      }
      __syncthreads();
      prefix = sh.prefix;
      need = sh.need;
      const int m = sh.count;
      if (shift == 0) {
        threshold = prefix;
      } else if (m <= kEvictFew) {
        // Few keys share the digits so far: collect them and rank each among them.
        each_tile([&](int) {
#pragma unroll
          for (int i = 0; i < kEvictPer; ++i)
            if (ranked(k[i]) && (k[i] >> shift) == prefix) sh.few[atomicAdd(&sh.num_few, 1)] = k[i];
        });
        evict_sync(ctas);
        for (int r = 0, at = 0; r < ctas; ++r) {
          const int c = cluster_load(&sh.num_few, r);
          if (tid < c) sh.all_few[at + tid] = cluster_load(&sh.few[tid], r);
          at += c;
        }
        __syncthreads();
        for (int c = warp; c < m; c += kEvictWarps) {
          const uint32_t mine = sh.all_few[c];
          int above = 0, equal = 0;
          for (int i = lane; i < m; i += 32) {
            above += sh.all_few[i] > mine;
            equal += sh.all_few[i] == mine;
          }
          above = __reduce_add_sync(0xffffffffu, above);
          equal = __reduce_add_sync(0xffffffffu, equal);
          if (lane == 0 && above < need && need <= above + equal) {  // every equal of the threshold writes the same
            sh.prefix = mine;
            sh.need = need - above;
          }
        }
        __syncthreads();
        threshold = sh.prefix;
        need = sh.need;
        break;
      }
    }
  }
  // Kept: keys above the threshold (the ends' among them) and the first `need` equal to it.
  const bool any = threshold != kKeyEnd;
  const uint32_t above = any ? threshold : kKeyEnd - 1u;
  int x = 0, y = 0;
  auto count = [&] {
    x = y = 0;
#pragma unroll
    for (int i = 0; i < kEvictPer; ++i) {
      x += k[i] > above;
      y += any && k[i] == threshold;
    }
  };
  int2 carry = make_int2(0, 0), total, at = make_int2(0, 0);
  if (one_tile || ctas > 1) {
    each_tile([&](int) {
      count();
      at = evict_scan(sh, x, y, &total);
      carry.x += total.x;
      carry.y += total.y;
    });
  }
  if (ctas > 1) {
    if (tid == 0) {
      sh.cta_sum[0] = carry.x;
      sh.cta_sum[1] = carry.y;
    }
    cluster_barrier();
  }
  carry = make_int2(0, 0);
  for (int r = 0; r < rank; ++r) {
    carry.x += cluster_load(&sh.cta_sum[0], r);
    carry.y += cluster_load(&sh.cta_sum[1], r);
  }
  each_tile([&](int tile) {
    if (!one_tile) {
      count();
      at = evict_scan(sh, x, y, &total);
    }
    int eq = carry.y + at.y, place = carry.x + at.x + min(eq, need);
    const int t = tile + tid * kEvictPer;
#pragma unroll
    for (int i = 0; i < kEvictPer; ++i) {
      const bool is_eq = any && k[i] == threshold;
      if (k[i] > above || (is_eq && eq < need)) kept[place++] = t + i;
      eq += is_eq;
    }
    if (!one_tile) {
      carry.x += total.x;
      carry.y += total.y;
    }
  });
}

// grid (cluster, kv heads, sequences). In the move a strip is 16 << log_lanes bytes of the head's key or value
// row, and a step is one strip of a round, kMoveUnroll loads of 32 >> log_lanes rows a warp and CTA. The scores
// move with the rows.
__global__ void __launch_bounds__(kEvictThreads, kEvictPerSm)
evict_kernel(const EvictArgs a) {
  __shared__ EvictShared sh;
  grid_dependency_wait();
  grid_dependents_launch();
  const int rank = blockIdx.x, ctas = gridDim.x, h = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const size_t rowi = static_cast<size_t>(s) * a.num_kv_heads + h;
  int32_t* kept = a.kept + rowi * a.budget;
  const int L = a.context_lens[s];
  if (evict_len_invalid(L, a)) {  // the whole cluster alike
    if (tid == 0 && rank == 0) {
      atomicOr(a.error_word, PA_DEVERR_CONTEXT_LEN);
      if (h == 0) a.new_lens[s] = 0;
    }
    for (int j = rank * kEvictThreads + tid; j < a.budget; j += ctas * kEvictThreads) kept[j] = -1;
    return;
  }
  const float* w = a.scores + rowi * a.score_stride;
  float* wo = a.scores_out + rowi * a.score_stride;
  const int n = min(L, a.budget), bs = a.block_size, blocks = n > 0 ? (n - 1) / bs + 1 : 0;
  const int32_t* src = a.block_tables + static_cast<size_t>(s) * a.max_blocks_per_seq;
  const int32_t* dst = a.dst_tables + static_cast<size_t>(s) * a.max_dst_blocks_per_seq;
  const int from0 = tid < blocks ? src[tid] : 0, to0 = tid < blocks ? dst[tid] : -1;  // compared after the selection
  if (L <= a.budget) {
    for (int j = rank * kEvictThreads + tid; j < n; j += ctas * kEvictThreads) kept[j] = j;
  } else {
    evict_select(sh, a, L, rank, ctas, w, kept);
  }
  evict_sync(ctas);  // kept is complete; nothing reads this CTA's shared memory any more
  const int strips = (a.row_bytes + (16 << a.log_lanes) - 1) / (16 << a.log_lanes);
  const int rows = 32 >> a.log_lanes;                        // of one load
  const int log_round = kMoveLogLoads + 5 - a.log_lanes, round = 1 << log_round;  // rows of this CTA and round
  const size_t token_bytes = static_cast<size_t>(a.num_kv_heads) * a.row_bytes;
  const int log_bs = a.log_block;
  // Whether a slot that is written may be one that is read: every CTA of the cluster finds the same.
  bool same_block = from0 == to0;
  for (int i = tid + kEvictThreads; i < blocks; i += kEvictThreads) same_block = same_block || src[i] == dst[i];
  const bool over = __syncthreads_or(same_block);
  auto in_block = [&](int t) { return log_bs >= 0 ? t >> log_bs : t / bs; };
  const int row0 = warp * (kMoveUnroll * rows) + (lane >> a.log_lanes);
  const int lane_col = (lane & ((1 << a.log_lanes) - 1)) * 16;
  const int stage_rounds = kMoveStage / round;
  for (int lo = 0; lo < n; lo += stage_rounds * ctas * round) {
    // The stage's rounds are dealt over the CTAs in turn: row i of this CTA is token j.
    const int rounds = min(stage_rounds, (n - lo + ctas * round - 1) / (ctas * round));
    if (lo > 0) __syncthreads();
#pragma unroll 4
    for (int i = tid; i < rounds * round; i += kEvictThreads) {
      const int j = lo + (((i >> log_round) * ctas + rank) << log_round) + (i & (round - 1));
      uint32_t f = kNoMove;
      if (j < n) {
        const int t = kept[j];
        sh.score[i] = w[t];
        const int tb = in_block(t), jb = in_block(j);
        const int sb = src[tb], db = dst[jb];
        const uint32_t d = static_cast<uint32_t>(db) * bs + (j - jb * bs);
        if (sb < 0 || sb >= a.num_blocks || db < 0 || db >= a.num_blocks)
          atomicOr(a.error_word, PA_DEVERR_BLOCK_ID);
        else if ((f = static_cast<uint32_t>(sb) * bs + (t - tb * bs)) == d)
          f = kNoMove;
        sh.slots[kMoveStage + i] = d;
      }
      sh.slots[i] = f;
    }
    evict_sync(wo == w ? ctas : 1);  // in place, every CTA has read the stage's scores, which are now written over
    // Step = (round, strip); loads and stores have a cursor each, and go two steps at a time (keys and values are an
    // even number). The rows of later rounds come from slots above.
    struct Cursor {
      int round, strip;
      const uint32_t* from;
    };
    auto column = [&](int strip) {  // this lane's column of the strip; null when it has none
      const bool value = strip >= strips;
      const int col = ((value ? strip - strips : strip) << (a.log_lanes + 4)) + lane_col;
      if (col >= a.row_bytes) return static_cast<uint8_t*>(nullptr);
      return (value ? a.value_cache : a.key_cache) + static_cast<size_t>(h) * a.row_bytes + col;
    };
    auto next = [&](Cursor& c) {
      if (++c.strip == 2 * strips) {
        c.strip = 0;
        ++c.round;
        c.from += round;
      }
    };
    auto load = [&](uint4 (&x)[kMoveUnroll], Cursor& c) {
      if (c.round < rounds) {
        const uint8_t* base = column(c.strip);
#pragma unroll
        for (int i = 0; i < kMoveUnroll; ++i) {
          const uint32_t f = c.from[rows * i];
          if (base && f != kNoMove) x[i] = __ldcg(reinterpret_cast<const uint4*>(base + f * token_bytes));
        }
      }
      next(c);
    };
    auto store = [&](const uint4 (&x)[kMoveUnroll], Cursor& c) {
      uint8_t* base = column(c.strip);
#pragma unroll
      for (int i = 0; i < kMoveUnroll; ++i) {
        if (base && c.from[rows * i] != kNoMove)
          *reinterpret_cast<uint4*>(base + (c.from + kMoveStage)[rows * i] * token_bytes) = x[i];
      }
      next(c);
    };
    uint4 x0[kMoveUnroll], x1[kMoveUnroll];
    Cursor in{0, 0, sh.slots + row0}, out = in;
    while (out.round < rounds) {
      load(x0, in);
      load(x1, in);
      if (over) evict_sync(ctas);
      store(x0, out);
      store(x1, out);
    }
    for (int i = tid; i < rounds * round; i += kEvictThreads) {
      const int j = lo + (((i >> log_round) * ctas + rank) << log_round) + (i & (round - 1));
      if (j < n) wo[j] = sh.score[i];
    }
  }
  if (h == 0 && tid == 0 && rank == 0) a.new_lens[s] = n;
  for (int j = n + rank * kEvictThreads + tid; j < a.budget; j += ctas * kEvictThreads) kept[j] = -1;
  // The rest of the row starts from zero: every score has been read.
  for (int j = n + rank * kEvictThreads + tid; j < a.score_stride; j += ctas * kEvictThreads) wo[j] = 0.f;
}

}  // namespace pa
