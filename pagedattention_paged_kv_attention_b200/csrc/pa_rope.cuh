// pa_rope.cuh -- rotary positions with several axes, applied on the way into the paged cache.
//
// Rotary embedding turns pair i of a head's first R elements by the angle pos * inv_freq[i]. With several
// axes (time, height and width of an image or video token) the position of pair i is the token's
// position on axis freq_axis[i], so one table covers sections laid end to end, interleaved sections and
// frequency ladders of their own per axis:
//     a = positions[freq_axis[i]][token] * inv_freq[i]
//     (x, y) -> (x cos a - y sin a, y cos a + x sin a)
// for (x, y) = elements (i, i + R/2), or (2i, 2i + 1) when interleaved; elements R and above pass through.
//
// Angles. A 32-bit product pos * inv_freq is off by up to 2^-24 |a|: 0.03 rad at position 500,000. The
// turn count pos * inv_freq / (2 pi) is formed in 64 bits and reduced to [-1/2, 1/2] there, where it is
// exact to about 1e-10 turns; its sine and cosine are then taken in 32 bits (sincospif of twice the
// fraction, no argument reduction left to do). Rotation is in 32 bits, rounded once to the output type,
// or divided by the scale and rounded once to E4M3 (the division correctly rounded, as
// reshape_and_cache_kernel's), so an FP8 key never passes through a 16-bit rounding first.
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kRopeMaxRotary = 512;   // cos/sin table in shared memory
constexpr int kRopeThreads = 256;

struct RopeArgs {
  void* query_out;                    // rows of num_heads * head_size, query_out_stride apart (may be query itself)
  const void* query;
  const void* key;
  const void* value;
  void* key_cache;
  void* value_cache;
  const float* k_scale;
  const float* v_scale;
  const int64_t* slot_mapping;        // [num_tokens]
  const int32_t* positions;           // [num_axes][num_tokens]
  const float* inv_freq;              // [rotary / 2]
  const int32_t* freq_axis;           // [rotary / 2]
  int64_t query_out_stride, query_stride, key_stride, value_stride;  // elements between tokens
  int num_tokens, num_axes, num_heads, num_kv_heads, head_size, rotary, block_size, num_blocks, scale_stride;
};

// 8 floats as 8 elements of the cache: 16-bit (16 bytes) or E4M3 codes of x / scale (8 bytes).
template <typename T, typename KVT>
__device__ __forceinline__ void store8(KVT* dst, const float (&x)[8], float scale) {
  if constexpr (sizeof(KVT) == 1) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(
          make_float2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale)), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(
          make_float2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale)), __NV_SATFINITE, __NV_E4M3);
      w[i] = (lo & 0xffffu) | (hi << 16);
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
  }
}

template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&x)[8]) {
  const uint4 p = *reinterpret_cast<const uint4*>(src);
  float2 f[4];
  Elem<T>::to_float(p, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = f[i].x;
    x[2 * i + 1] = f[i].y;
  }
}

// One CTA per token: its cosines and sines go to shared memory once, then each thread turns units of 8
// pairs (two 16-byte vectors half a rotary width apart, or one vector of 4 interleaved pairs).
template <typename T, typename KVT, bool IL>
__global__ void __launch_bounds__(kRopeThreads)
rope_reshape_and_cache_kernel(const RopeArgs a) {
  __shared__ float cs[kRopeMaxRotary / 2], sn[kRopeMaxRotary / 2];
  const int64_t token = blockIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  const int half = a.rotary / 2;
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    const int axis = a.freq_axis[i];
    // An axis outside the table has no position: its pairs stay as they are.
    const int pos = axis >= 0 && axis < a.num_axes ? a.positions[static_cast<int64_t>(axis) * a.num_tokens + token] : 0;
    const double turns = static_cast<double>(pos) * (static_cast<double>(a.inv_freq[i]) * 0.15915494309189535);
    sincospif(2.0f * static_cast<float>(turns - rint(turns)), &sn[i], &cs[i]);
  }
  __syncthreads();
  const int64_t slot = a.slot_mapping[token];
  const bool cached = slot >= 0 && slot < static_cast<int64_t>(a.num_blocks) * a.block_size;
  const int64_t blk = cached ? slot / a.block_size : 0;
  const int d = a.head_size;
  const int64_t row = static_cast<int64_t>(a.num_kv_heads) * d;
  const T* q = static_cast<const T*>(a.query) + token * a.query_stride;
  T* qo = static_cast<T*>(a.query_out) + token * a.query_out_stride;
  const T* k = static_cast<const T*>(a.key) + token * a.key_stride;
  const T* v = static_cast<const T*>(a.value) + token * a.value_stride;
  KVT* kc = static_cast<KVT*>(a.key_cache) + (cached ? slot : 0) * row;
  KVT* vc = static_cast<KVT*>(a.value_cache) + (cached ? slot : 0) * row;

  // Units of a rotated head: rotary/16 pair units (or rotary/8 interleaved ones), then plain vectors.
  const int turned = IL ? a.rotary / 8 : a.rotary / 16;
  const int per_head = turned + (d - a.rotary) / 8;
  const int q_units = a.num_heads * per_head, k_units = a.num_kv_heads * per_head;
  const int v_units = static_cast<int>(row / 8);
  for (int u = threadIdx.x; u < q_units + (cached ? k_units + v_units : 0); u += blockDim.x) {
    if (u >= q_units + k_units) {  // values: moved (and encoded), not turned
      const int e = (u - q_units - k_units) * 8;
      float x[8];
      load8(v + e, x);
      store8<T>(vc + e, x, sizeof(KVT) == 1 ? a.v_scale[blk * a.scale_stride + e / d] : 1.f);
      continue;
    }
    const bool is_q = u < q_units;
    const int r = is_q ? u : u - q_units;
    const int h = r / per_head, j = r - h * per_head;
    const T* src = (is_q ? q : k) + h * d;
    const float scale = (sizeof(KVT) == 1 && !is_q) ? a.k_scale[blk * a.scale_stride + h] : 1.f;
    float x[8], y[8];
    int e0, e1 = -1;
    if (j >= turned) {
      e0 = a.rotary + (j - turned) * 8;
      load8(src + e0, x);
    } else if constexpr (IL) {
      e0 = j * 8;
      load8(src + e0, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float c = cs[j * 4 + i], s = sn[j * 4 + i], p = x[2 * i], o = x[2 * i + 1];
        x[2 * i] = p * c - o * s;
        x[2 * i + 1] = o * c + p * s;
      }
    } else {
      e0 = j * 8;
      e1 = e0 + half;
      load8(src + e0, x);
      load8(src + e1, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = cs[e0 + i], s = sn[e0 + i], p = x[i], o = y[i];
        x[i] = p * c - o * s;
        y[i] = o * c + p * s;
      }
    }
    if (is_q) {
      store8<T>(qo + h * d + e0, x, 1.f);
      if (e1 >= 0) store8<T>(qo + h * d + e1, y, 1.f);
    } else {
      store8<T>(kc + h * d + e0, x, scale);
      if (e1 >= 0) store8<T>(kc + h * d + e1, y, scale);
    }
  }
}

}  // namespace pa
