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
constexpr int kRopeMaxHead = 8192;    // so that inv_units is exact: unit count x units of a head <= 2^32
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
  int num_tokens, num_axes, num_heads, num_kv_heads, head_size, rotary, block_size, num_blocks, scale_stride,
      units;                          // of a head: those of rotated pairs, and plain vectors
  // ceil(2^32 / units) (0: one unit) and ceil(2^32 / (head_size / 8)): a quotient is a product's high word.
  unsigned inv_units, inv_plain;
};

// E4M3 codes of x / scale, as __fdiv_rn and a conversion give them. The product with 1 / scale is within 2 units
// of the last place of the quotient, so both round to one code unless it lies that near a border between
// codes (a midpoint of 4-bit significands), or below the normal range, where borders sit elsewhere; then, for
// about 1 unit of 8 values in 500, the division is made.
__device__ __forceinline__ uint2 encode8(float (&x)[8], float scale) {
  const float inv = 1.0f / scale;
  float q[8];
  bool near = !(inv > 1e-30f && inv < 1e30f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = x[i] * inv;
    near = near || (__float_as_uint(q[i]) & 0xfffffu) - 0x7fffcu <= 8u || fabsf(q[i]) < 0.03125f;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(x[i], scale);
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i], q[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[4 * i + 2], q[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
    w[i] = (lo & 0xffffu) | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& p, float (&x)[8]) {
  float2 f[4];
  Elem<T>::to_float(p, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = f[i].x;
    x[2 * i + 1] = f[i].y;
  }
}

// One CTA per token. Its threads turn units of 8 pairs (two 16-byte vectors half a rotary width apart) or of 4
// interleaved pairs (one vector), and move plain vectors. A CTA lives for two chains of loads, positions ->
// cosines and sines (in shared memory) and the token's vectors, so a thread fetches its first unit before
// the cosines are formed. Threads per CTA: 96 to 256 measure alike (16384 tokens, 64 / 8 heads: 105 us, 97% of the copy
// bandwidth), 512 a fifth slower, 1024 half as slow again: fewer CTAs are at different points of their chains.
template <typename T, typename KVT, bool IL>
__global__ void __launch_bounds__(kRopeThreads, 8)
rope_reshape_and_cache_kernel(const RopeArgs a) {
  __shared__ __align__(16) float cs[kRopeMaxRotary / 2], sn[kRopeMaxRotary / 2];
  constexpr bool kFp8 = sizeof(KVT) == 1;
  const int64_t token = blockIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  const int d = a.head_size, half = a.rotary / 2;
  const int64_t row = static_cast<int64_t>(a.num_kv_heads) * d;
  // Units of a rotated head: rotary/16 pair units (or rotary/8 interleaved ones), then plain vectors.
  const int turned = IL ? a.rotary / 8 : a.rotary / 16;
  const int per_head = a.units;
  const int q_units = a.num_heads * per_head, qk_units = q_units + a.num_kv_heads * per_head;
  const int all_units = qk_units + static_cast<int>(row / 8);  // values: moved (and encoded), not turned
  // Unit u: its first element, and its second vector's (-1: none), from the start of its head's tensor.
  struct Unit {
    int h, j, e0, e1;
  };
  auto place = [&](int u) {
    Unit w;
    if (u >= qk_units) {
      w.e0 = (u - qk_units) * 8;
      w.h = static_cast<int>(__umulhi(u - qk_units, a.inv_plain));  // (u - qk_units) / (d / 8)
      w.j = turned;
      w.e1 = -1;
      return w;
    }
    const int r = u < q_units ? u : u - q_units;
    w.h = a.inv_units ? static_cast<int>(__umulhi(r, a.inv_units)) : r;  // r / per_head
    w.j = r - w.h * per_head;
    w.e0 = w.h * d + (w.j >= turned ? a.rotary + (w.j - turned) * 8 : w.j * 8);
    w.e1 = !IL && w.j < turned ? w.e0 + half : -1;
    return w;
  };
  uint4 p0, p1;
  auto fetch = [&](int u, const Unit& w) {
    const T* src = u >= qk_units  ? static_cast<const T*>(a.value) + token * a.value_stride
                   : u >= q_units ? static_cast<const T*>(a.key) + token * a.key_stride
                                  : static_cast<const T*>(a.query) + token * a.query_stride;
    p0 = *reinterpret_cast<const uint4*>(src + w.e0);
    if (w.e1 >= 0) p1 = *reinterpret_cast<const uint4*>(src + w.e1);
  };
  int u = threadIdx.x;
  Unit w = place(u);
  if (u < all_units) fetch(u, w);
  const int64_t slot = a.slot_mapping[token];
  for (int i = threadIdx.x; i < half; i += blockDim.x) {
    const int axis = a.freq_axis[i];
    // An axis outside the table has no position: its pairs are turned by 0, whatever their frequency holds.
    const bool known = axis >= 0 && axis < a.num_axes;
    const int pos = known ? a.positions[static_cast<int64_t>(axis) * a.num_tokens + token] : 0;
    const float freq = known ? a.inv_freq[i] : 0.f;
    const double turns = static_cast<double>(pos) * (static_cast<double>(freq) * 0.15915494309189535);
    sincospif(2.0f * static_cast<float>(turns - rint(turns)), &sn[i], &cs[i]);
  }
  __syncthreads();
  const bool cached = slot >= 0 && slot < static_cast<int64_t>(a.num_blocks) * a.block_size;
  const int units = cached ? all_units : q_units;
  while (u < units) {
    float x[8], y[8];
    if (kFp8 || w.j < turned) {
      unpack8<T>(p0, x);
      if (!IL && w.e1 >= 0) unpack8<T>(p1, y);
    }
    if (w.j < turned) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        if constexpr (IL) {
          const float2 c = *reinterpret_cast<const float2*>(&cs[w.j * 4 + i / 2]);
          const float2 s = *reinterpret_cast<const float2*>(&sn[w.j * 4 + i / 2]);
          float q = x[i], o = x[i + 1];
          x[i] = q * c.x - o * s.x;
          x[i + 1] = o * c.x + q * s.x;
          q = x[i + 2], o = x[i + 3];
          x[i + 2] = q * c.y - o * s.y;
          x[i + 3] = o * c.y + q * s.y;
        } else {
          const float4 c4 = *reinterpret_cast<const float4*>(&cs[w.j * 8 + i]);
          const float4 s4 = *reinterpret_cast<const float4*>(&sn[w.j * 8 + i]);
          const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float q = x[i + k], o = y[i + k];
            x[i + k] = q * c[k] - o * s[k];
            y[i + k] = o * c[k] + q * s[k];
          }
        }
      }
      p0 = make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
      if constexpr (!IL)
        p1 = make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
    }
    if (!kFp8 || u < q_units) {
      T* dst = u < q_units ? static_cast<T*>(a.query_out) + token * a.query_out_stride
                           : static_cast<T*>(u < qk_units ? a.key_cache : a.value_cache) + slot * row;
      *reinterpret_cast<uint4*>(dst + w.e0) = p0;
      if (w.e1 >= 0) *reinterpret_cast<uint4*>(dst + w.e1) = p1;
    } else {
      const float scale =
          (u < qk_units ? a.k_scale : a.v_scale)[slot / a.block_size * a.scale_stride + w.h];
      uint8_t* dst = static_cast<uint8_t*>(u < qk_units ? a.key_cache : a.value_cache) + slot * row;
      *reinterpret_cast<uint2*>(dst + w.e0) = encode8(x, scale);
      if (w.e1 >= 0) *reinterpret_cast<uint2*>(dst + w.e1) = encode8(y, scale);
    }
    u += blockDim.x;
    if (u >= units) break;
    w = place(u);
    fetch(u, w);
  }
}

}  // namespace pa
