// Vectors of neighbouring row values, bf16 or fp32 in memory and fp32 in registers.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace mla {

__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }

// a in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// two E4M3 codes, a in the low byte (nearest, ties to even, saturating at +-448)
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  uint32_t c;
  asm("{ .reg .b16 t; cvt.rn.satfinite.e4m3x2.f32 t, %1, %2; cvt.u32.u16 %0, t; }" : "=r"(c) : "f"(b), "f"(a));
  return c;
}
// max(a, |b|, |c|), and NaN if one of them is
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Eight values as loaded, in pairs: W neighbouring ones at p, W more at p + step, and so on while
// they lie before `left` values from p.
template <typename T, int W>
struct Raw8;
template <int W>
struct Raw8<__nv_bfloat16, W> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int step, int left) {
#pragma unroll
    for (int c = 0; c < 8 / W; ++c) {
      const __nv_bfloat16* q = p + (int64_t)c * step;
      const bool in = c * step < left;
      if constexpr (W == 8) {
        const uint4 u = in ? *reinterpret_cast<const uint4*>(q) : make_uint4(0, 0, 0, 0);
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
      } else if constexpr (W == 4) {
        const uint2 u = in ? *reinterpret_cast<const uint2*>(q) : make_uint2(0, 0);
        w[2 * c] = u.x; w[2 * c + 1] = u.y;
      } else if constexpr (W == 2) {
        w[c] = in ? *reinterpret_cast<const uint32_t*>(q) : 0u;
      } else {
        const uint32_t u = in ? *reinterpret_cast<const uint16_t*>(q) : 0u;
        w[c >> 1] = c & 1 ? w[c >> 1] | u << 16 : u;
      }
    }
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  // m = max(m, |values|), NaN above all (as their bits order them, two at a time)
  __device__ __forceinline__ void largest(float& m) const {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) a = __vmaxu2(a, w[i] & 0x7FFF7FFFu);
    m = max_abs_nan(m, __uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u));
  }
};
template <int W>
struct Raw8<float, W> {
  float2 v[4];
  __device__ __forceinline__ void load(const float* p, int step, int left) {
#pragma unroll
    for (int c = 0; c < 8 / W; ++c) {
      const float* q = p + (int64_t)c * step;
      const bool in = c * step < left;
      if constexpr (W >= 4) {
#pragma unroll
        for (int h = 0; h < W / 4; ++h) {
          const float4 a = in ? reinterpret_cast<const float4*>(q)[h] : make_float4(0.f, 0.f, 0.f, 0.f);
          v[c * W / 2 + 2 * h] = make_float2(a.x, a.y);
          v[c * W / 2 + 2 * h + 1] = make_float2(a.z, a.w);
        }
      } else if constexpr (W == 2) {
        v[c] = in ? *reinterpret_cast<const float2*>(q) : make_float2(0.f, 0.f);
      } else {
        const float a = in ? *q : 0.f;
        if (c & 1) v[c >> 1].y = a;
        else v[c >> 1].x = a;
      }
    }
  }
  __device__ __forceinline__ float2 pair(int i) const { return v[i]; }
  __device__ __forceinline__ void largest(float& m) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max_abs_nan(m, v[i].x, v[i].y);
  }
};

template <int W>
__device__ __forceinline__ void store_pairs(float* p, int step, int left, const float2 (&v)[4]) {
#pragma unroll
  for (int c = 0; c < 8 / W; ++c) {
    if (c * step >= left) continue;
    float* q = p + (int64_t)c * step;
    if constexpr (W >= 4) {
#pragma unroll
      for (int h = 0; h < W / 4; ++h) {
        const float2 a = v[c * W / 2 + 2 * h], b = v[c * W / 2 + 2 * h + 1];
        reinterpret_cast<float4*>(q)[h] = make_float4(a.x, a.y, b.x, b.y);
      }
    } else if constexpr (W == 2) {
      *reinterpret_cast<float2*>(q) = v[c];
    } else {
      *q = c & 1 ? v[c >> 1].y : v[c >> 1].x;
    }
  }
}
template <int W>
__device__ __forceinline__ void store_pairs(__nv_bfloat16* p, int step, int left, const float2 (&v)[4]) {
#pragma unroll
  for (int c = 0; c < 8 / W; ++c) {
    if (c * step >= left) continue;
    __nv_bfloat16* q = p + (int64_t)c * step;
    if constexpr (W == 8)
      *reinterpret_cast<uint4*>(q) = make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y),
                                                pack_bf16(v[2].x, v[2].y), pack_bf16(v[3].x, v[3].y));
    else if constexpr (W == 4)
      *reinterpret_cast<uint2*>(q) = make_uint2(pack_bf16(v[2 * c].x, v[2 * c].y), pack_bf16(v[2 * c + 1].x, v[2 * c + 1].y));
    else if constexpr (W == 2)
      *reinterpret_cast<uint32_t*>(q) = pack_bf16(v[c].x, v[c].y);
    else
      *q = __float2bfloat16_rn(c & 1 ? v[c >> 1].y : v[c >> 1].x);
  }
}
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace mla
