// Rows on their way into an int8 product:
//
//   add_norm_q8     r = x + residual (fp32), residual_out = r in the residual's type
//                   y = r / sqrt(mean(r^2) + eps) * gamma                          (bf16)
//                   codes, scale with code * scale = y to half a code
//   quantize_rows   codes, scale of x itself
//
// The row's own factor rstd = 1/sqrt(mean(r^2) + eps) is common to all its values, so it cancels
// from the codes: with t = r * gamma and m = max|t|, code = round(127 t / m) and
// scale = m rstd / 127. The sum of squares and the maximum are therefore taken in one reduction
// over values that stay in registers (one pass over memory), and the codes depend on no sum:
// they are the exact nearest integers (ties to even) of 127 t / m for the fp32 t and m, the same
// on every run and for every block size. The quotient is first taken in fp32 (its error is under
// 127 * 4 * 2^-24 = 3.1e-5); only a value within 1e-4 of a border between two codes is decided
// again by comparing 127 t with (j + 1/2) m, both exact in fp64 (24 + 8 bits each).
//
// One block per row; a thread holds NV vectors of 8 neighbouring values (or, for rows that are
// not 16-byte aligned, 16 values a block apart). Bound by HBM: per value the bytes of x, the
// residual in and out, one code, and y where it is wanted.
#include <algorithm>
#include <type_traits>

#include "mla_internal.cuh"
#include "rows.cuh"

namespace mla {
namespace {

struct NormParams {
  const void* x;
  const void* res;        // nullptr: none
  void* res_out;
  const __nv_bfloat16* gamma;
  __nv_bfloat16* y;       // nullptr: not wanted
  int8_t* codes;          // nullptr: not wanted
  float* scales;
  int64_t x_stride, res_stride, res_out_stride, y_stride, codes_stride;   // elements
  int d;
  float eps;
};

struct NoResidual {};

// The low byte is the code: the integer nearest to 127 t / m (ties to even), with inv = 127 / m.
__device__ __forceinline__ uint32_t code_of(float t, float m, float inv) {
  constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer
  const float v = t * inv;
  float k = v + kMagic;
  if (fabsf(v - (k - kMagic)) > 0.4999f) {
    const double j = floor((double)v);   // the border is j + 1/2: fp32's v is within 1e-4 of it
    const double a = (double)t * 127.0, c = (double)m * (j + 0.5);
    const bool up = a > c || (a == c && fmod(j, 2.0) != 0.0);
    k = (float)(j + (up ? 1.0 : 0.0)) + kMagic;
  }
  return __float_as_uint(k);
}

// RT: the residual's type, or NoResidual. kVec: every row's pointers are aligned for 8 values at
// a time and d is a multiple of 8; value i of thread `tid`, vector n, is 8 (n blockDim + tid) + i,
// otherwise (8 n + i) blockDim + tid.
template <typename XT, typename RT, bool kNorm, int NV, bool kVec>
__global__ void __launch_bounds__(1024)
norm_q8_kernel(const NormParams p) {
  constexpr bool kRes = !std::is_same<RT, NoResidual>::value;
  __shared__ float part_ss[32];
  __shared__ uint32_t part_m[32];
  __shared__ double part_d[32];
  const int tid = threadIdx.x, nthr = blockDim.x, warp = tid >> 5, lane = tid & 31, warps = nthr >> 5;
  const int64_t row = blockIdx.x;
  const XT* x = static_cast<const XT*>(p.x) + row * p.x_stride;
  grid_dependency_wait();
  allow_dependent_launch();

  float r[NV][8], g[NV][8];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    if constexpr (kVec) {
      const int e = 8 * (n * nthr + tid);
      const bool in = e < p.d;
#pragma unroll
      for (int i = 0; i < 8; ++i) r[n][i] = 0.f, g[n][i] = 0.f;
      if (in) load8(x + e, r[n]);
      if constexpr (kNorm)
        if (in) load8(p.gamma + e, g[n]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = (8 * n + i) * nthr + tid;
        r[n][i] = e < p.d ? load1(x + e) : 0.f;
        if constexpr (kNorm) g[n][i] = e < p.d ? load1(p.gamma + e) : 0.f;
      }
    }
  }
  if constexpr (kRes) {
    const RT* res = static_cast<const RT*>(p.res) + row * p.res_stride;
    RT* out = static_cast<RT*>(p.res_out) + row * p.res_out_stride;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      if constexpr (kVec) {
        const int e = 8 * (n * nthr + tid);
        if (e < p.d) {
          float a[8];
          load8(res + e, a);
#pragma unroll
          for (int i = 0; i < 8; ++i) r[n][i] += a[i];
          store8(out + e, r[n]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = (8 * n + i) * nthr + tid;
          if (e < p.d) {
            r[n][i] += load1(res + e);
            store1(out + e, r[n][i]);
          }
        }
      }
    }
  }

  // one reduction: the sum of squares, and the largest |t| as the bits of a float, an order in
  // which infinity and NaN lie above every finite value
  float ss = 0.f;
  uint32_t mb = 0;
#pragma unroll
  for (int n = 0; n < NV; ++n)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (kNorm) ss = fmaf(r[n][i], r[n][i], ss);
      const float t = kNorm ? r[n][i] * g[n][i] : r[n][i];
      mb = max(mb, __float_as_uint(fabsf(t)));
    }
  if constexpr (kNorm) ss = warp_sum(ss);
  mb = __reduce_max_sync(0xffffffffu, mb);
  if (lane == 0) {
    part_ss[warp] = ss;
    part_m[warp] = mb;
  }
  __syncthreads();
  if constexpr (kNorm) ss = warp_sum(lane < warps ? part_ss[lane] : 0.f);
  mb = __reduce_max_sync(0xffffffffu, lane < warps ? part_m[lane] : 0u);

  float rstd = 1.f;
  if constexpr (kNorm) {
    rstd = 1.f / sqrtf(ss / (float)p.d + p.eps);
    // the squares of values over 1e19 or under 1e-19 leave fp32's range: sum them in fp64
    // (the same for all threads of the block)
    if (!(ss > 1e-30f && ss < 3e38f)) {
      double dd = 0.0;
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) dd += (double)r[n][i] * r[n][i];
      dd = warp_sum(dd);
      if (lane == 0) part_d[warp] = dd;
      __syncthreads();
      dd = warp_sum(lane < warps ? part_d[lane] : 0.0);
      rstd = (float)(1.0 / sqrt(dd / p.d + (double)p.eps));
    }
  }

  if (kNorm && p.y != nullptr) {
    __nv_bfloat16* y = p.y + row * p.y_stride;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = r[n][i] * rstd * g[n][i];
      if constexpr (kVec) {
        const int e = 8 * (n * nthr + tid);
        if (e < p.d) store8(y + e, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = (8 * n + i) * nthr + tid;
          if (e < p.d) store1(y + e, v[i]);
        }
      }
    }
  }
  if (p.codes == nullptr) return;
  const float m = __uint_as_float(mb);
  const bool finite = mb < 0x7F800000u;
  if (tid == 0)
    p.scales[row] = !finite ? __uint_as_float(0x7FC00000u) : m > 0.f ? m * rstd / 127.f : 0.f;
  // rows of very small values are scaled up by a power of two (exact), so that 127 / m is finite
  const float lift = m < 1e-30f ? 0x1p64f : 1.f;
  const float ml = m * lift, inv = finite && m > 0.f ? 127.f / ml : 0.f;
  int8_t* codes = p.codes + row * p.codes_stride;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = kNorm ? r[n][i] * g[n][i] : r[n][i];
      c[i] = inv > 0.f ? code_of(t * lift, ml, inv) : 0u;
    }
    if constexpr (kVec) {
      const int e = 8 * (n * nthr + tid);
      if (e < p.d) {
        const uint32_t lo = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        const uint32_t hi = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
        *reinterpret_cast<uint2*>(codes + e) = make_uint2(lo, hi);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = (8 * n + i) * nthr + tid;
        if (e < p.d) codes[e] = (int8_t)(c[i] & 0xFFu);
      }
    }
  }
}

bool rows_aligned(const void* p, int64_t stride, int elem, int rows_bytes) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % rows_bytes == 0 && stride * elem % rows_bytes == 0);
}

template <typename XT, typename RT, bool kNorm>
cudaError_t launch_typed(const NormParams& p, int64_t n_rows, cudaStream_t s) {
  constexpr bool kRes = !std::is_same<RT, NoResidual>::value;
  constexpr int res_size = kRes ? (std::is_same<RT, float>::value ? 4 : 2) : 1;
  const bool vec = p.d % 8 == 0 && rows_aligned(p.x, p.x_stride, sizeof(XT), 16) &&
                   rows_aligned(p.res, p.res_stride, res_size, 16) &&
                   rows_aligned(p.res_out, p.res_out_stride, res_size, 16) &&
                   rows_aligned(p.gamma, 0, 2, 16) && rows_aligned(p.y, p.y_stride, 2, 16) &&
                   rows_aligned(p.codes, p.codes_stride, 1, 8);
  const dim3 grid((unsigned)n_rows);
  const bool one = vec && p.d <= 8192;   // a vector of 8 per thread, else two
  const int per = one ? 8 : 16;
  const int threads = std::max(32, ((p.d + per - 1) / per + 31) / 32 * 32);
  if (one) return launch_pdl(norm_q8_kernel<XT, RT, kNorm, 1, true>, grid, dim3(threads), 0, s, p);
  if (vec) return launch_pdl(norm_q8_kernel<XT, RT, kNorm, 2, true>, grid, dim3(threads), 0, s, p);
  return launch_pdl(norm_q8_kernel<XT, RT, kNorm, 2, false>, grid, dim3(threads), 0, s, p);
}

}  // namespace

cudaError_t launch_norm_q8(const NormArgs& a, cudaStream_t s) {
  NormParams p{};
  p.x = a.x;
  p.res = a.residual;
  p.res_out = a.residual_out;
  p.gamma = a.gamma;
  p.y = a.y;
  p.codes = a.codes;
  p.scales = a.scales;
  p.x_stride = a.x_stride;
  p.res_stride = a.residual_stride;
  p.res_out_stride = a.residual_out_stride;
  p.y_stride = a.y_stride;
  p.codes_stride = a.codes_stride;
  p.d = a.d;
  p.eps = a.eps;
  if (a.gamma == nullptr)
    return a.x_f32 ? launch_typed<float, NoResidual, false>(p, a.n_rows, s)
                   : launch_typed<__nv_bfloat16, NoResidual, false>(p, a.n_rows, s);
  if (a.residual == nullptr)
    return a.x_f32 ? launch_typed<float, NoResidual, true>(p, a.n_rows, s)
                   : launch_typed<__nv_bfloat16, NoResidual, true>(p, a.n_rows, s);
  if (a.residual_f32)
    return a.x_f32 ? launch_typed<float, float, true>(p, a.n_rows, s)
                   : launch_typed<__nv_bfloat16, float, true>(p, a.n_rows, s);
  return a.x_f32 ? launch_typed<float, __nv_bfloat16, true>(p, a.n_rows, s)
                 : launch_typed<__nv_bfloat16, __nv_bfloat16, true>(p, a.n_rows, s);
}

}  // namespace mla
