// Rows on their way into an int8 product:
//
//   add_norm_q8     r = x + residual (fp32), residual_out = r in the residual's type
//                   t = r * gamma (fp32), rstd = 1 / sqrt(mean(r^2) + eps), y = t * rstd (bf16)
//                   codes, scale with code * scale = y to half a code
//   quantize_rows   codes, scale of t = x itself, rstd = 1
//
// rstd is common to a row's values, so it cancels from the codes: with m = max|t|,
// code = round(127 t / m) and scale = m rstd / 127. The sum of squares and the maximum are therefore
// taken in one reduction over values that stay in registers (one pass over memory), and the codes
// depend on no sum: they are the nearest integers (ties to even) of 127 t / m for the fp32 t and m,
// the same on every run and for every layout. The integer is first taken from t * (127 / m) in fp32,
// off by the reciprocal's rounding, under 127 * 2^-24 = 7.6e-6; where the distance to it exceeds
// 0.49998 the side of the border is decided by 127 t - border * m, exact in fp64.
//
// A group of threads takes a row: 8, 16 or 32 lanes up to 1024 values, a block of its own beyond. A
// thread holds NV vectors of 8 values of t (neighbours where rows are 16-byte aligned) and nothing
// else across the reduction. Bound by HBM: per value the bytes of x, the residual in and out, one
// code, and y where it is wanted; rows of bf16 without a residual also by the issue slots (11
// instructions per value with packed fp32 pairs and two- and three-way maxima). Measured: 4096 x 5120
// bf16 with an fp32 residual and y 42.4 us (6430 GB/s); 2048 x 16384 bf16 quantised 19.8 us (5090 GB/s),
// the same in fp32 26.3 us (6390 GB/s); one row of 5120 2.1 us, the launch and one round trip. Rows of odd
// width, one value at a time, take up to twice as long (4882 x 4095 against 4096, bf16: 22.7 and 13.0 us).
#include <algorithm>
#include <type_traits>

#include "mla_internal.cuh"
#include "rows.cuh"
#include "sm100_i8.cuh"

namespace mla {
namespace {

constexpr int kGroupThreads = 256;   // threads of a block whose lanes take a row in groups

struct NormParams {
  int64_t n_rows;
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

template <int W>
__device__ __forceinline__ void store_codes(int8_t* p, int step, int left, uint2 v) {
#pragma unroll
  for (int c = 0; c < 8 / W; ++c) {
    if (c * step >= left) continue;
    int8_t* q = p + (int64_t)c * step;
    if constexpr (W == 8) *reinterpret_cast<uint2*>(q) = v;
    else if constexpr (W == 4) *reinterpret_cast<uint32_t*>(q) = c ? v.y : v.x;
    else if constexpr (W == 2) *reinterpret_cast<uint16_t*>(q) = (uint16_t)((c & 2 ? v.y : v.x) >> (16 * (c & 1)));
    else *q = (int8_t)((c & 4 ? v.y : v.x) >> (8 * (c & 3)));
  }
}

// A row's statistics so far. The squares of values over 1e15 or under 1e-13 go to an fp64 sum, so
// that none of them leaves fp32's range and none is lost.
struct Stats {
  float ss = 0.f, m = 0.f;
  double dd = 0.0;
  __device__ __forceinline__ void squares(const float2 (&r)[4]) {
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) s2 = sm100::ffma2(r[i], r[i], s2);
    const float s = s2.x + s2.y;
    if (s > 1e-25f && s < 1e30f) {
      ss += s;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) dd = fma((double)r[i].x, (double)r[i].x, fma((double)r[i].y, (double)r[i].y, dd));
    }
  }
  __device__ __forceinline__ void largest(const float2 (&t)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max_abs_nan(m, t[i].x, t[i].y);
  }
};

constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer in the low bits

// The same integer for a value near the border between two, decided by the sign of 127 t - border * m
// (24 + 8 bits each: exact in fp64), ties to even. k: kMagic + the nearest integer by fp32.
__device__ __forceinline__ float at_border(float k, float t, float m, float inv) {
  const float j = k - kMagic, e = fmaf(t, inv, -j);
  if (!(fabsf(e) > 0.49998f)) return k;
  const double over = fma(-(double)m, (double)(j + copysignf(0.5f, e)), (double)t * 127.0);
  const bool odd = __float_as_uint(k) & 1u;
  if (e > 0.f) return over > 0.0 || (over == 0.0 && odd) ? k + 1.f : k;
  return over < 0.0 || (over == 0.0 && odd) ? k - 1.f : k;
}

// Eight codes, the integers nearest to 127 t / m, ties to even; inv = 127 / m (0: a row of zeros).
__device__ __forceinline__ uint2 codes8(const float2 (&t)[4], float m, float inv) {
  const float2 inv2 = make_float2(inv, inv), magic = make_float2(kMagic, kMagic), minus = make_float2(-1.f, -1.f);
  float2 k[4];
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    k[i] = sm100::ffma2(t[i], inv2, magic);
    const float2 j = sm100::ffma2(k[i], minus, magic);   // minus the integer
    const float2 e = sm100::ffma2(t[i], inv2, j);
    off = max_abs(off, e.x, e.y);
  }
  if (off > 0.49998f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      k[i].x = at_border(k[i].x, t[i].x, m, inv);
      k[i].y = at_border(k[i].y, t[i].y, m, inv);
    }
  }
  const auto pack = [](const float2& a, const float2& b) {
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
  };
  return make_uint2(pack(k[0], k[1]), pack(k[2], k[3]));
}

// RT: the residual's type, or NoResidual. G: the lanes that share a row, or 0: a block per row. W:
// the values that all rows' pointers are aligned for (d is a multiple). With nthr threads per row,
// vector n of thread `tid` is 8/W pieces, piece c the W values from W ((8/W n + c) nthr + tid) on.
template <typename XT, typename RT, bool kNorm, int NV, int W, int G>
__global__ void __launch_bounds__(G > 0 ? kGroupThreads : NV > 2 ? 512 : 1024,
                                  G > 0 ? 1 : NV > 2 ? (!kNorm && sizeof(XT) == 2 ? 3 : 2) : 1)
norm_q8_kernel(const NormParams p) {
  constexpr bool kRes = !std::is_same<RT, NoResidual>::value;
  using Res = typename std::conditional<kRes, RT, float>::type;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tid = G > 0 ? (int)threadIdx.x % (G > 0 ? G : 1) : (int)threadIdx.x, nthr = G > 0 ? G : (int)blockDim.x;
  int64_t row = blockIdx.x;
  if (G > 0) row = row * (kGroupThreads / (G > 0 ? G : 1)) + threadIdx.x / (G > 0 ? G : 1);
  grid_dependency_wait();
  allow_dependent_launch();
  // groups behind the last row take part in the warp's exchanges, with nothing to read or write
  const int d = G == 0 || row < p.n_rows ? p.d : 0;
  const XT* x = static_cast<const XT*>(p.x) + row * p.x_stride;
  const Res* res = static_cast<const Res*>(p.res) + row * p.res_stride;
  Res* res_out = static_cast<Res*>(p.res_out) + row * p.res_out_stride;
  const int step = W * nthr;

  // what stays in registers across the reduction: t, or x as loaded where that is t
  float2 t[kNorm ? NV : 1][4];
  Raw8<XT, W> rx[NV];
  Stats st;
  if constexpr (!kNorm) {
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int e = W * (8 / W * n * nthr + tid);
      rx[n].load(x + e, step, d - e);
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) rx[n].largest(st.m);
  } else {
    Raw8<Res, W> rr[NV];
    Raw8<__nv_bfloat16, W> rg[NV];
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int e = W * (8 / W * n * nthr + tid);
      rx[n].load(x + e, step, d - e);
      if constexpr (kRes) rr[n].load(res + e, step, d - e);
      rg[n].load(p.gamma + e, step, d - e);
    }
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int e = W * (8 / W * n * nthr + tid);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t[n][i] = rx[n].pair(i);
        if constexpr (kRes) t[n][i] = sm100::fadd2(t[n][i], rr[n].pair(i));
      }
      if constexpr (kRes) store_pairs<W>(res_out + e, step, d - e, t[n]);
      st.squares(t[n]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 g = rg[n].pair(i);
        t[n][i] = sm100::fmul2(t[n][i], g);
      }
      st.largest(t[n]);
    }
  }

  // the row's maximum and sum of squares
  uint32_t mb = __float_as_uint(st.m);   // NaN above infinity above all
  float ss = st.ss;
  bool wide = st.dd != 0.0;   // NaN too
  double dd = st.dd;
  if constexpr (G > 0) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    if constexpr (kNorm) {
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      wide = __any_sync(0xffffffffu, wide);
      if (wide) {
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1) dd += __shfl_xor_sync(0xffffffffu, dd, o);
      }
    }
  } else {
    __shared__ float part_ss[32];
    __shared__ uint32_t part_m[32];
    const int warps = nthr >> 5;
    mb = __reduce_max_sync(0xffffffffu, mb);
    if constexpr (kNorm) ss = warp_sum(ss);
    if (lane == 0) {
      part_ss[warp] = ss;
      part_m[warp] = mb;
    }
    if constexpr (kNorm) wide = __syncthreads_or(wide);
    else __syncthreads();
    mb = __reduce_max_sync(0xffffffffu, lane < warps ? part_m[lane] : 0u);
    if constexpr (kNorm) {
      ss = warp_sum(lane < warps ? part_ss[lane] : 0.f);
      if (wide) {   // the same for the whole block
        __shared__ double part_d[32];
        dd = warp_sum(dd);
        if (lane == 0) part_d[warp] = dd;
        __syncthreads();
        dd = warp_sum(lane < warps ? part_d[lane] : 0.0);
      }
    }
  }
  float rstd = 1.f;
  if constexpr (kNorm) {
    rstd = 1.f / sqrtf(ss / (float)p.d + p.eps);
    // Without an eps 1 / rms of a row of subnormal values lies beyond fp32: minus 2^-64 times it stands for
    // it, and the 2^64 go onto t and m by themselves (exact): with another product for y, or in place for
    // odd widths, whose kernels have no registers left (13000 x 1537 fp32, bf16 residual 79.5 us with the
    // product, 74.0 in place, 72.8 without either; 4096 x 5120 bf16 16.5, 17.1 and 16.4).
    if (wide && dd != 0.0) {
      const double exact = 1.0 / sqrt((dd + (double)ss) / p.d + (double)p.eps);
      rstd = (float)(exact > 0x1p100 ? exact * -0x1p-64 : exact);
    }
    if constexpr (W == 1) {
      if (rstd < 0.f) {
        rstd = -rstd;
        if (mb < 0x7F800000u) mb = __float_as_uint(__uint_as_float(mb) * 0x1p64f);
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) t[n][i] = make_float2(t[n][i].x * 0x1p64f, t[n][i].y * 0x1p64f);
      }
    }
    if (p.y != nullptr) {
      __nv_bfloat16* y = p.y + row * p.y_stride;
      const float up = rstd < 0.f ? 0x1p64f : 1.f;
      const float size = W == 1 ? rstd : fabsf(rstd);
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int e = W * (8 / W * n * nthr + tid);
        float2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = sm100::fmul2(W == 1 ? t[n][i] : sm100::fmul2(t[n][i], make_float2(up, up)), make_float2(size, size));
        store_pairs<W>(y + e, step, d - e, v);
      }
    }
    if (p.codes == nullptr) return;
  }
  float m = __uint_as_float(mb);
  const bool finite = mb < 0x7F800000u;
  if (tid == 0 && d > 0)
    p.scales[row] = !finite ? __uint_as_float(0x7FC00000u)
                    : m > 0.f ? (W > 1 && rstd < 0.f ? m * 0x1p64f * -rstd : m * rstd) / 127.f : 0.f;
  // below 1e-30, where 127 / m may overflow, the row is scaled up by a power of two (exact)
  float lift = 1.f;
  if (m < 1e-30f) {
    lift = 0x1p100f;
    m *= lift;
  }
  const float inv = finite && m > 0.f ? 127.f / m : 0.f;
  int8_t* codes = p.codes + row * p.codes_stride;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int e = W * (8 / W * n * nthr + tid);
    uint2 c = make_uint2(0u, 0u);
    float2(&v)[4] = t[kNorm ? n : 0];
    if constexpr (!kNorm) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = rx[n].pair(i);
    }
    if (finite) {
      if (lift != 1.f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = make_float2(v[i].x * lift, v[i].y * lift);
      }
      c = codes8(v, m, inv);
    }
    store_codes<W>(codes + e, step, d - e, c);
  }
}

template <typename XT, typename RT, bool kNorm, int NV, int W, int G>
cudaError_t launch_shape(const NormParams& p, cudaStream_t s) {
  const auto kernel = norm_q8_kernel<XT, RT, kNorm, NV, W, G>;
  if constexpr (G > 0) {
    constexpr int kRows = kGroupThreads / G;
    return launch_pdl(kernel, dim3((unsigned)((p.n_rows + kRows - 1) / kRows)), dim3(kGroupThreads), 0, s, p);
  } else {
    constexpr int per = 8 * NV;
    return launch_pdl(kernel, dim3((unsigned)p.n_rows), dim3(((p.d + per - 1) / per + 31) / 32 * 32), 0, s, p);
  }
}

// Rows with less than 16-byte alignment. Four values at a time against two: 1200 x 16380 bf16 with an fp32
// residual and y 44.7 and 52.0 us, 4882 x 4100 bf16 quantised 15.9 and 16.9; two against one: 10000 x 1022
// with the residual and y 22.4 and 37.3 us, 2441 x 8194 bf16 quantised 18.7 and 51.0.
template <typename XT, typename RT, bool kNorm, int W>
cudaError_t launch_narrow(const NormParams& p, cudaStream_t s) {
  if (p.d <= 256) return launch_shape<XT, RT, kNorm, 1, W, 32>(p, s);
  if (p.d <= 512) return launch_shape<XT, RT, kNorm, 2, W, 32>(p, s);
  if (p.d <= 1024) return launch_shape<XT, RT, kNorm, 4, W, 32>(p, s);
  // (4882 x 4095 bf16 quantised 22.7 against 27.7 us, in fp32 22.9 against 19.7; 2441 x 8191 36 against 31)
  if constexpr (sizeof(XT) == 2)
    if (p.d <= 4096) return launch_shape<XT, RT, kNorm, 1, W, 0>(p, s);
  return launch_shape<XT, RT, kNorm, 2, W, 0>(p, s);
}

template <typename XT, typename RT, bool kNorm>
cudaError_t launch_typed(const NormParams& p, int num_sms, cudaStream_t s) {
  constexpr bool kRes = !std::is_same<RT, NoResidual>::value;
  constexpr int kResSize = kRes ? (std::is_same<RT, float>::value ? 4 : 2) : 1;
  // the largest W for which d is a multiple and each row starts on W values or 16 bytes
  int w = 8;
  const auto fit = [&w](const void* q, int64_t stride, int elem) {
    while (q != nullptr && w > 1) {
      const int bytes = std::min(16, w * elem);
      if (reinterpret_cast<uintptr_t>(q) % bytes == 0 && stride * elem % bytes == 0) break;
      w /= 2;
    }
  };
  while (p.d % w != 0) w /= 2;
  fit(p.x, p.x_stride, sizeof(XT));
  fit(p.res, p.res_stride, kResSize);
  fit(p.res_out, p.res_out_stride, kResSize);
  fit(p.gamma, 0, 2);
  fit(p.y, p.y_stride, 2);
  fit(p.codes, p.codes_stride, 1);
  if (w == 4) return launch_narrow<XT, RT, kNorm, 4>(p, s);
  if (w == 2) return launch_narrow<XT, RT, kNorm, 2>(p, s);
  if (w == 1) return launch_narrow<XT, RT, kNorm, 1>(p, s);
  if (p.d <= 64) return launch_shape<XT, RT, kNorm, 1, 8, 8>(p, s);
  if (p.d <= 128) return launch_shape<XT, RT, kNorm, 1, 8, 16>(p, s);
  if (p.d <= 256) return launch_shape<XT, RT, kNorm, 1, 8, 32>(p, s);
  if (p.d <= 512) return launch_shape<XT, RT, kNorm, 2, 8, 32>(p, s);
  if (p.d <= 768) return launch_shape<XT, RT, kNorm, 3, 8, 32>(p, s);
  if (p.d <= 1024) return launch_shape<XT, RT, kNorm, 4, 8, 32>(p, s);
  // A little over 1024 values fill a block of their own badly: five vectors a lane where rows are many
  // and no residual takes registers (16276 x 1232 bf16 quantised 13.2 against 18.1 us; with an fp32
  // residual 35.1 against 34.3 us; 2048 values in eight vectors 15.3 against 12.8 us).
  if constexpr (!kRes)
    if (p.d <= 1280 && p.n_rows >= 32 * num_sms) return launch_shape<XT, RT, kNorm, 5, 8, 32>(p, s);
  // Block per row. A row alone on its SM is bound by latency, and more threads with a vector each
  // shorten it (1 x 5120: 1.95 against 2.3 us). Many rows want two vectors in flight per thread (2441 x
  // 8192 bf16 quantised 13.4 against 16.9 us), and where nothing is fp32 beside a residual four, with half
  // the threads, so that rows load while others are stored: 4096 x 5120 bf16, normed, 16.4 against 19.4
  // us, with a bf16 residual 23.7 against 25.6; with fp32 in it 43.9 against 42.2 (registers), and
  // 2000 x 4096 quantised 7.5 against 6.9 (too few rows to fill the SMs with small blocks).
  if (p.n_rows <= num_sms && p.d <= 8192) return launch_shape<XT, RT, kNorm, 1, 8, 0>(p, s);
  constexpr bool kFour = !kRes || (sizeof(XT) == 2 && kResSize == 2);
  if constexpr (kFour)
    if (p.d >= 2048 && p.n_rows * p.d >= (int64_t)num_sms * 81920)
      return launch_shape<XT, RT, kNorm, 4, 8, 0>(p, s);
  return launch_shape<XT, RT, kNorm, 2, 8, 0>(p, s);
}

}  // namespace

cudaError_t launch_norm_q8(const mla_decode_s& h, const NormArgs& a, cudaStream_t s) {
  NormParams p{};
  p.n_rows = a.n_rows;
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
  using BF = __nv_bfloat16;
  const int sms = h.num_sms;
  if (a.gamma == nullptr)
    return a.x_f32 ? launch_typed<float, NoResidual, false>(p, sms, s) : launch_typed<BF, NoResidual, false>(p, sms, s);
  if (a.residual == nullptr)
    return a.x_f32 ? launch_typed<float, NoResidual, true>(p, sms, s) : launch_typed<BF, NoResidual, true>(p, sms, s);
  if (a.residual_f32)
    return a.x_f32 ? launch_typed<float, float, true>(p, sms, s) : launch_typed<BF, float, true>(p, sms, s);
  return a.x_f32 ? launch_typed<float, BF, true>(p, sms, s) : launch_typed<BF, BF, true>(p, sms, s);
}

}  // namespace mla
