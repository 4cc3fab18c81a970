// The cache write of rows that are projected already (the 576 columns [W_DKV ; W_KR] h of a
// fused down-projection):
//
//   row = [ x[0:512] / sqrt(mean(x[0:512]^2) + eps) * gamma ; RoPE_p(x[512:576]) ]
//
// as bf16, or as E4M3 codes with the row's smallest power-of-two scale, at token p of its
// sequence. Rows are ragged: row i belongs to the sequence b with row_starts[b] <= i <
// row_starts[b+1], at position p = kv_lens[b] - row_starts[b+1] + i, so prompts, single tokens
// and sequences with nothing new share one call; rows outside every sequence write nothing.
//
// A warp takes a row: lane l holds latent values 8 l .. 8 l + 7 of each half and the pair l of
// the 32 rotated ones, so every load and store of a warp is contiguous and the row needs one
// warp reduction. The sequence is found by a 32-way search (two rounds of one coalesced load for
// 1024 sequences). Bound by HBM: the row in, the cache row out.
//
// The angle p theta_m is reduced to a part of a turn in fp64 and its sine and cosine are taken
// in fp32 (error under 2^-22, against 2^-9 of a bf16 result). A quantised row's exponent is read
// off the bits of its largest fp32 value; next to the border between two exponents the row is
// taken again in fp64, so that the exponent is the one of the definition.
#include <cmath>

#include "mla_internal.cuh"
#include "rows.cuh"

namespace mla {
namespace {

constexpr int kWarps = 4;   // rows per block

struct RowsParams {
  const void* x;
  int64_t x_stride;
  int n_rows, batch, q_len;
  const int32_t* starts;   // nullptr: q_len rows per sequence
  const int32_t* kv_lens;
  int64_t max_kv_len;
  const __nv_bfloat16* gamma;
  float eps;
  CacheView cv;
  __nv_bfloat16* c_kv;
  __nv_bfloat16* k_r;
  uint8_t* codes;
  int8_t* kv_exp;
  double turns[kDRope / 2];   // pair frequencies over 2 pi (0: no rotation)
  uint32_t* err;
};

// The last b in 0..batch with starts[b] <= i (-1 if none): three rounds at most for 1024
// sequences, each one load of 32 entries a power of 32 apart. All lanes take part.
__device__ __forceinline__ int find_sequence(const int32_t* starts, int batch, int i, int lane) {
  int lo = 0, step = 1;
  while (32 * (int64_t)step < batch + 1) step *= 32;
  for (; step >= 1; step /= 32) {
    const int at = lo + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, at <= batch && starts[at] <= i);
    if (le == 0) return -1;
    lo += (31 - __clz(le)) * step;
  }
  return lo;
}

// The sum of the row's 512 squares in fp64 (all lanes take part).
__device__ __noinline__ double square_sum(const float (&v)[2][8]) {
  double ss = 0.0;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fma((double)v[h][j], (double)v[h][j], ss);
  return warp_sum(ss);
}

// The quantised row's exponent with the whole row in fp64 (all lanes take part; x is read again).
template <typename XT>
__device__ __noinline__ int exact_exponent(const XT* x, const __nv_bfloat16* gamma, float eps, double turns,
                                           bool rotate, int lane) {
  double ss = 0.0, most = 0.0;
  for (int f = lane; f < kDLatent; f += 32) {
    const double v = load1(x + f);
    ss = fma(v, v, ss);
    most = fmax(most, fabs(v * (double)load1(gamma + f)));
  }
  ss = warp_sum(ss);
  const float2 k = load2(x + kDLatent + 2 * lane);
  double sn = 0.0, cs = 1.0;
  if (rotate) sincospi(2.0 * (turns - rint(turns)), &sn, &cs);
  most = fmax(most / sqrt(ss / kDLatent + (double)eps),
              fmax(fabs(k.x * cs - k.y * sn), fabs(k.x * sn + k.y * cs)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmax(most, __shfl_xor_sync(0xffffffffu, most, o));
  const long long b = __double_as_longlong(most);
  return (int)(b >> 52) - 1023 - 8 + ((b & 0xFFFFFFFFFFFFFll) > 0xC000000000000ll ? 1 : 0);
}

template <typename XT, bool kFp8>
__global__ void __launch_bounds__(32 * kWarps)
append_rows_kernel(const RowsParams p) {
  const int lane = threadIdx.x & 31;
  const int i = blockIdx.x * kWarps + (threadIdx.x >> 5);
  grid_dependency_wait();
  allow_dependent_launch();
  if (i >= p.n_rows) return;
  const XT* x = static_cast<const XT*>(p.x) + (int64_t)i * p.x_stride;
  float v[2][8];
  load8(x + 8 * lane, v[0]);
  load8(x + 256 + 8 * lane, v[1]);
  const float2 kr = load2(x + kDLatent + 2 * lane);

  // the sequence and position
  int b;
  int64_t back;   // rows from this one to the end of its sequence
  if (p.starts == nullptr) {
    b = i / p.q_len;
    back = (int64_t)(b + 1) * p.q_len - i;
  } else {
    b = find_sequence(p.starts, p.batch, i, lane);
    if (b < 0 || b >= p.batch) return;   // before the first or behind the last sequence
    back = (int64_t)p.starts[b + 1] - i;
    if (back <= 0) {                     // only where row_starts decreases
      if (lane == 0) atomicOr(p.err, kErrBadKvLen);
      return;
    }
  }
  const int64_t L = p.kv_lens[b], pos = L - back;
  if (pos < 0 || L > p.max_kv_len) {     // no room for the new tokens
    if (lane == 0) atomicOr(p.err, kErrBadKvLen);
    return;
  }
  int64_t row;
  if (p.cv.page_table == nullptr) {
    row = (int64_t)b * p.cv.seq_stride + pos;
  } else {
    const int32_t page = p.cv.page_table[(int64_t)b * p.cv.max_pages + pos / p.cv.page_size];
    if (page < 0 || page >= p.cv.num_pages) {
      if (lane == 0) atomicOr(p.err, kErrBadPage);
      return;
    }
    row = (int64_t)page * p.cv.page_size + pos % p.cv.page_size;
  }

  // RoPE of the pair (2 lane, 2 lane + 1)
  float2 k = kr;
  const double turn = p.turns[lane];
  if (turn != 0.0) {
    const double a = (double)pos * turn;
    float sn, cs;
    sincospif(2.f * (float)(a - rint(a)), &sn, &cs);
    k = make_float2(kr.x * cs - kr.y * sn, kr.x * sn + kr.y * cs);
  }

  float g[2][8];
  load8(p.gamma + 8 * lane, g[0]);
  load8(p.gamma + 256 + 8 * lane, g[1]);
  float ss = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[h][j], v[h][j], ss);
  ss = warp_sum(ss);
  float rstd = 1.f / sqrtf(ss / kDLatent + p.eps);
  if (!(ss > 1e-30f && ss < 3e38f))   // squares that leave fp32's range: sum them in fp64
    rstd = (float)(1.0 / sqrt(square_sum(v) / kDLatent + (double)p.eps));
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[h][j] = v[h][j] * rstd * g[h][j];

  if constexpr (!kFp8) {
    __nv_bfloat16* out = p.c_kv + row * p.cv.row_stride;
    store8(out + 8 * lane, v[0]);
    store8(out + 256 + 8 * lane, v[1]);
    *reinterpret_cast<uint32_t*>(p.k_r + row * p.cv.row_stride + 2 * lane) = pack_bf16(k.x, k.y);
  } else {
    float most = fmaxf(fabsf(k.x), fabsf(k.y));
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(v[h][j]));
    const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    // most = f * 2^q with 1 <= f < 2, and 448 = 1.75 * 2^8: the smallest e with most <= 448 * 2^e
    // is q - 8, or q - 7 where f > 1.75
    int e = 0;
    const int mant = (int)(bits & 0x7FFFFFu) - 0x600000;
    if (bits != 0) {
      e = (int)(bits >> 23) - 127 - 8 + (mant > 0 ? 1 : 0);
      if (abs(mant) < 128)   // within 2^-16 of the border: decide it from the row in fp64
        e = exact_exponent<XT>(x, p.gamma, p.eps, (double)pos * turn, turn != 0.0, lane);
      e = min(max(e, -126), 127);
    }
    const float q = exp2f((float)-e);
    uint8_t* out = p.codes + row * p.cv.row_stride;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo = pack_e4m3(v[h][0] * q, v[h][1] * q) | pack_e4m3(v[h][2] * q, v[h][3] * q) << 16;
      const uint32_t hi = pack_e4m3(v[h][4] * q, v[h][5] * q) | pack_e4m3(v[h][6] * q, v[h][7] * q) << 16;
      *reinterpret_cast<uint2*>(out + 256 * h + 8 * lane) = make_uint2(lo, hi);
    }
    *reinterpret_cast<uint16_t*>(out + kDLatent + 2 * lane) = (uint16_t)pack_e4m3(k.x * q, k.y * q);
    if (lane == 0) p.kv_exp[row] = (int8_t)e;
  }
}

}  // namespace

cudaError_t launch_append_rows(const mla_decode_s& h, int batch, int n_rows, const void* x, bool x_f32,
                               int64_t x_stride, const __nv_bfloat16* gamma, float eps, const CacheView& cv,
                               __nv_bfloat16* c_kv, __nv_bfloat16* k_r, const int32_t* kv_lens,
                               const int32_t* row_starts, cudaStream_t s) {
  RowsParams p{};
  p.x = x;
  p.x_stride = x_stride;
  p.n_rows = n_rows;
  p.batch = batch;
  p.q_len = h.q_len;
  p.starts = row_starts;
  p.kv_lens = kv_lens;
  p.max_kv_len = h.cfg.max_kv_len;
  p.gamma = gamma;
  p.eps = eps;
  p.cv = cv;
  p.c_kv = c_kv;
  p.k_r = k_r;
  if (cv.kv_exp != nullptr) {
    p.codes = reinterpret_cast<uint8_t*>(c_kv);
    p.kv_exp = const_cast<int8_t*>(cv.kv_exp);
  }
  for (int m = 0; m < kDRope / 2; ++m) p.turns[m] = h.theta[m] / 6.283185307179586476925;
  p.err = h.ws.err;
  const dim3 grid((n_rows + kWarps - 1) / kWarps), block(32 * kWarps);
  if (cv.kv_exp != nullptr)
    return x_f32 ? launch_pdl(append_rows_kernel<float, true>, grid, block, 0, s, p)
                 : launch_pdl(append_rows_kernel<__nv_bfloat16, true>, grid, block, 0, s, p);
  return x_f32 ? launch_pdl(append_rows_kernel<float, false>, grid, block, 0, s, p)
               : launch_pdl(append_rows_kernel<__nv_bfloat16, false>, grid, block, 0, s, p);
}

}  // namespace mla
