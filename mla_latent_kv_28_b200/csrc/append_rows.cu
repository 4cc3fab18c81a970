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
// A warp or half of one takes a row, all its loads first; every load and store is contiguous over the
// row's lanes, and a row needs one reduction. A lane per row looks the rows' places up: the window of
// 32 sequences around them, starts and lengths in one round of loads (1024 sequences: two more).
// Bound by HBM (the row in, the cache row out) and, for quantised rows, by the issue slots: 65536 bf16
// rows into a bf16 cache 26.0 us (5800 GB/s), into an E4M3 cache 26.1 us; 64 rows 2.4 us.
//
// The angle p theta_m is kept as an integer part of a turn (p times the frequency's 64-bit fraction,
// which drops whole turns by itself): positions to 2^30 lose 2^-34 of a turn, beside 2^-25 by the
// rounding of the frequency as an fp64 number, and nothing but one conversion to fp32 is left for the
// units of fp64 and conversions, which bound an earlier form. A quantised row's exponent is read off
// the bits of its largest fp32 value; next to the border between two exponents the row is taken again
// in fp64, so that the exponent is the one of the definition.
#include <type_traits>

#include "mla_internal.cuh"
#include "rows.cuh"
#include "sm100_i8.cuh"

namespace mla {
namespace {

constexpr int kWarps = 4;   // warps per block
constexpr int kPage = 64;   // rows per page (the only size a handle takes)

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
  const uint64_t* turns;   // pair frequencies over 2 pi, the part of a turn in 2^-64 (0: no rotation)
  uint32_t* err;
};

// The last multiple of 32, b, in 0..batch with starts[b] <= i (0 if none): two rounds at most for 1024
// sequences, each one load of 32 entries a power of 32 apart. All lanes take part.
__device__ __forceinline__ int find_window(const int32_t* starts, int batch, int i, int lane) {
  int lo = 0, step = 1;
  while (32 * (int64_t)step < batch + 1) step *= 32;
  for (; step >= 32; step /= 32) {
    const int at = lo + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, at <= batch && starts[at] <= i);
    if (le == 0) return 0;
    lo += (31 - __clz(le)) * step;
  }
  return lo;
}

// Sine and cosine of an angle given as a part of a turn, in 2^-64 of one (signed: -1/2 .. 1/2). The
// nearest quarter turn is taken off; Taylor's polynomials of the rest, |a| <= pi/4, leave out
// a^11 / 11! < 2^-29 and a^12 / 12! < 2^-32.
__device__ __forceinline__ void sine_cosine(int64_t angle, float& sn, float& cs) {
  const int32_t top = (int32_t)(angle >> 32);
  const uint32_t quarter = ((uint32_t)top + 0x20000000u) >> 30;
  const float a = (float)(int32_t)((uint32_t)top - (quarter << 30)) * (float)(6.283185307179586476925 / 4294967296.0);
  const float z = a * a;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -0.16666667f);
  s = fmaf(z * s, a, a);
  float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  c = fmaf(z, c, -1.3888889e-3f);
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const bool swap = quarter & 1;
  sn = swap ? c : s;
  cs = swap ? s : c;
  if (quarter & 2) sn = -sn;              // the third and fourth quarter
  if ((quarter + 1) & 2) cs = -cs;        // the second and third
}

// Neighbouring pairs of the key part, from pair l or 2 l on.
__device__ __forceinline__ void store_key(__nv_bfloat16* p, int l, const float2 (&k)[1]) {
  reinterpret_cast<uint32_t*>(p)[l] = pack_bf16(k[0].x, k[0].y);
}
__device__ __forceinline__ void store_key(__nv_bfloat16* p, int l, const float2 (&k)[2]) {
  reinterpret_cast<uint2*>(p)[l] = make_uint2(pack_bf16(k[0].x, k[0].y), pack_bf16(k[1].x, k[1].y));
}
template <int G, typename T>
__device__ __forceinline__ T group_sum(T v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int G, typename T>
__device__ __forceinline__ T group_max(T v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// 1 / sqrt(mean square + eps) of a row in fp64 (lane l of G; the whole warp takes part). Without an eps that of
// a row of subnormal values lies beyond fp32: it comes as minus 2^-64 times it, and the caller puts the
// 2^64 on the values (exact).
template <typename XT, int G>
__device__ __noinline__ float wide_rstd(const XT* x, float eps, int l) {
  double ss = 0.0;
  for (int f = l; f < kDLatent; f += G) {
    const double v = load1(x + f);
    ss = fma(v, v, ss);
  }
  const double rstd = 1.0 / sqrt(group_sum<G>(ss) / kDLatent + (double)eps);
  return (float)(rstd > 0x1p100 ? rstd * -0x1p-64 : rstd);
}

// A quantised row's exponent with the whole row in fp64, its angles at `position` (as above).
template <typename XT, int G>
__device__ __noinline__ int exact_exponent(const XT* x, const __nv_bfloat16* gamma, float eps, const uint64_t* turns,
                                           uint64_t position, int l) {
  double ss = 0.0, most = 0.0;
  for (int f = l; f < kDLatent; f += G) {
    const double v = load1(x + f);
    ss = fma(v, v, ss);
    most = fmax(most, fabs(v * (double)load1(gamma + f)));
  }
  most /= sqrt(group_sum<G>(ss) / kDLatent + (double)eps);
  for (int m = l; m < kDRope / 2; m += G) {
    const float2 k = load2(x + kDLatent + 2 * m);
    double sn, cs;
    sincospi((double)(int64_t)(position * turns[m]) * 0x1p-63, &sn, &cs);
    most = fmax(most, fmax(fabs(k.x * cs - k.y * sn), fabs(k.x * sn + k.y * cs)));
  }
  const long long b = __double_as_longlong(group_max<G>(most));
  return (int)(b >> 52) - 1023 - 8 + ((b & 0xFFFFFFFFFFFFFll) > 0xC000000000000ll ? 1 : 0);
}

// G lanes take a row, 32 / G rows a warp. Lane l of a row holds the latent values 8 (l + G c) .. + 7,
// c < 64 / G, and 32 / G neighbouring pairs of the rotated ones from pair 32 / G l on.
template <typename XT, bool kFp8, int G>
__global__ void __launch_bounds__(32 * kWarps)
append_rows_kernel(const RowsParams p) {
  constexpr int kRows = 32 / G, kChunks = 64 / G, kPairs = 32 / G;
  const int lane = threadIdx.x & 31, l = lane % G, mine = lane / G;
  const int i0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRows;
  grid_dependency_wait();
  allow_dependent_launch();
  if (i0 >= p.n_rows) return;
  const int rows = min(kRows, p.n_rows - i0);
  const bool in = mine < rows;
  // (a group behind the last row reads the last one again and writes nothing)
  const XT* x = static_cast<const XT*>(p.x) + (int64_t)(i0 + (in ? mine : 0)) * p.x_stride;
  Raw8<XT, 8> raw[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) raw[c].load(x + 8 * (l + G * c), 0, 1);
  float2 k[kPairs];
#pragma unroll
  for (int c = 0; c < kPairs; ++c) k[c] = load2(x + kDLatent + 2 * (kPairs * l + c));
  uint64_t turn[kPairs];
#pragma unroll
  for (int c = 0; c < kPairs; ++c) turn[c] = p.turns[kPairs * l + c];

  // Each row's place: lane r looks row r up in a window of 32 neighbouring sequences, whose starts
  // and lengths arrive together. at < 0: nothing to write.
  int64_t pos = 0, at = -1;
  int b = -1, end = 0, len = 0;
  if (p.starts == nullptr) {
    b = (i0 + lane) / p.q_len;
    if (lane < rows) {
      end = (b + 1) * p.q_len;
      len = p.kv_lens[b];
    }
  } else {
    int lo = find_window(p.starts, p.batch, i0, lane);
    int start = lo + lane <= p.batch ? p.starts[lo + lane] : INT32_MAX;
    int lens = lo + lane < p.batch ? p.kv_lens[lo + lane] : 0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      uint32_t le = __ballot_sync(0xffffffffu, start <= i0 + r);
      if (r > 0 && le == 0xffffffffu && lo + 31 < p.batch) {   // the next rows may belong behind the window
        lo = find_window(p.starts, p.batch, i0 + r, lane);
        start = lo + lane <= p.batch ? p.starts[lo + lane] : INT32_MAX;
        lens = lo + lane < p.batch ? p.kv_lens[lo + lane] : 0;
        le = __ballot_sync(0xffffffffu, start <= i0 + r);
      }
      const int in = 31 - __clz(le);   // -1 where no sequence starts at or before the row
      const int l = __shfl_sync(0xffffffffu, lens, in & 31);
      int next = __shfl_sync(0xffffffffu, start, (in + 1) & 31);
      if (in == 31 && lo + 32 <= p.batch) next = p.starts[lo + 32];
      if (lane == r && in >= 0) {
        b = lo + in;
        end = next;
        len = l;
      }
    }
  }
  if (lane < rows && b >= 0 && b < p.batch) {   // else before the first or behind the last sequence
    pos = (int64_t)len - ((int64_t)end - (i0 + lane));
    // a row behind its sequence's end (row_starts decreases), or no room for the new tokens
    if (end <= i0 + lane || pos < 0 || len > p.max_kv_len) {
      atomicOr(p.err, kErrBadKvLen);
    } else if (p.cv.page_table == nullptr) {
      at = (int64_t)b * p.cv.seq_stride + pos;
    } else {
      const int32_t page = p.cv.page_table[(int64_t)b * p.cv.max_pages + pos / kPage];
      if (page >= 0 && page < p.cv.num_pages) at = (int64_t)page * kPage + pos % kPage;
      else atomicOr(p.err, kErrBadPage);
    }
  }

  const int64_t row = __shfl_sync(0xffffffffu, at, mine);
  const uint64_t position = (uint64_t)__shfl_sync(0xffffffffu, pos, mine);
  if (__all_sync(0xffffffffu, row < 0)) return;

  // RoPE
#pragma unroll
  for (int c = 0; c < kPairs; ++c) {
    if (turn[c] != 0) {
      float sn, cs;
      sine_cosine((int64_t)(position * turn[c]), sn, cs);
      k[c] = make_float2(k[c].x * cs - k[c].y * sn, k[c].x * sn + k[c].y * cs);
    }
  }
  float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) s2 = sm100::ffma2(raw[c].pair(j), raw[c].pair(j), s2);
  const float ss = group_sum<G>(s2.x + s2.y);
  float rstd = 1.f / sqrtf(ss / kDLatent + p.eps);
  const bool wide = !(ss > 1e-30f && ss < 3e38f);   // squares that leave fp32's range: sum them in fp64
  if (__any_sync(0xffffffffu, wide)) {
    const float w = wide_rstd<XT, G>(x, p.eps, l);
    if (wide) rstd = w;
  }
  float2 v[kChunks][4];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    Raw8<__nv_bfloat16, 8> gamma;
    gamma.load(p.gamma + 8 * (l + G * c), 0, 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[c][j] = sm100::fmul2(sm100::fmul2(raw[c].pair(j), make_float2(rstd, rstd)), gamma.pair(j));
  }
  if (rstd < 0.f) {   // (read again: kept, the values cost registers that rows in earnest pay for)
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      Raw8<XT, 8> again;
      Raw8<__nv_bfloat16, 8> gamma;
      again.load(x + 8 * (l + G * c), 0, 1);
      gamma.load(p.gamma + 8 * (l + G * c), 0, 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 r = sm100::fmul2(again.pair(j), make_float2(0x1p64f, 0x1p64f));
        v[c][j] = sm100::fmul2(sm100::fmul2(r, make_float2(-rstd, -rstd)), gamma.pair(j));
      }
    }
  }
  if constexpr (!kFp8) {
    if (row < 0) return;
    __nv_bfloat16* out = p.c_kv + row * p.cv.row_stride;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) store_pairs<8>(out + 8 * (l + G * c), 0, 1, v[c]);
    store_key(p.k_r + row * p.cv.row_stride, l, k);
  } else {
    float most = 0.f;
#pragma unroll
    for (int c = 0; c < kPairs; ++c) most = max_abs(most, k[c].x, k[c].y);
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) most = max_abs(most, v[c][j].x, v[c][j].y);
    const uint32_t bits = group_max<G>(__float_as_uint(most));
    // most = f * 2^q with 1 <= f < 2, and 448 = 1.75 * 2^8: the smallest e with most <= 448 * 2^e
    // is q - 8, or q - 7 where f > 1.75
    const int mant = (int)(bits & 0x7FFFFFu) - 0x600000;
    int e = (int)(bits >> 23) - 127 - 8 + (mant > 0 ? 1 : 0);
    const bool border = bits != 0 && abs(mant) < 32;   // within 2^-18 (fp32 is off by 2^-20): fp64 decides
    if (__any_sync(0xffffffffu, border)) {
      const int f = exact_exponent<XT, G>(x, p.gamma, p.eps, p.turns, position, l);
      if (border) e = f;
    }
    e = bits == 0 ? 0 : bits == 0x7F800000u ? 127 : min(max(e, -126), 127);   // (an infinity: the largest)
    if (row < 0) return;
    const float q = exp2f((float)-e);
    uint8_t* out = p.codes + row * p.cv.row_stride;
    const float2 q2 = make_float2(q, q);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 u = sm100::fmul2(v[c][j], q2);
        w[j] = pack_e4m3(u.x, u.y);
      }
      *reinterpret_cast<uint2*>(out + 8 * (l + G * c)) =
          make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
    }
#pragma unroll
    for (int c = 0; c < kPairs; ++c)
      *reinterpret_cast<uint16_t*>(out + kDLatent + 2 * (kPairs * l + c)) = (uint16_t)pack_e4m3(k[c].x * q, k[c].y * q);
    if (l == 0) p.kv_exp[row] = (int8_t)e;
  }
}

template <typename XT, bool kFp8>
cudaError_t launch_typed(const RowsParams& p, int num_sms, cudaStream_t s) {
  // Two rows a warp halve what each row costs beside its values (look-up, statistics, exponent): 65536
  // bf16 rows into an E4M3 cache 26.1 against 30.2 us. Few rows are bound by a row's latency, which a
  // whole warp makes shorter (64 rows: 2.40 against 2.83 us; 2000 rows: 3.0 against 3.25 us).
  const bool many = p.n_rows >= 32 * num_sms;
  const int per = kWarps * (many ? 2 : 1);
  const dim3 grid((p.n_rows + per - 1) / per), block(32 * kWarps);
  return many ? launch_pdl(append_rows_kernel<XT, kFp8, 16>, grid, block, 0, s, p)
              : launch_pdl(append_rows_kernel<XT, kFp8, 32>, grid, block, 0, s, p);
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
  p.turns = h.ws.turns;
  p.err = h.ws.err;
  const int sms = h.num_sms;
  if (cv.kv_exp != nullptr)
    return x_f32 ? launch_typed<float, true>(p, sms, s) : launch_typed<__nv_bfloat16, true>(p, sms, s);
  return x_f32 ? launch_typed<float, false>(p, sms, s) : launch_typed<__nv_bfloat16, false>(p, sms, s);
}

}  // namespace mla
