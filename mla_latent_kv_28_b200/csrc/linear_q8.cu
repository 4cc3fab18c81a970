// The int8 projection: out[i, j] = (sum_k a[i, k] w[j, k]) * w_scale[j] * a_scale[i], with a the
// int8 codes of the tokens (a scale per token) and w those of an nn.Linear weight [n, k] (a scale
// per output channel). The sum is exact in 32-bit integers (|sum| <= 2^14 k < 2^31 for k < 131072),
// so a result does not depend on how the sum is split; it is rounded when it becomes fp32, at each
// of the two scales, and to the output's type.
//
// Few tokens (linear_few): bound by reading the weights. A cluster takes 128 output channels (the
// M = 128 operand) times up to 128 tokens (N); its CTAs share the sum's length, each streaming its
// part of the weights through a ring of TMA boxes into tcgen05 MMAs (kind::i8, int32 in tensor
// memory), and meet in distributed shared memory, where each adds and scales a part of the tile.
//
// Many tokens (linear_many): bound by the tensor core. A pair of CTAs (cta_group::2) takes 256
// tokens x up to 256 channels: each CTA holds 128 of the tokens and half of the channels, so a
// pair reads 64 KB per 128 steps of k for 256 x 256 results. Persistent, with the accumulator
// double-buffered in tensor memory: eight warps scale and store a tile while the next is summed.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "mla_internal.cuh"
#include "rows.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kBoxK = 128;                      // codes (bytes) of k per box: one swizzle row
constexpr uint32_t kWBox = 128 * kBoxK;         // 128 rows of a box
constexpr int kMaxSplits = 8;                   // portable cluster size
constexpr long long kWaitLimit = 2000000000LL;  // cycles: about a second

struct FewParams {
  int rows, n, n_tile, splits, kblocks, stages;
  uint32_t ring;         // bytes of the ring, at least those of the partial tile
  uint32_t idesc;
  const float* a_scale;
  const float* w_scale;
  void* out;
  int64_t out_stride;
  bool vec;              // 4 neighbouring outputs can be stored at once
  uint32_t* err;
};

__device__ __forceinline__ void store4(float* p, const float (&v)[4], int n, bool vec) {
  if (vec && n >= 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < n) p[j] = v[j];
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4], int n, bool vec) {
  if (vec && n >= 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < n) p[j] = __float2bfloat16_rn(v[j]);
}

// smem: ring of stages [128 x 128 weight box | n_tile x 128 token box], then the barriers. The
// ring is reused for the CTA's partial sums [token][128 channels] once its MMAs are done.
template <typename OT>
__global__ void __launch_bounds__(256)
linear_few(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a,
           const FewParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t stage_bytes = kWBox + (uint32_t)p.n_tile * kBoxK;
  const uint32_t bars = sbase + p.ring;   // full[stages], empty[stages], done
  const uint32_t done = bars + 16 * p.stages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (done + 8 - sbase));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + (done + 12 - sbase));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = p.splits > 1 ? (int)cluster_ctarank() : 0;
  const int f0 = (blockIdx.x / p.splits) * 128, t0 = blockIdx.y * p.n_tile;
  const int kb0 = (int)((int64_t)p.kblocks * rank / p.splits);
  const int kb1 = (int)((int64_t)p.kblocks * (rank + 1) / p.splits);
  const uint32_t tmem_cols = p.n_tile < 32 ? 32u : (uint32_t)p.n_tile;   // a power of two
  const WaitGuard guard{abort_flag, p.err, kErrTimeout, kWaitLimit};

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bars + 8 * s, 1);
      mbar_init(bars + 8 * (p.stages + s), 1);
    }
    mbar_init(done, 1);
    fence_mbarrier_init_cluster();
    *abort_flag = 0;
    prefetch_tmap(&tmap_w);
    prefetch_tmap(&tmap_a);
    // the first weights into L2 while the kernel before finishes (a hint only)
    for (int kb = kb0; kb < kb1 && kb < kb0 + p.stages; ++kb) tma_prefetch_2d(&tmap_w, kb * kBoxK, f0);
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  allow_dependent_launch();

  if (tid == 0) {
    int issued = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++issued) {
      const int s = issued % p.stages;
      if (!wait_bounded(bars + 8 * (p.stages + s), ((issued / p.stages) & 1) ^ 1, guard)) break;
      const uint32_t full = bars + 8 * s, dst = sbase + s * stage_bytes;
      mbar_arrive_expect_tx(full, stage_bytes);
      tma_load_2d(dst, &tmap_w, kb * kBoxK, f0, full);
      tma_load_2d(dst + kWBox, &tmap_a, kb * kBoxK, t0, full);
    }
    if (*abort_flag) {   // never leave with copies in flight
      for (int u = std::max(0, issued - p.stages); u < issued; ++u) {
        const long long t = clock64();
        while (!mbar_test(bars + 8 * (u % p.stages), (u / p.stages) & 1) && clock64() - t < kWaitLimit) {}
      }
    }
  } else if (warp == 1 && lane == 0) {
    for (int u = 0; u < kb1 - kb0; ++u) {
      const int s = u % p.stages;
      if (!wait_bounded(bars + 8 * s, (u / p.stages) & 1, guard)) break;
      tc_fence_after();
      const uint32_t w = sbase + s * stage_bytes, a = w + kWBox;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_i8_ss(tmem, smem_desc(w + 32 * k, 16, 1024, 2), smem_desc(a + 32 * k, 16, 1024, 2), p.idesc,
                  (u | k) != 0 ? 1u : 0u);
      mma_commit(bars + 8 * (p.stages + s));
    }
    mma_commit(done);
  }
  __syncwarp();
  wait_bounded(done, 0, guard);
  tc_fence_after();
  // wait_bounded returns per thread; the warp-wide loads below need the warp together
  __syncwarp();
  // (all boxes of this CTA have been read by its MMAs: the ring is free)
  {
    int32_t* part = reinterpret_cast<int32_t*>(smem);
    const int f = 32 * (warp & 3) + lane;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const int cols = p.n_tile < 16 ? 16 : p.n_tile;
    for (int c0 = 16 * (warp >> 2); c0 < cols; c0 += 32) {
      uint32_t r[16];
      tmem_ld16_sync(lanes | (tmem + c0), r);
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(c0 + j) * 128 + f] = (int32_t)r[j];
    }
  }
  tc_fence_before();
  if (p.splits > 1) cluster_sync();
  else __syncthreads();

  const int rows = min(p.n_tile, p.rows - t0);
  const int items = rows * 32;   // 4 channels of one token each
  for (int it = rank * 256 + tid; it < items; it += 256 * p.splits) {
    const int t = it >> 5, q = it & 31, f = f0 + 4 * q;
    if (f >= p.n) continue;
    int32_t acc[4] = {0, 0, 0, 0};
    const uint32_t at = sbase + (uint32_t)it * 16;
    for (int s = 0; s < p.splits; ++s) {
      int4 v;
      ld_cluster_v4(p.splits > 1 ? map_to_rank(at, s) : at, v);
      acc[0] += v.x; acc[1] += v.y; acc[2] += v.z; acc[3] += v.w;
    }
    const float as = p.a_scale[t0 + t];
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = f + j < p.n ? (float)acc[j] * p.w_scale[f + j] * as : 0.f;
    store4(static_cast<OT*>(p.out) + (int64_t)(t0 + t) * p.out_stride + f, o, p.n - f, p.vec);
  }
  if (p.splits > 1) cluster_sync();   // no CTA leaves while another reads its shared memory
  else __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, tmem_cols);
}

// ------------------------------------------------------------------ many tokens

constexpr int kManyStages = 6;
constexpr uint32_t kManyStage = 2 * kWBox;                  // 128 tokens + up to 128 channels
constexpr int kEpiWarps = 8;
constexpr uint32_t kEpiBox = 32 * 128;                      // 32 rows x 128 bytes per warp
constexpr int kManyThreads = 32 * (4 + kEpiWarps);
constexpr uint32_t kManySmem = kManyStages * kManyStage + kEpiWarps * kEpiBox + 256 + 1024;

struct ManyParams {
  int rows, n, n_tile, kblocks, tiles_m, tiles_n, group;
  uint32_t idesc;
  const float* a_scale;
  const float* w_scale;
  void* out;
  int64_t out_stride;
  bool vec;              // rows of the output are 16-byte aligned
  uint32_t* err;
};

// Tile t in groups of `group` channel tiles: within a group the token tiles run first, so that the
// pairs that run together share few weight tiles and few token tiles.
__device__ __forceinline__ void tile_at(const ManyParams& p, int t, int& tm, int& tn) {
  const int per = p.group * p.tiles_m, g = t / per, first = g * p.group;
  const int width = min(p.group, p.tiles_n - first), r = t - g * per;
  tm = r / width;
  tn = first + r % width;
}

template <typename OT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kManyThreads, 1)
linear_many(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a,
            const ManyParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t epi = kManyStages * kManyStage;
  const uint32_t bars = sbase + epi + kEpiWarps * kEpiBox;
  const uint32_t full = bars, empty = bars + 8 * kManyStages, acc_full = empty + 8 * kManyStages,
                 acc_empty = acc_full + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (acc_empty + 16 - sbase));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + (acc_empty + 20 - sbase));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster = (int)cluster_id_x(), clusters = (int)num_clusters_x();
  const int tiles = p.tiles_m * p.tiles_n;
  const WaitGuard guard{abort_flag, p.err, kErrTimeout, kWaitLimit};

  if (tid == 0) {
    for (int s = 0; s < kManyStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(acc_full + 8 * s, 1);
      mbar_init(acc_empty + 8 * s, 2 * kEpiWarps);
    }
    fence_mbarrier_init_cluster();
    *abort_flag = 0;
    prefetch_tmap(&tmap_w);
    prefetch_tmap(&tmap_a);
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();   // the peer's barriers and tensor memory are ready too
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  allow_dependent_launch();

  const uint32_t half_n = (uint32_t)p.n_tile / 2;
  if (warp == 0 && lane == 0) {
    // producer: this CTA's tokens and its half of the channels; both CTAs' copies count toward
    // the first CTA's barrier, where the MMAs are issued
    const uint32_t bytes = 2 * (kWBox + half_n * kBoxK);
    int u = 0;
    for (int t = cluster; t < tiles && !*abort_flag; t += clusters) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int y_a = tm * 256 + (int)rank * 128, y_w = tn * p.n_tile + (int)(rank * half_n);
      for (int kb = 0; kb < p.kblocks; ++kb, ++u) {
        const int s = u % kManyStages;
        if (!wait_bounded(empty + 8 * s, ((u / kManyStages) & 1) ^ 1, guard)) break;
        if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, bytes);
        const uint32_t bar = map_to_rank(full + 8 * s, 0), dst = sbase + s * kManyStage;
        tma_load_2d_pair(dst, &tmap_a, kb * kBoxK, y_a, bar);
        tma_load_2d_pair(dst + kWBox, &tmap_w, kb * kBoxK, y_w, bar);
      }
    }
    // the last boxes have been read, so no copy and no signal is still on its way to this CTA
    for (int v = max(0, u - kManyStages); v < u; ++v)
      if (!wait_bounded(empty + 8 * (v % kManyStages), (v / kManyStages) & 1, guard)) break;
    if (*abort_flag && rank == 0) {   // bounded: let both CTAs' copies land
      for (int v = max(0, u - kManyStages); v < u; ++v) {
        const long long t0 = clock64();
        while (!mbar_test(full + 8 * (v % kManyStages), (v / kManyStages) & 1) && clock64() - t0 < kWaitLimit) {}
      }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    int u = 0, it = 0;
    for (int t = cluster; t < tiles && !*abort_flag; t += clusters, ++it) {
      const int as = it & 1;
      if (!wait_bounded(acc_empty + 8 * as, ((it >> 1) & 1) ^ 1, guard, true)) break;
      tc_fence_after();
      bool ok = true;
      for (int kb = 0; kb < p.kblocks; ++kb, ++u) {
        const int s = u % kManyStages;
        if (!(ok = wait_bounded(full + 8 * s, (u / kManyStages) & 1, guard))) break;
        tc_fence_after();
        const uint32_t a = sbase + s * kManyStage, w = a + kWBox;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_i8_ss_pair(tmem + 256 * as, smem_desc(a + 32 * k, 16, 1024, 2), smem_desc(w + 32 * k, 16, 1024, 2),
                         p.idesc, (kb | k) != 0 ? 1u : 0u);
        mma_commit_pair(empty + 8 * s);
      }
      if (!ok) break;
      mma_commit_pair(acc_full + 8 * as);
    }
  } else if (warp >= 4) {
    // epilogue: warp w reads tensor memory lanes 32 (w % 4) .. + 32 (one token each) and half of
    // the tile's columns, a box of 32 tokens x 128 bytes at a time
    constexpr int kCols = 128 / (int)sizeof(OT);   // columns per box
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    const uint32_t box = sbase + epi + (uint32_t)(warp - 4) * kEpiBox;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const int per = p.n_tile / 2;
    int it = 0;
    for (int t = cluster; t < tiles; t += clusters, ++it) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int as = it & 1;
      const bool ok = wait_bounded(acc_full + 8 * as, (it >> 1) & 1, guard);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const int row0 = tm * 256 + (int)rank * 128 + 32 * quarter, row = row0 + lane;
      const float a_scale = row < p.rows ? p.a_scale[row] : 0.f;
      for (int c = 0; c < per; c += kCols) {
        const int col0 = tn * p.n_tile + part * per + c;
        const int width = min(kCols, per - c);
#pragma unroll
        for (int h = 0; h < kCols; h += 32) {
          if (h >= width) break;
          uint32_t r[32];
          tmem_ld32_sync(lanes | (tmem + 256 * as + part * per + c + h), r);
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            float4 w;
            if (col0 + h + j + 3 < p.n) {
              w = make_float4(p.w_scale[col0 + h + j], p.w_scale[col0 + h + j + 1], p.w_scale[col0 + h + j + 2],
                              p.w_scale[col0 + h + j + 3]);
            } else {
              w.x = col0 + h + j < p.n ? p.w_scale[col0 + h + j] : 0.f;
              w.y = col0 + h + j + 1 < p.n ? p.w_scale[col0 + h + j + 1] : 0.f;
              w.z = col0 + h + j + 2 < p.n ? p.w_scale[col0 + h + j + 2] : 0.f;
              w.w = 0.f;
            }
            v[j] = (float)(int32_t)r[j] * w.x * a_scale;
            v[j + 1] = (float)(int32_t)r[j + 1] * w.y * a_scale;
            v[j + 2] = (float)(int32_t)r[j + 2] * w.z * a_scale;
            v[j + 3] = (float)(int32_t)r[j + 3] * w.w * a_scale;
          }
          // 16-byte units of row `lane`, swizzled so that both directions are free of conflicts
          constexpr int kUnits = 32 * (int)sizeof(OT) / 16;
#pragma unroll
          for (int u = 0; u < kUnits; ++u) {
            const uint32_t at = box + lane * 128 + (((h * (int)sizeof(OT) / 16 + u) ^ (lane & 7)) << 4);
            if constexpr (sizeof(OT) == 2)
              st_shared_v4(at, pack_bf16(v[8 * u], v[8 * u + 1]), pack_bf16(v[8 * u + 2], v[8 * u + 3]),
                           pack_bf16(v[8 * u + 4], v[8 * u + 5]), pack_bf16(v[8 * u + 6], v[8 * u + 7]));
            else
              st_shared_v4(at, __float_as_uint(v[4 * u]), __float_as_uint(v[4 * u + 1]),
                           __float_as_uint(v[4 * u + 2]), __float_as_uint(v[4 * u + 3]));
          }
        }
        __syncwarp();
        const int unit = lane & 7, col = col0 + unit * (16 / (int)sizeof(OT));
        const bool mine = unit * (16 / (int)sizeof(OT)) < width;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + (lane >> 3);
          if (row0 + rr >= p.rows || !mine) continue;
          const uint4 q = *reinterpret_cast<const uint4*>(smem + (box - sbase) + rr * 128 + ((unit ^ (rr & 7)) << 4));
          OT* o = static_cast<OT*>(p.out) + (int64_t)(row0 + rr) * p.out_stride + col;
          if (p.vec && col + 16 / (int)sizeof(OT) <= p.n) {
            *reinterpret_cast<uint4*>(o) = q;
          } else {
            const OT* e = reinterpret_cast<const OT*>(&q);
#pragma unroll
            for (int j = 0; j < 16 / (int)sizeof(OT); ++j)
              if (col + j < p.n) o[j] = e[j];
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      if (lane == 0) mbar_arrive_remote(map_to_rank(acc_empty + 8 * as, 0));
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool found = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess;
    return found ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
  }();
  return fn;
}

// int8 codes [rows, k], rows `stride` bytes apart, as a TMA source of {128 codes, box_rows} boxes
// with the 128-byte swizzle (the K-major operand layout of the MMAs); what lies outside reads as 0.
bool encode(CUtensorMap* m, const int8_t* base, uint64_t rows, uint64_t k, uint64_t stride, uint32_t box_rows) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {k, rows};
  const cuuint64_t strides[1] = {stride};
  const cuuint32_t box[2] = {(cuuint32_t)kBoxK, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// cudaFuncSetAttribute acts on the current device: once for each (a second call does no harm).
template <auto kKernel>
cudaError_t allow_smem(int device, uint32_t bytes) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = device < 64 ? 1ull << device : 0;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

constexpr uint32_t kFewSmem = 108 * 1024;   // two CTAs per SM

template <typename OT>
cudaError_t launch_few(const mla_decode_s& h, const LinearArgs& a, cudaStream_t s) {
  const int n_tile = a.rows <= 16 ? 16 : a.rows <= 32 ? 32 : a.rows <= 64 ? 64 : 128;
  const int kblocks = (a.k + kBoxK - 1) / kBoxK;
  const int blocks = (a.n + 127) / 128, row_tiles = (a.rows + n_tile - 1) / n_tile;
  const uint32_t stage = kWBox + (uint32_t)n_tile * kBoxK;
  int splits = 1;
  while (splits < kMaxSplits && blocks * row_tiles * splits < h.num_sms && kblocks >= 4 * splits) splits *= 2;
  const int stages = std::min((int)((kFewSmem - 2048) / stage), std::max((kblocks + splits - 1) / splits, 1));
  // the ring also holds the partial tile
  const uint32_t ring = std::max(stages * stage, (uint32_t)n_tile * 512);
  const uint32_t smem = ring + 16 * stages + 64 + 1024;
  CUtensorMap tw, ta;
  if (!encode(&tw, a.w_codes, (uint64_t)a.n, (uint64_t)a.k, (uint64_t)a.w_stride, 128) ||
      !encode(&ta, a.codes, (uint64_t)a.rows, (uint64_t)a.k, (uint64_t)a.codes_stride, (uint32_t)n_tile))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<linear_few<OT>>(h.device, kFewSmem);
  if (e != cudaSuccess) return e;
  FewParams p{};
  p.rows = a.rows;
  p.n = a.n;
  p.n_tile = n_tile;
  p.splits = splits;
  p.kblocks = kblocks;
  p.stages = stages;
  p.ring = ring;
  p.idesc = idesc_i8_s32(128, n_tile);
  p.a_scale = a.scales;
  p.w_scale = a.w_scales;
  p.out = a.out;
  p.out_stride = a.out_stride;
  p.vec = reinterpret_cast<uintptr_t>(a.out) % (4 * sizeof(OT)) == 0 && a.out_stride % 4 == 0;
  p.err = h.ws.err;
  return launch_pdl_cluster(linear_few<OT>, dim3(blocks * splits, row_tiles), dim3(256), smem, splits, s, tw, ta, p);
}

template <typename OT>
cudaError_t launch_many(const mla_decode_s& h, const LinearArgs& a, cudaStream_t s) {
  ManyParams p{};
  p.n_tile = 256;
  p.rows = a.rows;
  p.n = a.n;
  p.kblocks = (a.k + kBoxK - 1) / kBoxK;
  p.tiles_m = (a.rows + 255) / 256;
  p.tiles_n = (a.n + p.n_tile - 1) / p.n_tile;
  p.group = 8;
  p.idesc = idesc_i8_s32(256, p.n_tile);
  p.a_scale = a.scales;
  p.w_scale = a.w_scales;
  p.out = a.out;
  p.out_stride = a.out_stride;
  p.vec = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.out_stride * sizeof(OT) % 16 == 0;
  p.err = h.ws.err;
  CUtensorMap tw, ta;
  if (!encode(&tw, a.w_codes, (uint64_t)a.n, (uint64_t)a.k, (uint64_t)a.w_stride, (uint32_t)p.n_tile / 2) ||
      !encode(&ta, a.codes, (uint64_t)a.rows, (uint64_t)a.k, (uint64_t)a.codes_stride, 128))
    return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<linear_many<OT>>(h.device, kManySmem);
  if (e != cudaSuccess) return e;
  const int clusters = std::min(h.num_sms / 2, p.tiles_m * p.tiles_n);
  return launch_pdl(linear_many<OT>, dim3(2 * clusters), dim3(kManyThreads), kManySmem, s, tw, ta, p);
}

}  // namespace

cudaError_t launch_linear_q8(const mla_decode_s& h, const LinearArgs& a, cudaStream_t s) {
  if (a.rows <= 128) return a.out_f32 ? launch_few<float>(h, a, s) : launch_few<__nv_bfloat16>(h, a, s);
  return a.out_f32 ? launch_many<float>(h, a, s) : launch_many<__nv_bfloat16>(h, a, s);
}

}  // namespace mla
