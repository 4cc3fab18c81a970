// The int8 projection: out[i, j] = (sum_k a[i, k] w[j, k]) * w_scale[j] * a_scale[i], with a the
// int8 codes of the tokens (a scale per token) and w those of an nn.Linear weight [n, k] (a scale
// per output channel). The sum is exact in 32-bit integers (|sum| <= 2^14 k < 2^31 for k < 131072),
// so a result does not depend on how the sum is split; it is rounded when it becomes fp32, at each
// of the two scales, and to the output's type.
//
// Few tokens (linear_few): bound by reading the weights. A cluster takes 128 output channels (the M = 128
// operand) times up to 128 tokens (N); its CTAs share the sum's length, each streaming its part of the
// weights through a ring of TMA boxes into tcgen05 MMAs (kind::i8, int32 in tensor memory). Each CTA then
// sends its partial sums to the CTAs that finish them (asynchronous stores into their shared memory,
// counted by a barrier there: no second meeting), which add, scale and store. 33 x 16384 -> 5120 16.8 us
// (5000 GB/s), 64 x 1536 -> 16384 7.8 us, 1 x 5120 -> 2112 4.9 us (2 us of launch, 1.5 us until the boxes
// are here and multiplied, 1 us of exchange).
//
// More tokens (linear_many): bound by the tensor core, and by the power that it takes, where tokens and sums
// are long; between 129 and some 2000 tokens by what tiles of 256 tokens in whole rounds over the pairs
// leave idle, and by set-up (512 x 5120 -> 2112 11.9 us for 3.3 us of products, 1048 x 7376 -> 5576 at least
// 49.5 for 25.7). A pair of CTAs (cta_group::2) takes 256 tokens x up to 256 channels: each CTA holds 128 of
// the tokens and half of the channels, so a pair reads 64 KB per 128 steps of k for 256 x 256 results.
// Persistent, with the accumulator double-buffered in tensor memory: eight warps scale and store a tile
// while the next is summed. 2048 x 16384 -> 5120 115 us (2980 TOP/s; 135 us at the clocks of a long run), 8192 x 512 -> 8192
// 40 us (its 134 MB of results), 333 x 1000 -> 777 6 to 8 us.
//
// In both the loops that issue copies and MMAs are run by whole warps with one elected lane, so that
// descriptors and barriers stay in uniform registers: with a lone thread the 730 cycles of its own
// instructions per k block were what bound them (512 of MMA).
#include <cudaTypedefs.h>

#include <algorithm>

#include "mla_internal.cuh"
#include "rows.cuh"
#include "sm100_i8.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kBoxK = 128;                      // codes (bytes) of k per box: one swizzle row
constexpr uint32_t kWBox = 128 * kBoxK;         // 128 rows of a box
constexpr int kFewRows = 128;                   // tokens of linear_few: the MMA's N, in one piece
constexpr int kMaxFewStages = 12;
constexpr long long kWaitLimit = 2000000000LL;  // cycles: about a second

// A ring position: the stage and how often the ring has been passed, mod 2.
struct RingPos {
  uint32_t stage = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t stages) {
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// wait_bounded by a whole warp, with one answer for it, whose first probe takes no clock: a ring's stages
// follow each other within a few hundred cycles, and the issuing warps' own instructions count.
__device__ __forceinline__ bool wait_ring(uint32_t bar, uint32_t parity, const WaitGuard& g) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, g));
}

struct FewParams {
  int rows, n, n_tile, splits, kblocks, stages;
  uint32_t ring;         // bytes of the ring
  uint32_t recip;        // ceil(2^18 / splits)
  uint32_t pitch;        // bytes between a part's groups of four tokens: 16 for each of its channels
  uint32_t idesc;
  const float* a_scale;
  const float* w_scale;
  void* out;
  int64_t out_stride;
  uint32_t* err;
};

// 32 of a token's results into row `lane` of a box of 32 rows of 128 bytes (in bf16 half of the row, the
// half-th), in the TMA's swizzle: 16-byte units, free of bank conflicts.
__device__ __forceinline__ void put_row(uint32_t box, int lane, int, const float (&v)[32], const float*) {
#pragma unroll
  for (int u = 0; u < 8; ++u)
    st_shared_v4(box + lane * 128 + ((u ^ (lane & 7)) << 4), __float_as_uint(v[4 * u]), __float_as_uint(v[4 * u + 1]),
                 __float_as_uint(v[4 * u + 2]), __float_as_uint(v[4 * u + 3]));
}
__device__ __forceinline__ void put_row(uint32_t box, int lane, int half, const float (&v)[32], const __nv_bfloat16*) {
#pragma unroll
  for (int u = 0; u < 4; ++u)
    st_shared_v4(box + lane * 128 + (((u + 4 * half) ^ (lane & 7)) << 4), pack_bf16(v[8 * u], v[8 * u + 1]),
                 pack_bf16(v[8 * u + 2], v[8 * u + 3]), pack_bf16(v[8 * u + 4], v[8 * u + 5]),
                 pack_bf16(v[8 * u + 6], v[8 * u + 7]));
}
// Value `col` of row `row` of such a box.
template <typename OT>
__device__ __forceinline__ OT get_one(const uint8_t* box, int row, int col) {
  const int byte = col * (int)sizeof(OT);
  return *reinterpret_cast<const OT*>(box + row * 128 + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15));
}

// smem: the barriers, the scales, a ring of stages [128 x 128 weight box | n_tile x 128 token box], the
// partial sums that this CTA receives. Of the tile's 128 channels CTA r of the cluster finishes those from
// ceil(128 r / splits) on: it gets from each CTA pieces of 16 bytes, [4 tokens][its channels], so that what
// a warp sends at a time, and what one reads, is contiguous (128 x 16384 -> 5120 22.8 us; with a channel's
// tokens together 24.4, 64 x 5120 -> 2112 7.0 and 8.0 us).
// kTiles: the tokens are cut into tiles too, one for each blockIdx.y (of its own, because the kernel of a few
// microseconds was up to 0.7 us slower with the tile's offset in it: 128 x 1536 -> 16384).
template <typename OT, bool kTiles>
__global__ void __launch_bounds__(256)
linear_few(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a,
           const FewParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t stages = p.stages, stage_bytes = kWBox + (uint32_t)p.n_tile * kBoxK;
  const uint32_t full = sbase, empty = full + 8 * kMaxFewStages, done = empty + 8 * kMaxFewStages, received = done + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 16 * kMaxFewStages + 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 16 * kMaxFewStages + 20);
  float* a_scale = reinterpret_cast<float*>(smem + 1024);   // the tokens' scales, the tile's channels'
  float* w_scale = a_scale + kFewRows;
  const uint32_t ring = sbase + 2048, parts = ring + p.ring;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int splits = p.splits, rank = splits > 1 ? (int)cluster_ctarank() : 0;
  // x / splits for x <= 2^13 (kblocks is 1024 at most, splits 8): 2^18 / splits rounded up is close enough
  const auto share = [&](int x) { return (int)((uint32_t)x * p.recip >> 18); };
  const int f0 = (int)cluster_id_x() * 128, t0 = kTiles ? blockIdx.y * p.n_tile : 0;
  const int kb0 = share(p.kblocks * rank), kb1 = share(p.kblocks * (rank + 1));
  const uint32_t tmem_cols = p.n_tile <= 32 ? 32u : p.n_tile <= 64 ? 64u : 128u;
  const int rows = kTiles ? min(p.n_tile, p.rows - t0) : p.rows, quads = (rows + 3) / 4;
  const int c_begin = share(128 * rank + splits - 1), c_count = share(128 * (rank + 1) + splits - 1) - c_begin;
  const uint32_t part = (uint32_t)quads * p.pitch;   // bytes between the parts
  const WaitGuard guard{abort_flag, p.err, kErrTimeout, kWaitLimit};

  if (tid == 0) {
    for (uint32_t s = 0; s < stages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    mbar_init(done, 1);
    mbar_init(received, 1);
    fence_mbarrier_init_cluster();
    if (splits > 1) mbar_arrive_expect_tx(received, (uint32_t)(splits * c_count * quads * 16));
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
  if (splits > 1) cluster_arrive();   // this CTA may be written to
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  allow_dependent_launch();

  if (warp == 0) {
    RingPos at;
    int issued = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++issued) {
      if (!wait_ring(empty + 8 * at.stage, at.phase ^ 1, guard)) break;
      if (elect_one()) {
        const uint32_t bar = full + 8 * at.stage, dst = ring + at.stage * stage_bytes;
        mbar_arrive_expect_tx(bar, stage_bytes);
        tma_load_2d(dst, &tmap_w, kb * kBoxK, f0, bar);
        tma_load_2d(dst + kWBox, &tmap_a, kb * kBoxK, t0, bar);
      }
      at.next(stages);
    }
    if (*abort_flag) {   // never leave with copies in flight
      for (int u = max(0, issued - p.stages); u < issued; ++u) {
        const long long t = clock64();
        while (!mbar_test(full + 8 * (u % p.stages), (u / p.stages) & 1) && clock64() - t < kWaitLimit) {}
      }
    }
  } else if (warp == 1) {
    RingPos at;
    const uint64_t w_desc = smem_desc(ring, 16, 1024, 2), a_desc = smem_desc(ring + kWBox, 16, 1024, 2);
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!wait_ring(full + 8 * at.stage, at.phase, guard)) break;
      tc_fence_after();
      const uint64_t off = (at.stage * stage_bytes) >> 4;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)   // 32 codes each
          mma_i8_ss(tmem, w_desc + off + 2 * k, a_desc + off + 2 * k, p.idesc, kb != kb0 || k != 0 ? 1u : 0u);
        mma_commit(empty + 8 * at.stage);
      }
      at.next(stages);
    }
    if (elect_one()) mma_commit(done);
  } else if (warp >= 4) {
    // the scales arrive while the tile is summed
    const int i = tid - 128;
    a_scale[i] = i < rows ? p.a_scale[t0 + i] : 0.f;
    w_scale[i] = f0 + i < p.n ? p.w_scale[f0 + i] : 0.f;
  }
  __syncwarp();
  bool ok = wait_bounded(done, 0, guard);
  __syncthreads();
  tc_fence_after();

  const int f = 32 * (warp & 3) + lane;   // this lane's channel of the tile
  const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
  if (splits == 1) {
    const float w = w_scale[f];
    for (int c0 = 16 * (warp >> 2); c0 < rows; c0 += 32) {
      uint32_t r[16];
      tmem_ld16_sync(lanes | (tmem + c0), r);
      OT* out = static_cast<OT*>(p.out) + (int64_t)(t0 + c0) * p.out_stride + f0 + f;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c0 + j < rows && f0 + f < p.n)
          store1(out + j * p.out_stride, (float)(int32_t)r[j] * w * a_scale[c0 + j]);
    }
  } else {
    const int owner = f * splits >> 7, c = f - share(128 * owner + splits - 1);
    cluster_wait();   // the others have set their barriers up
    const uint32_t to = map_to_rank(parts + rank * part + c * 16, owner), bar = map_to_rank(received, owner);
    for (int c0 = 16 * (warp >> 2); c0 < rows; c0 += 32) {
      uint32_t r[16];
      tmem_ld16_sync(lanes | (tmem + c0), r);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c0 + 4 * j < rows) st_async_v4(to + (c0 / 4 + j) * p.pitch, r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3], bar);
    }
    ok = wait_bounded(received, 0, guard, true) && ok;
    const int count = min(c_count, p.n - f0 - c_begin);   // may be negative
    if (ok && count > 0) {
      for (int it = tid; it < count * quads; it += 256) {
        const int q = it / count, ch = it - q * count, col = f0 + c_begin + ch;
        int32_t acc[4] = {0, 0, 0, 0};
        const uint8_t* from = smem + (parts - sbase) + ch * 16 + q * p.pitch;
        for (int src = 0; src < splits; ++src) {
          const int4 v = *reinterpret_cast<const int4*>(from + src * part);
          acc[0] += v.x; acc[1] += v.y; acc[2] += v.z; acc[3] += v.w;
        }
        const float w = w_scale[c_begin + ch];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 4 * q + j;
          if (t < rows)
            store1(static_cast<OT*>(p.out) + (int64_t)(t0 + t) * p.out_stride + col, (float)acc[j] * w * a_scale[t]);
        }
      }
    }
  }
  tc_fence_before();
  const bool failed = __syncthreads_or(!ok);
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, tmem_cols);
  // having received from every CTA, none writes here any more; after a wait that ran out one might
  if (failed && splits > 1) cluster_sync();
}

// ------------------------------------------------------------------ many tokens

constexpr int kMaxManyStages = 10;
constexpr int kEpiWarps = 8;
constexpr int kEpiParts = kEpiWarps / 4, kPartCols = 256 / kEpiParts;   // the warps of a quarter share the columns
constexpr int kManyThreads = 32 * (4 + kEpiWarps);
// smem: a ring of boxes [128 tokens | half of the channels], the warps' channel scales, the barriers, and for
// each warp a box of 32 rows of 128 bytes of results.
constexpr uint32_t kManyRing = 11 * kWBox, kManyScales = kManyRing;
constexpr uint32_t kManyBars = kManyScales + kEpiWarps * kPartCols * 4, kManyBoxes = kManyBars + 1024;
constexpr uint32_t kManySmem = kManyBoxes + kEpiWarps * 4096 + 1024;

struct ManyParams {
  int rows, n, n_tile, kblocks, tiles_m, tiles_n, group, stages;
  uint32_t idesc;
  const float* a_scale;
  const float* w_scale;
  void* out;
  int64_t out_stride;
  bool tma;              // the output's rows are aligned for TMA stores
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
            const __grid_constant__ CUtensorMap tmap_out, const ManyParams p) {
  constexpr int kCols = 128 / (int)sizeof(OT);   // columns of a box of results
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t stage_bytes = kWBox + (uint32_t)p.n_tile / 2 * kBoxK;
  const uint32_t stages = p.stages;
  const uint32_t bars = sbase + kManyBars;
  const uint32_t full = bars, empty = bars + 8 * kMaxManyStages, acc_full = empty + 8 * kMaxManyStages,
                 acc_empty = acc_full + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + (acc_empty + 16 - sbase));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + (acc_empty + 20 - sbase));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster = (int)cluster_id_x(), clusters = (int)num_clusters_x();
  const int tiles = p.tiles_m * p.tiles_n;
  const WaitGuard guard{abort_flag, p.err, kErrTimeout, kWaitLimit};

  if (tid == 0) {
    for (uint32_t s = 0; s < stages; ++s) {
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
    if (p.tma) prefetch_tmap(&tmap_out);
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
  if (warp == 0) {
    // producer: this CTA's tokens and its half of the channels; both CTAs' copies count toward
    // the first CTA's barrier, where the MMAs are issued
    const uint32_t bytes = 2 * (kWBox + half_n * kBoxK), lead_full = map_to_rank(full, 0);
    RingPos at;
    int u = 0;
    bool ok = true;
    for (int t = cluster; t < tiles && ok; t += clusters) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int y_a = tm * 256 + (int)rank * 128, y_w = tn * p.n_tile + (int)(rank * half_n);
      for (int kb = 0; kb < p.kblocks; ++kb, ++u) {
        if (!(ok = wait_ring(empty + 8 * at.stage, at.phase ^ 1, guard))) break;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(full + 8 * at.stage, bytes);
          const uint32_t bar = lead_full + 8 * at.stage, dst = sbase + at.stage * stage_bytes;
          tma_load_2d_pair(dst, &tmap_a, kb * kBoxK, y_a, bar);
          tma_load_2d_pair(dst + kWBox, &tmap_w, kb * kBoxK, y_w, bar);
        }
        at.next(stages);
      }
    }
    // the last boxes have been read, so no copy and no signal is still on its way to this CTA
    const int ring = (int)stages;
    for (int v = max(0, u - ring); v < u; ++v)
      if (!wait_bounded(empty + 8 * (v % ring), (v / ring) & 1, guard)) break;
    if (*abort_flag && rank == 0) {   // bounded: let both CTAs' copies land
      for (int v = max(0, u - ring); v < u; ++v) {
        const long long t0 = clock64();
        while (!mbar_test(full + 8 * (v % ring), (v / ring) & 1) && clock64() - t0 < kWaitLimit) {}
      }
    }
  } else if (warp == 1 && rank == 0) {
    RingPos at;
    int it = 0;
    bool ok = true;
    const uint64_t a_desc = smem_desc(sbase, 16, 1024, 2), w_desc = smem_desc(sbase + kWBox, 16, 1024, 2);
    for (int t = cluster; t < tiles && ok; t += clusters, ++it) {
      const int as = it & 1;
      if (!__all_sync(0xffffffffu, wait_bounded(acc_empty + 8 * as, ((it >> 1) & 1) ^ 1, guard, true))) break;
      tc_fence_after();
      for (int kb = 0; kb < p.kblocks; ++kb) {
        if (!(ok = wait_ring(full + 8 * at.stage, at.phase, guard))) break;
        tc_fence_after();
        const uint64_t off = (at.stage * stage_bytes) >> 4;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)   // 32 codes each
            mma_i8_ss_pair(tmem + 256 * as, a_desc + off + 2 * k, w_desc + off + 2 * k, p.idesc,
                           (kb | k) != 0 ? 1u : 0u);
          mma_commit_pair(empty + 8 * at.stage);
        }
        at.next(stages);
      }
      if (ok && elect_one()) mma_commit_pair(acc_full + 8 * as);
    }
  } else if (warp >= 4) {
    // Epilogue: warp w reads tensor memory lanes 32 (w % 4) .. + 32 (one token each) and every second of
    // the tile's blocks of 128 bytes of columns. Its results go into a box and leave by TMA; where the
    // output's rows are not aligned for that, or a tile ends inside a block, the warp stores them a row at
    // a time. The scales of the next tile are on their way while this one is worked on, the channels' in
    // shared memory, read by all lanes at once. (Rolled: a tile of a small product runs through here once,
    // and instructions that are read once cost more than the rest.) 6244 x 320 -> 4704 in bf16 20.1 us:
    // the chain of a block from tensor memory to its box, twice per SM sub-partition; with sixteen warps
    // 18.6, but 120 against 115 us for 2048 x 16384 -> 5120, whose ring then has less room. Handing the
    // accumulator back with a release at cluster scope, which waits for the stores, took 24.8.
    const int quarter = warp & 3, part = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    const uint32_t box = sbase + kManyBoxes + (uint32_t)(warp - 4) * 4096;
    float* w_scale = reinterpret_cast<float*>(smem + kManyScales) + kPartCols * (warp - 4);
    // (this warp's i-th 32 columns of a tile: its blocks are kEpiParts apart)
    const auto column = [&](int i) {
      return kCols * (part + kEpiParts * (32 * i / kCols)) + 32 * i % kCols;
    };
    float a_next = 0.f, w_next[kPartCols / 32];
    const auto fetch = [&](int t) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int row = tm * 256 + (int)rank * 128 + 32 * quarter + lane;
      a_next = row < p.rows ? p.a_scale[row] : 0.f;
#pragma unroll
      for (int i = 0; i < kPartCols / 32; ++i) {
        const int c = column(i), col = tn * p.n_tile + c + lane;
        w_next[i] = c < p.n_tile && col < p.n ? p.w_scale[col] : 0.f;
      }
    };
    if (cluster < tiles) fetch(cluster);
    int it = 0;
    for (int t = cluster; t < tiles; t += clusters, ++it) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int as = it & 1, row0 = tm * 256 + (int)rank * 128 + 32 * quarter;
      const int begin = tn * p.n_tile;
      const float a_scale = a_next;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPartCols / 32; ++i) w_scale[32 * i + lane] = w_next[i];
      __syncwarp();
      if (t + clusters < tiles) fetch(t + clusters);
      const bool ok = wait_bounded(acc_full + 8 * as, (it >> 1) & 1, guard);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
#pragma unroll 1
      for (int q = 0; q < kPartCols / 32; ++q) {
        const int c = column(q), half = 32 * q % kCols / 32;
        if (c >= p.n_tile) break;
        uint32_t r[32];
        tmem_ld32_sync(lanes | (tmem + 256 * as + c), r);
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 w = *reinterpret_cast<const float4*>(w_scale + 32 * q + j);
          v[j] = (float)(int32_t)r[j] * w.x * a_scale;
          v[j + 1] = (float)(int32_t)r[j + 1] * w.y * a_scale;
          v[j + 2] = (float)(int32_t)r[j + 2] * w.z * a_scale;
          v[j + 3] = (float)(int32_t)r[j + 3] * w.w * a_scale;
        }
        if (half == 0) {
          if (lane == 0) bulk_wait_group_read<0>();   // the last store has read the box
          __syncwarp();
        }
        put_row(box, lane, half, v, static_cast<const OT*>(nullptr));
        const int c0 = c - 32 * half, width = min(kCols, p.n_tile - c0);   // of the box
        if (c + 32 < c0 + width) continue;   // its other half comes first
        if (p.tma && width == kCols) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            // (what lies outside the output is not written)
            if (begin + c0 < p.n && row0 < p.rows) tma_store_2d(&tmap_out, box, begin + c0, row0);
            bulk_commit_group();
          }
        } else {
          __syncwarp();
          const int rows = min(32, p.rows - row0);
#pragma unroll 1
          for (int l = lane; l < width && begin + c0 + l < p.n; l += 32) {
            OT* out = static_cast<OT*>(p.out) + (int64_t)row0 * p.out_stride + begin + c0 + l;
#pragma unroll 1
            for (int r0 = 0; r0 < rows; r0 += 8) {
              OT o[8];   // (reads before stores: the compiler keeps their order)
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = get_one<OT>(smem + (box - sbase), r0 + i, l);
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (r0 + i < rows) out[(r0 + i) * p.out_stride] = o[i];
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_relaxed(map_to_rank(acc_empty + 8 * as, 0));   // the accumulator is free
    }
    if (lane == 0) bulk_wait_group0();   // the boxes are read before the block ends
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

// The output as a destination of boxes of 32 rows of 128 bytes.
template <typename OT>
bool encode_out(CUtensorMap* m, const LinearArgs& a) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)a.n, (cuuint64_t)a.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)a.out_stride * sizeof(OT)};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / sizeof(OT)), 32};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, sizeof(OT) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, a.out, dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr uint32_t kFewHead = 3 * 1024;   // barriers and scales, 1024 bytes each, and what aligns them
constexpr uint32_t kFewSmem = 113 * 1024, kFewSmemOne = 227 * 1024;   // two CTAs per SM, or one

// How linear_few cuts its work: the tokens of a tile, the CTAs that share its sum, the stages of their
// rings, and about how long it takes.
struct FewShape {
  int n_tile, row_tiles, splits, stages;
  uint32_t ring, smem;
  int64_t ns = INT64_MAX, capped_ns = INT64_MAX;
};
FewShape few_shape(const mla_decode_s& h, const LinearArgs& a) {
  const int row_tiles = (a.rows + kFewRows - 1) / kFewRows, kblocks = (a.k + kBoxK - 1) / kBoxK;
  const int n_tile = ((a.rows + row_tiles - 1) / row_tiles + 15) / 16 * 16;
  const int64_t tiles = (int64_t)((a.n + 127) / 128) * row_tiles;
  const uint32_t stage = kWBox + (uint32_t)n_tile * kBoxK;
  FewShape best{};
  // (tokens in several tiles only where the sum is shared: of a short sum linear_many's tiles read less and
  // their results leave while the next is summed: 2821 x 192 -> 1520 6.2 against 9.4 us)
  for (int splits = row_tiles > 1 ? 2 : 1; splits <= kMaxSplits && (splits == 1 || kblocks >= 2 * splits); ++splits)
    for (const bool two : {false, true}) {
      const uint32_t channels = (128 + splits - 1) / splits;   // of a CTA, at most
      const uint32_t parts = splits == 1 ? 0 : splits * channels * ((uint32_t)n_tile / 4) * 16;
      const int per = (kblocks + splits - 1) / splits;
      const uint32_t limit = two ? kFewSmem : kFewSmemOne;
      if (limit < parts + kFewHead + stage) continue;
      FewShape f{n_tile, row_tiles, splits};
      f.stages = std::min({kMaxFewStages, (int)((limit - parts - kFewHead) / stage), per});
      if (f.stages < std::min(3, per)) continue;
      f.ring = f.stages * stage;
      f.smem = kFewHead + f.ring + parts;
      // A k block arrives at some 110 bytes a nanosecond (two CTAs on an SM slow each other down, the more
      // tokens the more), as often as not all clusters fit at once; set-up, and the exchange of the
      // partial sums at 16 bytes a store.
      const int one = h.few_clusters[splits], clusters = one * (f.smem <= kFewSmem ? 2 : 1);
      if (clusters < 1) continue;
      const int64_t waves = (tiles + clusters - 1) / clusters, at_once = std::min<int64_t>(tiles, clusters);
      const int64_t arrival = waves * per * (int64_t)(stage / 110) * (at_once > one ? 10 + n_tile / 8 : 10) / 10;
      const int64_t rest = (row_tiles > 1 ? 2300 : 1600) + waves * 1400 + (splits > 1 ? 340 + 18 * n_tile : 10 * n_tile);
      if (arrival + rest >= best.ns) continue;
      best = f;
      best.ns = arrival + rest;
      // (against linear_many, not between the splits: all CTAs together get some 9600 bytes a nanosecond)
      best.capped_ns = std::max<int64_t>(arrival, waves * per * (int64_t)stage * at_once * splits / 9600) + rest;
    }
  return best;
}

template <typename OT>
cudaError_t launch_few(const mla_decode_s& h, const LinearArgs& a, const FewShape& f, cudaStream_t s) {
  FewParams p{};
  p.rows = a.rows;
  p.n = a.n;
  p.n_tile = f.n_tile;
  p.kblocks = (a.k + kBoxK - 1) / kBoxK;
  p.splits = f.splits;
  p.stages = f.stages;
  p.ring = f.ring;
  p.recip = ((1u << 18) + f.splits - 1) / f.splits;
  p.pitch = (128 + f.splits - 1) / f.splits * 16;
  CUtensorMap tw, ta;
  if (!encode(&tw, a.w_codes, (uint64_t)a.n, (uint64_t)a.k, (uint64_t)a.w_stride, 128) ||
      !encode(&ta, a.codes, (uint64_t)a.rows, (uint64_t)a.k, (uint64_t)a.codes_stride, (uint32_t)p.n_tile))
    return cudaErrorInvalidValue;
  p.idesc = idesc_i8_s32(128, p.n_tile);
  p.a_scale = a.scales;
  p.w_scale = a.w_scales;
  p.out = a.out;
  p.out_stride = a.out_stride;
  p.err = h.ws.err;
  const auto kernel = f.row_tiles > 1 ? linear_few<OT, true> : linear_few<OT, false>;
  return launch_pdl_cluster(kernel, dim3((a.n + 127) / 128 * p.splits, f.row_tiles), dim3(256), f.smem, p.splits, s, tw,
                            ta, p);
}

// linear_many's channels per tile, and about how long it takes: the pairs work in rounds, a tile each, so
// what a round takes counts as often as there are rounds.
struct ManyShape {
  int n_tile = 0;
  int64_t ns = INT64_MAX;
};
ManyShape many_shape(const mla_decode_s& h, const LinearArgs& a) {
  const int64_t kblocks = (a.k + kBoxK - 1) / kBoxK, tiles_m = (a.rows + 255) / 256, clusters = h.num_sms / 2;
  ManyShape best;
  for (int tile = 256; tile >= 32; tile -= 32) {
    const int64_t tiles = tiles_m * ((a.n + tile - 1) / tile), rounds = (tiles + clusters - 1) / clusters;
    // cycles, as measured: a k block of a tile (2 x tile of them are the MMAs' at tile 256; narrower tiles
    // read as many tokens for less), and its results' way out, beside the next tile's sum but for the last;
    // in ns at 1.75 GHz (the longest products run at less, where linear_few is no choice)
    const int64_t sum = kblocks * (220 + 14 * tile / 10), store = 400 + (tile + 63) / 64 * 850;
    const int64_t ns = 3800 + (rounds * std::max(sum, store) + std::min(sum, store)) * 4 / 7;
    if (ns < best.ns) best = ManyShape{tile, ns};
  }
  return best;
}

template <typename OT>
cudaError_t launch_many(const mla_decode_s& h, const LinearArgs& a, int n_tile, cudaStream_t s) {
  ManyParams p{};
  p.rows = a.rows;
  p.n = a.n;
  p.kblocks = (a.k + kBoxK - 1) / kBoxK;
  p.tiles_m = (a.rows + 255) / 256;
  p.n_tile = n_tile;
  p.tiles_n = (a.n + p.n_tile - 1) / p.n_tile;
  p.group = 8;
  p.idesc = idesc_i8_s32(256, p.n_tile);
  p.a_scale = a.scales;
  p.w_scale = a.w_scales;
  p.out = a.out;
  p.out_stride = a.out_stride;
  p.tma = (reinterpret_cast<uintptr_t>(a.out) | (uint64_t)a.out_stride * sizeof(OT)) % 16 == 0;
  p.stages = std::min<int>(kMaxManyStages, kManyRing / (kWBox + p.n_tile / 2 * kBoxK));
  p.err = h.ws.err;
  CUtensorMap tw, ta, to{};
  if (p.tma && !encode_out<OT>(&to, a)) return cudaErrorInvalidValue;
  if (!encode(&tw, a.w_codes, (uint64_t)a.n, (uint64_t)a.k, (uint64_t)a.w_stride, (uint32_t)p.n_tile / 2) ||
      !encode(&ta, a.codes, (uint64_t)a.rows, (uint64_t)a.k, (uint64_t)a.codes_stride, 128))
    return cudaErrorInvalidValue;
  const int clusters = std::min(h.num_sms / 2, p.tiles_m * p.tiles_n);
  return launch_pdl(linear_many<OT>, dim3(2 * clusters), dim3(kManyThreads), kManySmem, s, tw, ta, to, p);
}

}  // namespace

cudaError_t init_linear_q8(mla_decode_s& h) {
  const struct { const void* kernel; uint32_t smem; } need[] = {
      {reinterpret_cast<const void*>(linear_few<float, false>), kFewSmemOne},
      {reinterpret_cast<const void*>(linear_few<float, true>), kFewSmemOne},
      {reinterpret_cast<const void*>(linear_few<__nv_bfloat16, false>), kFewSmemOne},
      {reinterpret_cast<const void*>(linear_few<__nv_bfloat16, true>), kFewSmemOne},
      {reinterpret_cast<const void*>(linear_many<float>), kManySmem},
      {reinterpret_cast<const void*>(linear_many<__nv_bfloat16>), kManySmem}};
  for (const auto& k : need) {
    const cudaError_t e = cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)k.smem);
    if (e != cudaSuccess) return e;
  }
  // A cluster stays within a group of SMs, so how many fit depends on the groups' sizes. Asked for one
  // CTA per SM: for two of a kernel that takes tensor memory the answer is still one, while two do run
  // (1 x 5120 -> 2112 over 17 clusters of 8: 4.8 us, where 15 fit with one; 9 us over clusters of 7
  // that leave room for one).
  for (int splits = 1; splits <= kMaxSplits; ++splits) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(splits);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = kFewSmemOne;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaOccupancyMaxActiveClusters(&h.few_clusters[splits], linear_few<float, false>, &cfg);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_linear_q8(const mla_decode_s& h, const LinearArgs& a, cudaStream_t s) {
  // Up to 64 tokens always linear_few, a pair's tile of 256 being mostly empty (it was ahead for every one of
  // nine weights, 512 -> 512, 64 -> 131072 and 2048 -> 128 among them: 1 x 5120 -> 2112 4.9 us against 17.5,
  // 64 x 16384 -> 5120 18.2 against 27.8, 64 x 512 -> 512 3.7 against 3.9); of more, the one that should be
  // done first: few channels under a long sum are one pair's work for long, while clusters share it (us,
  // linear_few against linear_many: 491 x 14864 -> 172 10.6 and 27.3, 128 x 1536 -> 16384 8.8 and 10.1,
  // 195 x 15913 -> 2655 23 and 36; 512 x 5120 -> 2112 15 and 11.7, 2821 x 192 -> 1520 9.4 and 6.2).
  const FewShape f = few_shape(h, a);
  const ManyShape m = a.rows <= 64 ? ManyShape{} : many_shape(h, a);
  if (f.capped_ns < m.ns) return a.out_f32 ? launch_few<float>(h, a, f, s) : launch_few<__nv_bfloat16>(h, a, f, s);
  if (m.n_tile == 0) return cudaErrorInvalidValue;
  return a.out_f32 ? launch_many<float>(h, a, m.n_tile, s) : launch_many<__nv_bfloat16>(h, a, m.n_tile, s);
}

}  // namespace mla
