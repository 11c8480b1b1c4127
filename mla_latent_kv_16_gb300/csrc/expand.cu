// The expansion of a windowed prefill: per-head keys and values from the latent
// rows, K[t] = W_UK c_KV[t] and V[t] = W_UV c_KV[t] for all heads, both weights
// and both row regions (the sinks and the window's rows, see prefill_window.cu) in one
// launch.
//
// The product is [rows x 512] x [512 x H*128], twice: K = 512 is short, so a
// 128 x 256 tile per CTA needs 384 KB of operands for 4,096 cycles of MMAs, and
// the generic linear layer is bound by what the SMs can take in from L2 (119 us for
// both weights at 4096 rows and 128 heads: 13 TB/s). Here a pair of CTAs computes
// 256 x 256 tiles with cta_group::2 MMAs, each CTA streaming its 128 token rows and
// its half of the weight tile: 256 KB per 4,096 cycles through a ring of six 32 KB
// stages. 96 us at the same size, 1.43 PFLOP/s, 11 TB/s from L2 beside the 2.8 TB/s
// of outputs (75 us with the stores left out). Measured and not kept: the token
// rows resident in shared memory (half the L2 traffic, but only 64 KB left in
// flight: 107 us), five stages and two staging areas per epilogue warp (97 us).
//
// The products accumulate in fp32 and are rounded to bf16 once: they are operands of
// the attention's bf16 MMAs.
//
// Warps of each CTA: 0 = TMA producer, 1 = MMA issue (leader CTA only), 2-9 =
// epilogue (two per TMEM lane quarter, 128 of the tile's 256 outputs each): the
// rows are packed to bf16, staged (4 KB per warp, 128-byte swizzle) and stored by
// TMA, whose maps end where a region ends. TMEM: two accumulators of 256 columns.
//
// The loads of both CTAs complete on the leader's barriers; the leader's commits
// release the slots in both. Every wait is bounded: on a timeout a CTA raises
// MLA_DEVERR_TIMEOUT and leaves, and so does its peer when its own waits run out.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "host.h"
#include "launchers.h"
#include "tc_ptx.cuh"

namespace mla {
namespace {

using namespace tc;

constexpr int kExThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kPairRows = 256;          // token rows of a pair's tile (128 per CTA)
constexpr int kOutTile = 256;           // outputs of a tile
constexpr int kChunks = kDC / 64;       // K chunks of 64 columns
constexpr int kBoxBytes = 128 * 128;    // 128 rows x 64 bf16, 128-byte swizzled
constexpr int kStages = 6;              // ring of K chunks: 128 token rows and 128 weight rows
constexpr int kStoreBytes = 32 * 128;   // 32 rows x 64 bf16
constexpr uint32_t kAccCols = 256;

struct __align__(1024) ExSmem {
  uint8_t a[kStages][kBoxBytes];
  uint8_t b[kStages][kBoxBytes];
  uint8_t st[kEpiWarps][kStoreBytes];
  uint64_t full[kStages], empty[kStages];        // full: the leader's counts
  uint64_t acc_full[2], acc_empty[2];            // empty: the leader's counts
  uint64_t drain;
  uint32_t tmem_base;
  int32_t abort_flag;
};
constexpr size_t kExSmemBytes = sizeof(ExSmem) + 1024;
static_assert(kExSmemBytes <= 232448, "shared memory budget of one CTA");

// Rows of both regions (0: the sinks, 1: the window's rows), the weights, and the
// outputs of each weight in each region.
struct ExMaps {
  CUtensorMap rows[2];
  CUtensorMap w[2];
  CUtensorMap out[2][2];  // [weight][region]
};

struct ExArgs {
  int32_t region_rows[2];
  int32_t n_out;          // H * 128
  int32_t out_tiles;      // per weight
  int32_t units;          // row tiles x 2 weights x out_tiles
  int32_t* dev_error;
};

// ---- cta_group::2 forms

__device__ __forceinline__ void tmem_alloc_pair(uint32_t holder_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(holder_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Load into this CTA's shared memory, completing on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, uint32_t cluster_bar, int32_t x,
                                                 int32_t y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void mma_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs once the issued MMAs complete.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// Unit u: row tiles outermost, so that a pair's consecutive units share their rows.
struct Unit {
  int region, row0, weight, out0, row_tile;
};
__device__ __forceinline__ Unit unit_at(const ExArgs& a, int u) {
  Unit r;
  const int per = 2 * a.out_tiles;
  r.row_tile = u / per;
  const int j = u - r.row_tile * per;
  r.weight = j / a.out_tiles;
  r.out0 = (j - r.weight * a.out_tiles) * kOutTile;
  const int tiles0 = (a.region_rows[0] + kPairRows - 1) / kPairRows;
  r.region = r.row_tile < tiles0 ? 0 : 1;
  r.row0 = (r.row_tile - (r.region ? tiles0 : 0)) * kPairRows;
  return r;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kExThreads, 1)
    expand_kernel(const __grid_constant__ ExMaps maps, const ExArgs a) {
  extern __shared__ uint8_t smem_raw[];
  ExSmem* sm = reinterpret_cast<ExSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int u0 = static_cast<int>(static_cast<int64_t>(pair) * a.units / pairs);
  const int u1 = static_cast<int>(static_cast<int64_t>(pair + 1) * a.units / pairs);
  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&sm->full[s]), 1);
      mbar_init(smem_u32(&sm->empty[s]), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&sm->acc_full[x]), 1);
      mbar_init(smem_u32(&sm->acc_empty[x]), 2 * kEpiWarps);
    }
    mbar_init(smem_u32(&sm->drain), 1);
    sm->abort_flag = 0;
    fence_mbar_init_cluster();
    for (int x = 0; x < 2; ++x) {
      prefetch_tmap(&maps.rows[x]);
      prefetch_tmap(&maps.w[x]);
    }
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&sm->tmem_base), 2 * kAccCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  volatile int32_t* abort_flag = &sm->abort_flag;
  pdl_wait();

  if (warp == 0) {
    if (lane == 0) {
      // ---- TMA producer
      const uint32_t full = map_to_rank(smem_u32(&sm->full[0]), 0);
      const uint64_t keep = l2_evict_last_policy();  // read by many pairs, while the outputs stream past them
      const int mine = 128 * static_cast<int>(rank);
      uint32_t g = 0;  // chunks requested so far
      bool ok = true;
      for (int u = u0; ok && u < u1; ++u) {
        const Unit w = unit_at(a, u);
        for (int k = 0; k < kChunks; ++k, ++g) {
          const int s = static_cast<int>(g % kStages);
          if (g >= kStages)
            ok = mbar_wait<2>(smem_u32(&sm->empty[s]), ((g / kStages) & 1) ^ 1, abort_flag, a.dev_error);
          if (!ok) break;
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sm->full[s]), 4 * kBoxBytes);
          tma_load_2d_pair(smem_u32(sm->a[s]), &maps.rows[w.region], full + 8 * s, 64 * k, w.row0 + mine, keep);
          tma_load_2d_pair(smem_u32(sm->b[s]), &maps.w[w.weight], full + 8 * s, 64 * k, w.out0 + mine, keep);
        }
      }
      if (rank == 0) {
        // what was requested lands before the CTAs go (after an abort nobody consumes it)
        volatile int32_t never = 0;
        const uint32_t from = g > kStages ? g - kStages : 0;
        for (uint32_t q = from; q < g; ++q)
          mbar_wait<2>(smem_u32(&sm->full[q % kStages]), (q / kStages) & 1, &never, nullptr);
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      // ---- MMA issuer, for both CTAs
      constexpr uint32_t kId = idesc_bf16_f32(kPairRows, kOutTile, false, false);
      const uint64_t da = sdesc_sw128(smem_u32(sm->a[0]), 16, 1024), db = sdesc_sw128(smem_u32(sm->b[0]), 16, 1024);
      uint32_t g = 0;
      bool ok = true;
      for (int u = u0; ok && u < u1; ++u) {
        const int i = u - u0, x = i & 1;
        if (i >= 2) ok = mbar_wait<2>(smem_u32(&sm->acc_empty[x]), ((i >> 1) - 1) & 1, abort_flag, a.dev_error);
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(x) * kAccCols;
        for (int k = 0; ok && k < kChunks; ++k, ++g) {
          const int s = static_cast<int>(g % kStages);
          ok = mbar_wait<2>(smem_u32(&sm->full[s]), (g / kStages) & 1, abort_flag, a.dev_error);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (uint32_t kk = 0; kk < 4; ++kk)
            mma_ss_pair(d, da + ((s * kBoxBytes + kk * 32u) >> 4), db + ((s * kBoxBytes + kk * 32u) >> 4), kId,
                        (k > 0 || kk > 0) ? 1u : 0u);
          mma_commit_pair(smem_u32(&sm->empty[s]));
        }
        if (!ok) break;
        mma_commit_pair(smem_u32(&sm->acc_full[x]));
      }
      // every MMA this thread issued completes before TMEM is freed
      mma_commit_pair(smem_u32(&sm->drain));
      volatile int32_t never = 0;
      mbar_wait<2>(smem_u32(&sm->drain), 0, &never, nullptr);
    }
  } else {
    // ---- epilogue: warp e has TMEM lane quarter q4 and outputs [128 half, +128) of the tile
    const int e = warp - 2, q4 = warp & 3, half = e >> 2;
    const uint32_t lanes = static_cast<uint32_t>(q4 * 32) << 16;
    const uint32_t acc_empty = map_to_rank(smem_u32(&sm->acc_empty[0]), 0);
    const uint64_t pol = l2_evict_first_policy();  // (larger than L2 where the speed counts)
    uint8_t* st = sm->st[e];
    for (int u = u0; u < u1; ++u) {
      const int i = u - u0, x = i & 1;
      const Unit w = unit_at(a, u);
      if (!__all_sync(0xffffffffu, mbar_wait<0>(smem_u32(&sm->acc_full[x]), (i >> 1) & 1, abort_flag, a.dev_error)))
        break;
      tc_fence_after();
      const int row = w.row0 + 128 * static_cast<int>(rank) + q4 * 32;
#pragma unroll
      for (int c = 0; c < 128; c += 64) {
        float v[64];
        tmem_ld64_sync(tmem + static_cast<uint32_t>(x) * kAccCols + lanes + 128u * half + c, v);
        if (c == 64) {  // this warp has read its part of the accumulator
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(acc_empty + 8 * x);
        }
        if (lane == 0) bulk_wait_group_read0();  // the staging area's last store has been read
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<uint4*>(st + lane * 128 + ((j ^ (lane & 7)) << 4)) =
              make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                         pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
        fence_proxy_async_smem();
        __syncwarp();
        const int out = w.out0 + 128 * half + c;
        if (lane == 0 && row < a.region_rows[w.region] && out < a.n_out) {
          tma_store_2d(&maps.out[w.weight][w.region], smem_u32(st), out, row, pol);
          bulk_commit_group();
        }
      }
    }
    if (lane == 0) bulk_wait_group_read0();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // nothing of either CTA is in flight towards the other
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * kAccCols);
  }
}

// [rows][cols] bf16 with row stride `stride` elements, 64 x box_rows boxes, 128-byte swizzle
bool ex_map(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint64_t stride, uint32_t box_rows) {
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {stride * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_expand(const ExpandArgs& x, cudaStream_t s) {
  if (tensor_map_encoder() == nullptr) return cudaErrorNotSupported;
  const uint64_t hd = static_cast<uint64_t>(x.heads) * 128;
  ExMaps maps;
  ExArgs a{};
  const auto at = [](const void* base, int64_t row, int64_t stride) {
    return static_cast<const char*>(base) + row * stride * 2;
  };
  const int32_t from[2] = {0, x.lo}, to[2] = {0, x.rows_a}, n[2] = {x.rows_a, x.rows_b};
  const void* w[2] = {x.w_uk, x.w_uv};
  void* out[2] = {x.k_nope, x.v};
  for (int r = 1; r >= 0; --r) {
    a.region_rows[r] = n[r];
    if (n[r] == 0) {  // no such region: never visited
      maps.rows[r] = maps.rows[1];
      for (int k = 0; k < 2; ++k) maps.out[k][r] = maps.out[k][1];
      continue;
    }
    if (!ex_map(&maps.rows[r], at(x.rows, from[r], kRow), static_cast<uint64_t>(n[r]), kDC, kRow, 128))
      return cudaErrorInvalidValue;
    for (int k = 0; k < 2; ++k)
      if (!ex_map(&maps.out[k][r], at(out[k], to[r], static_cast<int64_t>(hd)), static_cast<uint64_t>(n[r]), hd, hd, 32))
        return cudaErrorInvalidValue;
  }
  for (int k = 0; k < 2; ++k)
    if (!ex_map(&maps.w[k], w[k], hd, kDC, kDC, 128)) return cudaErrorInvalidValue;
  a.n_out = static_cast<int32_t>(hd);
  a.out_tiles = (a.n_out + kOutTile - 1) / kOutTile;
  const int64_t row_tiles = (n[0] + kPairRows - 1) / kPairRows + (n[1] + kPairRows - 1) / kPairRows;
  a.units = static_cast<int32_t>(row_tiles * 2 * a.out_tiles);
  a.dev_error = x.dev_error;
  static SmemOptIn opt_in;
  const cudaError_t e = opt_in(kExSmemBytes, expand_kernel);
  if (e != cudaSuccess) return e;
  const int pairs = device_sm_count() / 2;
  const unsigned grid = 2u * static_cast<unsigned>(a.units < pairs ? a.units : pairs);
  return launch_pdl(expand_kernel, dim3(grid), dim3(kExThreads), kExSmemBytes, s, maps, a);
}

}  // namespace mla
