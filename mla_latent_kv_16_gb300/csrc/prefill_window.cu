// Windowed prefill attention in the MHA form on the 5th-generation tensor cores
// (mla_prefill_window), after the expansion of K and V (expand.cu).
//
// The query at position p = n_tokens - n_queries + j sees the keys t <= p with
// p - t < window or t < sinks:
//   o_h[j] = sum_t softmax_t(q_h[j] . [K_nope_h[t] ; k_R[t]] * scale) V_h[t]
//
// Only rows that some query of the call sees are expanded and loaded: the sinks
// (region A) and [lo, n_tokens) (region B, lo = the first query's first window
// row), or all rows as one region when the two meet. Each region has tensor maps of
// its own, which end where it ends, so the ends of the last tiles read as zeros (a
// hidden row's V must not be Inf or NaN: 0 * NaN is not 0).
//
// Persistent, one CTA per SM; a work item is (head, 128 queries). Per tile of 128
// keys S = Q K^T (M = 128, N = 128, K = 192: 12 MMAs) and O += P V (N = 128, K = 128: 8
// MMAs, P in TMEM as the A operand). S and P are double-buffered, so the products of
// the neighbouring tiles run under a tile's softmax, which is what a tile takes: a
// chain of scores, maximum, exponentials and P. Sixteen warps share it (four per TMEM
// lane quarter, thread = query row, 32 of the tile's keys each), which meet once per
// tile to agree on the row maxima; scales and sums take two values per instruction.
// The rings and buffers run on from one item to the next: its first K and its Q (on
// their way into L2 an item ahead) are loaded as soon as the last item's last QK is
// done, and that item's outputs are written behind the new item's first tile, when O
// has long been complete and the new PV can wait a tile for it.
//
// Measured (4096 tokens, 128 heads, window 1024, 64 sinks: 35,200 tiles): 294 us, about
// 2,100 cycles per tile against 1,290 of MMAs, 3,000 cycles per item besides (its three
// tiles with an edge of the mask cost 600 to 800 more each). Steps to it: an item's
// outputs before the next item's first tile, Q asked for behind the last V, and one
// 16-byte piece of 32 rows per store instead of four of eight rows 326 (6,200 cycles
// between items); the softmax warps finding their items themselves 309 (1,000 cycles
// of divisions); one value per instruction 299. Not kept: one CTA per item 373;
// eight softmax warps 328 against 323; two query tiles per CTA, a warpgroup each, with
// P over S 410-555; the outputs' code out of line 335 against 309.
//
// Scores, maxima, sums and O are fp32. K, V (by the expansion) and P are rounded to bf16,
// the type of the MMAs' operands: with the output's own rounding o is within 0.0031 of
// the exact value in relative L2, where fp32 products rounded once have 0.0017. Two
// bf16 terms for each operand would take that away for twice to four times the MMAs.
//
// Which tiles: the sinks' tiles, then region B's from the query tile's own first
// window row on. Where an edge of the mask crosses a tile its hidden keys are found
// by a bit per key. A row may see nothing of a tile it visits, the first one
// included: its running max stays -inf and its weights there are taken relative to 0.
//
// Warps: 0-15 softmax, 16 = TMA (K and V rings of two tiles), 17 = QK issue, 18 = PV
// issue (an issuing thread stays busy while the tensor pipe takes its MMAs: one for
// each product). TMEM (512 columns): two S buffers [0,128) [128,256), O [256,384),
// two P buffers [384,448) [448,512) (bf16 pairs).
//
// Every wait is bounded; on a timeout the CTA raises MLA_DEVERR_TIMEOUT, lets its
// own copies and MMAs land, writes NaN outputs for its rows and frees TMEM.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include "common.cuh"
#include "host.h"
#include "launchers.h"
#include "tc_ptx.cuh"

namespace mla {
namespace {

using namespace tc;

constexpr int kTile = 128;  // queries of a tile, keys of a tile
constexpr int kParts = 4;   // softmax warps per lane quarter
constexpr int kKeys = kTile / kParts;  // keys of a tile per softmax warp
constexpr int kSmxWarps = 4 * kParts;
static_assert(kKeys == 32, "one TMEM load, one word of mask bits");
constexpr int kTmaWarp = kSmxWarps, kQkWarp = kSmxWarps + 1, kPvWarp = kSmxWarps + 2;
constexpr int kPwThreads = 32 * (kSmxWarps + 3);
constexpr int kBox = 128 * 128;  // 128 rows x 64 bf16
constexpr int kStagesK = 2, kStagesV = 2;
constexpr uint32_t kTmS = 0, kTmO = 256, kTmP = 384;
constexpr float kRescaleLog2 = 8.0f;
constexpr int kHeadGroup = 16;
constexpr int kItemSlots = 8;  // (five are enough)

// A work item's tiles as the softmax warps walk them. Tile j begins at key j * 128, from j =
// n_a on at j * 128 + k0_b. No edge of the mask crosses the tiles [0, a_full) and [b_lo, b_hi).
struct __align__(16) ItemTiles {
  int n_kt, a_full, b_lo, b_hi;
  int pos0, n_a, k0_b;
  int h, q0;
};

struct __align__(1024) PwSmem {
  uint8_t q[3][kBox];
  uint8_t k[kStagesK][3][kBox];
  uint8_t v[kStagesV][2][kBox];
  uint64_t q_full, q_empty;
  uint64_t k_full[kStagesK], k_empty[kStagesK];
  uint64_t v_full[kStagesV], v_empty[kStagesV];
  uint64_t s_full[2], s_free[2];  // S of tile j in buffer j & 1: written by QK / read by the softmax warps
  uint64_t p_full[2];             // P of tile j in buffer j & 1 (and any O rescale) complete
  uint64_t p_free[2];             // PV of the tile that last used P buffer x is done
  uint64_t o_done, o_free;        // O of an item complete / read by the softmax warps
  uint64_t item_full[kItemSlots];  // items[x] written
  uint64_t drain, drain_pv;
  float mx_part[2][kParts][128];  // tile j's row max over a warp's keys, in [j & 1]
  float lsum[2][kParts][128];     // item i's row sum over each softmax warp's keys, in [i & 1]
  float mlast[2][128];            // and its row maximum
  ItemTiles items[kItemSlots];    // what the softmax warps need of item i, in [i % kItemSlots]
  uint32_t tmem_base;
  int32_t abort_flag;
};
constexpr size_t kPwSmemBytes = sizeof(PwSmem) + 1024;
static_assert(kPwSmemBytes <= 232448, "shared memory budget of one CTA");

// q, qr: the queries; k, kr, v: the rows of region 0 (the sinks) and 1 (the window's).
struct PwMaps {
  CUtensorMap q, qr;
  CUtensorMap k[2], kr[2], v[2];
};

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// Two fp32 values in a register pair, and both lanes' a b + c and a + b (each rounded as the
// single instruction rounds).
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bits [0, n) of 32, n clamped to 0..32.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

__device__ __forceinline__ void pw_drain(uint32_t bar, uint32_t parity, int32_t* dev_error) {
  volatile int32_t never = 0;
  mbar_wait<2>(bar, parity, &never, dev_error);
}

// A work item: 128 queries of one head, and the key tiles they see.
struct Item {
  int h, q0;
  int pos0;         // position of the first query
  int n_a;          // key tiles of the sinks; then region B's (which starts at row w.lo) from b_first on
  int b_first;
  int n_kt;
  // row of tile j in its region's maps
  __device__ __forceinline__ int row(int j) const { return (j < n_a ? j : j - n_a + b_first) * kTile; }
};

__device__ __forceinline__ Item item_at(const PrefillArgs& a, const PrefillWindow& w, int n_qt, int u) {
  // Heads go in groups of up to 16, whose K and V stay in L2 while neighbouring
  // query tiles read them; within a group the last query tiles go first.
  const int G = min(kHeadGroup, a.heads);
  const int grp = u / (G * n_qt);
  const int gh = min(G, a.heads - grp * G);  // heads in this group (fewer in a last, partial one)
  const int r = u - grp * G * n_qt;
  Item it;
  it.h = grp * G + r % gh;
  it.q0 = (n_qt - 1 - r / gh) * kTile;
  it.pos0 = a.n_tokens - a.n_queries + it.q0;
  const int last = min(a.n_tokens - 1, it.pos0 + kTile - 1);
  const int first_key = max(0, it.pos0 - a.window + 1);
  it.n_a = (min(a.sinks, w.split ? a.sinks : last + 1) + kTile - 1) / kTile;
  it.b_first = w.split ? (first_key - w.lo) / kTile : max(it.n_a, first_key / kTile);
  it.n_kt = it.n_a + max(0, (last - w.lo) / kTile + 1 - it.b_first);
  return it;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t par, PwSmem* sm, int32_t* dev_error) {
  return __all_sync(0xffffffffu, mbar_wait<0>(smem_u32(bar), par, &sm->abort_flag, dev_error));
}

// The four warps of a lane quarter meet, and learn whether all of them are well.
__device__ __forceinline__ bool meet(int q4, bool v) {
  switch (q4) {
    case 0: return bar_red_and<1, 32 * kParts>(v);
    case 1: return bar_red_and<2, 32 * kParts>(v);
    case 2: return bar_red_and<3, 32 * kParts>(v);
    default: return bar_red_and<4, 32 * kParts>(v);
  }
}

// The four warps of a row quarter hold 32 outputs each of 32 rows, 64 bytes of a row per
// lane: w[16]. Groups of four lanes exchange their 16-byte pieces so that a store
// writes 64 bytes of eight rows instead of 16 bytes of 32. Afterwards piece k belongs
// to row (lane & ~3) + k and lies (lane & 3) * 16 bytes into it.
__device__ __forceinline__ void transpose4(uint32_t (&w)[16], int lane) {
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int step = 1 << b;
    const bool up = lane & step;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c & step) continue;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t& lo = w[4 * c + x];
        uint32_t& hi = w[4 * (c + step) + x];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, step);
        lo = up ? got : lo;
        hi = up ? hi : got;
      }
    }
  }
}

__global__ void __launch_bounds__(kPwThreads, 1)
    prefill_window_kernel(const __grid_constant__ PwMaps maps, const PrefillArgs a, const PrefillWindow w,
                          const int n_qt, const int units) {
  extern __shared__ uint8_t smem_raw[];
  PwSmem* sm = reinterpret_cast<PwSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sm->q_full), 1);
    mbar_init(smem_u32(&sm->q_empty), 1);
    for (int s = 0; s < kStagesK; ++s) {
      mbar_init(smem_u32(&sm->k_full[s]), 1);
      mbar_init(smem_u32(&sm->k_empty[s]), 1);
    }
    for (int s = 0; s < kStagesV; ++s) {
      mbar_init(smem_u32(&sm->v_full[s]), 1);
      mbar_init(smem_u32(&sm->v_empty[s]), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&sm->s_full[x]), 1);
      mbar_init(smem_u32(&sm->s_free[x]), kSmxWarps);
      mbar_init(smem_u32(&sm->p_full[x]), kSmxWarps);
      mbar_init(smem_u32(&sm->p_free[x]), 1);
    }
    mbar_init(smem_u32(&sm->o_done), 1);
    mbar_init(smem_u32(&sm->o_free), kSmxWarps);
    for (int x = 0; x < kItemSlots; ++x) mbar_init(smem_u32(&sm->item_full[x]), 1);
    mbar_init(smem_u32(&sm->drain), 1);
    mbar_init(smem_u32(&sm->drain_pv), 1);
    sm->abort_flag = 0;
    fence_mbar_init_cluster();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.qr);
    prefetch_tmap(&maps.k[1]);
    prefetch_tmap(&maps.kr[1]);
    prefetch_tmap(&maps.v[1]);
  }
  if (warp == kQkWarp) tmem_alloc(smem_u32(&sm->tmem_base), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = sm->tmem_base;
  volatile int32_t* abort_flag = &sm->abort_flag;

  // In every role g counts the key tiles over all of this CTA's items (it sets the
  // ring slots, the S and P buffers and their phases), i the items.
  if (warp == kTmaWarp) {
    // ================= TMA producer: per item Q, then K(0), then K(j + 1) before V(j)
    if (lane == 0) {
      int gk = 0, gv = 0, i = 0;
      bool ok = true;
      auto load_k = [&](const Item& it, int j) -> bool {
        const int s = gk % kStagesK;
        if (gk >= kStagesK && !mbar_wait<2>(smem_u32(&sm->k_empty[s]), ((gk / kStagesK) & 1) ^ 1, abort_flag,
                                            a.dev_error))
          return false;
        const uint32_t bar = smem_u32(&sm->k_full[s]);
        const int r = j < it.n_a && w.split ? 0 : 1, y = it.row(j);
        mbar_arrive_expect_tx(bar, 3 * kBox);
        tma_load_2d_nohint(smem_u32(sm->k[s][0]), &maps.k[r], bar, it.h * 128, y);
        tma_load_2d_nohint(smem_u32(sm->k[s][1]), &maps.k[r], bar, it.h * 128 + 64, y);
        tma_load_2d_nohint(smem_u32(sm->k[s][2]), &maps.kr[r], bar, 512, y);
        ++gk;
        return true;
      };
      auto load_v = [&](const Item& it, int j) -> bool {
        const int s = gv % kStagesV;
        if (gv >= kStagesV && !mbar_wait<2>(smem_u32(&sm->v_empty[s]), ((gv / kStagesV) & 1) ^ 1, abort_flag,
                                            a.dev_error))
          return false;
        const uint32_t bar = smem_u32(&sm->v_full[s]);
        const int r = j < it.n_a && w.split ? 0 : 1, y = it.row(j);
        mbar_arrive_expect_tx(bar, 2 * kBox);
        tma_load_2d_nohint(smem_u32(sm->v[s][0]), &maps.v[r], bar, it.h * 128, y);
        tma_load_2d_nohint(smem_u32(sm->v[s][1]), &maps.v[r], bar, it.h * 128 + 64, y);
        ++gv;
        return true;
      };
      auto load_q = [&](const Item& it) {
        const uint32_t bar = smem_u32(&sm->q_full);
        mbar_arrive_expect_tx(bar, 3 * kBox);
        tma_load_2d_nohint(smem_u32(sm->q[0]), &maps.q, bar, it.h * 128, it.q0);
        tma_load_2d_nohint(smem_u32(sm->q[1]), &maps.q, bar, it.h * 128 + 64, it.q0);
        tma_load_2d_nohint(smem_u32(sm->q[2]), &maps.qr, bar, it.h * 64, it.q0);
        ++i;
      };
      Item it = item_at(a, w, n_qt, blockIdx.x);
      ok = load_k(it, 0);
      load_q(it);
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
        const bool more = u + static_cast<int>(gridDim.x) < units;
        Item next = it;
        for (int j = 0; ok && j < it.n_kt; ++j) {
          if (j + 1 < it.n_kt) ok = load_k(it, j + 1);
          if (more && j == min(2, it.n_kt - 1)) {  // (behind the item's first loads)
            next = item_at(a, w, n_qt, u + gridDim.x);
            if (j + 1 < it.n_kt) {  // Q comes from HBM, once: on its way into L2
              tma_prefetch_l2_2d(&maps.q, next.h * 128, next.q0);
              tma_prefetch_l2_2d(&maps.q, next.h * 128 + 64, next.q0);
              tma_prefetch_l2_2d(&maps.qr, next.h * 64, next.q0);
            }
          }
          if (ok && more && j + 1 == it.n_kt) {
            // the next item's first loads, as soon as this one's last QK is done with Q
            ok = load_k(next, 0) && mbar_wait<2>(smem_u32(&sm->q_empty), (i - 1) & 1, abort_flag, a.dev_error);
            if (ok) load_q(next);
          }
          if (ok) ok = load_v(it, j);
        }
        it = next;
      }
      // our own loads land before the CTA tears down
      for (int j = max(0, gk - kStagesK); j < gk; ++j)
        pw_drain(smem_u32(&sm->k_full[j % kStagesK]), (j / kStagesK) & 1, a.dev_error);
      for (int j = max(0, gv - kStagesV); j < gv; ++j)
        pw_drain(smem_u32(&sm->v_full[j % kStagesV]), (j / kStagesV) & 1, a.dev_error);
      if (i > 0) pw_drain(smem_u32(&sm->q_full), (i - 1) & 1, a.dev_error);
    }
  } else if (warp == kQkWarp) {
    // ================= QK issue: S(g) = Q K(g)^T as soon as K(g) has landed and score
    // buffer g & 1 has been read out
    if (lane == 0) {
      constexpr uint32_t kIdQK = idesc_bf16_f32(128, 128, false, false);
      const uint64_t dQ = sdesc_sw128(smem_u32(sm->q[0]), 16, 1024);
      const uint64_t dK = sdesc_sw128(smem_u32(sm->k[0][0]), 16, 1024);
      int g = 0, i = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x, ++i) {
        const Item it = item_at(a, w, n_qt, u);
        const int n_kt = it.n_kt;
        {
          // This thread is ahead of the softmax warps, which would divide for a thousand
          // cycles between items. Its slot is free: the last QK of item i - 1 waited for scores of
          // item i - 3 or later to be read, so every warp is done with item i - 4, and the outputs
          // of item i - 5 are written.
          ItemTiles t;
          t.pos0 = it.pos0, t.n_a = it.n_a, t.n_kt = it.n_kt, t.h = it.h, t.q0 = it.q0;
          t.k0_b = (it.b_first - it.n_a) * kTile + w.lo;
          t.a_full = min(it.n_a, min(a.sinks, it.pos0 + 1) / kTile);
          t.b_lo = max(it.n_a, ((it.pos0 + kTile - 1 - a.window - t.k0_b) >> 7) + 1);
          t.b_hi = ((it.pos0 - (kTile - 1) - t.k0_b) >> 7) + 1;
          sm->items[i % kItemSlots] = t;
          mbar_arrive(smem_u32(&sm->item_full[i % kItemSlots]));
        }
        ok = mbar_wait<2>(smem_u32(&sm->q_full), i & 1, abort_flag, a.dev_error);
        for (int j = 0; ok && j < n_kt; ++j, ++g) {
          const int s = g % kStagesK, sb = g & 1;
          ok = mbar_wait<2>(smem_u32(&sm->k_full[s]), (g / kStagesK) & 1, abort_flag, a.dev_error);
          if (ok && g >= 2) ok = mbar_wait<2>(smem_u32(&sm->s_free[sb]), ((g - 2) >> 1) & 1, abort_flag, a.dev_error);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + kTmS + static_cast<uint32_t>(sb) * 128u;
          const uint64_t dk = dK + static_cast<uint64_t>((s * 3 * kBox) >> 4);
#pragma unroll
          for (uint32_t kk = 0; kk < 12; ++kk) {
            const uint32_t off = ((kk >> 2) * kBox + (kk & 3u) * 32u) >> 4;
            mma_ss(d, dQ + off, dk + off, kIdQK, kk > 0 ? 1u : 0u);
          }
          mma_commit(smem_u32(&sm->s_full[sb]));
          mma_commit(smem_u32(&sm->k_empty[s]));
          if (j == n_kt - 1) mma_commit(smem_u32(&sm->q_empty));
        }
      }
      mma_commit(smem_u32(&sm->drain));
      pw_drain(smem_u32(&sm->drain), 0, a.dev_error);
    }
  } else if (warp == kPvWarp) {
    // ================= PV issue: O += P(g) V(g) once P(g) is complete
    if (lane == 0) {
      constexpr uint32_t kIdPV = idesc_bf16_f32(128, 128, false, true);
      const uint64_t dV = sdesc_sw128(smem_u32(sm->v[0][0]), kBox, 1024);  // MN-major: boxes of 64 d apart
      int g = 0, i = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < units; u += gridDim.x, ++i) {
        const int n_kt = item_at(a, w, n_qt, u).n_kt;
        for (int j = 0; ok && j < n_kt; ++j, ++g) {
          const int s = g % kStagesV, pb = g & 1;
          ok = mbar_wait<2>(smem_u32(&sm->v_full[s]), (g / kStagesV) & 1, abort_flag, a.dev_error);
          // O of the last item has been read
          if (ok && j == 0 && i > 0) ok = mbar_wait<2>(smem_u32(&sm->o_free), (i - 1) & 1, abort_flag, a.dev_error);
          if (ok) ok = mbar_wait<2>(smem_u32(&sm->p_full[pb]), (g >> 1) & 1, abort_flag, a.dev_error);
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv = dV + static_cast<uint64_t>((s * 2 * kBox) >> 4);
#pragma unroll
          for (uint32_t kk = 0; kk < 8; ++kk)
            mma_ts<kIdPV>(tmem + kTmO, tmem + kTmP + static_cast<uint32_t>(pb) * 64u + kk * 8u,
                          dv + ((kk * 16u * 128u) >> 4), (j > 0 || kk > 0) ? 1u : 0u);
          mma_commit(smem_u32(&sm->p_free[pb]));
          if (j == n_kt - 1) mma_commit(smem_u32(&sm->o_done));
          mma_commit(smem_u32(&sm->v_empty[s]));
        }
      }
      mma_commit(smem_u32(&sm->drain_pv));
      pw_drain(smem_u32(&sm->drain_pv), 0, a.dev_error);
    }
  } else {
    // ================= softmax and epilogue. Warp `part` of a lane quarter takes the key
    // columns [32 part, +32) of every tile, thread = query row. The four warps of a quarter
    // meet once per tile, to combine their row maxima (each then derives the same running
    // max); a failed wait is carried to the next meeting, so they fail together. An item's
    // outputs are written behind the next item's first tile: O is complete by then, and
    // the next item's PV has the time of a tile to wait for it.
    const int q4 = warp & 3, part = warp >> 2;
    const int row = q4 * 32 + lane;
    const uint32_t base = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
    const float c2 = a.softmax_scale * kLog2e;  // > 0
    // Item n's o = O / l (bf16) and lse; NaN after a failure. (The warps of a quarter hold
    // the same running max, so the row sum is the sum of theirs.)
    auto write_outputs = [&](int n, bool ok) -> bool {
      const int x = n & 1;
      ok = ok && warp_wait(&sm->o_done, x, sm, a.dev_error);
      tc_fence_after();
      float l_row = sm->lsum[x][0][row];
#pragma unroll
      for (int k = 1; k < kParts; ++k) l_row += sm->lsum[x][k][row];
      const float scale = ok ? 1.0f / l_row : CUDART_NAN_F;
      uint32_t w16[16];
      {
        float o[32];
        tmem_ld32_sync(base + kTmO + static_cast<uint32_t>(kKeys * part), o);
#pragma unroll
        for (int k = 0; k < 16; ++k) w16[k] = pack_bf16x2(o[2 * k] * scale, o[2 * k + 1] * scale);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm->o_free));
      transpose4(w16, lane);
      const int h = sm->items[n % kItemSlots].h, q0 = sm->items[n % kItemSlots].q0;
      const int q = q0 + q4 * 32 + (lane & ~3);
      uint8_t* out = static_cast<uint8_t*>(a.o) + (static_cast<int64_t>(q) * a.heads + h) * 256 + part * kKeys * 2 +
                     (lane & 3) * 16;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (q + k < a.n_queries)
          *reinterpret_cast<uint4*>(out + static_cast<int64_t>(k) * a.heads * 256) =
              make_uint4(w16[4 * k], w16[4 * k + 1], w16[4 * k + 2], w16[4 * k + 3]);
      if (part == 0 && a.lse != nullptr && q0 + row < a.n_queries)
        a.lse[static_cast<int64_t>(q0 + row) * a.heads + h] =
            ok ? (sm->mlast[x][row] + log2f(l_row)) * kLn2 : CUDART_NAN_F;
      return ok;
    };
    const int n_items = (units - 1 - static_cast<int>(blockIdx.x)) / static_cast<int>(gridDim.x) + 1;
    int g = 0, i = 0;
    bool ok = true, well = true, behind = false;  // behind: stopped with two items' outputs to write
    for (; i < n_items; ++i) {
      ok = ok && warp_wait(&sm->item_full[i % kItemSlots], (i / kItemSlots) & 1, sm, a.dev_error);
      // (read where it is used: the registers are all taken)
      const volatile ItemTiles* t = &sm->items[i % kItemSlots];
      float m = -CUDART_INF_F, l = 0.0f;
      for (int j = 0;; ++j, ++g) {
        const int sb = g & 1;
        int n_kt, a_full, b_lo, b_hi;
        asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(n_kt), "=r"(a_full), "=r"(b_lo), "=r"(b_hi)
                     : "r"(smem_u32(&sm->items[i % kItemSlots])));
        const bool edge = (j >= a_full) & ((j < b_lo) | (j >= b_hi)), end = j + 1 >= n_kt;
        const bool good = ok && warp_wait(&sm->s_full[sb], (g >> 1) & 1, sm, a.dev_error);
        float s[kKeys];
        if (good) {
          tc_fence_after();
          // raw scores; the scale into log2 units is folded into each exponent's FMA below
          tmem_ld32_sync(base + kTmS + static_cast<uint32_t>(sb * kTile + kKeys * part), s);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm->s_free[sb]));
          if (edge) {
            // An edge of the mask crosses the tile: of its keys [0, 128), those in [sk, lo) and
            // those past hi are hidden from this row. (Region A apart from B holds the sinks
            // alone: its rows past them are not loaded.)
            const bool in_a = j < t->n_a;
            const int k0 = j * kTile + (in_a ? 0 : t->k0_b);
            const int hi = t->pos0 + row - k0, lo = w.split && in_a ? kTile : hi - a.window + 1, sk = a.sinks - k0;
            const int c = kKeys * part;
            const uint32_t vis = below(hi + 1 - c) & ~(below(lo - c) & ~below(sk - c));
            if (__any_sync(0xffffffffu, vis != 0xffffffffu)) {
#pragma unroll
              for (int x = 0; x < kKeys; ++x)
                if ((vis & (1u << x)) == 0u) s[x] = -CUDART_INF_F;
            }
          }
          float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int x = 4; x + 4 < kKeys; x += 8)
#pragma unroll
            for (int y = 0; y < 4; ++y) mx4[y] = max3(mx4[y], s[x + y], s[x + 4 + y]);
          sm->mx_part[sb][part][row] =
              max3(max3(mx4[0], mx4[1], s[28]), max3(mx4[2], mx4[3], s[29]), fmaxf(s[30], s[31])) * c2;
        }
        well = meet(q4, good);
        if (!well) {
          behind = j == 0 && i > 0;
          break;
        }
        float mx = sm->mx_part[sb][0][row];
#pragma unroll
        for (int x = 1; x < kParts; ++x) mx = fmaxf(mx, sm->mx_part[sb][x][row]);
        const bool first = (j == 0);
        const float m_prev = m;
        const float m_new = fmaxf(m_prev, mx);
        const bool resc = !first && (m_new > m_prev + kRescaleLog2);
        const float m_use = (first || resc) ? m_new : m_prev;
        const float ref = m_use == -CUDART_INF_F ? 0.0f : m_use;  // a row that has seen nothing yet
        uint32_t pw[kKeys / 2];
        uint64_t rsum[2] = {0, 0};  // (two pairs of zeros)
        const uint64_t c2_2 = pair(c2, c2), ref_2 = pair(-ref, -ref);
#pragma unroll
        for (int x = 0; x < kKeys / 2; ++x) {
          const float2 e = unpair(fma2(pair(s[2 * x], s[2 * x + 1]), c2_2, ref_2));
          const float p0 = fast_exp2(e.x), p1 = fast_exp2(e.y);
          pw[x] = pack_bf16x2(p0, p1);
          // (before the rounding for PV: the two differ by at most one rounding)
          rsum[x & 1] = add2(rsum[x & 1], pair(p0, p1));
        }
        const float2 rs = unpair(add2(rsum[0], rsum[1]));
        const bool resc_any = __any_sync(0xffffffffu, resc);
        const float alpha = resc ? fast_exp2(m_prev - ref) : 1.0f;
        l = (first ? 0.0f : l * alpha) + (rs.x + rs.y);
        m = m_use;
        // P of this tile: the buffer was last read by PV(g - 2)
        if (g >= 2) ok = warp_wait(&sm->p_free[sb], ((g - 2) >> 1) & 1, sm, a.dev_error);
        tc_fence_after();
        if (ok) tmem_st16(base + kTmP + static_cast<uint32_t>(sb * (kTile / 2) + kKeys / 2 * part), pw);
        // O rows (this warp's 32 of the 128 columns) rescale only after PV(g - 1) (phase
        // (g - 1) >> 1 of p_free[(g - 1) & 1])
        if (resc_any) {
          ok = ok && warp_wait(&sm->p_free[(g - 1) & 1], ((g - 1) >> 1) & 1, sm, a.dev_error);
          if (ok) {
            tc_fence_after();
            const uint32_t at_o = base + kTmO + static_cast<uint32_t>(kKeys * part);
            float o[32];
            tmem_ld32_sync(at_o, o);
            uint32_t w32[32];
#pragma unroll
            for (int k = 0; k < 32; ++k) w32[k] = __float_as_uint(o[k] * alpha);
            tmem_st32(at_o, w32);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(smem_u32(&sm->p_full[sb]));
        if (j == 0 && i > 0) {
          ok = write_outputs(i - 1, ok);
        }
        if (end) break;
      }
      if (!well) break;
      ++g;
      sm->lsum[i & 1][part][row] = l;
      if (part == 0) sm->mlast[i & 1][row] = m;
    }
    if (meet(q4, ok && well)) {
      write_outputs(n_items - 1, true);
    } else {
      // the four warps fail together, at the same item
      const uint32_t nan2 = pack_bf16x2(CUDART_NAN_F, CUDART_NAN_F);
      for (int n = behind || i == n_items ? i - 1 : i; n < n_items; ++n) {
        const Item it = item_at(a, w, n_qt, static_cast<int>(blockIdx.x) + n * static_cast<int>(gridDim.x));
        const int q = it.q0 + row;
        if (q >= a.n_queries) continue;
        uint4* out = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.o) +
                                              (static_cast<int64_t>(q) * a.heads + it.h) * 256 + part * kKeys * 2);
        for (int k = 0; k < 4; ++k) out[k] = make_uint4(nan2, nan2, nan2, nan2);
        if (part == 0 && a.lse != nullptr) a.lse[static_cast<int64_t>(q) * a.heads + it.h] = CUDART_NAN_F;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kQkWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// [rows][cols] bf16 with row stride `stride` elements, 64 x 128 boxes, 128-byte swizzle
bool pw_map(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint64_t stride) {
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {stride * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(kTile)};
  const cuuint32_t estr[2] = {1, 1};
  return tensor_map_encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

PrefillWindow prefill_window_regions(int32_t n_tokens, int32_t n_queries, int32_t window, int32_t sinks) {
  PrefillWindow w;
  const int64_t first = static_cast<int64_t>(n_tokens) - n_queries;  // position of the first query
  const int64_t lo = first - window + 1 > 0 ? first - window + 1 : 0;
  w.split = lo > sinks;
  w.lo = w.split ? static_cast<int32_t>(lo) : 0;
  w.rows_a = w.split ? sinks : 0;
  w.rows_b = n_tokens - w.lo;
  return w;
}

cudaError_t launch_prefill_window(const PrefillArgs& a, cudaStream_t s) {
  if (tensor_map_encoder() == nullptr) return cudaErrorNotSupported;
  const PrefillWindow w = prefill_window_regions(a.n_tokens, a.n_queries, a.window, a.sinks);
  cudaError_t e = launch_expand(
      ExpandArgs{a.rows, a.w_uk, a.w_uv, a.k_nope, a.v, w.lo, w.rows_a, w.rows_b, a.heads, a.dev_error}, s);
  if (e != cudaSuccess) return e;
  const int64_t H = a.heads;
  const uint64_t hd = static_cast<uint64_t>(H * 128);
  PwMaps maps;
  const auto at = [](const void* base, int64_t row, int64_t stride) {
    return static_cast<const char*>(base) + row * stride * 2;
  };
  const auto region = [&](int r, int64_t from, int32_t n, int64_t to) {
    return pw_map(&maps.k[r], at(a.k_nope, to, H * 128), static_cast<uint64_t>(n), hd, hd) &&
           pw_map(&maps.kr[r], at(a.rows, from, kRow), static_cast<uint64_t>(n), kRow, kRow) &&
           pw_map(&maps.v[r], at(a.v, to, H * 128), static_cast<uint64_t>(n), hd, hd);
  };
  if (!pw_map(&maps.q, a.q_nope, static_cast<uint64_t>(a.n_queries), hd, hd) ||
      !pw_map(&maps.qr, a.q_rope, static_cast<uint64_t>(a.n_queries), hd / 2, hd / 2) ||
      !region(1, w.lo, w.rows_b, w.rows_a) || (w.rows_a > 0 && !region(0, 0, w.rows_a, 0)))
    return cudaErrorInvalidValue;
  if (w.rows_a == 0) maps.k[0] = maps.k[1], maps.kr[0] = maps.kr[1], maps.v[0] = maps.v[1];
  static SmemOptIn opt_in;
  e = opt_in(kPwSmemBytes, prefill_window_kernel);
  if (e != cudaSuccess) return e;
  const int32_t n_qt = (a.n_queries + kTile - 1) / kTile;
  const int32_t units = n_qt * a.heads;  // at most 2^13 x 128
  const int32_t sms = device_sm_count();
  return launch_pdl(prefill_window_kernel, dim3(static_cast<unsigned>(units < sms ? units : sms)), dim3(kPwThreads),
                    kPwSmemBytes, s, maps, a, w, n_qt, units);
}

}  // namespace mla
