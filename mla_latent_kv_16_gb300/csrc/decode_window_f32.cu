// mla_decode_window in fp32 (fp32 activations and cache) on CUDA cores.
//
//   s[h][t] = (q_lat[h] . c_KV[t] + q_rope[h] . k_R[t]) * scale,  u[h] = sum_t softmax(s)_t c_KV[t]
// over the visible tokens of one query: the first `sinks` and the last `window`.
//
// Per cached token and head 1,088 FMAs against 2,304 bytes per token: with 16 heads
// 7.6 FMA per byte, so the 128 FMA lanes of an SM (78 TFLOP/s over the chip) and HBM
// take about the same time, and shared memory must not cost more than either. A
// CTA of 16 warps (one per SM) takes one query, 16 heads and a share of its list of
// visible tokens, in tiles of 32 tokens that arrive by cp.async in one of two
// buffers while the other is computed on:
//   QK: warp w takes columns [36 w, +36) of all 16 x 32 scores; a thread 4 heads x 4
//       tokens, so eight 16-byte loads feed 64 FMAs. Rows are 580 floats apart: eight
//       rows at one column fall into different banks. The 16 partial sums are added
//       in warp order.
//   softmax: warp w is head w, lane = token: running maximum and sum, P and the
//       rescale factor to shared memory.
//   PV: a thread has 8 heads x 8 latent columns of u in registers, for every fourth
//       token; per token four 16-byte loads, two of P (broadcast) and two of the row,
//       feed 64 FMAs. The four token groups' sums are added at the end, in order.
// The list of visible tokens has no hidden token in it, so there is no mask; entries
// past its end are zero rows with weight 0.
//
// Measured: 32 sequences, 16 heads, 4096 + 64 visible tokens: 188 us (303 MB, 4.6 GFLOP: the
// FMA lanes and HBM would take 60 and 45 us). On a busy SM the FMA pipe is 48 % busy, the
// shared-memory port 57 % and the issue slots 64 %: the three phases of a tile are short
// against the barriers between them, and there is no room for a second CTA beside 148 KB
// of tiles. (8 heads x 2 columns in PV, twice its port cycles: 205 us; the partial sums
// 32 floats apart, four-way conflicts: 199 us.)
#include <math_constants.h>

#include "common.cuh"
#include "host.h"
#include "launchers.h"

namespace mla {
namespace {

constexpr int kThreads = 512, kWarps = 16;
constexpr int kHeads = 16;   // heads of a CTA
constexpr int kTok = 32;     // tokens of a tile
constexpr int kPad = 580;    // floats between rows in shared memory
constexpr int kSlice = kRow / kWarps;  // QK columns of a warp: 36
constexpr int kChunks = kRow / 4;      // 16-byte chunks of a row

struct __align__(16) F32Smem {
  float rows[2][kTok][kPad];
  float q[kHeads][kPad];
  float part[kWarps][kHeads][kTok + 8];  // (+ 8: four heads' rows fall into different banks)
  float p[kTok][kHeads];
  float alpha[kHeads];
};
static_assert(sizeof(F32Smem) <= 232448, "shared memory budget of one CTA");
static_assert(sizeof(F32Smem::rows) >= 4 * kHeads * kDC * sizeof(float), "the sums of four token groups");

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}

__global__ void __launch_bounds__(kThreads, 1) decode_window_f32_kernel(const DecodeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  F32Smem& sm = *reinterpret_cast<F32Smem*>(smem_raw);
  const int split = blockIdx.x, h0 = blockIdx.y * kHeads, bj = blockIdx.z;
  const int b = bj / a.q_len, j = bj % a.q_len;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const int heads = min(kHeads, a.heads - h0);
  const int L = a.seq_lens[b], P = a.page_size;
  int n_vis = L - a.q_len + j + 1;
  if (L < a.q_len || static_cast<int64_t>(L) > static_cast<int64_t>(a.max_pages) * P) {
    if (threadIdx.x == 0) flag_error(a.dev_error, MLA_DEVERR_BAD_SEQLEN);
    n_vis = 0;
  }
  // the visible tokens as a list: [0, gap_at) and [gap_at + gap, n_vis)
  const int win_lo = max(0, n_vis - a.window);
  const int gap_at = min(a.sinks, win_lo), gap = win_lo - gap_at;
  const int share = (n_vis - gap + a.num_splits - 1) / a.num_splits;
  const int begin = split * share;
  int end = min(n_vis - gap, begin + share);
  const int32_t* bt = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  auto token = [&](int v) { return v + (v >= gap_at ? gap : 0); };
  {
    int bad = 0;
    for (int v = begin + static_cast<int>(threadIdx.x); v < end; v += kThreads) {
      const int32_t page = bt[token(v) / P];
      bad |= page < 0 || page >= a.num_pages;
    }
    if (__syncthreads_or(bad)) {
      if (threadIdx.x == 0) flag_error(a.dev_error, MLA_DEVERR_BAD_PAGE);
      end = begin;
    }
  }
  // rows [v0, v0 + 32) of the list into a buffer: warp w copies rows 2 w and 2 w + 1
  auto load = [&](int v0, int buf) {
#pragma unroll
    for (int r = 0; r < kTok / kWarps; ++r) {
      const int row = warp * (kTok / kWarps) + r, v = v0 + row;
      const bool valid = v < end;
      const int tok = valid ? token(v) : 0;
      const int64_t slot = valid ? static_cast<int64_t>(bt[tok / P]) * P + tok % P : 0;
      const float* src = static_cast<const float*>(a.cache) + slot * kRow;
#pragma unroll
      for (int k = 0; k < (kChunks + 31) / 32; ++k) {
        const int c = lane + 32 * k;
        if (c < kChunks) cp_async16(&sm.rows[buf][row][4 * c], src + 4 * c, valid);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (begin < end) load(begin, 0);

  // the queries, scaled into log2 units; heads past the last are zero
  const float qscale = a.softmax_scale * kLog2e;
  for (int e = threadIdx.x; e < kHeads * kRow; e += kThreads) {
    const int h = e / kRow, k = e % kRow;
    const int64_t qi = static_cast<int64_t>(bj) * a.heads + h0 + h;
    float v = 0.0f;
    if (h < heads)
      v = k < kDC ? static_cast<const float*>(a.q_lat)[qi * kDC + k]
                  : static_cast<const float*>(a.q_rope)[qi * kDRope + (k - kDC)];
    sm.q[h][k] = v * qscale;
  }

  // QK: 4 heads hg + 4 i, 4 tokens tg + 8 i
  const int hg = lane >> 3, tg = lane & 7;
  // PV: the tokens pt + 4 i, 8 heads from 8 ph, the columns from 4 pc and from 256 + 4 pc
  const int pt = warp >> 2, ph = (warp >> 1) & 1, pc = (warp & 1) * 32 + lane;
  float acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[i][x] = 0.0f;
  float m = -CUDART_INF_F, l = 0.0f;  // of head `warp`

  int buf = 0;
  for (int v0 = begin; v0 < end; v0 += kTok, buf ^= 1) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the tile has landed for all, and the other buffer is no longer read
    if (v0 + kTok < end) load(v0 + kTok, buf ^ 1);
    {
      float s[4][4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) s[x][y] = 0.0f;
      const int k0 = warp * kSlice;
#pragma unroll
      for (int k = k0; k < k0 + kSlice; k += 4) {
        float4 q4[4], c4[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) q4[x] = *reinterpret_cast<const float4*>(&sm.q[hg + 4 * x][k]);
#pragma unroll
        for (int y = 0; y < 4; ++y) c4[y] = *reinterpret_cast<const float4*>(&sm.rows[buf][tg + 8 * y][k]);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            s[x][y] = fmaf(q4[x].x, c4[y].x, s[x][y]);
            s[x][y] = fmaf(q4[x].y, c4[y].y, s[x][y]);
            s[x][y] = fmaf(q4[x].z, c4[y].z, s[x][y]);
            s[x][y] = fmaf(q4[x].w, c4[y].w, s[x][y]);
          }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) sm.part[warp][hg + 4 * x][tg + 8 * y] = s[x][y];
    }
    __syncthreads();
    {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sm.part[w][warp][lane];
      if (v0 + lane >= end) s = -CUDART_INF_F;
      const float m_new = fmaxf(m, warp_max(s));
      const float alpha = fast_exp2(m - m_new);  // (0 on the first tile)
      const float p = fast_exp2(s - m_new);
      l = l * alpha + warp_sum(p);
      m = m_new;
      sm.p[lane][warp] = p;
      if (lane == 0) sm.alpha[warp] = alpha;
    }
    __syncthreads();
    bool moved = false;  // (the same for all threads of a warp)
    float al[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      al[i] = sm.alpha[8 * ph + i];
      moved |= al[i] != 1.0f;
    }
    if (moved) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[i][x] *= al[i];
    }
#pragma unroll 4
    for (int t = pt; t < kTok; t += 4) {
      const float4 pa = *reinterpret_cast<const float4*>(&sm.p[t][8 * ph]);
      const float4 pb = *reinterpret_cast<const float4*>(&sm.p[t][8 * ph + 4]);
      const float4 ca = *reinterpret_cast<const float4*>(&sm.rows[buf][t][4 * pc]);
      const float4 cb = *reinterpret_cast<const float4*>(&sm.rows[buf][t][256 + 4 * pc]);
      const float pv[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
      const float cv[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[i][x] = fmaf(pv[i], cv[x], acc[i][x]);
    }
  }
  __syncthreads();  // (no tile is read any more)
  // the four token groups' sums, added in order; a warp takes a head
  float(*red)[kHeads][kDC] = reinterpret_cast<float(*)[kHeads][kDC]>(&sm.rows[0][0][0]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float* d = red[pt][8 * ph + i];
    *reinterpret_cast<float4*>(d + 4 * pc) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    *reinterpret_cast<float4*>(d + 256 + 4 * pc) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
  }
  __syncthreads();
  if (warp >= heads) return;
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  const int64_t row = static_cast<int64_t>(bj) * a.heads + h0 + warp;
  const int64_t prow = (static_cast<int64_t>(bj) * a.num_splits + split) * a.heads + h0 + warp;
  float* u = a.num_splits == 1 ? static_cast<float*>(a.u_out) + row * kDC : a.part_u + prow * kDC;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = 4 * (lane + 32 * k);
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float4 x = *reinterpret_cast<const float4*>(red[g][warp] + c);
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    *reinterpret_cast<float4*>(u + c) = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
  }
  if (lane == 0) {
    const float lse = l > 0.0f ? (m + log2f(l)) * kLn2 : -CUDART_INF_F;
    if (a.num_splits > 1)
      a.part_lse[prow] = lse;
    else if (a.lse_out != nullptr)
      a.lse_out[row] = lse;
  }
}

}  // namespace

cudaError_t launch_decode_window_f32(const DecodeArgs& a, cudaStream_t s) {
  static SmemOptIn opt_in;
  const cudaError_t e = opt_in(sizeof(F32Smem), decode_window_f32_kernel);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.num_splits, (a.heads + kHeads - 1) / kHeads, a.batch * a.q_len);
  return launch_pdl(decode_window_f32_kernel, grid, dim3(kThreads), sizeof(F32Smem), s, a);
}

}  // namespace mla
