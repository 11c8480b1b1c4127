// The page bookkeeping of the latent cache on the device: mla_cache_extend (fork
// and grow), mla_cache_free, mla_cache_compact.
//
// State: block_table [num_seqs][max_pages] (physical page of each logical page,
// -1 for none), seq_lens [num_seqs], ref_counts [num_pages] (holders of each
// page; 0 = free). There is no free list: the counts alone say what is free, so
// giving pages back is a decrement and its order cannot matter, and pages are
// handed out lowest number first, so every result is a function of the state.
//
// These calls move a few hundred kilobytes at most; what they cost is launches
// and round trips. extend and compact are a plan by one cluster of eight CTAs,
// which counts the pool's free (or live) pages in warp-wide segments, joins the
// counts once over distributed shared memory and ranks the pages in a second pass
// over the segments, and an apply, which writes the table. extend's first CTA
// checks the requests while the others count. Up to kFusedWork table entries the
// same cluster applies its plan after a cluster barrier (one launch); beyond, a
// second kernel does with as many CTAs as there is table.
//
// Measured (device, with the 1 to 2 us copy that restores the state before each
// call): 64 sequences grown 7.3 us, 192 forked 9.7, pages of 64 windows given back
// 4.4, a pool of 2,048 pages compacted 6.5, one of 65,536 10.6. The forks and the
// large compaction took 18.5 and 15 with three launches, 11.3 and 11.5 with the
// requests checked before the count and every load awaited by itself.
#include "common.cuh"
#include "host.h"
#include "launchers.h"
#include "tc_ptx.cuh"

namespace mla {
namespace {

constexpr int kPlanCtas = 8;  // one cluster
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kApplyThreads = 256;
constexpr int kBatch = 4;          // table entries a thread requests at once
constexpr int64_t kFusedWork = 1 << 15;

// Pages per warp of the plan's CTAs from kFirst on: a multiple of 128 (32 lanes x 4 pages).
template <int kFirst>
__device__ __forceinline__ int64_t segment_pages(int32_t num_pages) {
  const int64_t warps = (kPlanCtas - kFirst) * kPlanWarps;
  return ((num_pages + warps * 128 - 1) / (warps * 128)) * 128;
}

// Bit k of the result: ref_counts[p + k] is zero (kFree) or positive (!kFree); p + k < num_pages.
template <bool kFree>
__device__ __forceinline__ uint32_t page_bits(const int32_t* refs, int64_t p, int32_t num_pages) {
  int32_t v[4];
  if (p + 3 < num_pages) {
    const int4 x = *reinterpret_cast<const int4*>(refs + p);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = p + k < num_pages ? refs[p + k] : (kFree ? 1 : 0);
  }
  uint32_t b = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) b |= (kFree ? v[k] == 0 : v[k] > 0) ? 1u << k : 0u;
  return b;
}

struct PlanShared {
  int32_t warp_count[kPlanWarps];
  int32_t cta_count[kPlanCtas];  // every CTA's total, written by the CTAs themselves
  int32_t need;                  // extend: pages that the requests ask for (from CTA 0)
  int32_t scan[kPlanWarps];
};

// Counts this warp's pages (the CTAs from kFirst on have some), joins the counts over the cluster (one cluster
// barrier) and returns how many of the counted pages precede the warp's segment;
// *total gets the pool's. `need` of CTA 0's PlanShared is broadcast on the way.
template <bool kFree, int kFirst>
__device__ int32_t count_pages(const int32_t* refs, int32_t num_pages, PlanShared* sm, uint32_t rank, int32_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t seg = segment_pages<kFirst>(num_pages);
  const int64_t p0 = (static_cast<int64_t>(rank) - kFirst) * kPlanWarps * seg + warp * seg;
  int32_t n = 0;
  for (int64_t p = p0; static_cast<int>(rank) >= kFirst && p < p0 + seg && p < num_pages; p += 128)
    n += p + 4 * lane < num_pages ? __popc(page_bits<kFree>(refs, p + 4 * lane, num_pages)) : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if (lane == 0) sm->warp_count[warp] = n;
  __syncthreads();
  if (warp == 0) {
    int32_t t = sm->warp_count[lane];
    int32_t incl = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    sm->warp_count[lane] = incl - t;  // counted pages of the CTA's earlier warps
    const int32_t mine = __shfl_sync(0xffffffffu, incl, 31);
    if (lane < kPlanCtas)
      tc::st_cluster_u32(tc::map_to_rank(tc::smem_u32(&sm->cta_count[rank]), static_cast<uint32_t>(lane)),
                         static_cast<uint32_t>(mine));
    if (rank == 0 && lane > 0 && lane < kPlanCtas)
      tc::st_cluster_u32(tc::map_to_rank(tc::smem_u32(&sm->need), static_cast<uint32_t>(lane)),
                         static_cast<uint32_t>(sm->need));
  }
  __syncwarp();
  tc::cluster_sync();
  int32_t before = sm->warp_count[warp], all = 0;
#pragma unroll
  for (int r = 0; r < kPlanCtas; ++r) {
    const int32_t t = sm->cta_count[r];
    if (r < static_cast<int>(rank)) before += t;
    all += t;
  }
  *total = all;
  return before;
}

// Calls f(page, rank) for each counted page of this warp's segment, rank = the
// counted pages before it. All lanes stay together; f runs per lane.
template <bool kFree, int kFirst, typename F>
__device__ void rank_pages(const int32_t* refs, int32_t num_pages, uint32_t cta, int32_t before, int32_t stop, F f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t seg = segment_pages<kFirst>(num_pages);
  const int64_t p0 = (static_cast<int64_t>(cta) - kFirst) * kPlanWarps * seg + warp * seg;
  for (int64_t p = p0; static_cast<int>(cta) >= kFirst && p < p0 + seg && p < num_pages && before < stop; p += 128) {
    const int64_t mine = p + 4 * lane;
    const uint32_t bits = mine < num_pages ? page_bits<kFree>(refs, mine, num_pages) : 0u;
    const int32_t c = __popc(bits);
    int32_t incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    int32_t r = before + incl - c;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool is = (bits >> k) & 1u;
      f(mine + k, is, r);
      r += is ? 1 : 0;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
}

// Inclusive sum over the CTA's 1024 threads of a 64-bit value; *all gets the sum
// of all. Every warp adds up the warps' sums itself: one barrier less.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* buf, int64_t* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  if (lane == 31) buf[warp] = v;
  __syncthreads();
  int64_t t = buf[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += up;
  }
  const int64_t before = __shfl_sync(0xffffffffu, t, warp > 0 ? warp - 1 : 0);
  *all = __shfl_sync(0xffffffffu, t, 31);
  return warp > 0 ? v + before : v;
}

// ------------------------------------------------------------------ extend

// One request as the plan leaves it for the apply kernel.
struct __align__(16) ExtendItem {
  int32_t len;        // tokens of the source before the call; -1: refused
  int32_t n_new;      // tokens whose outputs the request owns (refused ones too)
  int32_t page_at;    // index of its first page in the list of free pages
  int32_t token_at;   // index of its first new token
};

// Writes request i's part of the state: this thread takes the entries at, at + step, ...
// (its first ones are loaded together: what follows is a chain of round trips to L2)
__device__ void extend_apply(const ExtendArgs& a, int i, int at, int step, int32_t free_total) {
  const ExtendItem it = static_cast<const ExtendItem*>(a.items)[i];
  const int32_t s = a.src[i], d = a.dst[i];
  const int32_t P = a.page_size;
  const int64_t width = a.max_pages;
  const int32_t* from = a.block_table + s * width;
  int32_t* to = a.block_table + d * width;
  const int32_t* fresh = a.free_list + it.page_at;  // [need - keep]
  bool ok = it.len >= 0;
  const bool fork = ok && s != d;
  int32_t full = 0, keep = 0, need = 0, bad = 0;
  bool cut = false;  // the source's last page is partly filled: its rows are copied, or new ones follow them
  if (ok) {
    full = it.len / P;
    keep = fork ? full : (it.len + P - 1) / P;  // the first page that is newly allocated
    need = static_cast<int32_t>((static_cast<int64_t>(it.len) + it.n_new + P - 1) / P);
    cut = it.len % P != 0 && (fork || it.n_new > 0);
    if (need > keep && static_cast<int64_t>(it.page_at) + (need - keep) > free_total) bad = MLA_DEVERR_NO_PAGE;
  }
  int32_t last = -1, tail_to = -1, e_fresh = -1, e_slot = -1;
  int32_t shared[kBatch];  // entries at, at + step, ... of the pages that a fork shares (a given-back page stays none)
  auto load_shared = [&](int p0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) shared[k] = p0 + k * step < keep ? from[p0 + k * step] : -1;
  };
  // (no request of the call writes `last`: growths write the pages past it, forks the rows of empty sequences)
  if (cut) last = from[full];
  if (bad == 0) {
    if (fork && cut && at == 0) tail_to = fresh[0];
    if (keep + at < need) e_fresh = fresh[at];
    const int32_t page = (it.len + at) / P;
    if (ok && at < it.n_new && page >= keep) e_slot = fresh[page - keep];
  }
  if (fork) load_shared(at);
  if (cut && (last < 0 || last >= a.num_pages)) bad |= MLA_DEVERR_BAD_PAGE;
  if (bad != 0) {
    ok = false;
    if (at == 0) flag_error(a.dev_error, bad);
  }
  // page of new token k: a growth's first tokens go to the last page, the others to new ones
  auto page_of = [&](int k) -> int32_t {
    const int32_t page = (it.len + k) / P;
    return page < keep ? last : (k == at ? e_slot : fresh[page - keep]);
  };
  if (ok && fork)
    for (int p0 = at; p0 < keep; p0 += kBatch * step) {
      if (p0 > at) load_shared(p0);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (p0 + k * step >= keep) break;
        if (shared[k] >= a.num_pages) flag_error(a.dev_error, MLA_DEVERR_BAD_PAGE);
        const bool valid = shared[k] >= 0 && shared[k] < a.num_pages;
        to[p0 + k * step] = valid ? shared[k] : -1;
        if (valid) atomicAdd(&a.ref_counts[shared[k]], 1);
      }
    }
  if (at == 0) {
    const bool tail = ok && fork && cut;
    a.copy_src[i] = tail ? last : -1;
    a.copy_dst[i] = tail ? tail_to : -1;
    a.copy_rows[i] = tail ? it.len % P : 0;
    if (ok) a.seq_lens[d] = it.len + it.n_new;
  }
  if (ok)
    for (int p = keep + at; p < need; p += step) {
      const int32_t e = p == keep + at ? e_fresh : fresh[p - keep];
      to[p] = e;
      a.ref_counts[e] = 1;
    }
  // (n_new may come within a step of 2^31: the counter is unsigned)
  for (uint32_t t = at; t < static_cast<uint32_t>(it.n_new); t += step) {
    const int32_t k = static_cast<int32_t>(t), pos = it.len + k;
    a.positions[it.token_at + k] = ok ? pos : 0;
    a.slots[it.token_at + k] = ok ? static_cast<int64_t>(page_of(k)) * P + pos % P : -1;
  }
}

template <bool kFused>
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    extend_plan_kernel(ExtendArgs a) {
  extern __shared__ int32_t first[];  // [num_seqs]: the first request that names the sequence as its destination
  __shared__ PlanShared sm;
  __shared__ int64_t scan_buf[2][kPlanWarps];  // tokens, pages
  const uint32_t rank = tc::cluster_ctarank();
  pdl_trigger();
  tc::cluster_sync();  // every CTA of the cluster has started: its shared memory may be written
  pdl_wait();
  ExtendItem* items = static_cast<ExtendItem*>(a.items);
  if (rank == 0) {
    // ---- the requests: checks, pages and tokens of each, and their running sums
    // (the first kPlanThreads requests are loaded ahead of the barriers)
    struct Request {
      int32_t s, d, g;
      int32_t len_s, len_d;  // of sequences in the table
    };
    auto in_table = [&](int32_t q) -> bool { return q >= 0 && q < a.num_seqs; };
    auto load = [&](int i) -> Request {
      Request q{-1, -1, 0, 0, 0};
      if (i < a.n) {
        q.s = a.src[i], q.d = a.dst[i], q.g = a.n_new[i];
        if (in_table(q.s)) q.len_s = a.seq_lens[q.s];
        if (in_table(q.d)) q.len_d = a.seq_lens[q.d];
      }
      return q;
    };
    Request q = load(threadIdx.x);
    for (int i = threadIdx.x; i < a.num_seqs; i += kPlanThreads) first[i] = 0x7fffffff;
    __syncthreads();
    if (in_table(q.d)) atomicMin(&first[q.d], static_cast<int32_t>(threadIdx.x));
    for (int i = kPlanThreads + static_cast<int>(threadIdx.x); i < a.n; i += kPlanThreads) {
      const int32_t d = a.dst[i];
      if (in_table(d)) atomicMin(&first[d], i);
    }
    __syncthreads();
    int64_t pages_before = 0, tokens_before = 0;
    const int64_t capacity = static_cast<int64_t>(a.max_pages) * a.page_size;
    for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
      const int i = i0 + static_cast<int>(threadIdx.x);
      ExtendItem it{-1, 0, 0, 0};
      int64_t pages = 0;
      int32_t bad = 0;
      if (i0 > 0) q = load(i);
      if (i < a.n) {
        const int32_t s = q.s, d = q.d, g = q.g;
        it.n_new = max(g, 0);
        if (!in_table(s) || !in_table(d) || first[d] != i) {
          bad = MLA_DEVERR_BAD_SEQ;
        } else {
          const int64_t len = q.len_s;
          if (s != d && q.len_d != 0) bad = MLA_DEVERR_BAD_SEQ;
          if (g < 0 || len < 0 || len + it.n_new > capacity) bad |= MLA_DEVERR_BAD_SEQLEN;
          if (bad == 0) {
            it.len = static_cast<int32_t>(len);
            const int64_t need = (len + g + a.page_size - 1) / a.page_size;
            pages = need - (s != d ? len / a.page_size : (len + a.page_size - 1) / a.page_size);
          }
        }
      }
      int64_t all_tokens = 0, all_pages = 0;
      const int64_t tokens_incl = block_scan(it.n_new, scan_buf[0], &all_tokens);
      const int64_t token_at = tokens_before + tokens_incl - it.n_new;
      if (i < a.n && token_at + it.n_new > a.max_new) {
        // no room for its outputs: refused, and it writes none
        bad |= MLA_DEVERR_BAD_SLOT;
        it.len = -1;
        it.n_new = token_at < a.max_new ? static_cast<int32_t>(a.max_new - token_at) : 0;
        pages = 0;
      }
      const int64_t pages_incl = block_scan(pages, scan_buf[1], &all_pages);
      if (i < a.n) {
        const int64_t page_at = pages_before + pages_incl - pages;
        // more pages than the pool has cannot be served: the apply kernel sees the sum
        it.page_at = page_at + pages > 0x7ffffffe ? 0x7ffffffe : static_cast<int32_t>(page_at);
        it.token_at = token_at < a.max_new ? static_cast<int32_t>(token_at) : a.max_new;
        items[i] = it;
        if (bad != 0) flag_error(a.dev_error, bad);
      }
      pages_before += all_pages;
      tokens_before += all_tokens;
      // scan_buf[0] of the next pass is written after every warp has passed the
      // barrier of this pass's second scan, i.e. has read scan_buf[0]; scan_buf[1]
      // after the barrier of the next pass's first scan
    }
    if (threadIdx.x == 0) sm.need = static_cast<int32_t>(min(pages_before, static_cast<int64_t>(a.num_pages)));
    __syncthreads();
  }
  // ---- the lowest free pages, as many as are asked for
  int32_t total = 0;
  const int32_t before = count_pages<true, 1>(a.ref_counts, a.num_pages, &sm, rank, &total);
  const int32_t need = sm.need;
  int32_t* free_list = a.free_list;
  rank_pages<true, 1>(a.ref_counts, a.num_pages, rank, before, need, [&](int64_t p, bool is, int32_t r) {
    if (is && r < need) free_list[r] = static_cast<int32_t>(p);
  });
  if constexpr (kFused) {
    __syncwarp();
    tc::cluster_sync();  // the plan and the list of free pages are written
    const int warps = kPlanCtas * kPlanWarps;
    // one warp per request, requests spread over the CTAs first
    for (int i = (threadIdx.x >> 5) * kPlanCtas + rank; i < a.n; i += warps)
      extend_apply(a, i, threadIdx.x & 31, 32, total);
  } else if (rank == 0 && threadIdx.x == 0) {
    *a.free_total = total;
  }
}

// grid (requests, parts of the row)
__global__ void __launch_bounds__(kApplyThreads) extend_apply_kernel(ExtendArgs a) {
  pdl_trigger();
  pdl_wait();
  extend_apply(a, blockIdx.x, blockIdx.y * kApplyThreads + threadIdx.x, gridDim.y * kApplyThreads, *a.free_total);
}

// ------------------------------------------------------------------ free

// grid (listed sequences, parts of the row). An entry is taken out of the table
// with an exchange, so a sequence that is listed twice gives each page back once.
__global__ void __launch_bounds__(kApplyThreads) free_kernel(FreeArgs a) {
  pdl_trigger();
  pdl_wait();
  const int32_t b = a.seqs[blockIdx.x];
  const int at = blockIdx.y * kApplyThreads + threadIdx.x, step = gridDim.y * kApplyThreads;
  if (b < 0 || b >= a.num_seqs) {
    if (at == 0) flag_error(a.dev_error, MLA_DEVERR_BAD_SEQ);
    return;
  }
  int32_t lo = 0, hi = a.max_pages;
  if (a.window > 0) {
    // tokens [sinks, dead) are behind every later query's window
    const int64_t dead = static_cast<int64_t>(a.seq_lens[b]) - a.window;
    lo = static_cast<int32_t>((static_cast<int64_t>(a.sinks) + a.page_size - 1) / a.page_size);
    hi = static_cast<int32_t>(min(static_cast<int64_t>(a.max_pages), dead > 0 ? dead / a.page_size : 0));
  } else if (at == 0) {
    a.seq_lens[b] = 0;  // (not read on this path)
  }
  int32_t* row = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  for (int64_t p = static_cast<int64_t>(lo) + at; p < hi; p += step) {
    if (row[p] < 0) continue;
    const int32_t e = atomicExch(&row[p], -1);
    if (e < 0) continue;
    if (e >= a.num_pages || atomicSub(&a.ref_counts[e], 1) <= 0) {
      if (e < a.num_pages) atomicAdd(&a.ref_counts[e], 1);  // nobody held it
      flag_error(a.dev_error, MLA_DEVERR_BAD_PAGE);
    }
  }
}

// ------------------------------------------------------------------ compact

// With L live pages, the live pages from L on (there are as many as free pages
// below L) go, highest first, to the free pages below L, lowest first.

// Table entries at, at + step, ...: kBatch of them (-1 past the table).
struct Entries {
  int32_t e[kBatch];
};
__device__ __forceinline__ Entries load_entries(const CompactArgs& a, int64_t at, int64_t step) {
  const int64_t entries = static_cast<int64_t>(a.num_seqs) * a.max_pages;
  Entries r;
#pragma unroll
  for (int x = 0; x < kBatch; ++x) r.e[x] = at + x * step < entries ? a.block_table[at + x * step] : -1;
  return r;
}

// `now`: the thread's first entries, loaded by the caller
__device__ void compact_apply(const CompactArgs& a, int64_t at, int64_t step, int32_t live, Entries now) {
  const int64_t entries = static_cast<int64_t>(a.num_seqs) * a.max_pages;
  // this thread's first move, loaded beside the table's
  const int32_t src = at < a.max_moves ? a.move_src[at] : -1;
  const int32_t dst = at < a.max_moves ? a.move_dst[at] : -1;
  const int32_t held = src >= 0 ? a.ref_counts[src] : 0;
  for (int64_t i0 = at; i0 < entries; i0 += kBatch * step) {
    if (i0 > at) now = load_entries(a, i0, step);
    const int32_t(&e)[kBatch] = now.e;
    int32_t k[kBatch], to[kBatch];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) k[x] = e[x] >= live && e[x] < a.num_pages ? a.move_of[e[x]] : -1;
#pragma unroll
    for (int x = 0; x < kBatch; ++x) to[x] = k[x] >= 0 ? a.move_dst[k[x]] : -1;
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      if (k[x] >= 0) a.block_table[i0 + x * step] = to[x];
      if (e[x] >= a.num_pages) flag_error(a.dev_error, MLA_DEVERR_BAD_PAGE);
    }
  }
  if (src >= 0) {
    a.ref_counts[dst] = held;
    a.ref_counts[src] = 0;
  }
  for (int64_t k = at + step; k < a.max_moves; k += step) {
    const int32_t s = a.move_src[k];
    if (s < 0) continue;
    a.ref_counts[a.move_dst[k]] = a.ref_counts[s];
    a.ref_counts[s] = 0;
  }
}

template <bool kFused>
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads, 1)
    compact_plan_kernel(CompactArgs a) {
  __shared__ PlanShared sm;
  const uint32_t rank = tc::cluster_ctarank();
  pdl_trigger();
  tc::cluster_sync();  // every CTA of the cluster has started: its shared memory may be written
  pdl_wait();
  if (threadIdx.x == 0) sm.need = 0;
  const int64_t at = static_cast<int64_t>(rank) * kPlanThreads + threadIdx.x, step = kPlanCtas * kPlanThreads;
  Entries mine{};
  if constexpr (kFused) mine = load_entries(a, at, step);  // used after the second barrier
  for (int i = rank * kPlanThreads + threadIdx.x; i < a.max_moves; i += kPlanCtas * kPlanThreads)
    a.move_src[i] = a.move_dst[i] = -1;
  int32_t live = 0;
  // (the cluster barrier inside also orders the -1 above before the moves below)
  const int32_t before = count_pages<false, 0>(a.ref_counts, a.num_pages, &sm, rank, &live);
  // stats[1]: every live page lies below it once the listed moves are made
  if (rank == 0 && threadIdx.x == 0) a.stats[0] = live;
  rank_pages<false, 0>(a.ref_counts, a.num_pages, rank, before, 0x7fffffff, [&](int64_t p, bool is, int32_t r) {
    if (p >= a.num_pages) return;
    if (p < live) {
      const int64_t k = p - r;  // free pages before it
      if (!is && k < a.max_moves) a.move_dst[k] = static_cast<int32_t>(p);
    } else {
      const int32_t k = live - 1 - r;  // live pages after it
      a.move_of[p] = is && k < a.max_moves ? k : -1;
      if (is && k < a.max_moves) a.move_src[k] = static_cast<int32_t>(p);
      if (is && k == a.max_moves) a.stats[1] = static_cast<int32_t>(p) + 1;  // the highest page that stays
    }
    // the pool's live pages from `live` on number free pages below it: fewer than
    // max_moves of them is what leaves stats[1] at `live`
    const bool edge = p == live - 1 || (live == 0 && p == 0);
    if (edge) {
      const int32_t below = live == 0 ? 0 : r + (is ? 1 : 0);  // live pages below `live`
      if (live - below <= a.max_moves) a.stats[1] = live;
    }
  });
  if constexpr (kFused) {
    __syncwarp();
    tc::cluster_sync();  // every count has been read, every move is listed
    compact_apply(a, at, step, live, mine);
  }
}

__global__ void __launch_bounds__(kApplyThreads) compact_apply_kernel(CompactArgs a) {
  pdl_trigger();
  pdl_wait();
  const int64_t at = static_cast<int64_t>(blockIdx.x) * kApplyThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kApplyThreads;
  compact_apply(a, at, step, a.stats[0], load_entries(a, at, step));
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

unsigned parts(int64_t n, int64_t most) {
  const int64_t p = (n + kApplyThreads - 1) / kApplyThreads;
  return static_cast<unsigned>(p < 1 ? 1 : (p < most ? p : most));
}

}  // namespace

// Workspace of extend: the requests' plan, the count of free pages, the free pages handed out.
size_t extend_workspace_bytes(int32_t n, int64_t num_pages) {
  return align256(static_cast<size_t>(n) * sizeof(ExtendItem)) + 256 +
         align256(static_cast<size_t>(num_pages) * sizeof(int32_t));
}

cudaError_t launch_extend(ExtendArgs a, void* workspace, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  char* ws = static_cast<char*>(workspace);
  a.items = ws;
  a.free_total = reinterpret_cast<int32_t*>(ws + align256(static_cast<size_t>(a.n) * sizeof(ExtendItem)));
  a.free_list = a.free_total + 64;
  const size_t smem = static_cast<size_t>(a.num_seqs) * sizeof(int32_t);
  static SmemOptIn opt_in;
  cudaError_t e = opt_in(kMaxTableSeqs * sizeof(int32_t), extend_plan_kernel<true>, extend_plan_kernel<false>);
  if (e != cudaSuccess) return e;
  if (static_cast<int64_t>(a.n) * a.max_pages + a.max_new <= kFusedWork)
    return launch_pdl(extend_plan_kernel<true>, dim3(kPlanCtas), dim3(kPlanThreads), smem, s, a);
  e = launch_pdl(extend_plan_kernel<false>, dim3(kPlanCtas), dim3(kPlanThreads), smem, s, a);
  if (e != cudaSuccess) return e;
  const int64_t work = a.max_pages > a.max_new / a.n ? a.max_pages : a.max_new / a.n;
  return launch_pdl(extend_apply_kernel, dim3(static_cast<unsigned>(a.n), parts(work / 2, 16)), dim3(kApplyThreads), 0,
                    s, a);
}

cudaError_t launch_free(const FreeArgs& a, cudaStream_t s) {
  if (a.n == 0) return cudaSuccess;
  return launch_pdl(free_kernel, dim3(static_cast<unsigned>(a.n), parts(a.max_pages, 16)), dim3(kApplyThreads), 0, s,
                    a);
}

// Workspace of compact: each page's place in the list of moves.
size_t compact_workspace_bytes(int64_t num_pages) {
  return align256(static_cast<size_t>(num_pages) * sizeof(int32_t));
}

cudaError_t launch_compact(const CompactArgs& a, cudaStream_t s) {
  const int64_t entries = static_cast<int64_t>(a.num_seqs) * a.max_pages;
  if (entries + a.max_moves <= kFusedWork)
    return launch_pdl(compact_plan_kernel<true>, dim3(kPlanCtas), dim3(kPlanThreads), 0, s, a);
  const cudaError_t e = launch_pdl(compact_plan_kernel<false>, dim3(kPlanCtas), dim3(kPlanThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(compact_apply_kernel, dim3(parts(entries > a.max_moves ? entries : a.max_moves, 8 * device_sm_count())),
                    dim3(kApplyThreads), 0, s, a);
}

}  // namespace mla
