// tq_pages.cuh -- page operations of a packed cache on device tables: give and take pages
// (resize), share them with another sequence (fork), gather kept tokens (compact).
//
// State.  ref_counts[page] = number of block-table entries that name the page; a page is
// free when its count is 0.  Pages are given out lowest index first, to the requests in
// their order, so the result does not depend on how the grid runs.
//
// resize and fork plan and allocate in one cluster: it turns the counts into a bitmap of free
// pages in shared memory (each CTA a contiguous part of the pool), joins the CTAs' totals over
// distributed shared memory, and lets every free page find its rank (prefix sums of the
// bitmap's words) and the request of that rank (a search in the prefix sums of the demands).  What
// follows is long: page copies, shared or released table entries, count updates (integer atomics,
// so their order does not matter).  Where it is little (see kFusedChunks) the cluster's warps do
// it themselves after a cluster barrier, else a second launch with a CTA per sequence and layer.
// What that needs to know of the plan is in `moves`, a tensor of the caller: {from, to} of a page
// copy, {-1, -1} for none, {-2, -2} for a refused request.  No other state is kept between the
// launches or the calls.
//
// Bound: the plan by latency (a few dependent reads and cluster barriers; the pool is read
// once), the copies and compact by memory bandwidth.
#pragma once

#include <cooperative_groups.h>

#include "tq_device.cuh"

namespace tq {

constexpr int kPageTokens = 16;            // tokens per page block
constexpr int kMaxPageLayers = 128;        // pools one call copies pages of
constexpr int kMaxPageRequests = 8192;     // sequences of the table, pairs of a fork
constexpr int kMaxPoolPages = 1 << 21;
constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxCtas = 8;            // portable cluster size
constexpr int kPagesThreads = 256;

// What the cluster of the plan does itself: at most this many page pieces of kCopyPiece bytes to
// copy and runs of 128 table entries to go through, two rounds of its 256 warps, in at most
// kFusedLayers layers (a small kernel argument).  us on the GPU in one launch / in two, for a pair of
// calls: 128 runs 22.1 / 22.1, 512 29.4 / 28.8, 1,024 32.3 / 29.5, 1,152 pieces 21.3 / 17.0; from
// Python, where the host bounds small calls, 288 pieces 30 / 35, 1,024 runs 38.4 / 37.0.
constexpr int kFusedChunks = 512;
constexpr int kCopyPiece = 2048;
constexpr int kFusedLayers = 8;

// The pools that a call moves slots in (one per model layer).
template <int N>
struct PageLayersOf {
  int32_t count;
  uint8_t* base[N];
  int64_t blk_stride[N];                   // bytes between pages
  int32_t page_bytes[N];                   // a multiple of 128
};
using PageLayers = PageLayersOf<kMaxPageLayers>;
using FewLayers = PageLayersOf<kFusedLayers>;

struct PlanParams {
  int32_t* table;                          // [batch, cols]
  int64_t table_stride;
  int32_t cols;
  int32_t* seq_lens;
  int32_t batch;
  const int32_t* new_lens;                 // resize
  const int32_t* parents;                  // fork [requests]
  const int32_t* children;
  int32_t requests;
  int32_t* refs;                           // [pool]
  int32_t pool;
  int32_t* moves;                          // [requests, 2]
  int32_t window, sinks;                   // resize: pages out of the window are released
  unsigned int* err;
};

// Bitmap words of one CTA's part of the pool.
__host__ __device__ inline int plan_words(int pool, int ctas) {
  return ((pool + 31) / 32 + ctas - 1) / ctas;
}
// Shared memory of the plan: bitmap, its prefix sums, the demands' prefix sums, lengths and
// kinds, and (fork) the first pair of each child.
inline size_t plan_smem(int pool, int ctas, int requests, int owners) {
  return 4 * ((size_t)2 * plan_words(pool, ctas) + 2 + 2 * (size_t)requests + owners) + requests;
}

// Exclusive prefix sums over the block of one value a thread; *total receives the sum.
__device__ __forceinline__ unsigned block_scan(unsigned v, unsigned* warp_sums, unsigned* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();                         // warp_sums of an earlier scan are read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    unsigned w = warp_sums[lane];          // kPlanThreads / 32 = 32 warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned t = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += t;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  *total = warp_sums[31];
  return inc - v + (warp ? warp_sums[warp - 1] : 0u);
}

// The largest i in [0, n) with a[i] <= x (a[0] <= x, a ascending).
__device__ __forceinline__ int last_not_above(const unsigned* a, int n, unsigned x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__host__ __device__ __forceinline__ int pages_of(int tokens) {
  return tokens / kPageTokens + (tokens % kPageTokens != 0);
}

// What a request asks for: its pages, the length they are for, and its kind.
enum : uint8_t { kAsksNothing = 0, kAsksPages = 1, kAsksCopy = 2, kBadRequest = 4 };
struct Demand {
  int pages;
  int len;
  uint8_t kind;
};

// A growing sequence asks for the pages past its last one, and for one more, the first, where
// its partly filled last page is shared (copy on write).
__device__ __forceinline__ Demand resize_demand(const PlanParams& p, int b) {
  const int len = p.seq_lens[b], to = p.new_lens[b];
  const int64_t room = (int64_t)p.cols * kPageTokens;
  if (len < 0 || len > room || to < 0 || to > room) return Demand{0, 0, kBadRequest};
  Demand d{0, len, kAsksNothing};
  if (to <= len) return d;
  if (len % kPageTokens) {
    const int last = p.table[b * p.table_stride + len / kPageTokens];
    if (last >= 0 && last < p.pool && p.refs[last] > 1) d.kind |= kAsksCopy;
  }
  d.pages = pages_of(to) - pages_of(len) + ((d.kind & kAsksCopy) ? 1 : 0);
  if (d.pages) d.kind |= kAsksPages;
  return d;
}

// A fork asks for a page of its own where its parent's last page is partly filled.
// owner[c]: the first pair that names child c.
__device__ __forceinline__ Demand fork_demand(const PlanParams& p, int i, const int* owner) {
  const int from = p.parents[i], to = p.children[i];
  if (from < 0 || from >= p.batch || to < 0 || to >= p.batch || owner[to] != i)
    return Demand{0, 0, kBadRequest};
  const int len = p.seq_lens[from];
  if (p.seq_lens[to] != 0 || len < 0 || len > (int64_t)p.cols * kPageTokens)
    return Demand{0, 0, kBadRequest};
  Demand d{0, len, kAsksNothing};
  if (len % kPageTokens) {
    const int last = p.table[from * p.table_stride + len / kPageTokens];
    if (last >= 0 && last < p.pool) {
      d.kind = kAsksPages | kAsksCopy;
      d.pages = 1;
    }
  }
  return d;
}

// Entries c0 + t, c0 + t + n, ... (four of them, below the sequence's pages) of sequence b that
// a resize from len to want tokens releases: those past the new length, and with a window those
// whose tokens no query at a position >= min(len, want) sees.
__device__ __forceinline__ void release_entries(const PlanParams& p, int b, int len, int want, int c0,
                                                int n, int t) {
  const int have = pages_of(len), keep = pages_of(want), least = min(len, want);
  // all tokens >= sinks and < least - window + 1
  const int w0 = p.window > 0 ? pages_of(p.sinks) : 0;
  const int w1 = p.window > 0 ? max(0, least - p.window + 1) / kPageTokens : 0;
  int32_t* row = p.table + b * p.table_stride;
  int32_t id[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = c0 + t + j * n;
    id[j] = c < have && (c >= keep || (c >= w0 && c < w1)) ? row[c] : -1;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (id[j] < 0) continue;
    if (id[j] < p.pool) atomicSub(&p.refs[id[j]], 1);
    else report_error(p.err, TQ_DEVERR_BLOCK_RANGE);
    row[c0 + t + j * n] = -1;
  }
}

// Entries c0 + t, c0 + t + n, ... (four of them, below `end`) of the parent's row to the child's,
// their pages shared.
__device__ __forceinline__ void share_entries(const PlanParams& p, int parent, int child, int end, int c0,
                                              int n, int t) {
  const int32_t* src = p.table + parent * p.table_stride;
  int32_t* dst = p.table + child * p.table_stride;
  int32_t id[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) id[j] = c0 + t + j * n < end ? src[c0 + t + j * n] : -1;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (c0 + t + j * n >= end) continue;
    dst[c0 + t + j * n] = id[j];
    if (id[j] < 0) continue;
    if (id[j] < p.pool) atomicAdd(&p.refs[id[j]], 1);
    else report_error(p.err, TQ_DEVERR_BLOCK_RANGE);
  }
}

// 16-byte units [u0, u1) of a page, by n threads, four loads in flight each.
template <class Layers>
__device__ __forceinline__ void copy_units(const Layers& l, int layer, int from, int to, int u0, int u1,
                                           int n, int t) {
  const uint4* s = (const uint4*)(l.base[layer] + from * l.blk_stride[layer]);
  uint4* d = (uint4*)(l.base[layer] + to * l.blk_stride[layer]);
  for (int i0 = u0 + t; i0 < u1; i0 += 4 * n) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j * n < u1) v[j] = s[i0 + j * n];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j * n < u1) d[i0 + j * n] = v[j];
  }
}

// FUSED: the cluster also does what the second launch does otherwise.
template <bool FORK, bool FUSED>
__global__ void __launch_bounds__(kPlanThreads, 1)
pages_plan_kernel(const PlanParams p, const __grid_constant__ FewLayers layers, int pieces) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int words = plan_words(p.pool, ctas);
  extern __shared__ __align__(16) uint32_t plan_mem[];
  uint32_t* bitmap = plan_mem;                       // [words] free pages of this CTA's part
  unsigned* before = plan_mem + words;               // [words + 1] free pages before a word
  unsigned* need = before + words + 1;               // [requests + 1] pages asked before a request
  int* lens = (int*)(need + p.requests + 1);         // [requests]
  int* owner = lens + p.requests;                    // [batch] (fork)
  uint8_t* kind = (uint8_t*)(owner + (FORK ? p.batch : 0));   // [requests]
  __shared__ unsigned warp_sums[32];
  __shared__ unsigned cta_free;
  const int tid = threadIdx.x, lane = tid & 31;
  const int word0 = rank * words;

  // free pages of this part: one ballot a word, eight words' counts in flight
  for (int w0 = tid >> 5; w0 < words; w0 += 8 * (kPlanThreads / 32)) {
    int n[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int w = w0 + j * (kPlanThreads / 32);
      const int64_t page = (int64_t)(word0 + w) * 32 + lane;
      n[j] = w < words && page < p.pool ? p.refs[page] : 1;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int w = w0 + j * (kPlanThreads / 32);
      const uint32_t bits = __ballot_sync(0xffffffffu, n[j] == 0);
      if (lane == 0 && w < words) bitmap[w] = bits;
    }
  }
  if (FORK) {
    for (int b = tid; b < p.batch; b += kPlanThreads) owner[b] = 0x7fffffff;
    __syncthreads();
    for (int i = tid; i < p.requests; i += kPlanThreads) {
      const int to = p.children[i];
      if (to >= 0 && to < p.batch) atomicMin(&owner[to], i);
    }
  }
  __syncthreads();
  unsigned carry = 0;
  for (int w0 = 0; w0 < words; w0 += kPlanThreads) {
    const int w = w0 + tid;
    unsigned total;
    const unsigned pre = block_scan(w < words ? __popc(bitmap[w]) : 0, warp_sums, &total);
    if (w < words) before[w] = carry + pre;
    carry += total;
  }
  if (tid == 0) {
    before[words] = carry;
    cta_free = carry;
  }
  // the demands (every CTA: they are few next to the pool).  One above the pool counts as
  // pool + 1 and the sums stop at 2^30, which is refused all the same.
  constexpr unsigned kCap = 1u << 30;
  unsigned asked = 0;
  for (int i0 = 0; i0 < p.requests; i0 += kPlanThreads) {
    const int i = i0 + tid;
    Demand d{0, 0, kAsksNothing};
    if (i < p.requests) {
      d = FORK ? fork_demand(p, i, owner) : resize_demand(p, i);
      lens[i] = d.len;
      kind[i] = d.kind;
    }
    unsigned total;
    const unsigned pre = block_scan((unsigned)min(d.pages, p.pool + 1), warp_sums, &total);
    if (i < p.requests) need[i] = min(asked + pre, kCap);
    asked = min(asked + total, kCap);
  }
  if (tid == 0) need[p.requests] = asked;
  cluster.sync();        // the counts and lengths are read by every CTA, the totals are there
  unsigned first = 0, free_pages = 0;
  for (int c = 0; c < ctas; ++c) {
    const unsigned n = *cluster.map_shared_rank(&cta_free, c);
    if (c < rank) first += n;
    free_pages += n;
  }
  // the ranks [first, first + carry) of the demand are served from this part: a warp takes a
  // word of the bitmap, a lane a page of it
  for (int w = tid >> 5; w < words; w += kPlanThreads / 32) {
    if (first + before[w] >= asked) break;
    const uint32_t bits = bitmap[w];
    const unsigned r = first + before[w] + __popc(bits & ((1u << lane) - 1u));
    if (!((bits >> lane) & 1u) || r >= asked) continue;
    const int i = last_not_above(need, p.requests + 1, r);
    if (need[i + 1] > free_pages) continue;          // refused as a whole
    const int page = (word0 + w) * 32 + lane;
    const int k = (int)(r - need[i]);
    p.refs[page] = 1;
    const int seq = FORK ? p.children[i] : i;
    const int copies = (kind[i] & kAsksCopy) ? 1 : 0;
    int32_t* row = p.table + seq * p.table_stride;
    if (k < copies) {
      const int col = lens[i] / kPageTokens;
      const int from = p.table[(FORK ? p.parents[i] : seq) * p.table_stride + col];
      p.moves[2 * i] = from;
      p.moves[2 * i + 1] = page;
      row[col] = page;
    } else {
      row[pages_of(lens[i]) + k - copies] = page;
    }
  }
  if (rank == 0) {
    for (int i = tid; i < p.requests; i += kPlanThreads) {
      const uint8_t what = kind[i];
      const bool bad = what & kBadRequest;
      const bool refused = (what & kAsksPages) && need[i + 1] > free_pages;
      if (bad) report_error(p.err, FORK ? TQ_DEVERR_SEQ_INDEX : TQ_DEVERR_SEQLEN_RANGE);
      if (refused) report_error(p.err, TQ_DEVERR_NO_PAGES);
      if (bad || refused || !(what & kAsksCopy)) {
        const int mark = bad || refused ? -2 : -1;
        p.moves[2 * i] = mark;
        p.moves[2 * i + 1] = mark;
      }
      if (FORK && !bad && !refused) p.seq_lens[p.children[i]] = lens[i];
    }
  }
  cluster.sync();        // no CTA leaves while another may read its total
  if constexpr (FUSED) {
    const int warp = rank * (kPlanThreads / 32) + (tid >> 5), warps = ctas * (kPlanThreads / 32);
    auto served = [&](int i) {
      return !(kind[i] & kBadRequest) && !((kind[i] & kAsksPages) && need[i + 1] > free_pages);
    };
    const int runs = (p.cols + 127) / 128;
    for (int item = warp; item < p.requests * runs; item += warps) {
      const int i = item / runs, c0 = (item - i * runs) * 128;
      if (c0 >= pages_of(lens[i]) || !served(i)) continue;
      if (FORK) {
        // a partly filled last page without a copy is a hole (or out of range) in the parent too
        const int end = (kind[i] & kAsksCopy) ? lens[i] / kPageTokens : pages_of(lens[i]);
        share_entries(p, p.parents[i], p.children[i], end, c0, 32, lane);
      } else {
        release_entries(p, i, lens[i], p.new_lens[i], c0, 32, lane);
      }
    }
    for (int item = warp; item < p.requests * layers.count * pieces; item += warps) {
      const int i = item / (layers.count * pieces), rest = item - i * layers.count * pieces;
      const int layer = rest / pieces, piece = rest - layer * pieces;
      if (!(kind[i] & kAsksCopy) || !served(i)) continue;
      const int units = layers.page_bytes[layer] / 16, u0 = piece * (kCopyPiece / 16);
      copy_units(layers, layer, p.moves[2 * i], p.moves[2 * i + 1], u0, min(units, u0 + kCopyPiece / 16), 32,
                 lane);
    }
    if (!FORK && rank == 0) {                // every CTA read the old lengths before the barrier
      for (int i = tid; i < p.requests; i += kPlanThreads) {
        if (!served(i)) continue;
        if (kind[i] & kAsksCopy) atomicSub(&p.refs[p.moves[2 * i]], 1);
        p.seq_lens[i] = p.new_lens[i];
      }
    }
  }
}

__device__ __forceinline__ void copy_page(const PageLayers& l, int layer, int from, int to) {
  copy_units(l, layer, from, to, 0, l.page_bytes[layer] / 16, kPagesThreads, threadIdx.x);
}

// Second launch of resize: grid (batch, 1 + layers).  CTA (b, 0) releases sequence b's
// entries and gives it its length, CTA (b, 1 + l) makes its page copy in layer l.
static __global__ void __launch_bounds__(kPagesThreads)
pages_resize_kernel(const PlanParams p, const __grid_constant__ PageLayers layers) {
  const int b = blockIdx.x;
  const int from = p.moves[2 * b], to = p.moves[2 * b + 1];
  if (from == -2) return;
  if (blockIdx.y > 0) {
    if (from >= 0) copy_page(layers, blockIdx.y - 1, from, to);
    return;
  }
  const int len = p.seq_lens[b], want = p.new_lens[b];
  for (int c0 = 0; c0 < pages_of(len); c0 += 4 * kPagesThreads)
    release_entries(p, b, len, want, c0, kPagesThreads, threadIdx.x);
  __syncthreads();                         // the old length has been read
  if (threadIdx.x == 0) {
    if (from >= 0) atomicSub(&p.refs[from], 1);
    p.seq_lens[b] = want;
  }
}

constexpr int kForkChunk = 4 * kPagesThreads;   // table entries a CTA shares at a time
constexpr int kForkMostChunks = 32768;          // (chunks + layers is a grid's second dimension)

// Second launch of fork: grid (pairs, chunks of the table row + layers).  The entries of the
// parent's full pages are shared with the child, its partly filled one is copied.
static __global__ void __launch_bounds__(kPagesThreads)
pages_fork_kernel(const PlanParams p, const __grid_constant__ PageLayers layers, int chunks) {
  const int i = blockIdx.x;
  const int from = p.moves[2 * i], to = p.moves[2 * i + 1];
  if (from == -2) return;
  if ((int)blockIdx.y >= chunks) {
    if (from >= 0) copy_page(layers, blockIdx.y - chunks, from, to);
    return;
  }
  const int child = p.children[i];
  const int len = p.seq_lens[child];       // the parent's before the call
  // a partly filled last page without a copy is a hole (or out of range) in the parent too
  const int end = from >= 0 ? len / kPageTokens : pages_of(len);
  for (int c0 = blockIdx.y * kForkChunk; c0 < end; c0 += chunks * kForkChunk)
    share_entries(p, p.parents[i], child, end, c0, kPagesThreads, threadIdx.x);
}

struct CompactParams {
  const int32_t* src_table;
  int64_t src_stride;
  int32_t src_cols;
  const int32_t* src_lens;
  const int32_t* positions;                // [batch, max_keep]
  int64_t pos_stride;
  int32_t max_keep;
  const int32_t* counts;
  const int32_t* dst_table;
  int64_t dst_stride;
  int32_t dst_cols;
  int32_t pool;
  unsigned int* err;
};

// Rows [0, counts[b]) of sequence b in the destination pages <- its rows positions[b, .].
// One CTA per destination page, sequence and layer: its 16 rows' addresses are resolved
// once, then their U-byte units are copied with four loads in flight a thread.
template <typename U, class Layers>
__global__ void __launch_bounds__(kPagesThreads)
pages_compact_kernel(const CompactParams p, const __grid_constant__ Layers layers) {
  const int b = blockIdx.y, layer = blockIdx.z;
  const int count = p.counts[b], len = p.src_lens[b];
  if (count < 0 || count > p.max_keep || pages_of(count) > p.dst_cols || len < 0 ||
      len > (int64_t)p.src_cols * kPageTokens) {
    if (threadIdx.x == 0) report_error(p.err, TQ_DEVERR_SEQLEN_RANGE);
    return;
  }
  const int i0 = blockIdx.x * kPageTokens;
  if (i0 >= count) return;
  const int rows = min(kPageTokens, count - i0);
  const int row_units = layers.page_bytes[layer] / kPageTokens / (int)sizeof(U);
  __shared__ const U* src[kPageTokens];
  __shared__ U* dst_page;
  if ((int)threadIdx.x < rows) {
    const int t = p.positions[b * p.pos_stride + i0 + threadIdx.x];
    const U* s = nullptr;
    if (t < 0 || t >= len) {
      report_error(p.err, TQ_DEVERR_SLOT_RANGE);
    } else {
      const int id = p.src_table[b * p.src_stride + t / kPageTokens];
      if (id < 0 || id >= p.pool) report_error(p.err, TQ_DEVERR_BLOCK_RANGE);
      else s = (const U*)(layers.base[layer] + id * layers.blk_stride[layer]) +
               (t % kPageTokens) * row_units;
    }
    src[threadIdx.x] = s;
  }
  if (threadIdx.x == 32) {
    const int id = p.dst_table[b * p.dst_stride + blockIdx.x];
    if (id < 0 || id >= p.pool) {
      report_error(p.err, TQ_DEVERR_BLOCK_RANGE);
      dst_page = nullptr;
    } else {
      dst_page = (U*)(layers.base[layer] + id * layers.blk_stride[layer]);
    }
  }
  __syncthreads();
  U* d = dst_page;
  if (d == nullptr) return;
  const int n = rows * row_units;
  for (int u0 = threadIdx.x; u0 < n; u0 += 4 * kPagesThreads) {
    U v[4];
    bool ok[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int u = u0 + j * kPagesThreads;
      ok[j] = false;
      if (u < n) {
        const int r = u / row_units;
        const U* s = src[r];
        ok[j] = s != nullptr;
        if (ok[j]) v[j] = s[u - r * row_units];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (ok[j]) d[u0 + j * kPagesThreads] = v[j];
  }
}

}  // namespace tq
