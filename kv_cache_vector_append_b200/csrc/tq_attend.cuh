// tq_attend.cuh -- what the kernels of chunk and window attention over packed slots share:
// their parameters, and which keys a query sees.
//
// Query row (sequence b, token i of its n_q new ones, query head h) stands at position
// p = seq_lens[b] - n_q + i and sees key t when
//   t <= p  and  (window == 0  or  t > p - window  or  t < sinks).
// Rows of one KV head are counted r = i * group + g (g the head inside its group).
#pragma once

#include "tq_decode.cuh"

namespace tq {

struct AttendParams {
  const uint8_t* pages;
  int32_t num_blocks;
  int32_t h_kv;
  int32_t slot_stride;          // bytes between heads
  int64_t row_stride;           // bytes between tokens of a page
  int64_t blk_stride;           // bytes between pages
  const int32_t* block_table;
  int64_t bt_stride;
  int32_t max_blocks;
  const int32_t* seq_lens;
  int32_t batch;
  const int32_t* q_starts;      // [B + 1] rows of q of each sequence; null: row b alone
  int32_t num_rows;             // rows of q
  int32_t max_q;                // most new tokens of a sequence
  const void* q;                // [rows, H_q, D]
  int64_t q_rstride, q_hstride; // elements
  int32_t q_dtype;
  void* out;
  int64_t o_rstride, o_hstride;
  int32_t out_dtype;
  bool q_vec, out_vec;          // rows start on 16-byte boundaries
  int32_t group;
  float scale_log2;             // softmax scale * log2(e)
  uint64_t sign_seed;
  const float* kc;
  const float* vc;
  int32_t k_region;             // bytes of the K region (offset of the V region)
  int32_t window, sinks;
  int32_t tile_rows;            // rows a CTA of the tiles kernel takes
  int32_t row_tiles;            // row tiles of the longest chunk
  unsigned int* err;
  uint32_t wait_ms;
};

// One sequence of a call: its rows of q [row0, row0 + n_q) and its length.
struct AttendSeq {
  int32_t row0, n_q, len;
  bool skip;                    // a bad row range: nothing is written
};

// What a cluster works on.  The grid is one dimension of clusters: KV heads, then row tiles
// (the last first: it sees most keys), then sequences, the longest first where that pays (RANK)
// and a warp can rank them, so that what takes longest starts first.
struct AttendItem {
  int b, kvh, tile;
};
template <bool RANK>
__device__ __forceinline__ AttendItem attend_item(const AttendParams& p, int ctas) {
  const int lane = threadIdx.x & 31;
  int i = blockIdx.x / ctas;
  AttendItem it;
  it.kvh = i % p.h_kv;
  i /= p.h_kv;
  it.tile = p.row_tiles - 1 - i % p.row_tiles;
  it.b = i / p.row_tiles;
  if (RANK && p.batch > 1 && p.batch <= 32) {
    const int len = lane < p.batch ? p.seq_lens[lane] : -1;
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < p.batch; ++j) {
      const int other = __shfl_sync(0xffffffffu, len, j);
      rank += other > len || (other == len && j < lane);
    }
    it.b = __ffs(__ballot_sync(0xffffffffu, lane < p.batch && rank == it.b)) - 1;
  }
  return it;
}

__device__ __forceinline__ AttendSeq attend_seq(const AttendParams& p, int b, bool report) {
  AttendSeq s;
  s.row0 = b;
  s.n_q = 1;
  s.skip = false;
  if (p.q_starts != nullptr) {
    const int r0 = p.q_starts[b], r1 = p.q_starts[b + 1];
    s.skip = r0 < 0 || r1 < r0 || r1 > p.num_rows || r1 - r0 > p.max_q;
    s.row0 = r0;
    s.n_q = s.skip ? 0 : r1 - r0;
  }
  s.len = p.seq_lens[b];
  const bool bad = s.len < 0 || s.len > (int64_t)p.max_blocks * kBlockSize;
  if (bad) s.len = 0;           // its rows see nothing: 0
  if (report && (s.skip || bad)) report_error(p.err, TQ_DEVERR_SEQLEN_RANGE);
  return s;
}

// The keys [0, sink_end) and [win_begin, win_end), in units of `unit` tokens, that some
// query at a position in [p0, p1] sees (win_begin >= sink_end).
struct AttendSpan {
  int32_t sink_end, win_begin, win_end;
  __device__ __forceinline__ int count() const { return sink_end + win_end - win_begin; }
  __device__ __forceinline__ int at(int i) const { return i < sink_end ? i : win_begin + i - sink_end; }
};

__device__ __forceinline__ AttendSpan attend_span(const AttendParams& p, int p0, int p1, int unit) {
  AttendSpan s{0, 0, 0};
  if (p1 < 0) return s;
  s.win_end = p1 / unit + 1;
  if (p.window > 0) {
    s.win_begin = (int)max((int64_t)0, (int64_t)p0 - p.window + 1) / unit;
    s.sink_end = (int)min((int64_t)s.win_begin, ((int64_t)p.sinks + unit - 1) / unit);
  }
  return s;
}

// The factor 1 + j / 512 in [1, 2) under which the centroids of a table lie nearest to fp16 numbers
// (it leaves with the queries' scales).  The first: a warp's best of the factors of its threads, the
// least squared rounding (14 bits of it) with j below; the least of all warps' is the call's.
template <int BITS>
__device__ __forceinline__ unsigned centroid_factor_key(const float* c, int t, int threads) {
  float2 pair[1 << (BITS - 1)];
#pragma unroll
  for (int i = 0; i < 1 << (BITS - 1); ++i) pair[i] = make_float2(__ldg(c + 2 * i), __ldg(c + 2 * i + 1));
  unsigned key = ~0u;
  for (int j = t; j < 512; j += threads) {
    const float a = 1.0f + (float)j * (1.0f / 512);
    float e0 = 0.f, e1 = 0.f;
#pragma unroll
    for (int i = 0; i < 1 << (BITS - 1); ++i) {
      const float x = pair[i].x * a, y = pair[i].y * a;
      const float2 r = __half22float2(__floats2half2_rn(x, y));
      e0 = fmaf(r.x - x, r.x - x, e0);
      e1 = fmaf(r.y - y, r.y - y, e1);
    }
    key = min(key, (__float_as_uint((e0 + e1) / (a * a)) & ~511u) | (unsigned)j);
  }
  return __reduce_min_sync(0xffffffffu, key);
}
__device__ __forceinline__ float centroid_factor(unsigned key) {
  return 1.0f + (float)(key & 511u) * (1.0f / 512);
}

}  // namespace tq
