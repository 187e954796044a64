// tq_attend_tiles.cuh -- attention over packed slots for many query rows a KV head (chunks of
// new tokens), on the tcgen05 tensor cores.
//
// Math.  As in tq_attend_rows.cuh, in the rotated domain: S = q^ C~^T on the codes' centroids,
// x = S nK |q'| scale log2(e) per (row, key), P = 2^(x - M), O' += P V~, o = R^T O' / l;
// statistics and accumulators are fp32.  fp16 operands: unit queries (2^-12 off, as their sum
// over coordinates of either sign), centroids of keys times a factor in [1, 2) under which their
// roundings are smallest (a search over 512 factors; it leaves with the rows' scales), values
// c nV 2^-ev, P; 8-bit key centroids as hi + lo.  Together about 6e-4 of the output, a third of
// bf16's own rounding.  Key norms stay out of the operand: in it they would be rounded key by
// key, which costs 1e-3.
// M >= max(x + log2 nV): a tile whose V norms lie within 2^8 of each other and which every row
// sees takes the power 2^ev above its largest norm for all of them; in any other tile V~ = c,
// P = 2^(x - M) nV, and the bound goes key by key, masks included, so that what a row does not
// see never touches it.
//
// Layout.  A CTA holds two slots of 128 rows x N keys: two row tiles that share every key tile
// (256 rows), or, with 128 rows, one row tile whose key tiles alternate between the slots,
// each with its own (M, l, O'), joined at the end.  (D = 256: one O' fills the tensor
// memory; one softmax warpgroup, two score buffers.)  Warps 0-7 are the slots' softmax
// warpgroups (a thread = a row: scores from tensor memory, P back over them), warps 8-11 turn
// packed codes into fp16 tiles in shared memory (lookups of code pairs, one 256-byte row an
// entry, so that 32 lanes hit 32 banks; the next tile's codes are already on their way into
// registers), warps 12 and 13 issue the MMAs of a slot each: P V of an item of 64 keys, then Q K
// of the item after the next, so that a slot's softmax always finds scores.  Both operand tiles
// are rows of 64 columns with the 128-byte swizzle: K-major for Q K, MN-major for P V, the same
// bytes.  A cluster of CTAs may split the keys; partials are joined over distributed shared
// memory as in the rows kernel.
//
// Bound: shared memory, which operands (a step of 256 rows x 128 keys reads 256 KB for its
// MMAs), lookups, tiles and norms share: 805 TFLOP/s on 4,096 new tokens of 20,480 (32/8 heads
// of 128, 4/4 bits, 1,537 us), half of the measured matrix rate; the MMAs alone run at 1,267.
// Without the dequantization it took 9% less, without the softmax 14% less; no single part of
// the softmax is worth more than 5%.
#pragma once

#include <cooperative_groups.h>

#include "tq_append_dense.cuh"
#include "tq_attend.cuh"

namespace tq {

constexpr int kTileRows = 128;             // rows of a slot (the MMA's M)
constexpr int kTilesThreads = 512, kTilesWarps = kTilesThreads / 32;
constexpr int kDequantWarps = 4;
// registers a thread of the softmax, dequantizing and issuing warpgroups, from kTilesRegs each
constexpr int kTilesRegs = 128, kSoftmaxRegs = 152, kDequantRegs = 128, kIssueRegs = 80;
static_assert(2 * kSoftmaxRegs + kDequantRegs + kIssueRegs <= 4 * kTilesRegs, "registers of a CTA");

template <int D, int KB, int VB>
struct TilesCfg {
  static constexpr bool kTwoTiles = D <= 128;            // may hold two row tiles
  static constexpr bool kOneO = D == 256;                // one accumulator, one softmax warpgroup
  // 8-bit key centroids as fp16 hi + lo, two parts of a K tile: their cells are narrower than what
  // keys of one direction differ by, so that roundings do not cancel in the softmax as those of
  // coarser codes do (keys with channel means of 30 sigma: 6e-3 of the output without lo).  The
  // tiles are half as long then (4 x 512 new tokens at 8,192, 8/8 bits: 32/8 heads of 128 723
  // against 511 us, 16/4 heads of 256 1,128 against 856).
  static constexpr int KPARTS = KB == 8 ? 2 : 1, KPART = D / 64;   // (64-column blocks of a part)
  // bytes of a ring stage, keys of a tile
  static constexpr int STAGE = D == 64 ? 16384 * KPARTS : 32768, N = STAGE / (2 * D * KPARTS), RING = 3;
  static constexpr int PPT = N / kBlockSize;             // pages a tile
  // A slot works on items of NI keys of a tile, two score buffers in turn
  static constexpr int NI = N < 64 ? N : 64, H = N / NI;
  static constexpr int QTILE = kTileRows * D * 2;
  static constexpr int QBYTES = (kTwoTiles ? 2 : 1) * QTILE;
  static constexpr int PART = D + 4;                     // floats of a row's partial
  static constexpr int STAGING = (kOneO ? 1 : 2) * kTileRows * PART * 4;
  static constexpr int OPER = QBYTES + RING * STAGE > STAGING ? QBYTES + RING * STAGE : STAGING;
  static constexpr int LUT = kLutRow * (lut_entries(KB) > lut_entries(VB) ? lut_entries(KB) : lut_entries(VB));
  // norms [buffer][K, V][N]; a row tile whose key tiles alternate uses four buffers, at D <= 128
  // in the place of the second row tile's q
  static constexpr int NBUF = kOneO ? 4 : 2;
  // (and at the start, behind the first buffer, 256 scales of q)
  static constexpr int NORMS = 4 * (NBUF * N * 2 > N * 2 + 256 ? NBUF * N * 2 : N * 2 + 256);
  static constexpr int MISC = 1024;
  // more than half an SM: a CTA that holds all of tensor memory has the SM to itself
  static constexpr int RAW = OPER + LUT + NORMS + MISC;
  static constexpr int SMEM = RAW > 120 * 1024 ? RAW : 120 * 1024;
  // dequantization: 16 codes a lane
  static constexpr int LPR = D / 16, RPI = 32 / LPR, IT = N / kDequantWarps / RPI;
  // codes of both kinds a whole tile ahead in registers, or of the next kind only
  static constexpr int KW = KB == 2 ? 1 : KB == 8 ? 4 : 2, VW = VB == 2 ? 1 : VB == 8 ? 4 : 2;
  static constexpr bool kDeep = IT * (KW + VW) <= 32;
  static_assert(N % 16 == 0 && N <= 128 && IT >= 1 && N / kDequantWarps % RPI == 0, "tile geometry");
  static_assert(SMEM <= 232448, "shared memory");
};

// What the dequantizing warps know of their N / 4 keys of a tile: bounds of log2 nV, and whether
// every row of the CTA sees every key and all norms are finite.
struct TileMeta {
  int vmax, vmin, plain;
};
// And of the whole tile.  plain: no masks, V norms within 2^8 of each other; the operand then
// holds c nV 2^-ev, else c alone.
struct TileInfo {
  int plain;
  float ev;
};

struct TilesMisc {
  uint4 flip[32];                          // sign bits of the coordinates, as in a 16-bit row
  uint64_t s_full[2][2], p_ready[2][2], pv_done[2], norm_full[4], ring_full[3], ring_empty[3], o_done, q_ready;
  unsigned best;                           // the key centroids' factor (centroid_factor_key)
  float alpha;
  uint32_t tmem;
  int tok[4][8];                           // first token of a page of the tile; < 0: no page
  TileMeta meta[2][kDequantWarps];
  TileInfo info[4];
};
static_assert(sizeof(TilesMisc) <= 1024, "misc area");

__device__ __forceinline__ void umma_ts_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Descriptor of an MN-major operand in 64-column blocks of rows x 128 bytes, 128-byte swizzle:
// block_bytes between blocks (leading offset), 1024 between groups of 8 rows (stride offset).
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t block_bytes) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(block_bytes >> 4) << 16) | (64ull << 32) |
         (1ull << 46) | (2ull << 61);
}
// kind::f16, fp16 operands, fp32 accumulator, M = 128.
__host__ __device__ constexpr uint32_t f16_idesc(int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}
// Two fp32 at once.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " mul.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n"
      " add.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 w, {%6, %7};\n"
      " fma.rn.f32x2 z, x, y, w;\n mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int R>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(R)); }

// A lane's 16 codes of BITS bits at codes 16 l .. of a row's region (4-byte aligned).
template <int BITS>
struct Codes16 {
  static constexpr int W = BITS == 2 ? 1 : BITS == 8 ? 4 : 2;
  static __device__ __forceinline__ void load(uint32_t (&w)[4], const uint8_t* region, int l) {
    if constexpr (BITS == 3) {
      const int o = 6 * l;
      const uint32_t* a = (const uint32_t*)(region + (o & ~3));
      const int sh = 8 * (o & 3);                        // 0 or 16
      const uint32_t lo = a[0], hi = a[1];               // both inside the slot: the norm follows
      w[0] = __funnelshift_r(lo, hi, sh);
      w[1] = hi >> sh;
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j] = *(const uint32_t*)(region + 4 * W * l + 4 * j);
    }
  }
};

// Lookup tables of the tiles: entry e at row e, K in the first half of a row, V in the second,
// one copy a lane.  BITS <= 4: half2 of a code pair; 8 bits: half2(hi, lo) of a code.  A warp
// makes 32 entries at a time, one a lane, and writes each to its row.
template <int BITS, int HALF>
__device__ __forceinline__ void tiles_lut(uint8_t* lut, const float* c, float alpha, int warp, int warps,
                                          int lane) {
  constexpr int kEntries = lut_entries(BITS);
  for (int e0 = warp * 32; e0 < kEntries; e0 += warps * 32) {
    const int e = e0 + lane;
    uint32_t v = 0u;
    if (e < kEntries) {
      if constexpr (BITS <= 4) {
        v = pack_half2(c[e & ((1 << BITS) - 1)] * alpha, c[e >> BITS] * alpha);
      } else {
        const float hi = __half2float(__float2half_rn(c[e]));
        v = pack_half2(hi, c[e] - hi);
      }
    }
    uint32_t* row = (uint32_t*)(lut + e0 * kLutRow + HALF * 128) + lane;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < kEntries) row[j * (kLutRow / 4)] = __shfl_sync(0xffffffffu, v, j);
  }
}
// A row of D coordinates over D / 16 lanes: lane l of the group holds, in x[4 j + e], coordinate
// 4 (l + D / 16 j) + e, so that a group's accesses of 4 coordinates a lane are contiguous.
template <int D>
__device__ __forceinline__ int group_coord(int l, int j) { return 4 * (l + D / 16 * j); }
// FWHT of such a row (natural order, no scaling).
template <int D>
__device__ __forceinline__ void group_fwht(float (&x)[16], int l) {
#pragma unroll
  for (int h = 1; h < 16; h <<= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((i & h) == 0) {
        const float a = x[i], b = x[i + h];
        x[i] = a + b;
        x[i + h] = a - b;
      }
#pragma unroll
  for (int m = 1; m < D / 16; m <<= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float o = __shfl_xor_sync(0xffffffffu, x[i], m);
      x[i] = (l & m) ? o - x[i] : x[i] + o;
    }
}
// The signs of the coordinates that a lane holds (flip: sign bits in pairs of 16-bit fields).
template <int D>
__device__ __forceinline__ void group_flip(float (&x)[16], const uint4* flip, int l) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint2 f = ((const uint2*)flip)[group_coord<D>(l, j) / 4];
    const uint32_t m[4] = {f.x << 16, f.x, f.y << 16, f.y};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      x[4 * j + e] = __uint_as_float(__float_as_uint(x[4 * j + e]) ^ (m[e] & 0x80000000u));
  }
}
// Its elements from / to memory; vec: rows start on 16-byte boundaries.
template <int D>
__device__ __forceinline__ void group_load(float (&x)[16], const void* base, int64_t off, int32_t dtype,
                                           bool vec, int l) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t at = off + group_coord<D>(l, j);
    if (vec && dtype != TQ_F32) {
      const uint2 w = *(const uint2*)((const uint16_t*)base + at);
      if (dtype == TQ_BF16) {
        x[4 * j] = __uint_as_float(w.x << 16), x[4 * j + 1] = __uint_as_float(w.x & 0xffff0000u);
        x[4 * j + 2] = __uint_as_float(w.y << 16), x[4 * j + 3] = __uint_as_float(w.y & 0xffff0000u);
      } else {
        const float2 a = __half22float2(*(const __half2*)&w.x), b = __half22float2(*(const __half2*)&w.y);
        x[4 * j] = a.x, x[4 * j + 1] = a.y, x[4 * j + 2] = b.x, x[4 * j + 3] = b.y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * j + e] = load_as_f32(base, at + e, dtype);
    }
  }
}
template <int D>
__device__ __forceinline__ void group_store(const float (&x)[16], void* base, int64_t off, int32_t dtype,
                                            bool vec, int l) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t at = off + group_coord<D>(l, j);
    if (vec && dtype != TQ_F32) {
      uint2 w;
      if (dtype == TQ_BF16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[4 * j], x[4 * j + 1]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[4 * j + 2], x[4 * j + 3]);
        w = make_uint2(*(const uint32_t*)&a, *(const uint32_t*)&b);
      } else {
        w = make_uint2(pack_half2(x[4 * j], x[4 * j + 1]), pack_half2(x[4 * j + 2], x[4 * j + 3]));
      }
      *(uint2*)((uint16_t*)base + at) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) store_from_f32(base, at + e, dtype, x[4 * j + e]);
    }
  }
}

// FWHT over C consecutive values of a thread (natural order, no scaling).
template <int C>
__device__ __forceinline__ void thread_fwht(float* x) {
#pragma unroll
  for (int i = 0; i < C; i += 2) {
    const float a = x[i], b = x[i + 1];
    x[i] = a + b;
    x[i + 1] = a - b;
  }
  const float2 neg = make_float2(-1.0f, -1.0f);
#pragma unroll
  for (int h = 2; h < C; h <<= 1)
#pragma unroll
    for (int i = 0; i < C; i += 2)
      if ((i & h) == 0) {
        const float2 a = make_float2(x[i], x[i + 1]), b = make_float2(x[i + h], x[i + h + 1]);
        const float2 u = add2(a, b), v = fma2(b, neg, a);
        x[i] = u.x, x[i + 1] = u.y;
        x[i + h] = v.x, x[i + h + 1] = v.y;
      }
}

// mbar_wait for waits that are usually short: some polls before the clock is read.
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t parity, uint32_t limit_ms) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .u32 i;\n mov.u32 i, 0;\n"
      "POLL:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra DONE;\n"
      " add.u32 i, i, 1;\n setp.lt.u32 q, i, 256;\n @q bra POLL;\n"
      "DONE:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  if (done) return true;
  return mbar_wait(bar, parity, limit_ms);
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}

template <int D, int KB, int VB>
__global__ void __launch_bounds__(kTilesThreads, 1) attend_tiles_kernel(const AttendParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  using C = TilesCfg<D, KB, VB>;
  constexpr int N = C::N, NI = C::NI, PART = C::PART;
  constexpr int KPACK = D * KB / 8, VPACK = D * VB / 8;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* q_s = smem;                                   // [row tile][part][64-column blocks]
  uint8_t* ring_s = smem + C::QBYTES;
  uint8_t* lut = smem + C::OPER;
  float* norm_s = (float*)(lut + C::LUT);                // [buffer][K, V][N]
  TilesMisc* ms = (TilesMisc*)(lut + C::LUT + C::NORMS);
  float* part_s = (float*)smem;                          // [slot][row][PART], at the end
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = (int)cluster.num_blocks(), split = (int)cluster.block_rank();
  const AttendItem item = attend_item<true>(p, ctas);
  const int b = item.b, kvh = item.kvh, G = p.group;

  const AttendSeq sq = attend_seq(p, b, tid == 0 && split == 0 && kvh == 0 && item.tile == 0);
  const int tile_rows = p.tile_rows;                     // kTileRows, or twice that (kTwoTiles)
  const int r0 = item.tile * tile_rows;
  const int rows = min(tile_rows, sq.n_q * G - r0);
  if (rows <= 0) return;                                 // the whole cluster
  const int p0 = sq.len - sq.n_q;
  const int pos_first = p0 + r0 / G, pos_last = p0 + (r0 + rows - 1) / G;
  const AttendSpan span = attend_span(p, pos_first, pos_last, kBlockSize);
  const int steps = span.count();
  const int all_tiles = (steps + C::PPT - 1) / C::PPT;
  const int k_begin = (int)((int64_t)all_tiles * split / ctas);
  const int tiles = (int)((int64_t)all_tiles * (split + 1) / ctas) - k_begin;
  const bool two = C::kTwoTiles && rows > kTileRows;     // two row tiles, else key tiles alternate
  // tiles of slot j, and its i-th
  auto slot_tiles = [&](int j) { return two || C::kOneO ? (C::kOneO && j ? 0 : tiles) : (tiles + 1 - j) / 2; };
  auto slot_tile = [&](int j, int i) { return two || C::kOneO ? i : 2 * i + j; };

  if (smem_u32(smem) & 1023u) {                          // the same in every CTA of the kernel
    if (tid == 0) report_error(p.err, TQ_DEVERR_LAYOUT);
    return;
  }
  // One thread issues the MMAs of a slot, in the order P V (n - ahead), Q K (n); a shared O' has
  // one thread for all.
  constexpr int kIssuers = C::kOneO ? 1 : 2;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < 2; ++j) {
        mbar_init(&ms->s_full[i][j], 1);
        mbar_init(&ms->p_ready[i][j], 4);                // a warp's arrival each
      }
      mbar_init(&ms->pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&ms->norm_full[i], kDequantWarps);
    for (int i = 0; i < C::RING; ++i) {
      mbar_init(&ms->ring_full[i], kDequantWarps);
      mbar_init(&ms->ring_empty[i], two ? 2 : 1);
    }
    mbar_init(&ms->o_done, kIssuers);
    mbar_init(&ms->q_ready, 8);                          // the softmax warps
    ms->best = ~0u;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc(&ms->tmem, 512);
  if (warp == 13)
    for (int i = lane; i < D / 2; i += 32)
      ((uint32_t*)ms->flip)[i] = (sign_mask_at(p.sign_seed, 2 * i) >> 16) | sign_mask_at(p.sign_seed, 2 * i + 1);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem;
  const int srow = tid & (kTileRows - 1);                // a softmax thread's row in its slot
  const int myrow = two && warp < 8 ? (warp >> 2) * kTileRows + srow : srow;
  float qs = 0.f;                                        // |q'| |scale| log2(e) of the row
  float ak = 1.0f;                                       // the factor of the key centroids
  float* qs_s = C::kOneO ? (float*)(ring_s + (C::RING - 1) * C::STAGE) : norm_s + 2 * N;
  // q' of the rows, a group of lanes each: sign flips, FWHT, 1/sqrt(D), to unit length in fp16
  // into the operand; its scale to qs_s
  auto make_q = [&](int w, int warps) {
    const int l = lane % C::LPR;
    const int all = two ? 2 * kTileRows : kTileRows;
    auto load = [&](float (&x)[16], int r) {
      const int t = (r0 + r) / G, g = r0 + r - t * G;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.f;
      if (r < rows)
        group_load<D>(x, p.q, (int64_t)(sq.row0 + t) * p.q_rstride + (int64_t)(kvh * G + g) * p.q_hstride,
                      p.q_dtype, p.q_vec, l);
    };
    float next[16];
    load(next, w * C::RPI + lane / C::LPR);
#pragma unroll 1
    for (int rb = w * C::RPI; rb < all; rb += warps * C::RPI) {
      const int r = rb + lane / C::LPR;
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = next[i];
      load(next, rb + warps * C::RPI < all ? r + warps * C::RPI : rows);
      group_flip<D>(x, ms->flip, l);
      group_fwht<D>(x, l);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int m = 1; m < C::LPR; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
      const float nrm = sqrtf(ss), inv = nrm > 0.f ? copysignf(1.0f / nrm, p.scale_log2) : 0.f;
      uint8_t* qt = q_s + (r / kTileRows) * C::QTILE;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t at = sw128_offset(r % kTileRows, group_coord<D>(l, j), kTileRows);
        const float a = x[4 * j] * inv, b = x[4 * j + 1] * inv, c = x[4 * j + 2] * inv, d = x[4 * j + 3] * inv;
        *(uint2*)(qt + at) = make_uint2(pack_half2(a, b), pack_half2(c, d));
      }
      if (l == 0) qs_s[r] = nrm * inv_sqrt_dim<D>() * fabsf(p.scale_log2);
    }
  };
  // 16-bit rows instead come as they are, 16 bytes a lane, into the operand's place, where a
  // thread then turns each row into q' (without shuffles; a CTA's start 20 to 16 thousand clocks)
  const bool raw_q = !C::kOneO && p.q_dtype != TQ_F32;
  auto load_q = [&](int w, int warps) {
    constexpr int CH = D / 8;                            // 16-byte pieces of a row
    const int all = (two ? 2 * kTileRows : kTileRows) * CH, step = warps * 32, i0 = w * 32 + lane;
#pragma unroll 1
    for (int i = i0; i < all; i += 4 * step) {
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = (i + j * step) / CH, c = (i + j * step) % CH;
        v[j] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
          const int t = (r0 + r) / G, g = r0 + r - t * G;
          const uint16_t* at = (const uint16_t*)p.q + (int64_t)(sq.row0 + t) * p.q_rstride +
                               (int64_t)(kvh * G + g) * p.q_hstride + 8 * c;
          if (p.q_vec)
            v[j] = *(const uint4*)at;
          else
            v[j] = make_uint4(at[0] | (uint32_t)at[1] << 16, at[2] | (uint32_t)at[3] << 16,
                              at[4] | (uint32_t)at[5] << 16, at[6] | (uint32_t)at[7] << 16);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = (i + j * step) / CH, c = (i + j * step) % CH;
        if (i + j * step < all)
          *(uint4*)(q_s + r / kTileRows * C::QTILE + sw128_offset(r % kTileRows, 8 * c, kTileRows)) = v[j];
      }
    }
  };
  auto find_factor = [&](int t, int threads) {
    if constexpr (KB <= 4) {
      const unsigned key = centroid_factor_key<KB>(p.kc, t, threads);
      if (lane == 0) atomicMin(&ms->best, key);
    }
  };
  if constexpr (C::kOneO) {
    // D = 256: a thread cannot hold a row; every warp takes rows, then the tables
    find_factor(tid, kTilesThreads);
    make_q(warp, kTilesWarps);
    __syncthreads();                                     // the best factors are known
    if (KB <= 4) ak = centroid_factor(ms->best);
    tiles_lut<KB, 0>(lut, p.kc, ak, warp, kTilesWarps, lane);
    tiles_lut<VB, 1>(lut, p.vc, 1.0f, kTilesWarps - 1 - warp, kTilesWarps, lane);
    if (warp < 8) qs = qs_s[srow] / ak;
    fence_proxy_async_smem();                            // q is read by the tensor cores
    __syncthreads();
  }
  // tensor memory: O' of slot j at columns j D, its scores (and weights) at 256 + 128 j, 64 a buffer
  auto fail = [&]() {
    report_error(p.err, TQ_DEVERR_TIMEOUT);
  };
  // norm buffers
  float* norms = !C::kOneO && !two ? (float*)(q_s + C::QTILE) : norm_s;
  const int nmask = two ? 1 : 3, nshift = two ? 1 : 2;
  // ring position of a tile's K and V
  auto k_at = [&](int k) { return two ? 2 * k : (k == 0 ? 0 : 2 * k - 1); };
  auto v_at = [&](int k) { return two ? 2 * k + 1 : 2 * k + 2; };

  if (warp >= 12) {
    regs_dec<kIssueRegs>();
    if constexpr (!C::kOneO) {
      if (raw_q) load_q(warp - 4, 12);
      else make_q(warp - 4, 12);
      fence_proxy_async_smem();                          // q is read by the tensor cores
      asm volatile("bar.sync 2, 384;" ::: "memory");
    }
    // The whole warp walks the loop, so that descriptors stay in uniform registers; one thread
    // issues.
    const int uwarp = __shfl_sync(0xffffffffu, warp, 0);
    if (uwarp < 12 + kIssuers && tiles > 0) {
      const bool leader = elect_one();
      const int slot = uwarp - 12, items = slot_tiles(slot) * C::H;
      const uint32_t acc = tmem + slot * D, s_at = tmem + 256 + slot * 128;
      const uint64_t q = sw128_desc(smem_u32(q_s) + (two ? slot * C::QTILE : 0));
      const uint32_t ring_at = smem_u32(ring_s);
      bool ok = C::kOneO || tile_wait(&ms->q_ready, 0, p.wait_ms);
      // Q K runs ahead of P V by two items.  A slot that takes every other tile, of one item each,
      // runs one ahead: then it has seen V of its last tile full, and with it every earlier ring
      // position, before it waits for K's, so that no wait skips a phase of its barrier.
      const int ahead = two || C::kOneO || C::H > 1 ? 2 : 1;
      for (int n = 0; n < items + ahead && __all_sync(0xffffffffu, ok); ++n) {
        if (n >= ahead) {                                // P V of item n - ahead
          const int m = n - ahead, at = v_at(slot_tile(slot, m / C::H)), sl = at % C::RING, half = m % C::H;
          ok = (half || tile_wait(&ms->ring_full[sl], (uint32_t)(at / C::RING) & 1u, p.wait_ms)) &&
               tile_wait(&ms->p_ready[slot][m & 1], (uint32_t)(m >> 1) & 1u, p.wait_ms);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
          const uint64_t v = sw128_mn_desc(ring_at + sl * C::STAGE, N * 128) + half * (NI * 8);
          const uint32_t pw = s_at + (m & 1) * 64;
          if (leader) {
#pragma unroll
            for (int ks = 0; ks < NI / 16; ++ks)         // 16 keys: 2048 bytes of each block
              umma_ts_f16(acc, pw + ks * 8, v + ks * 128, f16_idesc(D, true), (ks > 0 || m > 0) ? 1u : 0u);
            umma_commit(&ms->pv_done[slot]);
            if (half == C::H - 1) umma_commit(&ms->ring_empty[sl]);
          }
        }
        if (n < items) {                                 // Q K of item n
          const int at = k_at(slot_tile(slot, n / C::H)), sl = at % C::RING, half = n % C::H;
          ok = half || tile_wait(&ms->ring_full[sl], (uint32_t)(at / C::RING) & 1u, p.wait_ms);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
          const uint64_t kd = sw128_desc(ring_at + sl * C::STAGE) + half * (NI * 8);
          if (leader) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {        // 16 coordinates: 32 bytes of a block
              const uint64_t qd = q + (ks >> 2) * (kTileRows * 8) + (ks & 3) * 2;
              const uint64_t ko = kd + (ks >> 2) * (N * 8) + (ks & 3) * 2;
              const uint32_t to = s_at + (n & 1) * 64;
              umma_bf16(to, qd, ko, f16_idesc(NI, false), ks > 0 ? 1u : 0u);
              if constexpr (C::KPARTS == 2)
                umma_bf16(to, qd, ko + C::KPART * (N * 8), f16_idesc(NI, false), 1u);
            }
            umma_commit(&ms->s_full[slot][n & 1]);
            if (half == C::H - 1) umma_commit(&ms->ring_empty[sl]);
          }
        }
      }
      __syncwarp();
      if (leader) umma_commit(&ms->o_done);
      ok = tile_wait(&ms->o_done, 0, p.wait_ms) && ok;   // what was issued is complete
      if (!ok && leader) fail();
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ---- codes to operand tiles ----
    regs_dec<kDequantRegs>();
    const int w = warp - 8;
    const int l = lane % C::LPR, rsub = lane / C::LPR;
    const int rbase = w * (N / kDequantWarps) + rsub;                // this lane's rows: rbase + i RPI
    const int low_last = p.window > 0 ? (int)max((int64_t)0, (int64_t)pos_last - p.window + 1) : 0;
    const int64_t head = (int64_t)kvh * p.slot_stride;
    // The pages of this warp's rows, WP a tile: a lane holds one table entry of a window of TW
    // tiles (and one of the next window), so that no entry is waited for.
    constexpr int NW = N / kDequantWarps;                // a warp's rows of a tile
    constexpr int WP = NW > kBlockSize ? NW / kBlockSize : 1, TW = 32 / WP;
    auto entry = [&](int k) -> int32_t {                 // this lane's entry of the window at tile k
      const int step = (k_begin + k + lane / WP) * C::PPT + w * NW / kBlockSize + lane % WP;
      if (k + lane / WP >= tiles || step >= steps) return -1;
      const int32_t id = p.block_table[(int64_t)b * p.bt_stride + span.at(step)];
      if (id >= 0 && id < p.num_blocks) return id;
      report_error(p.err, TQ_DEVERR_BLOCK_RANGE);
      return -1;
    };
    int32_t window = entry(0), window_next = entry(TW);
    struct Pages {
      int32_t id[WP];
    };
    auto fetch = [&](int k) {                            // of tiles 0, 1, 2, ... in turn
      if (k > 0 && k % TW == 0) {
        window = window_next;
        window_next = entry(k + TW);
      }
      Pages r;
#pragma unroll
      for (int j = 0; j < WP; ++j) r.id[j] = __shfl_sync(0xffffffffu, window, (k % TW) * WP + j);
      return r;
    };
    auto base_of = [&](int32_t id) -> const uint8_t* {
      return id < 0 ? nullptr : p.pages + (int64_t)id * p.blk_stride + head;
    };
    // Rows i of a unit from its pages, in turn (at: this lane's next row)
    constexpr int IPP = C::IT / WP;                      // rows of a lane in a page
    const int64_t row_step = C::RPI * p.row_stride;
    const int64_t lane_at = (int64_t)(rbase % kBlockSize) * p.row_stride;
    auto load_rows = [&](auto IV, auto& raw, int i, const Pages& from, const uint8_t*& at) {
      constexpr bool V = decltype(IV)::value;
      if (i % IPP == 0) {
        at = base_of(from.id[i / IPP]);
        if (at != nullptr) at += lane_at + (V ? p.k_region : 0);
      }
      uint32_t r[4] = {0u, 0u, 0u, 0u};
      if (at != nullptr) {
        if constexpr (V) Codes16<VB>::load(r, at, l);
        else Codes16<KB>::load(r, at, l);
        at += row_step;
      }
#pragma unroll
      for (int j = 0; j < (V ? C::VW : C::KW); ++j) raw[i][j] = r[j];
    };
    auto look = [&](uint32_t a) { return *(const uint32_t*)(lut + a); };
    const uint32_t lk = 4u * lane, lv = 128u + 4u * lane;
    // 16 codes to 16 halves (8 bits: and to what these leave)
    auto look_up = [&](auto IV, const auto& raw, int i, uint32_t (&h)[8], uint32_t (&rest)[8]) {
      constexpr bool V = decltype(IV)::value;
      constexpr int BITS = V ? VB : KB, W = V ? C::VW : C::KW;
      const uint32_t off = V ? lv : lk;
      uint32_t r[W];
#pragma unroll
      for (int j = 0; j < W; ++j) r[j] = raw[i][j];
      static_for<8>([&](auto JI) {
        constexpr int j = decltype(JI)::value;
        if constexpr (BITS <= 4) {
          h[j] = look(lut_addr<2 * j * BITS, 2 * BITS>(r, off));
        } else {
          const uint32_t a = look(lut_addr<2 * j * BITS, BITS>(r, off));
          const uint32_t b = look(lut_addr<(2 * j + 1) * BITS, BITS>(r, off));
          h[j] = __byte_perm(a, b, 0x5410);
          rest[j] = __byte_perm(a, b, 0x7632);
        }
      });
    };
    // ... stored as two 16-byte chunks of the row; the order in which a lane stores its two
    // keeps 8 lanes on 8 chunks
    auto store_row = [&](const uint32_t (&h)[8], int i, uint8_t* stage) {
      const int row = rbase + i * C::RPI;
      uint8_t* dst = stage + (l >> 2) * (N * 128) + row * 128;
      const int c0 = 2 * (l & 3), odd = D > 64 ? (l >> 2) & 1 : 0;
      const uint4 v0 = make_uint4(h[0], h[1], h[2], h[3]), v1 = make_uint4(h[4], h[5], h[6], h[7]);
      *(uint4*)(dst + (((c0 + odd) ^ (row & 7)) << 4)) = odd ? v1 : v0;
      *(uint4*)(dst + (((c0 + 1 - odd) ^ (row & 7)) << 4)) = odd ? v0 : v1;
    };
    // ... times the norm of the row (mul: this lane's row's, twice)
    auto scale_row = [&](uint32_t (&h)[8], uint32_t mul, int i) {
      const uint32_t m = __shfl_sync(0xffffffffu, mul, i * C::RPI + rsub);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __half2 x = __hmul2(*(const __half2*)&h[j], *(const __half2*)&m);
        h[j] = *(const uint32_t*)&x;
      }
    };
    using KI = std::false_type;
    using VI = std::true_type;
    // norms of row w N / 4 + lane, one tile ahead
    const int nrow = w * (N / kDequantWarps) + lane;
    float nk = 0.f, nv = 0.f;
    int first = -1;
    auto load_norms = [&](int k, const Pages& from) {
      nk = nv = 0.f;
      first = -1;
      const uint8_t* pg = base_of(from.id[WP > 1 ? lane / kBlockSize : 0]);
      if (lane < N / kDequantWarps && pg != nullptr) {
        first = span.at((k_begin + k) * C::PPT + nrow / kBlockSize) * kBlockSize;
        const uint8_t* sl = pg + (nrow % kBlockSize) * p.row_stride;
        nk = *(const float*)(sl + KPACK);
        nv = *(const float*)(sl + p.k_region + VPACK);
      }
    };
    // Norms and facts of tile k for the softmax warps; vmul: the factor of this lane's row in the
    // V operand, twice (1 where the softmax applies the norms).
    uint32_t vmul = 0x3c003c00u;
    auto publish = [&](int k) {
      // the second buffer holds the scales of q until they are read
      if (!C::kOneO && k == 1) tile_wait(&ms->q_ready, 0, p.wait_ms);
      const int buf = k & nmask, mb = k & 1;
      bool ok = true;
      int vmax = -100, vmin = 1000;
      if (lane < N / kDequantWarps) {
        norms[buf * 2 * N + nrow] = nk;
        norms[buf * 2 * N + N + nrow] = nv;
        if (nrow % kBlockSize == 0) ms->tok[buf][nrow / kBlockSize] = first;
        const int tok = first + nrow % kBlockSize;
        ok = first >= 0 && tok <= pos_first && (tok >= low_last || tok < p.sinks) && isfinite(nk) &&
             isfinite(nv);
        vmax = (int)ceilf(fmaxf(log2_bound(fabsf(nv)), -100.0f));
        if (nv != 0.f) vmin = vmax;
      }
      vmax = __reduce_max_sync(0xffffffffu, vmax);
      vmin = __reduce_min_sync(0xffffffffu, vmin);
      ok = __all_sync(0xffffffffu, ok);
      if (lane == 0) ms->meta[mb][w] = TileMeta{vmax, vmin, ok ? 1 : 0};
      asm volatile("bar.sync 1, 128;" ::: "memory");     // the dequantizing warps
#pragma unroll
      for (int i = 0; i < kDequantWarps; ++i) {
        const TileMeta m = ms->meta[mb][i];
        ok = ok && m.plain;
        vmax = max(vmax, m.vmax);
        vmin = min(vmin, m.vmin);
      }
      ok = ok && vmax - vmin <= 8 && abs(vmax) < 60;
      const float v = ok ? nv * __int_as_float((127 - vmax) << 23) : 1.0f;
      vmul = pack_half2(v, v);
      if (w == 0 && lane == 0) ms->info[buf] = TileInfo{ok ? 1 : 0, (float)vmax};
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->norm_full[buf]);
    };
    auto free_stage = [&](int at) {                      // wait until ring position `at` may be written
      return at < C::RING ||
             tile_wait(&ms->ring_empty[at % C::RING], (uint32_t)(at / C::RING - 1) & 1u, p.wait_ms);
    };
    auto load_all = [&](auto IV, auto& raw, const Pages& from) {
      const uint8_t* at = nullptr;
#pragma unroll
      for (int i = 0; i < C::IT; ++i) load_rows(IV, raw, i, from, at);
    };
    // The codes in raw to ring position pos, some rows' lookups in flight; as each is used its
    // registers take the codes of a coming unit (kind INV, from these pages).
    auto produce = [&](auto IV, auto& raw, auto INV, auto& coming, int pos, uint32_t mul, bool more,
                       const Pages& next) {
      constexpr bool V = decltype(IV)::value;
      uint8_t* stage = ring_s + (pos % C::RING) * C::STAGE;
      const uint8_t* at = nullptr;
      constexpr bool REST = !V && C::KPARTS == 2;
      constexpr int U = C::IT % 4 == 0 && !REST ? 4 : C::IT % 2 == 0 ? 2 : 1;   // rows in flight
#pragma unroll
      for (int i = 0; i < C::IT; i += U) {
        uint32_t h[U][8], rest[U][8];
#pragma unroll
        for (int u = 0; u < U; ++u) look_up(IV, raw, i + u, h[u], rest[u]);
        if constexpr (V) {
#pragma unroll
          for (int u = 0; u < U; ++u) scale_row(h[u], mul, i + u);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) store_row(h[u], i + u, stage);
        if constexpr (REST) {
#pragma unroll
          for (int u = 0; u < U; ++u) store_row(rest[u], i + u, stage + C::KPART * (N * 128));
        }
        if (more) {
#pragma unroll
          for (int u = 0; u < U; ++u) load_rows(INV, coming, i + u, next, at);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->ring_full[pos % C::RING]);
    };
    constexpr int RW = C::KW > C::VW ? C::KW : C::VW;
    uint32_t raw_k[C::IT][C::kDeep ? C::KW : RW];
    uint32_t raw_x[C::IT][C::kDeep ? C::VW : 1];
    auto& raw_v = [&]() -> auto& {
      if constexpr (C::kDeep) return raw_x;
      else return raw_k;
    }();
    bool ok = true;
    if (tiles > 0) {
      // pages of tiles k, k + 1, k + 2 (as far as they are needed)
      Pages b0 = fetch(0), b1 = b0, b2 = b0;
      load_norms(0, b0);
      load_all(KI{}, raw_k, b0);
      if constexpr (C::kDeep) load_all(VI{}, raw_v, b0);
      if constexpr (!C::kOneO) {                         // the tables, while these come in
        tiles_lut<VB, 1>(lut, p.vc, 1.0f, w, kDequantWarps, lane);
        find_factor(tid - 256, 128);
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (KB <= 4) ak = centroid_factor(ms->best);
        if (tid == 256) ms->alpha = ak;                  // read past norm_full
        tiles_lut<KB, 0>(lut, p.kc, ak, w, kDequantWarps, lane);
        asm volatile("bar.sync 1, 128;" ::: "memory");
      }
      if (two) {                                         // K(0), V(0), K(1), V(1), ...
        for (int k = 0; k < tiles; ++k) {
          const bool more = k + 1 < tiles;
          // the norms' buffer: item k - 2 of both slots is past its P V when V(k - 2)'s stage,
          // which K(k) takes, is free
          ok = free_stage(k_at(k));
          if (!ok) break;
          publish(k);
          if (more) {
            b1 = fetch(k + 1);
            load_norms(k + 1, b1);
          }
          if constexpr (C::kDeep) produce(KI{}, raw_k, KI{}, raw_k, k_at(k), 0u, more, b1);
          else produce(KI{}, raw_k, VI{}, raw_v, k_at(k), 0u, true, b0);
          ok = free_stage(v_at(k));
          if (!ok) break;
          if constexpr (C::kDeep) produce(VI{}, raw_v, VI{}, raw_v, v_at(k), vmul, more, b1);
          else produce(VI{}, raw_v, KI{}, raw_k, v_at(k), vmul, more, b1);
          b0 = b1;
        }
      } else {                                           // K(0), K(1), V(0), K(2), V(1), ...
        publish(0);
        uint32_t vmul_now = vmul;
        if (tiles > 1) {
          b1 = fetch(1);
          load_norms(1, b1);
        }
        produce(KI{}, raw_k, KI{}, raw_k, k_at(0), 0u, tiles > 1, b1);
        if (!C::kDeep && tiles == 1) load_all(VI{}, raw_v, b0);
        for (int k = 0; k < tiles; ++k) {
          vmul_now = vmul;
          const bool more1 = k + 1 < tiles, more2 = k + 2 < tiles;
          if (more2) b2 = fetch(k + 2);
          if (more1) {
            ok = free_stage(k_at(k + 1));
            if (!ok) break;
            // the norms' buffer: tile k - 3 is past its P V (its V's stage was K(k)'s)
            publish(k + 1);
            if (more2) load_norms(k + 2, b2);
            if constexpr (C::kDeep) produce(KI{}, raw_k, KI{}, raw_k, k_at(k + 1), 0u, more2, b2);
            else produce(KI{}, raw_k, VI{}, raw_v, k_at(k + 1), 0u, true, b0);
          }
          ok = free_stage(v_at(k));
          if (!ok) break;
          if constexpr (C::kDeep) {
            produce(VI{}, raw_v, VI{}, raw_v, v_at(k), vmul_now, more1, b1);
          } else {
            produce(VI{}, raw_v, KI{}, raw_k, v_at(k), vmul_now, more2, b2);
            if (more1 && !more2) load_all(VI{}, raw_v, b1);   // no K tile is left to fetch it under
          }
          b0 = b1;
          b1 = b2;
        }
      }
    }
    if (!ok) fail();
  } else {
    // ---- softmax: a thread = a row of slot warp / 4 ----
    regs_inc<kSoftmaxRegs>();
    const int slot = warp >> 2;
    if constexpr (!C::kOneO) {
      if (raw_q) {
        load_q(warp, 12);
        asm volatile("bar.sync 2, 384;" ::: "memory");   // the warps that loaded q
        if (two || slot == 0) {
          // q' of this thread's row, in place: sign flips, FWHT, 1/sqrt(D), to unit length in fp16
          uint8_t* qt = q_s + (two ? slot : 0) * C::QTILE;
          float x[D];
#pragma unroll
          for (int c = 0; c < D; c += 8) {
            const uint4 v = *(const uint4*)(qt + sw128_offset(srow, c, kTileRows));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            const uint4 f = ms->flip[c / 8];
            const uint32_t m[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t u = w[i] ^ m[i];
              if (p.q_dtype == TQ_BF16) {
                x[c + 2 * i] = __uint_as_float(u << 16);
                x[c + 2 * i + 1] = __uint_as_float(u & 0xffff0000u);
              } else {
                const float2 h = __half22float2(*(const __half2*)&u);
                x[c + 2 * i] = h.x;
                x[c + 2 * i + 1] = h.y;
              }
            }
          }
          thread_fwht<D>(x);
          float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int i = 0; i < D; i += 2) {
            const float2 v = make_float2(x[i], x[i + 1]);
            s2[i / 2 % 2] = fma2(v, v, s2[i / 2 % 2]);
          }
          const float nrm = sqrtf((s2[0].x + s2[1].x) + (s2[0].y + s2[1].y));
          const float inv = nrm > 0.f ? copysignf(1.0f / nrm, p.scale_log2) : 0.f;
          const float2 i2 = make_float2(inv, inv);
#pragma unroll
          for (int c = 0; c < D; c += 8) {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = mul2(make_float2(x[c + 2 * i], x[c + 2 * i + 1]), i2);
              h[i] = pack_half2(v.x, v.y);
            }
            *(uint4*)(qt + sw128_offset(srow, c, kTileRows)) = make_uint4(h[0], h[1], h[2], h[3]);
          }
          qs_s[myrow] = nrm * inv_sqrt_dim<D>() * fabsf(p.scale_log2);
        }
        asm volatile("bar.sync 3, 256;" ::: "memory");   // the softmax warps
      } else {
        make_q(warp, 12);
        asm volatile("bar.sync 2, 384;" ::: "memory");   // the warps that made q
      }
      qs = qs_s[myrow];
      fence_proxy_async_smem();                          // q is read by the tensor cores
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->q_ready);
    }
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // this warp's quarter of tensor memory
    float M = -INFINITY, sum = 0.f;
    const int pos = myrow < rows ? p0 + (r0 + myrow) / G : -1;
    const int low = p.window > 0 ? (int)max((int64_t)0, (int64_t)pos - p.window + 1) : 0;
    const uint32_t o_at = tmem + lanes + slot * D;
    const int items = slot_tiles(slot) * C::H;
    bool ok = true;
    for (int n = 0; n < items; ++n) {
      const int k = slot_tile(slot, n / C::H), nb = k & nmask, half = n % C::H;
      const uint32_t s_at = tmem + lanes + 256 + slot * 128 + (n & 1) * 64;
      ok = (half || tile_wait(&ms->norm_full[nb], (uint32_t)(k >> nshift) & 1u, p.wait_ms)) &&
           tile_wait(&ms->s_full[slot][n & 1], (uint32_t)(n >> 1) & 1u, p.wait_ms);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      if (!C::kOneO && n == 0) qs /= ms->alpha;
      tc_fence_after();
      float s[NI];
      const float* nks = norms + nb * 2 * N + half * NI;
      const float* nvs = nks + N;
      const TileInfo info = ms->info[nb];
      const bool plain = info.plain;
      // x of 16 columns at c, key by key: norms and masks here (a tile that is not plain)
      auto masked = [&](int c, float (&x)[16]) {
        tmem_ld16_nowait(s_at + c, x);
        const int first = ms->tok[nb][(half * NI + c) / kBlockSize];
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int tok = first + i;
          const bool see = first >= 0 && tok <= pos && (tok >= low || tok < p.sinks);
          x[i] = see ? x[i] * nks[c + i] * qs : -INFINITY;
        }
      };
      float z = -INFINITY;
      if (plain) {
        // the first half's maxima while the second half is read
        constexpr int HL = NI >= 32 ? NI / 2 : NI;
        float zz[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < HL; c += 16) tmem_ld16_nowait(s_at + c, s + c);
#pragma unroll
        for (int h = 0; h < NI; h += HL) {
          tmem_wait_ld();
          if (h + HL < NI) {
#pragma unroll
            for (int c = h + HL; c < h + 2 * HL; c += 16) tmem_ld16_nowait(s_at + c, s + c);
          }
#pragma unroll
          for (int c = h; c < h + HL; c += 8) {
#pragma unroll
            for (int i = c; i < c + 8; i += 4) {
              const float4 f = *(const float4*)(nks + i);
              const float2 u = mul2(make_float2(s[i], s[i + 1]), make_float2(f.x, f.y));
              const float2 v = mul2(make_float2(s[i + 2], s[i + 3]), make_float2(f.z, f.w));
              s[i] = u.x, s[i + 1] = u.y, s[i + 2] = v.x, s[i + 3] = v.y;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) zz[j] = max3(zz[j], s[c + 2 * j], s[c + 2 * j + 1]);
          }
        }
        z = fmaf(max3(fmaxf(zz[0], zz[1]), zz[2], zz[3]), qs, info.ev);
      } else {
#pragma unroll 1
        for (int c = 0; c < NI; c += 16) {
          float x[16];
          masked(c, x);
#pragma unroll
          for (int i = 0; i < 16; ++i) z = fmaxf(z, x[i] + fmaxf(log2_bound(nvs[c + i]), -100.0f));
        }
      }
      const bool raise = z > M + kLazyRescale;
      if (__any_sync(0xffffffffu, raise)) {
        const float to = raise ? z : M;
        const float f = M == -INFINITY ? 0.f : exp2f(M - to);
        sum *= f;
        M = to;
        if (n > 0) {                                     // until P V of the last item is done
          ok = tile_wait(&ms->pv_done[slot], (uint32_t)(n - 1) & 1u, p.wait_ms);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            float o[16];
            tmem_ld16_nowait(o_at + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= f;
            tmem_st8(o_at + c, (const uint32_t*)o);
            tmem_st8(o_at + c + 8, (const uint32_t*)o + 8);
          }
        }
      }
      const float ref = M == -INFINITY ? 0.f : M;
      uint32_t pk[8];
      if (plain) {
        // P = 2^(x + ev - M): the norms over 2^ev are in the operand
        const float shift = info.ev - ref;
        const float2 q2 = make_float2(qs, qs), m2 = make_float2(shift, shift);
        float2 l0 = make_float2(0.f, 0.f), l1 = l0, l2 = l0, l3 = l0;
#pragma unroll
        for (int c = 0; c < NI; c += 8) {
          float2 u[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) u[j] = fma2(make_float2(s[c + 2 * j], s[c + 2 * j + 1]), q2, m2);
#pragma unroll
          for (int j = 0; j < 4; ++j) u[j] = make_float2(ex2_approx(u[j].x), ex2_approx(u[j].y));
          l0 = add2(l0, u[0]);
          l1 = add2(l1, u[1]);
          l2 = add2(l2, u[2]);
          l3 = add2(l3, u[3]);
#pragma unroll
          for (int j = 0; j < 4; ++j) pk[c / 2 % 8 + j] = pack_half2(u[j].x, u[j].y);
          if (c % 16 == 8) tmem_st8(s_at + c / 16 * 8, pk);
        }
        l0 = add2(add2(l0, l1), add2(l2, l3));
        const float part = l0.x + l0.y;
        sum = fmaf(part, __int_as_float((127 - (int)info.ev) << 23), sum);
      } else {
#pragma unroll 1
        for (int c = 0; c < NI; c += 16) {                // P of a chunk lies over scores already read
          float x[16];
          masked(c, x);
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float w0 = ex2_approx(x[i] - ref), w1 = ex2_approx(x[i + 1] - ref);
            sum += w0 + w1;
            pk[i / 2] = pack_half2(x[i] == -INFINITY ? 0.f : w0 * nvs[c + i],
                                   x[i + 1] == -INFINITY ? 0.f : w1 * nvs[c + i + 1]);
          }
          tmem_st8(s_at + c / 2, pk);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->p_ready[slot][n & 1]);
    }
    if (ok && tiles > 0) ok = tile_wait(&ms->o_done, 0, p.wait_ms);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) fail();
    // every other reader of the operands is done: their place takes the partials
    tc_fence_after();
    if (!(C::kOneO && slot)) {
      float* rec = part_s + (slot * kTileRows + srow) * PART;
      // the stages of the inverse rotation inside a quarter of the row go here, before the join
      // (which is linear), the two others after it
      constexpr int Q = D / 4;
#pragma unroll 1
      for (int c = 0; c < D; c += Q) {
        float o[Q];
        if (items > 0 && ok) {
#pragma unroll
          for (int i = 0; i < Q; i += 16) tmem_ld16_nowait(o_at + c + i, o + i);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < Q; ++i) o[i] = 0.f;
        }
        thread_fwht<Q>(o);
#pragma unroll
        for (int i = 0; i < Q; i += 4) *(float4*)(rec + c + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
      }
      // a sum that is not a number must survive the join, which drops empty partials
      rec[D] = sum != sum && M == -INFINITY ? -3e38f : M;
      rec[D + 1] = sum;
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
  if (ctas > 1) cluster.sync();
  // row r is joined by CTA r % ctas of the cluster, by a group of lanes; records: CTAs x slots
  const int recs = two || C::kOneO ? 1 : 2, l = lane % C::LPR;
#pragma unroll 1
  for (int rb = warp * C::RPI; rb * ctas < rows; rb += kTilesWarps * C::RPI) {
    const int r = (rb + lane / C::LPR) * ctas + split, t = (r0 + r) / G, g = r0 + r - t * G;
    float o[16], sum = 0.f, top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.f;
    if (r < rows) {
      auto record = [&](int i) -> const float* {
        const float* from = part_s + ((recs == 2 ? (i & 1) * kTileRows : 0) + r) * PART;
        return ctas > 1 ? cluster.map_shared_rank(from, recs == 2 ? i >> 1 : i) : from;
      };
      if (ctas * recs > 1) {
#pragma unroll 1
        for (int i = 0; i < ctas * recs; ++i) top = fmaxf(top, record(i)[D]);
      }
#pragma unroll 1
      for (int i = 0; i < ctas * recs; ++i) {
        const float* from = record(i);
        const float m = from[D], w = ctas * recs == 1 ? 1.0f : m == -INFINITY ? 0.f : exp2f(m - top);
        sum = fmaf(w, from[D + 1], sum);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 v = *(const float4*)(from + group_coord<D>(l, j));
          o[4 * j] = fmaf(w, v.x, o[4 * j]);
          o[4 * j + 1] = fmaf(w, v.y, o[4 * j + 1]);
          o[4 * j + 2] = fmaf(w, v.z, o[4 * j + 2]);
          o[4 * j + 3] = fmaf(w, v.w, o[4 * j + 3]);
        }
      }
    }
    const float inv = sum == 0.f ? 0.f : inv_sqrt_dim<D>() / sum;   // a row that sees nothing: 0
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= inv;
#pragma unroll
    for (int h = 4; h < 16; h <<= 1)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if ((i & h) == 0) {
          const float a = o[i], c = o[i + h];
          o[i] = a + c;
          o[i + h] = a - c;
        }
    group_flip<D>(o, ms->flip, l);
    if (r < rows)
      group_store<D>(o, p.out, (int64_t)(sq.row0 + t) * p.o_rstride + (int64_t)(kvh * G + g) * p.o_hstride,
                     p.out_dtype, p.out_vec, l);
  }
  if (ctas > 1) cluster.sync();              // no CTA leaves while its partials may be read
}

}  // namespace tq
