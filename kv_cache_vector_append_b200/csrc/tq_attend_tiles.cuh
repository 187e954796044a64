// tq_attend_tiles.cuh -- attention over packed slots for many query rows a KV head (chunks of
// new tokens), on the tcgen05 tensor cores.
//
// Math.  As in tq_attend_rows.cuh, in the rotated domain: S = q^ C~^T on the codes' centroids,
// x = S nK |q'| scale log2(e) per (row, key), P = 2^(x - M) nV in fp16, O' += P V~,
// o = R^T O' / l.  Norms never enter an operand, so keys and values keep the precision of
// their centroids; statistics and accumulators are fp32.  The centroids are scaled by a factor
// in [1, 2) under which their fp16 roundings are smallest (a search over 512 factors; exact to
// about 2^-13 of the largest), which leaves with the scales of the rows.
//   PREC (out is f16 or f32): q^ = hi + lo (two fp16), and 8-bit keys too, so that scores are
//   right to about 2^-20; bf16 outputs take the fp16 operands alone (2^-12).
// M >= max(x + log2 nV): a tile whose V norms lie within 2^8 of each other and which every row
// sees takes the tile's largest norm for all of them, any other the bound key by key, masks
// included: what a row does not see never touches it.
//
// Layout.  A CTA holds two slots of 128 rows x N keys: two row tiles that share every key tile
// (256 rows), or, with 128 rows or in PREC, one row tile whose key tiles alternate between the
// slots, each with its own (M, l, O'), joined at the end.  (D = 256: one O' fills the tensor
// memory; one softmax warpgroup, two score buffers.)  Warps 0-7 are the slots' softmax
// warpgroups (a thread = a row: scores from tensor memory, P back over them), warps 8-11 turn
// packed codes into fp16 tiles in shared memory (lookups of code pairs, one 256-byte row an
// entry, so that 32 lanes hit 32 banks; the next tile's codes are already on their way into
// registers), warp 12 issues the MMAs: P V of an item, then Q K of the slot's next one, so that
// one slot's softmax runs under the other's MMAs.  Both operand tiles are rows of 64 columns with
// the 128-byte swizzle: K-major for Q K, MN-major for P V, the same bytes.  A cluster of CTAs
// may split the keys; partials are joined over distributed shared memory as in the rows kernel.
//
// Bound: exponentials (16 a clock an SM) and MMAs (8192 flop a clock), which take equally long
// at D = 128; next shared memory (operands, lookups, tiles).
#pragma once

#include <cooperative_groups.h>

#include "tq_append_dense.cuh"
#include "tq_attend.cuh"

namespace tq {

constexpr int kTileRows = 128;             // rows of a slot (the MMA's M)
constexpr int kTilesThreads = 512;
constexpr int kTilesMaxCtas = 8;
// registers a thread of the softmax, dequantizing and issuing warpgroups, from kTilesRegs each
constexpr int kTilesRegs = 128, kSoftmaxRegs = 168, kDequantRegs = 104, kIssueRegs = 72;
static_assert(2 * kSoftmaxRegs + kDequantRegs + kIssueRegs <= 4 * kTilesRegs, "registers of a CTA");

template <int D, int KB, int VB, bool PREC>
struct TilesCfg {
  static constexpr bool kTwoTiles = !PREC && D <= 128;   // may hold two row tiles
  static constexpr bool kOneO = D == 256;                // one accumulator, one softmax warpgroup
  static constexpr bool kKeyLo = PREC && KB == 8;
  static constexpr int QPARTS = PREC ? 2 : 1;
  static constexpr int KPARTS = kKeyLo ? 2 : 1;
  // bytes of a ring stage, keys of a tile
  static constexpr int STAGE = D == 64 ? 16384 * KPARTS : (D == 256 && PREC ? 16384 : 32768);
  static constexpr int N = STAGE / (2 * D * KPARTS);
  static constexpr int RING = D == 256 && PREC ? 2 : 3;
  static constexpr int PPT = N / kBlockSize;             // pages a tile
  static constexpr int QTILE = kTileRows * D * 2;        // one part of one row tile
  static constexpr int QBYTES = (kTwoTiles ? 2 : 1) * QPARTS * QTILE;
  static constexpr int PART = D + 4;                     // floats of a row's partial
  static constexpr int STAGING = (kOneO ? 1 : 2) * kTileRows * PART * 4;
  static constexpr int OPER = QBYTES + RING * STAGE > STAGING ? QBYTES + RING * STAGE : STAGING;
  static constexpr int LUT = kLutRow * (lut_entries(KB) > lut_entries(VB) ? lut_entries(KB) : lut_entries(VB));
  static constexpr int NORMS = 2 * N * 2 * 4;
  static constexpr int MISC = 512;
  // more than half an SM: a CTA that holds all of tensor memory has the SM to itself
  static constexpr int RAW = OPER + LUT + NORMS + MISC;
  static constexpr int SMEM = RAW > 120 * 1024 ? RAW : 120 * 1024;
  // dequantization: 16 codes a lane
  static constexpr int LPR = D / 16, RPI = 32 / LPR, IT = N / 4 / RPI;
  static_assert(N % 16 == 0 && N <= 128 && IT >= 1 && N / 4 % RPI == 0, "tile geometry");
  static_assert(SMEM <= 232448, "shared memory");
};

// Per-tile facts, one entry a dequantizing warp (its N / 4 keys).
struct TileMeta {
  float emax, emin;                        // bounds of log2 nV
  int plain;                               // every row of the CTA sees every key, finite norms
};

struct TilesMisc {
  uint64_t s_full[2], p_ready[2], norm_full[2], ring_full[3], ring_empty[3], o_done;
  uint32_t tmem;
  int dead;
  float alpha[2];
  int tok[2][8];                           // first token of a page of the tile; < 0: no page
  TileMeta meta[2][4];
  unsigned long long best[2];
};
static_assert(sizeof(TilesMisc) <= 512, "misc area");

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
// one copy a lane.  BITS <= 4: half2 of a code pair; 8 bits: half2(hi, lo) of a code.
template <int BITS, int HALF>
__device__ __forceinline__ void tiles_lut(uint8_t* lut, const float* c, float alpha, int tid) {
  for (int i = tid; i < lut_entries(BITS) * 32; i += kTilesThreads) {
    const int e = i >> 5, l = i & 31;
    uint32_t v;
    if constexpr (BITS <= 4) {
      v = pack_half2(c[e & ((1 << BITS) - 1)] * alpha, c[e >> BITS] * alpha);
    } else {
      const float hi = __half2float(__float2half_rn(c[e]));
      v = pack_half2(hi, c[e] - hi);
    }
    *(uint32_t*)(lut + e * kLutRow + HALF * 128 + 4 * l) = v;
  }
}
// The factor whose scaled centroids lie nearest to fp16 numbers: 1 + best / 512.
template <int BITS>
__device__ __forceinline__ void tiles_alpha(const float* c, int tid, unsigned long long* best) {
  if constexpr (BITS <= 4) {
    const float a = 1.0f + (float)tid * (1.0f / kTilesThreads);
    float err = 0.f;
    for (int i = 0; i < 1 << BITS; ++i) {
      const float x = c[i] * a, d = __half2float(__float2half_rn(x)) - x;
      err = fmaf(d, d, err);
    }
    unsigned long long key = ((unsigned long long)__float_as_uint(err / (a * a)) << 32) | (unsigned)tid;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, key, o);
      key = other < key ? other : key;
    }
    if ((tid & 31) == 0) atomicMin(best, key);
  }
}

template <int D, int KB, int VB, bool PREC>
__global__ void __launch_bounds__(kTilesThreads, 1) attend_tiles_kernel(const AttendParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  using C = TilesCfg<D, KB, VB, PREC>;
  constexpr int N = C::N, PART = C::PART, E = D / 32;
  constexpr int KPACK = D * KB / 8, VPACK = D * VB / 8;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* q_s = smem;                                   // [row tile][part][64-column blocks]
  uint8_t* ring_s = smem + C::QBYTES;
  uint8_t* lut = smem + C::OPER;
  float* norm_s = (float*)(lut + C::LUT);                // [2][K, V][N]
  TilesMisc* ms = (TilesMisc*)(lut + C::LUT + C::NORMS);
  float* part_s = (float*)smem;                          // [slot][row][PART], at the end
  float* qs_s = (float*)(ring_s + (C::RING - 1) * C::STAGE);   // until the first tiles come
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = (int)cluster.num_blocks(), split = (int)cluster.block_rank();
  const int b = blockIdx.x / ctas, kvh = blockIdx.y, G = p.group;

  const AttendSeq sq = attend_seq(p, b, tid == 0 && split == 0 && kvh == 0 && blockIdx.z == 0);
  // later rows see more keys: they start first
  const int tile_rows = p.tile_rows;                     // kTileRows, or twice that (kTwoTiles)
  const int r0 = ((int)gridDim.z - 1 - (int)blockIdx.z) * tile_rows;
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
  const int items = two ? 2 * tiles : tiles;

  if (smem_u32(smem) & 1023u) {                          // the same in every CTA of the kernel
    if (tid == 0) report_error(p.err, TQ_DEVERR_LAYOUT);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ms->s_full[i], 1);
      mbar_init(&ms->p_ready[i], kTileRows);
      mbar_init(&ms->norm_full[i], 128);
    }
    for (int i = 0; i < C::RING; ++i) {
      mbar_init(&ms->ring_full[i], 128);
      mbar_init(&ms->ring_empty[i], 1);
    }
    mbar_init(&ms->o_done, 1);
    ms->dead = 0;
    ms->best[0] = ms->best[1] = ~0ull;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc(&ms->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  tiles_alpha<KB>(p.kc, tid, &ms->best[0]);
  tiles_alpha<VB>(p.vc, tid, &ms->best[1]);
  // q' of a row by a warp: sign flips, FWHT, 1/sqrt(D), to unit length, fp16 (hi, lo)
  {
    uint32_t sgn[E];
#pragma unroll
    for (int i = 0; i < E; ++i)
      sgn[i] = sign_mask_at(p.sign_seed, lane * E + i) ^ (p.scale_log2 < 0.f ? 0x80000000u : 0u);
    constexpr int B = 4;
    const int all = two ? 2 * kTileRows : kTileRows;
    for (int rb = warp * B; rb < all; rb += 16 * B) {
      float x[B][E];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int r = rb + j, rr = r0 + r;
        const int64_t off = (int64_t)(sq.row0 + rr / G) * p.q_rstride +
                            (int64_t)(kvh * G + rr % G) * p.q_hstride + lane * E;
#pragma unroll
        for (int i = 0; i < E; ++i) x[j][i] = r < rows ? load_as_f32(p.q, off + i, p.q_dtype) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const int r = rb + j;
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) x[j][i] = __uint_as_float(__float_as_uint(x[j][i]) ^ sgn[i]);
        warp_fwht<E>(x[j], lane);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          x[j][i] *= inv_sqrt_dim<D>();
          ss = fmaf(x[j][i], x[j][i], ss);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float nrm = sqrtf(ss), inv = nrm > 0.f ? 1.0f / nrm : 0.f;
        uint8_t* qt = q_s + (r / kTileRows) * C::QPARTS * C::QTILE;
        const int row = r % kTileRows;
        uint32_t hi[E / 2], lo[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
          const float u = x[j][2 * i] * inv, v = x[j][2 * i + 1] * inv;
          hi[i] = pack_half2(u, v);
          const float2 h = __half22float2(*(const __half2*)&hi[i]);
          lo[i] = pack_half2(u - h.x, v - h.y);
        }
        // E consecutive columns: inside one 16-byte chunk
        uint32_t* dst = (uint32_t*)(qt + sw128_offset(row, lane * E, kTileRows));
#pragma unroll
        for (int i = 0; i < E / 2; ++i) dst[i] = hi[i];
        if constexpr (PREC) {
          dst = (uint32_t*)(qt + C::QTILE + sw128_offset(row, lane * E, kTileRows));
#pragma unroll
          for (int i = 0; i < E / 2; ++i) dst[i] = lo[i];
        }
        if (lane == 0) qs_s[r] = nrm * fabsf(p.scale_log2);
      }
    }
  }
  __syncthreads();                                       // the best factors are known
  const float ak = KB <= 4 ? 1.0f + (float)(unsigned)ms->best[0] * (1.0f / kTilesThreads) : 1.0f;
  const float av = VB <= 4 ? 1.0f + (float)(unsigned)ms->best[1] * (1.0f / kTilesThreads) : 1.0f;
  tiles_lut<KB, 0>(lut, p.kc, ak, tid);
  tiles_lut<VB, 1>(lut, p.vc, av, tid);
  const int srow = tid & (kTileRows - 1);                // a softmax thread's row in its slot
  float qs = 0.f;
  int myrow = srow;
  if (warp < 8) {
    myrow = two ? (warp >> 2) * kTileRows + srow : srow;
    qs = qs_s[myrow] / ak;
  }
  fence_proxy_async_smem();                              // q is read by the tensor cores
  __syncthreads();
  const uint32_t tmem = ms->tmem;
  constexpr uint32_t O_COL = 0, S_COL = 256;
  // O' of slot j at columns j D (D <= 128), its scores and weights at 256 + 128 j
  auto fail = [&]() {
    report_error(p.err, TQ_DEVERR_TIMEOUT);
    ms->dead = 1;
  };
  // ring position of a tile's K and V
  auto k_at = [&](int k) { return two ? 2 * k : (k == 0 ? 0 : 2 * k - 1); };
  auto v_at = [&](int k) { return two ? 2 * k + 1 : 2 * k + 2; };

  if (warp >= 12) {
    regs_dec<kIssueRegs>();
    if (warp == 12 && lane == 0 && items > 0) {
      bool ok = true;
      for (int n = 0; n < items + 2 && ok; ++n) {
        if (n >= 2) {                                    // P V of item n - 2
          const int m = n - 2, k = two ? m >> 1 : m, at = v_at(k), sl = at % C::RING;
          ok = mbar_wait(&ms->p_ready[m & 1], (uint32_t)(m >> 1) & 1u, p.wait_ms) &&
               mbar_wait(&ms->ring_full[sl], (uint32_t)(at / C::RING) & 1u, p.wait_ms);
          if (!ok) break;
          tc_fence_after();
          const uint32_t vb = smem_u32(ring_s + sl * C::STAGE);
          const uint32_t acc = tmem + O_COL + (C::kOneO ? 0 : (m & 1) * D);
          const bool first = C::kOneO ? m == 0 : m < 2;
#pragma unroll
          for (int ks = 0; ks < N / 16; ++ks)
            umma_ts_f16(acc, tmem + S_COL + (m & 1) * 128 + ks * 8,
                        sw128_mn_desc(vb + ks * 2048, N * 128), f16_idesc(D, true),
                        (ks > 0 || !first) ? 1u : 0u);
          if (!two || (m & 1)) umma_commit(&ms->ring_empty[sl]);
        }
        if (n < items) {                                 // Q K of item n
          const int k = two ? n >> 1 : n, at = k_at(k), sl = at % C::RING;
          if (!two || !(n & 1)) ok = mbar_wait(&ms->ring_full[sl], (uint32_t)(at / C::RING) & 1u, p.wait_ms);
          if (!ok) break;
          tc_fence_after();
          const uint32_t kb = smem_u32(ring_s + sl * C::STAGE);
          const uint32_t qb = smem_u32(q_s + (two ? (n & 1) * C::QPARTS * C::QTILE : 0));
          const uint32_t acc = tmem + S_COL + (n & 1) * 128;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t qo = (ks >> 2) * (kTileRows * 128) + (ks & 3) * 32;
            const uint32_t ko = (ks >> 2) * (N * 128) + (ks & 3) * 32;
            umma_bf16(acc, sw128_desc(qb + qo), sw128_desc(kb + ko), f16_idesc(N, false), ks > 0 ? 1u : 0u);
            if constexpr (PREC)
              umma_bf16(acc, sw128_desc(qb + C::QTILE + qo), sw128_desc(kb + ko), f16_idesc(N, false), 1u);
            if constexpr (C::kKeyLo)
              umma_bf16(acc, sw128_desc(qb + qo), sw128_desc(kb + (D / 64) * (N * 128) + ko),
                        f16_idesc(N, false), 1u);
          }
          umma_commit(&ms->s_full[n & 1]);
          if (!two || (n & 1)) umma_commit(&ms->ring_empty[sl]);
        }
      }
      umma_commit(&ms->o_done);
      ok = mbar_wait(&ms->o_done, 0, p.wait_ms) && ok;   // what was issued is complete
      if (!ok) fail();
    }
    __syncwarp();
  } else if (warp >= 8) {
    // ---- codes to operand tiles ----
    regs_dec<kDequantRegs>();
    const int w = warp - 8;
    const int l = lane % C::LPR, rsub = lane / C::LPR;
    const int rbase = w * (N / 4) + rsub;                // this lane's rows: rbase + i RPI
    const int low_last = p.window > 0 ? (int)max((int64_t)0, (int64_t)pos_last - p.window + 1) : 0;
    const int64_t head = (int64_t)kvh * p.slot_stride;
    uint32_t raw[C::IT][4];
    // The pages of this warp's rows, WP a tile: a lane holds one table entry of a window of TW
    // tiles (and one of the next window), so that no entry is waited for.
    constexpr int WP = N / 4 > kBlockSize ? N / 4 / kBlockSize : 1, TW = 32 / WP;
    auto entry = [&](int k) -> int32_t {                 // this lane's entry of the window at tile k
      const int step = (k_begin + k + lane / WP) * C::PPT + w * (N / 4) / kBlockSize + lane % WP;
      if (k + lane / WP >= tiles || step >= steps) return -1;
      const int32_t id = p.block_table[(int64_t)b * p.bt_stride + span.at(step)];
      if (id >= 0 && id < p.num_blocks) return id;
      report_error(p.err, TQ_DEVERR_BLOCK_RANGE);
      return -1;
    };
    int32_t window = entry(0), window_next = entry(TW);
    struct Bases {
      const uint8_t* at[WP];
    };
    auto fetch = [&](int k) {                            // of tiles 0, 1, 2, ... in turn
      if (k > 0 && k % TW == 0) {
        window = window_next;
        window_next = entry(k + TW);
      }
      Bases r;
#pragma unroll
      for (int j = 0; j < WP; ++j) {
        const int32_t id = __shfl_sync(0xffffffffu, window, (k % TW) * WP + j);
        r.at[j] = id < 0 ? nullptr : p.pages + (int64_t)id * p.blk_stride + head;
      }
      return r;
    };
    // Rows i of a unit from its pages: this lane's first row of page j at at[j]
    const int64_t row_step = C::RPI * p.row_stride;
    const int64_t lane_at = (int64_t)(rbase % kBlockSize) * p.row_stride;
    constexpr int IPP = C::IT / WP;                      // rows of a lane in a page
    auto load_rows = [&](auto IV, uint32_t (&r)[4], int i, const Bases& from, const uint8_t*& at) {
      constexpr bool V = decltype(IV)::value;
      if (i % IPP == 0) {
        at = from.at[i / IPP];
        if (at != nullptr) at += lane_at + (V ? p.k_region : 0);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = 0u;
      if (at != nullptr) {
        if constexpr (V) Codes16<VB>::load(r, at, l);
        else Codes16<KB>::load(r, at, l);
        at += row_step;
      }
    };
    auto look = [&](uint32_t a) { return *(const uint32_t*)(lut + a); };
    const uint32_t lk = 4u * lane, lv = 128u + 4u * lane;
    // 16 codes to 16 halves, stored as two 16-byte chunks of the row; the order in which a
    // lane stores its two keeps 8 lanes on 8 chunks
    auto store_one = [&](auto IV, auto IL, const uint32_t (&r)[4], int i, uint8_t* stage) {
      constexpr bool V = decltype(IV)::value, LO = decltype(IL)::value;
      constexpr int BITS = V ? VB : KB;
      const uint32_t off = V ? lv : lk;
      uint32_t h[8];
      static_for<8>([&](auto JI) {
        constexpr int j = decltype(JI)::value;
        if constexpr (BITS <= 4) {
          h[j] = look(lut_addr<2 * j * BITS, 2 * BITS>(r, off));
        } else {
          h[j] = __byte_perm(look(lut_addr<2 * j * BITS, BITS>(r, off)),
                             look(lut_addr<(2 * j + 1) * BITS, BITS>(r, off)), LO ? 0x7632 : 0x5410);
        }
      });
      const int row = rbase + i * C::RPI;
      uint8_t* dst = stage + (l >> 2) * (N * 128) + row * 128 + (LO ? (D / 64) * (N * 128) : 0);
      const int c0 = 2 * (l & 3), odd = D > 64 ? (l >> 2) & 1 : 0;
      const uint4 v0 = make_uint4(h[0], h[1], h[2], h[3]), v1 = make_uint4(h[4], h[5], h[6], h[7]);
      *(uint4*)(dst + (((c0 + odd) ^ (row & 7)) << 4)) = odd ? v1 : v0;
      *(uint4*)(dst + (((c0 + 1 - odd) ^ (row & 7)) << 4)) = odd ? v0 : v1;
    };
    using KI = std::false_type;
    using VI = std::true_type;
    // norms of row w N / 4 + lane, one tile ahead
    const int nrow = w * (N / 4) + lane;
    float nk = 0.f, nv = 0.f;
    int first = -1;
    auto load_norms = [&](int k, const Bases& from) {
      nk = nv = 0.f;
      first = -1;
      const uint8_t* pg = from.at[WP > 1 ? lane / kBlockSize : 0];
      if (lane < N / 4 && pg != nullptr) {
        first = span.at((k_begin + k) * C::PPT + nrow / kBlockSize) * kBlockSize;
        const uint8_t* sl = pg + (nrow % kBlockSize) * p.row_stride;
        nk = *(const float*)(sl + KPACK);
        nv = *(const float*)(sl + p.k_region + VPACK);
      }
    };
    auto store_norms = [&](int k) {
      const int buf = k & 1;
      bool ok = true;
      float hi = -100.0f, lo = 1e30f;
      if (lane < N / 4) {
        norm_s[buf * 2 * N + nrow] = nk;
        norm_s[buf * 2 * N + N + nrow] = nv;
        if (nrow % kBlockSize == 0) ms->tok[buf][nrow / kBlockSize] = first;
        const int tok = first + nrow % kBlockSize;
        ok = first >= 0 && tok <= pos_first && (tok >= low_last || tok < p.sinks) && isfinite(nk) &&
             isfinite(nv);
        hi = fmaxf(log2_bound(nv), -100.0f);
        if (nv != 0.f) lo = fmaxf(log2_bound(fabsf(nv)), -100.0f);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      }
      ok = __all_sync(0xffffffffu, ok);
      if (lane == 0) ms->meta[buf][w] = TileMeta{hi, lo, ok ? 1 : 0};
      __syncwarp();
      mbar_arrive(&ms->norm_full[buf]);
    };
    auto free_stage = [&](int at) {                      // wait until ring position `at` may be written
      return at < C::RING ||
             mbar_wait(&ms->ring_empty[at % C::RING], (uint32_t)(at / C::RING - 1) & 1u, p.wait_ms);
    };
    auto load_all = [&](auto IV, const Bases& from) {
      const uint8_t* at = nullptr;
#pragma unroll
      for (int i = 0; i < C::IT; ++i) load_rows(IV, raw[i], i, from, at);
    };
    // the codes in raw to ring position pos; as each is used its register takes the codes of
    // the next unit (kind INV, from these pages)
    auto produce = [&](auto IV, auto INV, int pos, bool more, const Bases& next) {
      uint8_t* stage = ring_s + (pos % C::RING) * C::STAGE;
      const uint8_t* at = nullptr;
#pragma unroll
      for (int i = 0; i < C::IT; ++i) {
        store_one(IV, std::false_type{}, raw[i], i, stage);
        if constexpr (C::kKeyLo && !decltype(IV)::value) store_one(IV, std::true_type{}, raw[i], i, stage);
        if (more) load_rows(INV, raw[i], i, next, at);
      }
      fence_proxy_async_smem();
      mbar_arrive(&ms->ring_full[pos % C::RING]);
    };
    bool ok = true;
    if (tiles > 0) {
      Bases bk = fetch(0), bv = bk;                      // of the latest K tile, of the next V tile
      load_norms(0, bk);
      load_all(KI{}, bk);
      if (two) {                                         // K(0), V(0), K(1), V(1), ...
        for (int k = 0; k < tiles; ++k) {
          ok = free_stage(k_at(k));
          if (!ok) break;
          store_norms(k);
          produce(KI{}, VI{}, k_at(k), true, bk);
          const bool more = k + 1 < tiles;
          if (more) {
            bk = fetch(k + 1);
            load_norms(k + 1, bk);
          }
          ok = free_stage(v_at(k));
          if (!ok) break;
          produce(VI{}, KI{}, v_at(k), more, bk);
        }
      } else {                                           // K(0), K(1), V(0), K(2), V(1), ...
        store_norms(0);
        if (tiles > 1) {
          bk = fetch(1);
          load_norms(1, bk);
        }
        produce(KI{}, KI{}, k_at(0), tiles > 1, bk);
        if (tiles == 1) load_all(VI{}, bv);
        for (int k = 0; k < tiles; ++k) {
          if (k + 1 < tiles) {
            ok = free_stage(k_at(k + 1));
            if (!ok) break;
            produce(KI{}, VI{}, k_at(k + 1), true, bv);
            // the norms' buffer is free once item k - 1 has its weights
            if (k >= 1) ok = mbar_wait(&ms->p_ready[(k - 1) & 1], (uint32_t)((k - 1) >> 1) & 1u, p.wait_ms);
            if (!ok) break;
            store_norms(k + 1);
          }
          bv = bk;
          const bool more = k + 2 < tiles;
          if (more) {
            bk = fetch(k + 2);
            load_norms(k + 2, bk);
          }
          ok = free_stage(v_at(k));
          if (!ok) break;
          produce(VI{}, KI{}, v_at(k), more, bk);
          if (k + 2 == tiles) load_all(VI{}, bv);        // no K tile is left to fetch it under
        }
      }
    }
    if (!ok) fail();
  } else {
    // ---- softmax: a thread = a row of slot warp / 4 ----
    regs_inc<kSoftmaxRegs>();
    const int slot = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // this warp's quarter of tensor memory
    float M = -INFINITY, sum = 0.f;
    const int pos = myrow < rows ? p0 + (r0 + myrow) / G : -1;
    const int low = p.window > 0 ? (int)max((int64_t)0, (int64_t)pos - p.window + 1) : 0;
    const uint32_t o_at = tmem + lanes + O_COL + (C::kOneO ? 0 : slot * D);
    const int step_n = C::kOneO ? 1 : 2;
    bool ok = true, any = false;
    for (int n = slot; n < items && !(C::kOneO && slot); n += step_n) {
      const int buf = n & 1, k = two ? n >> 1 : n, nb = k & 1;
      const uint32_t s_at = tmem + lanes + S_COL + buf * 128;
      ok = mbar_wait(&ms->norm_full[nb], (uint32_t)(k >> 1) & 1u, p.wait_ms) &&
           mbar_wait(&ms->s_full[buf], (uint32_t)(n >> 1) & 1u, p.wait_ms);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float s[N];
#pragma unroll
      for (int c = 0; c < N; c += 16) tmem_ld16_nowait(s_at + c, s + c);
      const float* nks = norm_s + nb * 2 * N;
      const float* nvs = nks + N;
      bool plain = true;
      float emax = -100.f, emin = 1e30f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const TileMeta m = ms->meta[nb][i];
        plain = plain && m.plain;
        emax = fmaxf(emax, m.emax);
        emin = fminf(emin, m.emin);
      }
      plain = plain && emax - emin <= 8.0f;
      tmem_wait_ld();
      float z = -INFINITY;
      if (plain) {
        float z1 = -INFINITY;
#pragma unroll
        for (int c = 0; c < N; c += 4) {
          const float4 f = *(const float4*)(nks + c);
          float2 u = mul2(make_float2(s[c], s[c + 1]), make_float2(f.x, f.y));
          float2 v = mul2(make_float2(s[c + 2], s[c + 3]), make_float2(f.z, f.w));
          s[c] = u.x, s[c + 1] = u.y, s[c + 2] = v.x, s[c + 3] = v.y;
          z = fmaxf(z, fmaxf(u.x, u.y));
          z1 = fmaxf(z1, fmaxf(v.x, v.y));
        }
        z = fmaf(fmaxf(z, z1), qs, emax);
      } else {
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const int first = ms->tok[nb][c / kBlockSize], tok = first + c % kBlockSize;
          const bool see = first >= 0 && tok <= pos && (tok >= low || tok < p.sinks);
          s[c] = see ? s[c] * nks[c] * qs : -INFINITY;
          z = fmaxf(z, s[c] + fmaxf(log2_bound(nvs[c]), -100.0f));
        }
      }
      const bool raise = z > M + kLazyRescale;
      if (__any_sync(0xffffffffu, raise)) {
        const float to = raise ? z : M;
        const float f = M == -INFINITY ? 0.f : exp2f(M - to);
        sum *= f;
        M = to;
        if (any) {
          // With a slot's own O', P V of its last item precedes Q K of this one.  A shared O'
          // may still be under P V of item n - 1: until that has freed its V tile.
          if constexpr (C::kOneO) {
            const int at = v_at(n - 1);
            ok = mbar_wait(&ms->ring_empty[at % C::RING], (uint32_t)(at / C::RING) & 1u, p.wait_ms);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
          }
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
      any = true;
      const float ref = M == -INFINITY ? 0.f : M;
      uint32_t pk[8];
      if (plain) {
        const float2 q2 = make_float2(qs, qs), m2 = make_float2(-ref, -ref);
        float2 l0 = make_float2(sum, 0.f), l1 = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < N; c += 4) {
          float2 u = fma2(make_float2(s[c], s[c + 1]), q2, m2);
          float2 v = fma2(make_float2(s[c + 2], s[c + 3]), q2, m2);
          u = make_float2(ex2_approx(u.x), ex2_approx(u.y));
          v = make_float2(ex2_approx(v.x), ex2_approx(v.y));
          l0 = add2(l0, u);
          l1 = add2(l1, v);
          const float4 f = *(const float4*)(nvs + c);
          u = mul2(u, make_float2(f.x, f.y));
          v = mul2(v, make_float2(f.z, f.w));
          pk[c / 2 % 8] = pack_half2(u.x, u.y);
          pk[c / 2 % 8 + 1] = pack_half2(v.x, v.y);
          if (c % 16 == 12) tmem_st8(s_at + c / 16 * 8, pk);
        }
        sum = (l0.x + l0.y) + (l1.x + l1.y);
      } else {
#pragma unroll
        for (int c = 0; c < N; c += 2) {
          const float w0 = ex2_approx(s[c] - ref), w1 = ex2_approx(s[c + 1] - ref);
          sum += w0 + w1;
          pk[c / 2 % 8] = pack_half2(s[c] == -INFINITY ? 0.f : w0 * nvs[c],
                                     s[c + 1] == -INFINITY ? 0.f : w1 * nvs[c + 1]);
          if (c % 16 == 14) tmem_st8(s_at + c / 16 * 8, pk);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&ms->p_ready[buf]);
    }
    if (ok && items > 0) ok = mbar_wait(&ms->o_done, 0, p.wait_ms);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) fail();
    // every other reader of the operands is done: their place takes the partials
    tc_fence_after();
    if (!(C::kOneO && slot)) {
      float* rec = part_s + (slot * kTileRows + srow) * PART;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        float o[16];
        if (any && ok) {
          tmem_ld16_nowait(o_at + c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4) *(float4*)(rec + c + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
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
  // row r is joined by CTA r % ctas of the cluster, by a warp; records: CTAs x slots
  const int recs = two || C::kOneO ? 1 : 2;
  for (int r = split + ctas * warp; r < rows; r += ctas * 16) {
    float Mr = -INFINITY, lr = 0.f, o[E];
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = 0.f;
    fold_records<E>(ctas * recs, [&](int j, float& m, float& ll, float (&v)[E]) {
      const float* from = part_s + ((recs == 2 ? (j & 1) * kTileRows : 0) + r) * PART;
      if (ctas > 1) from = cluster.map_shared_rank(from, recs == 2 ? j >> 1 : j);
      m = from[D];
      ll = from[D + 1];
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = from[lane * E + i];
    }, Mr, lr, o);
    const float inv = lr == 0.f ? 0.f : 1.0f / (lr * av);     // a row that sees nothing: 0
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] *= inv;
    warp_fwht<E>(o, lane);
    const int rr = r0 + r;
    const int64_t off = (int64_t)(sq.row0 + rr / G) * p.o_rstride +
                        (int64_t)(kvh * G + rr % G) * p.o_hstride + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i)
      store_from_f32(p.out, off + i, p.out_dtype,
                     __uint_as_float(__float_as_uint(o[i] * inv_sqrt_dim<D>()) ^
                                     sign_mask_at(p.sign_seed, lane * E + i)));
  }
  if (ctas > 1) cluster.sync();              // no CTA leaves while its partials may be read
}

}  // namespace tq
