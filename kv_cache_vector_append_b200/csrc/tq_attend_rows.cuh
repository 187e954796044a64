// tq_attend_rows.cuh -- attention over packed slots for few query rows a KV head: the
// single-token form with a sliding window and sinks, and chunks of a token or few.
//
// Math.  With R the rotation, a key is nK R^T cK[i], a value nV R^T cV[j], so with q' = R q
//   s_t = scale log2(e) nK_t <q', cK[i_t]>,   o = R^T (sum_t 2^(s_t - M) nV_t cV[j_t]) / l,
// l = sum_t 2^(s_t - M): the queries are rotated once and the output once, keys and values
// are never rebuilt.  Sums, maxima and l are fp32; the operands of the two contractions are
// fp16: unit queries and centroids (2^-12 off; key centroids times a factor in [1, 2) under which
// their roundings are smallest, 8-bit ones as hi + lo), and weights P = 2^(s - M) nV <= 2^9 with
// M >= max(s + log2 nV), so that the weights keep fp16's range whatever the norms are.
//
// Layout.  A cluster of CTAs serves 8 NT rows of one (sequence, KV head); its warps take the
// 16-token pages that some row sees in turn, each warp straight from global memory into
// registers (each part of a page is reloaded for the next as soon as it has been used), and
// both contractions run on mma.sync m16n8k16 (M = tokens or coordinates, N = 8 rows): the tile
// is 16 x 8 NT, far below what a tcgen05 tile needs, and a page's lookups serve its NT row
// tiles.  Codes become fp16 through the pair tables of tq_decode.cuh (one 256-byte row an
// entry, so the 32 lanes of a lookup hit 32 banks; 2-bit V codes four at a time).  Pages that
// every row sees skip the masks.  The warps' partials (M, l, O') are joined in shared memory,
// those of the cluster's CTAs over distributed shared memory: no workspace, no counters, the
// same order of sums every time.
//
// Bound: instruction issue (some 350 a page) and the L1 wavefronts of loads that touch eight
// rows each (75% of the active cycles).  64 windows of 4,096 tokens, 28/4 heads of 128, 4/2 bits:
// 50 us, 2.2 TB/s; a block's start and end take about 8 us of it.
#pragma once

#include <cooperative_groups.h>

#include "tq_attend.cuh"

namespace tq {

constexpr int kRowsWarps = 8;
// Most row tiles of 8 a CTA takes: 64 accumulators a thread (128 at D = 256, one tile's are 64).
__host__ __device__ constexpr int rows_tiles(int d) { return d == 64 ? 4 : d == 128 ? 2 : 1; }

// A thread's share of one row's packed codes, read from global memory with 4-byte loads.
// (Share::load reads shares that are no whole words byte by byte: here they come from the
// one or two words around them.)
template <int D, int BITS, int NT>
__device__ __forceinline__ void load_share(uint32_t (&w)[Share<D, BITS, NT>::NW],
                                           const uint8_t* region, int t) {
  using S = Share<D, BITS, NT>;
  if constexpr (S::kInterleaved || S::kContig) {
    S::load(w, region, t);
  } else {
    static_assert(S::BYTES <= 6 && S::NW <= 2, "a share of at most 6 bytes");
    const int o = S::BYTES * t;
    const uint32_t* a = (const uint32_t*)(region + (o & ~3));
    const int sh = 8 * (o & 3);
    const uint32_t lo = a[0];
    // the second word is inside the slot: the norm follows the codes
    const uint32_t hi = (o & 3) + S::BYTES > 4 ? a[1] : 0u;
    w[0] = __funnelshift_r(lo, hi, sh);
    if constexpr (S::NW == 2) w[1] = hi >> sh;
  }
}

// The K share of one of 4 threads: 8-byte pieces where the row has enough of them (K regions
// start on 8-byte boundaries), else Share's words.
template <int D, int BITS>
struct KeyShare {
  using S = Share<D, BITS, 4>;
  static constexpr bool kWide = 32 % BITS == 0 && D * BITS / 64 % 4 == 0;
  static constexpr int NW = S::NW, PW = S::PW;
  static __host__ __device__ constexpr int pos(int m) { return S::pos(m); }
  static __host__ __device__ constexpr int coord(int t, int m) {
    return kWide ? (2 * (t + 4 * (m / PW / 2)) + m / PW % 2) * PW + m % PW : S::coord(t, m);
  }
  static __device__ __forceinline__ void load(uint32_t (&w)[NW], const uint8_t* region, int t) {
    if constexpr (kWide) {
#pragma unroll
      for (int j = 0; j < NW / 2; ++j) {
        const uint2 v = *(const uint2*)(region + 8 * (t + 4 * j));
        w[2 * j] = v.x;
        w[2 * j + 1] = v.y;
      }
    } else {
      load_share<D, BITS, 4>(w, region, t);
    }
  }
};

// The tables of tq_decode.cuh, made by warps: a lane holds an entry, and eight lanes write each
// entry's half row with 16-byte stores.  VQUAD: 2-bit V codes four at a time, as
// lut_build_vquad lays them out.
template <int BITS, int HALF, bool VQUAD>
__device__ __forceinline__ void rows_lut(uint8_t* lut, const float* c, float factor, int warp, int lane) {
  constexpr int kEntries = VQUAD ? 256 : lut_entries(BITS);
  for (int e0 = warp * 32; e0 < kEntries; e0 += kRowsWarps * 32) {
    const int e = e0 + lane;
    uint32_t v = 0u, v2 = 0u;
    if (e < kEntries) {
      if constexpr (VQUAD) {
        v = pack_half2(c[e & 3], c[(e >> 4) & 3]);
        v2 = pack_half2(c[(e >> 2) & 3], c[e >> 6]);
      } else if constexpr (BITS <= 4) {
        v = pack_half2(c[e & ((1 << BITS) - 1)] * factor, c[e >> BITS] * factor);
      } else {
        const float hi = __half2float(__float2half_rn(c[e]));
        v = pack_half2(hi, c[e] - hi);
      }
    }
    uint8_t* dst = lut + (e0 + (lane >> 3)) * kLutRow + HALF * 128 + 16 * (lane & 7);
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const uint32_t a = __shfl_sync(0xffffffffu, v, j + (lane >> 3));
      const uint32_t b = VQUAD ? __shfl_sync(0xffffffffu, v2, j + (lane >> 3)) : a;
      if (e0 + j + (lane >> 3) < kEntries) *(uint4*)(dst + j * kLutRow) = make_uint4(a, b, a, b);
    }
  }
}

__host__ __device__ constexpr int rows_lut_bytes(int kb, int vb) {
  const int ek = lut_entries(kb), ev = vb == 2 ? 256 : lut_entries(vb);
  return (ek > ev ? ek : ev) * kLutRow;
}
__host__ __device__ constexpr int rows_part(int d) { return d + 4; }   // floats of a partial
// [tables, later the warps' partials | q' fp16 | |q'| scales | the CTA's partials]
__host__ __device__ constexpr int rows_smem(int d, int kb, int vb, int nt) {
  const int lut = rows_lut_bytes(kb, vb), part = kRowsWarps * 8 * nt * rows_part(d) * 4;
  return (lut > part ? lut : part) + 8 * nt * (d * 2 + 4 + rows_part(d) * 4);
}

template <int D, int KB, int VB, int NT>
__global__ void __launch_bounds__(kRowsWarps * 32, NT == 1 ? 2 : 1)
attend_rows_kernel(const AttendParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  using C = DecodeCfg<D, KB, VB>;
  using KS = KeyShare<D, KB>;
  using VS = typename C::VS;
  constexpr bool VQUAD = VS::kInterleaved && VB == 2;
  constexpr int E = D / 32, PART = rows_part(D), ROWS = 8 * NT;
  constexpr int kLut = rows_lut_bytes(KB, VB);
  constexpr int kWarpParts = kRowsWarps * ROWS * PART * 4;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* lut = smem;
  float* wpart = (float*)smem;                                  // [warps][rows][PART]
  __half* qh = (__half*)(smem + (kLut > kWarpParts ? kLut : kWarpParts));
  float* qsc = (float*)(qh + ROWS * D);
  float* cpart = qsc + ROWS;                                    // [rows][PART]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int ctas = (int)cluster.num_blocks(), split = (int)cluster.block_rank();
  const AttendItem item = attend_item<false>(p, ctas);
  const int b = item.b, kvh = item.kvh, G = p.group;

  const AttendSeq sq = attend_seq(p, b, tid == 0 && split == 0 && kvh == 0 && item.tile == 0);
  // while the sequence's numbers are on their way
  __shared__ unsigned factor_key[kRowsWarps];
  if constexpr (KB <= 4) {
    const unsigned key = centroid_factor_key<KB>(p.kc, tid, kRowsWarps * 32);
    if (lane == 0) factor_key[warp] = key;
  }
  // this cluster's rows [r0, r0 + rows) of the KV head's n_q * G
  const int r0 = item.tile * ROWS;
  const int rows = min(ROWS, sq.n_q * G - r0);
  if (rows <= 0) return;                    // the whole cluster
  const int p0 = sq.len - sq.n_q;           // position of row 0
  const int pos_first = p0 + r0 / G, pos_last = p0 + (r0 + rows - 1) / G;
  const AttendSpan span = attend_span(p, pos_first, pos_last, kBlockSize);
  const int low_last = p.window > 0 ? (int)max((int64_t)0, (int64_t)pos_last - p.window + 1) : 0;
  auto row_offset = [&](int r, int64_t rstride, int64_t hstride) {
    return (int64_t)(sq.row0 + (r0 + r) / G) * rstride + (int64_t)(kvh * G + (r0 + r) % G) * hstride;
  };

  // the queries (row r = warp + 8 j of this CTA) are on their way first
  float xq[NT][E];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int r = warp + kRowsWarps * j;
    const int64_t off = row_offset(r, p.q_rstride, p.q_hstride) + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) xq[j][i] = r < rows ? load_as_f32(p.q, off + i, p.q_dtype) : 0.f;
  }
  // This warp's pages are the steps first + i stride.  A lane holds the table entry of one of 32
  // of them (and one of the next 32), -1 past the end or where it is out of range.
  const int steps = span.count(), stride = ctas * kRowsWarps, first = split * kRowsWarps + warp;
  const int mine = first < steps ? (steps - first + stride - 1) / stride : 0;
  auto entry = [&](int i) -> int32_t {
    if (i + lane >= mine) return -1;
    const int32_t id = p.block_table[(int64_t)b * p.bt_stride + span.at(first + (i + lane) * stride)];
    if (id >= 0 && id < p.num_blocks) return id;
    report_error(p.err, TQ_DEVERR_BLOCK_RANGE);
    return -1;
  };
  int32_t window = entry(0), window_next = entry(32);
  auto fetch = [&](int i) -> int32_t {      // i = 0, 1, 2, ... in turn
    if (i > 0 && i % 32 == 0) {
      window = window_next;
      window_next = entry(i + 32);
    }
    return __shfl_sync(0xffffffffu, window, i % 32);
  };
  // A page in registers, reloaded for the next page part by part as its parts have been used.
  constexpr int KREG = C::KPACK + 4;                    // bytes of the K region
  uint32_t kw0[KS::NW], kw1[KS::NW], vw[4][VS::NW];
  float nK[2], nV[2];
  const uint8_t* k_lane = p.pages + (int64_t)kvh * p.slot_stride + gid * p.row_stride;
  const uint8_t* v_lane = p.pages + (int64_t)kvh * p.slot_stride + 2 * tig * p.row_stride + KREG;
  auto load_keys = [&](int32_t id) {
    const uint8_t* k = k_lane + (int64_t)id * p.blk_stride;
    KS::load(kw0, k, tig);
    KS::load(kw1, k + 8 * p.row_stride, tig);
  };
  auto load_rest = [&](int32_t id) {
    const uint8_t* k = k_lane + (int64_t)id * p.blk_stride;
    nK[0] = *(const float*)(k + C::KPACK);
    nV[0] = *(const float*)(k + KREG + C::VPACK);
    k += 8 * p.row_stride;
    nK[1] = *(const float*)(k + C::KPACK);
    nV[1] = *(const float*)(k + KREG + C::VPACK);
    const uint8_t* v = v_lane + (int64_t)id * p.blk_stride;
    load_share<D, VB, 8>(vw[0], v, gid);
    load_share<D, VB, 8>(vw[1], v + p.row_stride, gid);
    v += 8 * p.row_stride;
    load_share<D, VB, 8>(vw[2], v, gid);
    load_share<D, VB, 8>(vw[3], v + p.row_stride, gid);
  };

  // the first page is on its way while the tables and the queries are made
  int32_t cur = fetch(0);
  if (cur >= 0) {
    load_keys(cur);
    load_rest(cur);
  }

  rows_lut<VB, 1, VQUAD>(lut, p.vc, 1.0f, kRowsWarps - 1 - warp, lane);
  // q' of a row by a warp: sign flips, FWHT, 1/sqrt(D), then to unit length in fp16
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int r = warp + kRowsWarps * j;
    float (&x)[E] = xq[j];
#pragma unroll
    for (int i = 0; i < E; ++i)
      x[i] = __uint_as_float(__float_as_uint(x[i]) ^ sign_mask_at(p.sign_seed, lane * E + i));
    warp_fwht<E>(x, lane);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      x[i] *= inv_sqrt_dim<D>();
      ss = fmaf(x[i], x[i], ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float nrm = sqrtf(ss);
    const float inv = nrm > 0.f ? 1.0f / nrm : 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) qh[r * D + lane * E + i] = __float2half_rn(x[i] * inv);
    if (lane == 0) qsc[r] = nrm * p.scale_log2;
  }
  __syncthreads();
  float factor = 1.0f;                        // of the key centroids
  if constexpr (KB <= 4) {
    unsigned key = factor_key[0];
#pragma unroll
    for (int i = 1; i < kRowsWarps; ++i) key = min(key, factor_key[i]);
    factor = centroid_factor(key);
  }
  rows_lut<KB, 0, false>(lut, p.kc, factor, warp, lane);

  uint32_t qb[NT][C::KSTEPS][2];
  // this thread's rows 8 nt + 2 tig + e: scale, position, first key of the window
  float qscale[NT][2], M[NT][2], l[NT][2], acc[NT][C::MT][4];
  int pos[NT][2], low[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int ks = 0; ks < C::KSTEPS; ++ks) {
      qb[nt][ks][0] = *(const uint32_t*)(qh + (8 * nt + gid) * D + KS::coord(tig, 4 * ks));
      qb[nt][ks][1] = *(const uint32_t*)(qh + (8 * nt + gid) * D + KS::coord(tig, 4 * ks + 2));
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * nt + 2 * tig + e;
      qscale[nt][e] = qsc[r] / factor;
      pos[nt][e] = r < rows ? p0 + (r0 + r) / G : -1;
      low[nt][e] = p.window > 0 ? (int)max((int64_t)0, (int64_t)pos[nt][e] - p.window + 1) : 0;
      M[nt][e] = -INFINITY;
      l[nt][e] = 0.f;
    }
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[nt][mt][k] = 0.f;
  }
  __syncthreads();                            // the tables are there
  const uint32_t lk = 4u * lane, lv = 128u + (VQUAD ? 8u * (lane & 15) : 4u * lane);
  auto look = [&](uint32_t a) { return *(const uint32_t*)(lut + a); };
  auto look2 = [&](uint32_t a) { return *(const uint2*)(lut + a); };

  for (int i = 0; i < mine; ++i) {
    const int32_t id = i + 1 < mine ? fetch(i + 1) : -1;
    if (cur < 0) {
      if (id >= 0) {
        load_keys(id);
        load_rest(id);
      }
      cur = id;
      continue;
    }

    // ---- S^T = K~ . Qhat^T ----
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[nt][k] = 0.f;
    static_for<C::KSTEPS>([&](auto KSI) {
      constexpr int ks = decltype(KSI)::value;
      constexpr int b0 = KS::pos(4 * ks), b2 = KS::pos(4 * ks + 2);
      if constexpr (KB <= 4) {
        const uint32_t a0 = look(lut_addr<b0, 2 * KB>(kw0, lk)), a1 = look(lut_addr<b0, 2 * KB>(kw1, lk));
        const uint32_t a2 = look(lut_addr<b2, 2 * KB>(kw0, lk)), a3 = look(lut_addr<b2, 2 * KB>(kw1, lk));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816(s[nt], a0, a1, a2, a3, qb[nt][ks][0], qb[nt][ks][1]);
      } else {
        // 8-bit codes: the fp16 centroids, then what they leave (c - fp16(c)), as the
        // whole-sequence decode does
        uint32_t hi[4], lo[4];
        auto one = [&](int i, uint32_t ex, uint32_t ey) {
          hi[i] = __byte_perm(ex, ey, 0x5410);
          lo[i] = __byte_perm(ex, ey, 0x7632);
        };
        one(0, look(lut_addr<b0, KB>(kw0, lk)), look(lut_addr<b0 + KB, KB>(kw0, lk)));
        one(1, look(lut_addr<b0, KB>(kw1, lk)), look(lut_addr<b0 + KB, KB>(kw1, lk)));
        one(2, look(lut_addr<b2, KB>(kw0, lk)), look(lut_addr<b2 + KB, KB>(kw0, lk)));
        one(3, look(lut_addr<b2, KB>(kw1, lk)), look(lut_addr<b2 + KB, KB>(kw1, lk)));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816(s[nt], hi[0], hi[1], hi[2], hi[3], qb[nt][ks][0], qb[nt][ks][1]);
          mma_16816(s[nt], lo[0], lo[1], lo[2], lo[3], qb[nt][ks][0], qb[nt][ks][1]);
        }
      }
    });

    if (id >= 0) load_keys(id);

    // ---- online softmax: this thread's tokens gid + 8 r, rows 8 nt + 2 tig + e ----
    const int page0 = span.at(first + i * stride) * kBlockSize;
    // a page that every row sees whole needs no masks
    const bool full = page0 + kBlockSize - 1 <= pos_first &&
                      (page0 >= low_last || page0 + kBlockSize <= p.sinks);
    // floor at 2^-100 keeps 2^(s - M) finite for rows of (near) zero V norm
    const float eV[2] = {fmaxf(log2_bound(nV[0]), -100.0f), fmaxf(log2_bound(nV[1]), -100.0f)};
    float z[NT][2];
    bool need = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int r = 0; r < 2; ++r) s[nt][2 * r + e] *= nK[r] * qscale[nt][e];
        if (!full) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int tok = page0 + gid + 8 * r;
            if (!(tok <= pos[nt][e] && (tok >= low[nt][e] || tok < p.sinks))) s[nt][2 * r + e] = -INFINITY;
          }
        }
        z[nt][e] = fmaxf(s[nt][e] + eV[0], s[nt][2 + e] + eV[1]);
        need |= z[nt][e] > M[nt][e] + kLazyRescale;
      }
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = z[nt][e];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float to = top > M[nt][e] + kLazyRescale ? top : M[nt][e];
          const float f = M[nt][e] == -INFINITY ? 0.f : exp2f(M[nt][e] - to);
          l[nt][e] *= f;
          M[nt][e] = to;
#pragma unroll
          for (int mt = 0; mt < C::MT; ++mt) {
            acc[nt][mt][e] *= f;
            acc[nt][mt][2 + e] *= f;
          }
        }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float pv[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ref = M[nt][e] == -INFINITY ? 0.f : M[nt][e];   // a row that has seen nothing yet
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float w = ex2_approx(s[nt][2 * r + e] - ref);       // 0 for a key the row does not see
          l[nt][e] += w;
          // whose norm may be anything
          pv[e][r] = full || s[nt][2 * r + e] != -INFINITY ? w * nV[r] : 0.f;
        }
      }
      pb[nt][0] = movmatrix_trans(pack_half2(pv[0][0], pv[1][0]));
      pb[nt][1] = movmatrix_trans(pack_half2(pv[0][1], pv[1][1]));
    }

    // ---- O'^T += V~^T . P^T ----
    auto add = [&](auto MI, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
      constexpr int mt = decltype(MI)::value;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_16816(acc[nt][mt], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
    };
    if constexpr (VQUAD) {
      // codes of tokens A/B and C/D side by side by nibble (two codes each): lo the even
      // nibbles of a word, hi the odd; a lookup gives rows g and g + 8 of an m-tile
      static_for<VS::NW>([&](auto JI) {
        constexpr int j = decltype(JI)::value;
        constexpr uint32_t M1 = 0x0F0F0F0Fu;
        const uint32_t loAB = (vw[0][j] & M1) | ((vw[1][j] << 4) & ~M1);
        const uint32_t hiAB = ((vw[0][j] >> 4) & M1) | (vw[1][j] & ~M1);
        const uint32_t loCD = (vw[2][j] & M1) | ((vw[3][j] << 4) & ~M1);
        const uint32_t hiCD = ((vw[2][j] >> 4) & M1) | (vw[3][j] & ~M1);
        static_for<8>([&](auto KI) {
          constexpr int k = decltype(KI)::value;
          const uint2 ab = look2(lut_addr1<8 * (k >> 1), 8>((k & 1) ? hiAB : loAB, lv));
          const uint2 cd = look2(lut_addr1<8 * (k >> 1), 8>((k & 1) ? hiCD : loCD, lv));
          add(std::integral_constant<int, j * 8 + k>{}, ab.x, ab.y, cd.x, cd.y);
        });
      });
    } else if constexpr (VS::kInterleaved && VB == 4) {
      // codes of tokens A/B and C/D side by side: lo the even codes of a word, hi the odd
      static_for<VS::NW>([&](auto JI) {
        constexpr int j = decltype(JI)::value;
        constexpr uint32_t M1 = 0x0F0F0F0Fu;
        const uint32_t loAB = (vw[0][j] & M1) | ((vw[1][j] << 4) & ~M1);
        const uint32_t hiAB = ((vw[0][j] >> 4) & M1) | (vw[1][j] & ~M1);
        const uint32_t loCD = (vw[2][j] & M1) | ((vw[3][j] << 4) & ~M1);
        const uint32_t hiCD = ((vw[2][j] >> 4) & M1) | (vw[3][j] & ~M1);
        static_for<4>([&](auto KI) {
          constexpr int k = decltype(KI)::value;
          add(std::integral_constant<int, j * 4 + k>{}, look(lut_addr1<8 * k, 8>(loAB, lv)),
              look(lut_addr1<8 * k, 8>(hiAB, lv)), look(lut_addr1<8 * k, 8>(loCD, lv)),
              look(lut_addr1<8 * k, 8>(hiCD, lv)));
        });
      });
    } else {
      static_for<C::MT>([&](auto MI) {
        constexpr int mt = decltype(MI)::value;
        auto two = [&](auto PI, const uint32_t (&x)[VS::NW], const uint32_t (&y)[VS::NW]) {
          constexpr int at = decltype(PI)::value;
          if constexpr (VB <= 4) {
            return look(((field<at, VB>(x) | (field<at, VB>(y) << VB)) << 8) | lv);
          } else {
            return __byte_perm(look(lut_addr<at, VB>(x, lv)), look(lut_addr<at, VB>(y, lv)), 0x5410);
          }
        };
        using P0 = std::integral_constant<int, VS::pos(2 * mt)>;
        using P1 = std::integral_constant<int, VS::pos(2 * mt + 1)>;
        add(MI, two(P0{}, vw[0], vw[1]), two(P1{}, vw[0], vw[1]), two(P0{}, vw[2], vw[3]),
            two(P1{}, vw[2], vw[3]));
      });
    }
    if (id >= 0) load_rest(id);
    cur = id;
  }

  // ---- the warps' partials [row][O' in natural order, M, l] ----
  __syncthreads();                            // the tables are no longer read
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float sum = l[nt][e];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      float* rec = wpart + (warp * ROWS + 8 * nt + 2 * tig + e) * PART;
      if (gid == 0) {
        // a sum that is not a number must survive the join, which drops empty partials
        rec[D] = sum != sum && M[nt][e] == -INFINITY ? -3e38f : M[nt][e];
        rec[D + 1] = sum;
      }
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt) {
        rec[VS::coord(gid, 2 * mt)] = acc[nt][mt][e];
        rec[VS::coord(gid, 2 * mt + 1)] = acc[nt][mt][e + 2];
      }
    }
  __syncthreads();
  // warp r joins row r's partials: n records at rec(j)
  float Mr = -INFINITY, lr = 0.f, o[E];
  auto join = [&](int n, auto rec) {
    Mr = -INFINITY;
    lr = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = 0.f;
    fold_records<E>(n, [&](int j, float& m, float& ll, float (&v)[E]) {
      const float* r = rec(j);
      m = r[D];
      ll = r[D + 1];
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = r[lane * E + i];
    }, Mr, lr, o);
  };
  auto write = [&](int r) {
    const float inv = lr == 0.f ? 0.f : 1.0f / lr;        // a row that sees nothing: 0
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] *= inv;
    warp_fwht<E>(o, lane);
    const int64_t off = row_offset(r, p.o_rstride, p.o_hstride) + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i)
      store_from_f32(p.out, off + i, p.out_dtype,
                     __uint_as_float(__float_as_uint(o[i] * inv_sqrt_dim<D>()) ^
                                     sign_mask_at(p.sign_seed, lane * E + i)));
  };
  for (int r = warp; r < rows; r += kRowsWarps) {
    join(kRowsWarps, [&](int j) { return wpart + (j * ROWS + r) * PART; });
    if (ctas == 1) {
      write(r);
      continue;
    }
    float* rec = cpart + r * PART;
    if (lane == 0) {
      rec[D] = Mr;
      rec[D + 1] = lr;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) rec[lane * E + i] = o[i];
  }
  if (ctas > 1) {
    cluster.sync();
    // row r to CTA r % ctas
    for (int r = split + ctas * warp; r < rows; r += ctas * kRowsWarps) {
      join(ctas, [&](int j) { return cluster.map_shared_rank(cpart, j) + r * PART; });
      write(r);
    }
    cluster.sync();                           // no CTA leaves while its partials may be read
  }
}

}  // namespace tq
