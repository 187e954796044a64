// tq_attend_rows.cuh -- attention over packed slots for at most 8 query rows a KV head: the
// single-token form with a sliding window and sinks, and chunks of a token or few.
//
// Math.  With R the rotation, a key is nK R^T cK[i], a value nV R^T cV[j], so with q' = R q
//   s_t = scale log2(e) nK_t <q', cK[i_t]>,   o = R^T (sum_t 2^(s_t - M) nV_t cV[j_t]) / l,
// l = sum_t 2^(s_t - M): the queries are rotated once and the output once, keys and values
// are never rebuilt.  Sums, maxima and l are fp32; the operands of the two contractions are
// fp16: unit queries and centroids (2^-11 off at most), and weights P = 2^(s - M) nV <= 2^9
// with M >= max(s + log2 nV), so that the weights keep fp16's range whatever the norms are.
//
// Layout.  A cluster of CTAs serves one (sequence, KV head); its warps take the 16-token
// pages that some row sees in turn, each warp straight from global memory into registers,
// one page ahead, and both contractions run on mma.sync m16n8k16 (M = tokens or
// coordinates, N = the 8 rows): the tile is 16 x 8, far below what a tcgen05 tile needs.  Codes
// become fp16 through the pair tables of tq_decode.cuh (one 256-byte row an entry, so the 32
// lanes of a lookup hit 32 banks).  The warps' partials (M, l, O') are joined in shared
// memory, those of the cluster's CTAs over distributed shared memory: no workspace, no
// counters, the same order of sums every time.
//
// Bound: instruction issue next to the packed bytes, as the whole-sequence decode.
#pragma once

#include <cooperative_groups.h>

#include "tq_attend.cuh"

namespace tq {

constexpr int kRowsWarps = 8;
constexpr int kRowsMax = 8;                // query rows a KV head (the mma's N)
constexpr int kRowsMaxCtas = 8;            // CTAs of a cluster

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

__host__ __device__ constexpr int rows_lut_bytes(int kb, int vb) {
  const int ek = lut_entries(kb), ev = lut_entries(vb);
  return (ek > ev ? ek : ev) * kLutRow;
}
__host__ __device__ constexpr int rows_part(int d) { return d + 4; }   // floats of a partial
// [tables, later the warps' partials | q' fp16 | |q'| scales | the CTA's partials]
__host__ __device__ constexpr int rows_smem(int d, int kb, int vb) {
  const int lut = rows_lut_bytes(kb, vb), part = kRowsWarps * kRowsMax * rows_part(d) * 4;
  return (lut > part ? lut : part) + kRowsMax * d * 2 + kRowsMax * 4 + kRowsMax * rows_part(d) * 4;
}

template <int D, int KB, int VB>
__global__ void __launch_bounds__(kRowsWarps * 32)
attend_rows_kernel(const AttendParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  using C = DecodeCfg<D, KB, VB>;
  using KS = typename C::KS;
  using VS = typename C::VS;
  constexpr int E = D / 32, PART = rows_part(D);
  constexpr int kLut = rows_lut_bytes(KB, VB);
  constexpr int kWarpParts = kRowsWarps * kRowsMax * PART * 4;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* lut = smem;
  float* wpart = (float*)smem;                                  // [warps][rows][PART]
  __half* qh = (__half*)(smem + (kLut > kWarpParts ? kLut : kWarpParts));
  float* qsc = (float*)(qh + kRowsMax * D);
  float* cpart = qsc + kRowsMax;                                // [rows][PART]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int ctas = (int)cluster.num_blocks(), split = (int)cluster.block_rank();
  const int b = blockIdx.x / ctas, kvh = blockIdx.y, G = p.group;

  const AttendSeq sq = attend_seq(p, b, tid == 0 && split == 0 && kvh == 0);
  // this cluster's rows [r0, r0 + rows) of the KV head's n_q * G
  const int r0 = blockIdx.z * kRowsMax;
  const int rows = min(kRowsMax, sq.n_q * G - r0);
  if (rows <= 0) return;                    // the whole cluster
  const int p0 = sq.len - sq.n_q;           // position of row 0
  const AttendSpan span = attend_span(p, p0 + r0 / G, p0 + (r0 + rows - 1) / G, kBlockSize);
  auto row_offset = [&](int r, int64_t rstride, int64_t hstride) {
    return (int64_t)(sq.row0 + (r0 + r) / G) * rstride + (int64_t)(kvh * G + (r0 + r) % G) * hstride;
  };

  // page of step i of this cluster, -1 past the end or when its entry is out of range
  const int steps = span.count();
  auto page_id = [&](int i) -> int32_t {
    if (i >= steps) return -1;
    const int32_t id = p.block_table[(int64_t)b * p.bt_stride + span.at(i)];
    if (id >= 0 && id < p.num_blocks) return id;
    if (lane == 0) report_error(p.err, TQ_DEVERR_BLOCK_RANGE);
    return -1;
  };
  struct Tile {
    uint32_t kw0[KS::NW], kw1[KS::NW], vw[4][VS::NW];
    float nK[2], nV[2];
  };
  auto load_tile = [&](Tile& t, int32_t id) {
    const uint8_t* base = p.pages + (int64_t)id * p.blk_stride + (int64_t)kvh * p.slot_stride;
    load_share<D, KB, 4>(t.kw0, base + gid * p.row_stride, tig);
    load_share<D, KB, 4>(t.kw1, base + (gid + 8) * p.row_stride, tig);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint8_t* sl = base + (gid + 8 * r) * p.row_stride;
      t.nK[r] = *(const float*)(sl + C::KPACK);
      t.nV[r] = *(const float*)(sl + p.k_region + C::VPACK);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_share<D, VB, 8>(t.vw[i], base + (2 * tig + (i & 1) + 8 * (i >> 1)) * p.row_stride + p.k_region,
                           gid);
  };

  // the first pages are on their way while the tables and the queries are made
  const int stride = ctas * kRowsWarps;
  int step = split * kRowsWarps + warp;
  Tile next;
  int32_t id = page_id(step), id_next = page_id(step + stride);
  if (id >= 0) load_tile(next, id);

  lut_build<KB, 0>(lut, p.kc, tid, kRowsWarps * 32);
  lut_build<VB, 1>(lut, p.vc, tid, kRowsWarps * 32);
  // q' of row `warp`: sign flips, FWHT, 1/sqrt(D), then to unit length in fp16
  {
    float x[E];
    const bool in = warp < rows;
    const int64_t off = row_offset(warp, p.q_rstride, p.q_hstride) + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = in ? load_as_f32(p.q, off + i, p.q_dtype) : 0.f;
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
    for (int i = 0; i < E; ++i) qh[warp * D + lane * E + i] = __float2half_rn(x[i] * inv);
    if (lane == 0) qsc[warp] = nrm * p.scale_log2;
  }
  __syncthreads();

  uint32_t qb[C::KSTEPS][2];
#pragma unroll
  for (int ks = 0; ks < C::KSTEPS; ++ks) {
    qb[ks][0] = *(const uint32_t*)(qh + gid * D + KS::coord(tig, 4 * ks));
    qb[ks][1] = *(const uint32_t*)(qh + gid * D + KS::coord(tig, 4 * ks + 2));
  }
  // this thread's two rows 2 tig + e: scale, position, first key of the window
  float qscale[2], M[2], l[2];
  int pos[2], low[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 2 * tig + e;
    qscale[e] = qsc[r];
    pos[e] = r < rows ? p0 + (r0 + r) / G : -1;
    low[e] = p.window > 0 ? (int)max((int64_t)0, (int64_t)pos[e] - p.window + 1) : 0;
    M[e] = -INFINITY;
    l[e] = 0.f;
  }
  float acc[C::MT][4];
#pragma unroll
  for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[mt][k] = 0.f;
  const uint32_t lk = 4u * lane, lv = 128u + 4u * lane;
  auto look = [&](uint32_t a) { return *(const uint32_t*)(lut + a); };

  for (; step < steps; step += stride) {
    const Tile t = next;
    const int32_t cur = id;
    id = id_next;
    id_next = page_id(step + 2 * stride);
    if (id >= 0) load_tile(next, id);
    if (cur < 0) continue;

    // ---- S^T = K~ . Qhat^T ----
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    static_for<C::KSTEPS>([&](auto KSI) {
      constexpr int ks = decltype(KSI)::value;
      constexpr int b0 = KS::pos(4 * ks), b2 = KS::pos(4 * ks + 2);
      if constexpr (KB <= 4) {
        mma_16816(s, look(lut_addr<b0, 2 * KB>(t.kw0, lk)), look(lut_addr<b0, 2 * KB>(t.kw1, lk)),
                  look(lut_addr<b2, 2 * KB>(t.kw0, lk)), look(lut_addr<b2, 2 * KB>(t.kw1, lk)),
                  qb[ks][0], qb[ks][1]);
      } else {
        // 8-bit codes: the fp16 centroids, then what they leave (c - fp16(c)), as the
        // whole-sequence decode does
        uint32_t hi[4], lo[4];
        auto one = [&](int i, uint32_t ex, uint32_t ey) {
          hi[i] = __byte_perm(ex, ey, 0x5410);
          lo[i] = __byte_perm(ex, ey, 0x7632);
        };
        one(0, look(lut_addr<b0, KB>(t.kw0, lk)), look(lut_addr<b0 + KB, KB>(t.kw0, lk)));
        one(1, look(lut_addr<b0, KB>(t.kw1, lk)), look(lut_addr<b0 + KB, KB>(t.kw1, lk)));
        one(2, look(lut_addr<b2, KB>(t.kw0, lk)), look(lut_addr<b2 + KB, KB>(t.kw0, lk)));
        one(3, look(lut_addr<b2, KB>(t.kw1, lk)), look(lut_addr<b2 + KB, KB>(t.kw1, lk)));
        mma_16816(s, hi[0], hi[1], hi[2], hi[3], qb[ks][0], qb[ks][1]);
        mma_16816(s, lo[0], lo[1], lo[2], lo[3], qb[ks][0], qb[ks][1]);
      }
    });

    // ---- online softmax: this thread's tokens gid + 8 r, rows 2 tig + e ----
    const int t0 = span.at(step) * kBlockSize + gid;
    float sv[2][2], z[2];
    bool see[2][2], need = false;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      z[e] = -INFINITY;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int tok = t0 + 8 * r;
        see[e][r] = tok <= pos[e] && (tok >= low[e] || tok < p.sinks);
        sv[e][r] = see[e][r] ? s[2 * r + e] * t.nK[r] * qscale[e] : -INFINITY;
        // floor at 2^-100 keeps 2^(s - M) finite for rows of (near) zero V norm
        z[e] = fmaxf(z[e], sv[e][r] + fmaxf(log2_bound(t.nV[r]), -100.0f));
      }
      need |= z[e] > M[e] + kLazyRescale;
    }
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) z[e] = fmaxf(z[e], __shfl_xor_sync(0xffffffffu, z[e], o));
        const float to = z[e] > M[e] + kLazyRescale ? z[e] : M[e];
        const float f = M[e] == -INFINITY ? 0.f : exp2f(M[e] - to);
        l[e] *= f;
        M[e] = to;
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
          acc[mt][e] *= f;
          acc[mt][2 + e] *= f;
        }
      }
    }
    float pv[2][2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float ref = M[e] == -INFINITY ? 0.f : M[e];   // a row that has seen nothing yet
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float w = ex2_approx(sv[e][r] - ref);       // 0 for a key the row does not see
        l[e] += w;
        pv[e][r] = see[e][r] ? w * t.nV[r] : 0.f;         // whose norm may be anything
      }
    }
    const uint32_t pb0 = movmatrix_trans(pack_half2(pv[0][0], pv[1][0]));
    const uint32_t pb1 = movmatrix_trans(pack_half2(pv[0][1], pv[1][1]));

    // ---- O'^T += V~^T . P^T ----
    if constexpr (VS::kInterleaved && (VB == 4 || VB == 2)) {
      // codes of tokens A/B and C/D side by side: lo the even codes of a word, hi the odd
      constexpr uint32_t M1 = VB == 4 ? 0x0F0F0F0Fu : 0x33333333u;
      static_for<VS::NW>([&](auto JI) {
        constexpr int j = decltype(JI)::value;
        constexpr int PER = VS::PW / 2;
        const uint32_t loAB = (t.vw[0][j] & M1) | ((t.vw[1][j] << VB) & ~M1);
        const uint32_t hiAB = ((t.vw[0][j] >> VB) & M1) | (t.vw[1][j] & ~M1);
        const uint32_t loCD = (t.vw[2][j] & M1) | ((t.vw[3][j] << VB) & ~M1);
        const uint32_t hiCD = ((t.vw[2][j] >> VB) & M1) | (t.vw[3][j] & ~M1);
        static_for<PER>([&](auto KI) {
          constexpr int k = decltype(KI)::value;
          mma_16816(acc[j * PER + k], look(lut_addr1<2 * VB * k, 2 * VB>(loAB, lv)),
                    look(lut_addr1<2 * VB * k, 2 * VB>(hiAB, lv)),
                    look(lut_addr1<2 * VB * k, 2 * VB>(loCD, lv)),
                    look(lut_addr1<2 * VB * k, 2 * VB>(hiCD, lv)), pb0, pb1);
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
        mma_16816(acc[mt], two(P0{}, t.vw[0], t.vw[1]), two(P1{}, t.vw[0], t.vw[1]),
                  two(P0{}, t.vw[2], t.vw[3]), two(P1{}, t.vw[2], t.vw[3]), pb0, pb1);
      });
    }
  }

  // ---- the warps' partials [row][O' in natural order, M, l] ----
  __syncthreads();                            // the tables are no longer read
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float sum = l[e];
    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    float* rec = wpart + (warp * kRowsMax + 2 * tig + e) * PART;
    if (gid == 0) {
      // a sum that is not a number must survive the join, which drops empty partials
      rec[D] = sum != sum && M[e] == -INFINITY ? -3e38f : M[e];
      rec[D + 1] = sum;
    }
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) {
      rec[VS::coord(gid, 2 * mt)] = acc[mt][e];
      rec[VS::coord(gid, 2 * mt + 1)] = acc[mt][e + 2];
    }
  }
  __syncthreads();
  // warp r joins row r's partials: n records at rec(j)
  float Mr = -INFINITY, lr = 0.f, o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.f;
  auto join = [&](int n, auto rec) {
    fold_records<E>(n, [&](int j, float& m, float& ll, float (&v)[E]) {
      const float* r = rec(j);
      m = r[D];
      ll = r[D + 1];
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] = r[lane * E + i];
    }, Mr, lr, o);
  };
  if (warp < rows) join(kRowsWarps, [&](int j) { return wpart + (j * kRowsMax + warp) * PART; });
  if (ctas > 1) {
    if (warp < rows) {
      float* rec = cpart + warp * PART;
      if (lane == 0) {
        rec[D] = Mr;
        rec[D + 1] = lr;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) rec[lane * E + i] = o[i];
    }
    cluster.sync();
    if (warp < rows && warp % ctas == split) {
      Mr = -INFINITY;
      lr = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) o[i] = 0.f;
      join(ctas, [&](int j) { return cluster.map_shared_rank(cpart, j) + warp * PART; });
    }
    cluster.sync();                           // no CTA leaves while its partials may be read
  }
  if (warp < rows && warp % ctas == split) {
    const float inv = lr == 0.f ? 0.f : 1.0f / lr;        // a row that sees nothing: 0
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] *= inv;
    warp_fwht<E>(o, lane);
    const int64_t off = row_offset(warp, p.o_rstride, p.o_hstride) + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i)
      store_from_f32(p.out, off + i, p.out_dtype,
                     __uint_as_float(__float_as_uint(o[i] * inv_sqrt_dim<D>()) ^
                                     sign_mask_at(p.sign_seed, lane * E + i)));
  }
}

}  // namespace tq
