// tq_attend_launch.cuh -- host-side launch of the attention over chunks and windows.
#pragma once

#include <algorithm>

#include "tq_attend_rows.cuh"
#include "tq_attend_tiles.cuh"
#include "tq_launch.cuh"
#include "tq_memo.cuh"

namespace tq {

// Rows a KV head up to which the rows kernel is used.  us of the rows / tiles kernel, 8 sequences of
// 4,096 tokens: 16/2 heads of 64, 8/8 bits, 32 rows 26 / 45 (48 rows of 64 sequences of 500 38 / 36);
// 32/8 heads of 128, 4/4 bits, 32 rows 45 / 82, 48 rows 80 / 81; 16/4 heads of 256, 4/4 bits, where a
// block takes 8 rows, 16 rows 55 / 61, 24 rows 82 / 61 (and 85 / 64 of 16 windows of 2,048 tokens, 87 /
// 75 of 64 sequences of 500, but 122 / 173 of one of 32,768).
constexpr int rows_most(int dim) { return dim == 256 ? 16 : 32; }
constexpr int kAttendMaxCtas = 8;          // the portable cluster size

// Launches the kernel as clusters of 1 to 8 CTAs that split the keys of a group of rows.  Of the
// counts that leave a CTA `least` units of keys or more, the one is taken whose waves of CTAs
// times a CTA's time are least; alone and joined are the times of a CTA's start and end in
// units of keys, without and with a join.
template <auto kern>
tq_status launch_attend(AttendParams p, int64_t tiles, int threads, int smem, int64_t units,
                        int alone, int joined, int least, cudaStream_t st) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices ||
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return cuda_failed();
  tiles = std::max<int64_t>(tiles, 1);       // max_q = 0: ranges are still checked
  const int64_t groups = (int64_t)p.batch * p.h_kv * tiles;
  if (groups > 0x7fffffff / 8) return TQ_ERR_UNSUPPORTED;
  p.row_tiles = (int32_t)tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto grid = [&](int ctas) {
    attr[0].val.clusterDim.x = (unsigned)ctas;
    cfg.gridDim = dim3((unsigned)(groups * ctas));
  };
  // clusters of each size that the device holds at once (0: none of that size)
  static Memo<kMaxDevices * kAttendMaxCtas> fit;
  int best = 1;
  int64_t best_cost = 0;
  for (int ctas = 1; ctas <= kAttendMaxCtas; ++ctas) {
    if (ctas > 1 && units < (int64_t)ctas * least) break;
    int n = 0;
    const bool known = fit.get(dev * kAttendMaxCtas + ctas - 1, [&](int* a) {
      grid(ctas);
      return cudaOccupancyMaxActiveClusters(a, kern, &cfg) == cudaSuccess;
    }, &n);
    if (!known || n < 1) {
      if (ctas == 1) return cuda_failed();
      if (!known) cuda_failed();
      continue;
    }
    const int64_t cost = (groups + n - 1) / n * ((ctas > 1 ? joined : alone) + (units + ctas - 1) / ctas);
    if (ctas == 1 || cost < best_cost) {
      best = ctas;
      best_cost = cost;
    }
  }
  grid(best);
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return cuda_failed();
  return launch_status();
}

// Pages of the longest span of keys that `tokens` consecutive tokens may see.
inline int64_t attend_pages(const AttendParams& p, int64_t tokens) {
  if (p.window == 0) return p.max_blocks;
  return std::min<int64_t>(p.max_blocks, (p.window + tokens) / kBlockSize + 2 +
                                             ((int64_t)p.sinks + kBlockSize - 1) / kBlockSize);
}

template <int D, int KB, int VB, int NT>
tq_status launch_rows_t(const AttendParams& p, cudaStream_t st) {
  const int64_t rows = (int64_t)p.max_q * p.group;
  // start and end of a CTA: about 8 us, 48 pages of its eight warps
  return launch_attend<attend_rows_kernel<D, KB, VB, NT>>(
      p, (rows + 8 * NT - 1) / (8 * NT), kRowsWarps * 32, rows_smem(D, KB, VB, NT),
      attend_pages(p, 8 * NT), 48, 48, kRowsWarps, st);
}

template <int D, int KB, int VB>
tq_status launch_tiles_t(AttendParams p, cudaStream_t st) {
  using C = TilesCfg<D, KB, VB>;
  // the split of registers between the warpgroups counts on the launch's own number
  static Memo<1> regs;
  int n = 0;
  if (!regs.get(0, [](int* a) {
        cudaFuncAttributes f{};
        if (cudaFuncGetAttributes(&f, attend_tiles_kernel<D, KB, VB>) != cudaSuccess) return false;
        *a = f.numRegs;
        return true;
      }, &n))
    return cuda_failed();
  if (n != kTilesRegs) return TQ_ERR_CUDA;
  const int64_t rows = (int64_t)p.max_q * p.group;
  p.tile_rows = C::kTwoTiles && rows > kTileRows ? 2 * kTileRows : kTileRows;
  const int64_t units = (attend_pages(p, p.tile_rows / p.group) + C::PPT - 1) / C::PPT;
  // start and end of a CTA: about 16 us, or 35 us with a join, at 2.3 us a key tile
  return launch_attend<attend_tiles_kernel<D, KB, VB>>(p, (rows + p.tile_rows - 1) / p.tile_rows,
                                                       kTilesThreads, C::SMEM, units, 7, 15, 2, st);
}

// All V widths for one (head_dim, K width); instantiated in tq_attend_d<D>_k<KB>.cu so that
// the kernels compile in parallel.
template <int D, int KB, int VB>
tq_status launch_rows_n(const AttendParams& p, cudaStream_t st) {
  const int64_t rows = (int64_t)p.max_q * p.group;
  if constexpr (rows_tiles(D) == 4)
    if (rows > 16) return launch_rows_t<D, KB, VB, 4>(p, st);
  if constexpr (rows_tiles(D) >= 2)
    if (rows > 8) return launch_rows_t<D, KB, VB, 2>(p, st);
  return launch_rows_t<D, KB, VB, 1>(p, st);
}
template <int D, int KB>
tq_status launch_rows_kbits(int vb, const AttendParams& p, cudaStream_t st) {
  switch (vb) {
    case 2: return launch_rows_n<D, KB, 2>(p, st);
    case 3: return launch_rows_n<D, KB, 3>(p, st);
    case 4: return launch_rows_n<D, KB, 4>(p, st);
    case 8: return launch_rows_n<D, KB, 8>(p, st);
    default: return TQ_ERR_UNSUPPORTED;
  }
}

template <int D, int KB>
tq_status launch_tiles_kbits(int vb, const AttendParams& p, cudaStream_t st) {
  switch (vb) {
    case 2: return launch_tiles_t<D, KB, 2>(p, st);
    case 3: return launch_tiles_t<D, KB, 3>(p, st);
    case 4: return launch_tiles_t<D, KB, 4>(p, st);
    case 8: return launch_tiles_t<D, KB, 8>(p, st);
    default: return TQ_ERR_UNSUPPORTED;
  }
}

#define TQ_DECLARE_TILES(D_, KB_)                                                          \
  tq_status launch_tiles_d##D_##_k##KB_(int vb, const AttendParams& p, cudaStream_t st);
#define TQ_DEFINE_TILES(D_, KB_)                                                           \
  tq_status launch_tiles_d##D_##_k##KB_(int vb, const AttendParams& p, cudaStream_t st) { \
    return launch_tiles_kbits<D_, KB_>(vb, p, st);                                         \
  }
TQ_FOR_EACH_DECODE(TQ_DECLARE_TILES)

#define TQ_DECLARE_ROWS(D_, KB_)                                                          \
  tq_status launch_rows_d##D_##_k##KB_(int vb, const AttendParams& p, cudaStream_t st);
#define TQ_DEFINE_ROWS(D_, KB_)                                                           \
  tq_status launch_rows_d##D_##_k##KB_(int vb, const AttendParams& p, cudaStream_t st) {  \
    return launch_rows_kbits<D_, KB_>(vb, p, st);                                          \
  }
TQ_FOR_EACH_DECODE(TQ_DECLARE_ROWS)

inline tq_status launch_attend_any(int dim, int kb, int vb, const AttendParams& p, cudaStream_t st) {
  const bool tiles = (int64_t)p.max_q * p.group > rows_most(dim);
#define TQ_ROWS_CASE(D_, KB_)                                                             \
  if (dim == D_ && kb == KB_)                                                             \
    return tiles ? launch_tiles_d##D_##_k##KB_(vb, p, st) : launch_rows_d##D_##_k##KB_(vb, p, st);
  TQ_FOR_EACH_DECODE(TQ_ROWS_CASE)
#undef TQ_ROWS_CASE
  return TQ_ERR_UNSUPPORTED;
}

}  // namespace tq
