// tq_attend_launch.cuh -- host-side launch of the attention over chunks and windows.
#pragma once

#include "tq_attend_rows.cuh"
#include "tq_attend_tiles.cuh"
#include "tq_launch.cuh"

namespace tq {

template <int D, int KB, int VB>
tq_status launch_rows_t(const AttendParams& p, const DeviceInfo& di, cudaStream_t st) {
  auto kern = attend_rows_kernel<D, KB, VB>;
  constexpr int smem = rows_smem(D, KB, VB);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TQ_ERR_CUDA;
  // CTAs a cluster: enough for two CTAs an SM, as long as each warp keeps two pages or more
  const int tiles = (int)(((int64_t)p.max_q * p.group + kRowsMax - 1) / kRowsMax);
  int64_t steps = p.max_blocks;
  if (p.window > 0)
    steps = std::min(steps, ((int64_t)p.window + p.max_q - 1) / kBlockSize + 2 +
                                ((int64_t)p.sinks + kBlockSize - 1) / kBlockSize);
  const int64_t groups = (int64_t)p.batch * p.h_kv * tiles;
  int ctas = 1;
  while (ctas < kRowsMaxCtas && groups * ctas < 2 * di.num_sms &&
         (int64_t)ctas * kRowsWarps * 4 <= steps)
    ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * ctas), (unsigned)p.h_kv, (unsigned)tiles);
  cfg.blockDim = dim3(kRowsWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return TQ_ERR_CUDA;
  return launch_status();
}

template <int D, int KB, int VB>
tq_status launch_tiles_t(AttendParams p, const DeviceInfo& di, cudaStream_t st) {
  using C = TilesCfg<D, KB, VB>;
  auto kern = attend_tiles_kernel<D, KB, VB>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return TQ_ERR_CUDA;
  // the split of registers between the warpgroups counts on the launch's own number
  static const bool regs_ok = [&] {
    cudaFuncAttributes a{};
    return cudaFuncGetAttributes(&a, kern) == cudaSuccess && a.numRegs == kTilesRegs;
  }();
  if (!regs_ok) return TQ_ERR_CUDA;
  const int64_t rows = (int64_t)p.max_q * p.group;
  p.tile_rows = C::kTwoTiles && rows > kTileRows ? 2 * kTileRows : kTileRows;
  const int tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
  int64_t steps = p.max_blocks;
  if (p.window > 0)
    steps = std::min(steps, ((int64_t)p.window + p.tile_rows / p.group) / kBlockSize + 3 +
                                ((int64_t)p.sinks + kBlockSize - 1) / kBlockSize);
  // CTAs a cluster: until the grid fills the SMs twice, each keeping 512 keys or more
  const int64_t groups = (int64_t)p.batch * p.h_kv * tiles;
  int ctas = 1;
  while (ctas < kTilesMaxCtas && groups * ctas < 2 * di.num_sms && (int64_t)ctas * 64 <= steps) ctas *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.batch * ctas), (unsigned)p.h_kv, (unsigned)tiles);
  cfg.blockDim = dim3(kTilesThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return TQ_ERR_CUDA;
  return launch_status();
}

// All V widths for one (head_dim, K width); instantiated in tq_attend_d<D>_k<KB>.cu so that
// the kernels compile in parallel.
template <int D, int KB>
tq_status launch_rows_kbits(int vb, const AttendParams& p, const DeviceInfo& di, cudaStream_t st) {
  switch (vb) {
    case 2: return launch_rows_t<D, KB, 2>(p, di, st);
    case 3: return launch_rows_t<D, KB, 3>(p, di, st);
    case 4: return launch_rows_t<D, KB, 4>(p, di, st);
    case 8: return launch_rows_t<D, KB, 8>(p, di, st);
    default: return TQ_ERR_UNSUPPORTED;
  }
}

template <int D, int KB>
tq_status launch_tiles_kbits(int vb, const AttendParams& p, const DeviceInfo& di, cudaStream_t st) {
  switch (vb) {
    case 2: return launch_tiles_t<D, KB, 2>(p, di, st);
    case 3: return launch_tiles_t<D, KB, 3>(p, di, st);
    case 4: return launch_tiles_t<D, KB, 4>(p, di, st);
    case 8: return launch_tiles_t<D, KB, 8>(p, di, st);
    default: return TQ_ERR_UNSUPPORTED;
  }
}

#define TQ_DECLARE_TILES(D_, KB_)                                                          \
  tq_status launch_tiles_d##D_##_k##KB_(int vb, const AttendParams& p, const DeviceInfo& di, \
                                        cudaStream_t st);
#define TQ_DEFINE_TILES(D_, KB_)                                                           \
  tq_status launch_tiles_d##D_##_k##KB_(int vb, const AttendParams& p, const DeviceInfo& di, \
                                        cudaStream_t st) {                                  \
    return launch_tiles_kbits<D_, KB_>(vb, p, di, st);                                      \
  }
TQ_FOR_EACH_DECODE(TQ_DECLARE_TILES)

#define TQ_DECLARE_ROWS(D_, KB_)                                                          \
  tq_status launch_rows_d##D_##_k##KB_(int vb, const AttendParams& p, const DeviceInfo& di, \
                                       cudaStream_t st);
#define TQ_DEFINE_ROWS(D_, KB_)                                                           \
  tq_status launch_rows_d##D_##_k##KB_(int vb, const AttendParams& p, const DeviceInfo& di, \
                                       cudaStream_t st) {                                  \
    return launch_rows_kbits<D_, KB_>(vb, p, di, st);                                      \
  }
TQ_FOR_EACH_DECODE(TQ_DECLARE_ROWS)

inline tq_status launch_attend_any(int dim, int kb, int vb, const AttendParams& p,
                                   const DeviceInfo& di, cudaStream_t st) {
  const bool tiles = (int64_t)p.max_q * p.group > kRowsMax;
#define TQ_ROWS_CASE(D_, KB_)                                                             \
  if (dim == D_ && kb == KB_)                                                             \
    return tiles ? launch_tiles_d##D_##_k##KB_(vb, p, di, st) : launch_rows_d##D_##_k##KB_(vb, p, di, st);
  TQ_FOR_EACH_DECODE(TQ_ROWS_CASE)
#undef TQ_ROWS_CASE
  return TQ_ERR_UNSUPPORTED;
}

}  // namespace tq
