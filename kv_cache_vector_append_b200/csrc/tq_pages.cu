// Launches of the page operations (tq_pages.cuh).
#include "tq_pages_launch.cuh"

namespace tq {

namespace {

// At most kFusedLayers layers as a small kernel argument.
FewLayers few_layers(const PageLayers& layers) {
  FewLayers few{};
  few.count = layers.count;
  for (int l = 0; l < layers.count; ++l) {
    few.base[l] = layers.base[l];
    few.blk_stride[l] = layers.blk_stride[l];
    few.page_bytes[l] = layers.page_bytes[l];
  }
  return few;
}

// The plan runs as one cluster: a CTA per 8192 pages, at most the portable cluster size, which
// it has where it also does the rest (*fused).
template <bool FORK>
tq_status launch_plan(const PlanParams& p, const PageLayers& layers, const DeviceInfo& di,
                      cudaStream_t st, bool* fused) {
  int pieces = 1;
  for (int l = 0; l < layers.count; ++l)
    pieces = std::max(pieces, (layers.page_bytes[l] + kCopyPiece - 1) / kCopyPiece);
  *fused = layers.count <= kFusedLayers &&
           (int64_t)p.requests * layers.count * pieces <= kFusedChunks &&
           (int64_t)p.requests * ((p.cols + 127) / 128) <= kFusedChunks;
  const FewLayers few = *fused ? few_layers(layers) : FewLayers{};
  int ctas = *fused ? kPlanMaxCtas : 1;
  while (ctas < kPlanMaxCtas && (int64_t)ctas * 8192 < p.pool) ctas *= 2;
  const size_t smem = plan_smem(p.pool, ctas, p.requests, FORK ? p.batch : 0);
  if (smem + 1024 > (size_t)di.max_smem_optin) return TQ_ERR_UNSUPPORTED;
  auto kern = *fused ? pages_plan_kernel<FORK, true> : pages_plan_kernel<FORK, false>;
  // (48 KB with the static part need no opting in; the same value always, as threads may call
  // at once)
  if (smem > 40 * 1024 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               di.max_smem_optin - 1024) != cudaSuccess)
    return cuda_failed();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p, few, pieces) != cudaSuccess) return cuda_failed();
  return launch_status();
}

}  // namespace

tq_status launch_pages_resize(const PlanParams& p, const PageLayers& layers, const DeviceInfo& di,
                              cudaStream_t st) {
  bool fused = false;
  const tq_status s = launch_plan<false>(p, layers, di, st, &fused);
  if (s != TQ_OK || fused) return s;
  pages_resize_kernel<<<dim3(p.batch, 1 + layers.count), kPagesThreads, 0, st>>>(p, layers);
  return launch_status();
}

tq_status launch_pages_fork(const PlanParams& p, const PageLayers& layers, const DeviceInfo& di,
                            cudaStream_t st) {
  bool fused = false;
  const tq_status s = launch_plan<true>(p, layers, di, st, &fused);
  if (s != TQ_OK || fused) return s;
  const int chunks = std::min((p.cols + kForkChunk - 1) / kForkChunk, kForkMostChunks);
  pages_fork_kernel<<<dim3(p.requests, chunks + layers.count), kPagesThreads, 0, st>>>(p, layers,
                                                                                       chunks);
  return launch_status();
}

template <typename U, class Layers>
void launch_compact_t(const CompactParams& p, const Layers& layers, dim3 grid, cudaStream_t st) {
  pages_compact_kernel<U, Layers><<<grid, kPagesThreads, 0, st>>>(p, layers);
}

tq_status launch_pages_compact(const CompactParams& p, const PageLayers& layers, int batch,
                               cudaStream_t st) {
  const dim3 grid((p.max_keep + kPageTokens - 1) / kPageTokens, batch, layers.count);
  // rows of every layer in 16-byte units where they are multiples of 16 bytes, else 8
  bool wide = true;
  for (int l = 0; l < layers.count; ++l) wide = wide && layers.page_bytes[l] / kPageTokens % 16 == 0;
  if (layers.count <= kFusedLayers) {
    const FewLayers few = few_layers(layers);
    if (wide) launch_compact_t<uint4>(p, few, grid, st);
    else launch_compact_t<uint2>(p, few, grid, st);
  } else {
    if (wide) launch_compact_t<uint4>(p, layers, grid, st);
    else launch_compact_t<uint2>(p, layers, grid, st);
  }
  return launch_status();
}

}  // namespace tq
