// Launches of the page operations (tq_pages.cuh).
#include "tq_pages_launch.cuh"

namespace tq {

namespace {

// The plan runs as one cluster: a CTA per 8192 pages, at most the portable cluster size.
template <bool FORK>
tq_status launch_plan(const PlanParams& p, const DeviceInfo& di, cudaStream_t st) {
  int ctas = 1;
  while (ctas < kPlanMaxCtas && (int64_t)ctas * 8192 < p.pool) ctas *= 2;
  const size_t smem = plan_smem(p.pool, ctas, p.requests, FORK ? p.batch : 0);
  if (smem + 1024 > (size_t)di.max_smem_optin) return TQ_ERR_UNSUPPORTED;
  auto kern = pages_plan_kernel<FORK>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess)
    return TQ_ERR_CUDA;
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
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return TQ_ERR_CUDA;
  return launch_status();
}

}  // namespace

tq_status launch_pages_resize(const PlanParams& p, const PageLayers& layers, const DeviceInfo& di,
                              cudaStream_t st) {
  const tq_status s = launch_plan<false>(p, di, st);
  if (s != TQ_OK) return s;
  pages_resize_kernel<<<dim3(p.batch, 1 + layers.count), kPagesThreads, 0, st>>>(p, layers);
  return launch_status();
}

tq_status launch_pages_fork(const PlanParams& p, const PageLayers& layers, const DeviceInfo& di,
                            cudaStream_t st) {
  const tq_status s = launch_plan<true>(p, di, st);
  if (s != TQ_OK) return s;
  const int chunks = (p.cols + kForkChunk - 1) / kForkChunk;
  pages_fork_kernel<<<dim3(p.requests, chunks + layers.count), kPagesThreads, 0, st>>>(p, layers,
                                                                                       chunks);
  return launch_status();
}

tq_status launch_pages_compact(const CompactParams& p, const PageLayers& layers, int batch,
                               cudaStream_t st) {
  const dim3 grid((p.max_keep + kPageTokens - 1) / kPageTokens, batch, layers.count);
  // rows of every layer in 16-byte units where they are multiples of 16 bytes, else 8
  bool wide = true;
  for (int l = 0; l < layers.count; ++l) wide = wide && layers.page_bytes[l] / kPageTokens % 16 == 0;
  if (wide) pages_compact_kernel<uint4><<<grid, kPagesThreads, 0, st>>>(p, layers);
  else pages_compact_kernel<uint2><<<grid, kPagesThreads, 0, st>>>(p, layers);
  return launch_status();
}

}  // namespace tq
