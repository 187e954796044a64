// tq_pages_launch.cuh -- host-side launch functions of the page operations.
#pragma once

#include "tq_launch.cuh"
#include "tq_pages.cuh"

namespace tq {

tq_status launch_pages_resize(const PlanParams& p, const PageLayers& layers, const DeviceInfo& di,
                              cudaStream_t st);
tq_status launch_pages_fork(const PlanParams& p, const PageLayers& layers, const DeviceInfo& di,
                            cudaStream_t st);
tq_status launch_pages_compact(const CompactParams& p, const PageLayers& layers, int batch,
                               cudaStream_t st);

}  // namespace tq
