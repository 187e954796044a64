// Tile attention kernels for head_dim 128 with 2-bit K codes.
#include "tq_attend_launch.cuh"

namespace tq {
TQ_DEFINE_TILES(128, 2)
}
