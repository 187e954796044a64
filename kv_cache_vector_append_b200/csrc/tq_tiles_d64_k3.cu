// Tile attention kernels for head_dim 64 with 3-bit K codes.
#include "tq_attend_launch.cuh"

namespace tq {
TQ_DEFINE_TILES(64, 3)
}
