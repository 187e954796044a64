// Tile attention kernels for head_dim 256 with 4-bit K codes.
#include "tq_attend_launch.cuh"

namespace tq {
TQ_DEFINE_TILES(256, 4)
}
