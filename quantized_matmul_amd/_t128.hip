#include "csrc/attend_tile.h"
namespace qlin { namespace {
template __global__ void attend_tile_kernel<QLIN_F16,NVFP4,64,1,3,false>(TileArgs);
} }
