#include "csrc/attend_tile.h"
namespace qlin { namespace {
template __global__ void attend_tile_kernel<QLIN_BF16,AFFINE,128,2,1,true,4>(TileArgs);
} }
