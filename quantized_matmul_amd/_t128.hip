#include "csrc/attend_prompt.h"
namespace qlin { namespace {
template __global__ void attend_prompt_kernel<QLIN_BF16,128,2>(TileArgs, int64_t);
} }
