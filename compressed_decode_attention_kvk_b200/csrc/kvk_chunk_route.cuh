// kvk_chunk_route.cuh -- which kernel a chunk call takes.
#pragma once

#include "kvk.h"

namespace kvk {

// Registers a thread that the tensor-core kernel has to be launched with: its warpgroups hand
// registers to one another, and an increase would wait for ever for registers that the block does
// not hold.  Another compiler may come to another number.
constexpr int kChunkLaunchRegs = 128;

// The kernel of a chunk call, or -1: the tensor-core kernel where it takes the types and widths
// (`tensor`) and was built with the registers it needs (`regs`, what the device reports; negative:
// no device to ask), the CUDA-core kernel (`cuda_core`: it holds the widths) otherwise, as the
// layout's decode path allows.
inline int chunk_route(int decode_path, bool tensor, int regs, bool cuda_core) {
  if (decode_path != KVK_PATH_CUDA_CORE && tensor && (regs < 0 || regs == kChunkLaunchRegs))
    return KVK_PATH_TENSOR;
  if (decode_path == KVK_PATH_TENSOR || decode_path == KVK_PATH_TENSOR_GENERAL) return -1;
  return cuda_core ? KVK_PATH_CUDA_CORE : -1;
}

}  // namespace kvk
