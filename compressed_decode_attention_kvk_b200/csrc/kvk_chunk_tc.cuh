// kvk_chunk_tc.cuh -- host interface and workspace of the tensor-core chunk attention.
#pragma once

#include "kvk_paged.cuh"

namespace kvk {

constexpr int kPieceCost = 2;   // cost of a row tile beside its 128-token blocks

// Header of one partial row tile (two per cluster: the tile its slice starts within, and the one
// that it starts but does not finish).
struct ChunkPartial {
  int32_t valid, seq, flat0, row0, rows, b1, nblk, pad;
};

struct ChunkWork {
  ChunkPartial* head;   // [G][2]
  float* ml;            // [G][2][128][2]: reference (log2 units) and weight sum of each row
  float* o;             // [G][2][128][d]: un-normalised outputs
  int G;                // clusters
};

// Bytes of the workspace; carves it when base != nullptr.
size_t chunk_workspace(int d, int G, void* base, ChunkWork* w);
bool chunk_tc_supported(const kvk_layout* L, const AnchorDesc& A, int dtype);
cudaError_t launch_chunk_tc(const ChunkArgs& a, const ChunkWork& w, int dtype, cudaStream_t st);

// two outputs as one 32-bit word of bf16 or f16
__device__ __forceinline__ uint32_t pack_out(int bf16, float x, float y) {
  if (bf16) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __half2 r = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&r);
}

}  // namespace kvk
