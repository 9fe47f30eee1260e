// kvk_chunk_tc.cuh -- host interface and workspace of the tensor-core chunk attention.
#pragma once

#include "kvk_paged.cuh"

namespace kvk {

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
  // expanded rows (nullptr: the kernel converts the packed rows itself): operand rows
  // [pool_slots][64 row_atoms] of 16-bit elements, their low parts, and a mark per slot
  void* hi;
  void* lo;
  float* mark;
  int pool_slots;
};

// 64-element atoms of an operand row: the latent part padded to whole 128 elements (a CTA of the
// pair supplies half of it to the output MMA), then the RoPE part padded to 64.
inline int latent_atoms(int d) { return (d + 127) / 128 * 2; }
inline int row_atoms(int d, int d_rope) { return latent_atoms(d) + (d_rope + 63) / 64; }
// Whether the score operand has a low part (16-bit codes, group scales).
inline bool chunk_split(int b, int group) { return b == 16 || group != 0; }

// Bytes of the workspace, with or without the expanded rows; carves it when base != nullptr.
size_t chunk_workspace(const AnchorDesc& A, int d_rope, int group, int64_t slots, int G, bool expand,
                       void* base, ChunkWork* w);
// Expands the rows of every sequence that has queries (kvk_chunk_expand.cu).
cudaError_t launch_chunk_expand(const ChunkArgs& a, const ChunkWork& w, cudaStream_t st);
bool chunk_tc_supported(const kvk_layout* L, const AnchorDesc& A, int dtype);
// Registers a thread that the kernel's two instances for these rows (converting, expanded) were
// built with; 0 where they differ, or the device does not tell.
int chunk_tc_regs(int b, int group);
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
