// kvk_chunk_expand.cu -- the pool's rows as tensor-core operands, ahead of the chunk attention.
//
// A sequence with many query rows is read by many row tiles, and converting its packed rows in
// each of them costs more issue slots than the MMAs leave.  This kernel converts every token of
// the sequences with queries once, into rows of 16-bit elements (and their low parts) at the
// token's own slot of a scratch pool, from where the attention kernel loads whole atoms with
// the tensor memory accelerator.  Sequences that share a page write the same values.
//
// One warp per 8 tokens, 16 elements a lane and step (32-byte stores, consecutive lanes
// consecutive): memory bound, row_bytes read and 128 bytes per atom (and part) written a token.
#include <math_constants.h>

#include <algorithm>

#include "kvk_chunk_convert.cuh"
#include "kvk_chunk_tc.cuh"

namespace kvk {
namespace {

using namespace chunk;

constexpr int kExpandWarps = 8;
constexpr int kTokens = 8;   // per warp and round

template <int BITS, bool GROUP>
__global__ void __launch_bounds__(kExpandWarps * 32)
chunk_expand_kernel(const __grid_constant__ ChunkArgs a, uint8_t* __restrict__ hi_p,
                    uint8_t* __restrict__ lo_p, float* __restrict__ mark, int NL, int NA) {
  constexpr bool kBf16 = BITS == KVK_BITS_BF16;
  constexpr bool kLo = kSplit<BITS, GROUP>;
  const int lane = threadIdx.x & 31, seq = blockIdx.y;
  bool bad;
  const ChunkSeq s = chunk_seq(a, seq, &bad);
  if (s.count == 0) return;
  const int units = NA * 4;
  const int step = gridDim.x * kExpandWarps * kTokens;
  for (int64_t t0 = ((int64_t)blockIdx.x * kExpandWarps + (threadIdx.x >> 5)) * kTokens; t0 < s.len;
       t0 += step) {
    const int t = (int)t0 + lane;
    int slot = -1;
    if (lane < kTokens && t < s.len) slot = chunk_slot(a, seq, t);
    uint32_t odd = 0;   // tokens with a non-finite element
    for (int i0 = 0; i0 < kTokens * units; i0 += 32) {
      const int i = i0 + lane;
      const int tok = i / units, u = i - tok * units;     // (8 units are whole rounds of 32)
      const int sl = __shfl_sync(0xffffffffu, slot, tok & (kTokens - 1));
      if (sl < 0) continue;
      const int at = u >> 2, x = (at < NL ? at : at - NL) * 64 + 16 * (u & 3);
      const int e = at < NL ? (x < a.d ? x : -1) : (x < a.d_rope ? a.d + x : -1);
      uint32_t hi[8], lo[8];
      if (e >= 0) {
        Unit<BITS, GROUP> v;
        load_unit<BITS, GROUP>(a, row_of<GROUP>(a, sl), e, v);
        convert16<BITS, GROUP, kLo>(v.w, v.s, hi, lo);
        if constexpr (kBf16 || GROUP) {
          if (nonfinite16<kBf16>(hi)) {
            odd |= 1u << tok;
            replace_nonfinite<kBf16>(hi, 0u);
            if constexpr (kLo) replace_nonfinite<kBf16>(lo, 0u);
          }
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) hi[k] = 0u, lo[k] = 0u;
      }
      const int64_t to = (int64_t)sl * NA * 128 + u * 32;
      uint4* ph = reinterpret_cast<uint4*>(hi_p + to);
      ph[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      ph[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
      if constexpr (kLo) {
        uint4* pl = reinterpret_cast<uint4*>(lo_p + to);
        pl[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        pl[1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
      }
    }
    odd = __reduce_or_sync(0xffffffffu, odd);
    if (slot >= 0) mark[slot] = odd >> lane & 1 ? CUDART_NAN_F : 0.0f;
  }
}

// The rows between a sequence's end and the end of the last box that it reads hold anything, NaN
// among it, which a zero weight does not silence: they become zero, ahead of the conversion (the
// page may be shared with a longer sequence, whose rows are written after it).
__global__ void __launch_bounds__(256)
chunk_tail_kernel(const __grid_constant__ ChunkArgs a, uint8_t* __restrict__ hi_p,
                  uint8_t* __restrict__ lo_p, int NA, int box) {
  bool bad;
  const ChunkSeq s = chunk_seq(a, blockIdx.x, &bad);
  const int rest = -s.len & (box - 1);
  if (s.count == 0 || rest == 0) return;
  const int slot = chunk_slot(a, blockIdx.x, s.len - 1);
  if (slot < 0) return;
  const int64_t from = (int64_t)(slot + 1) * NA * 8;      // 16-byte words
  for (int i = threadIdx.x; i < rest * NA * 8; i += blockDim.x) {
    reinterpret_cast<uint4*>(hi_p)[from + i] = make_uint4(0u, 0u, 0u, 0u);
    if (lo_p) reinterpret_cast<uint4*>(lo_p)[from + i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

template <int BITS, bool GROUP>
cudaError_t launch(const ChunkArgs& a, const ChunkWork& w, cudaStream_t st) {
  // about four CTAs per SM over the whole batch, each at least one round of a sequence
  const int box = std::min(1 << a.page_shift, 64);
  chunk_tail_kernel<<<dim3(a.batch), dim3(256), 0, st>>>(
      a, static_cast<uint8_t*>(w.hi), static_cast<uint8_t*>(w.lo), row_atoms(a.d, a.d_rope), box);
  const int per_round = kExpandWarps * kTokens;
  const int rounds = (a.cap + per_round - 1) / per_round;
  const int gx = std::max(1, std::min(rounds, (8 * 2 * w.G + a.batch - 1) / a.batch));
  chunk_expand_kernel<BITS, GROUP><<<dim3(gx, a.batch), dim3(kExpandWarps * 32), 0, st>>>(
      a, static_cast<uint8_t*>(w.hi), static_cast<uint8_t*>(w.lo), w.mark, latent_atoms(a.d),
      row_atoms(a.d, a.d_rope));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk_expand(const ChunkArgs& a, const ChunkWork& w, cudaStream_t st) {
  if (a.group) {
    if (a.b == 2) return launch<2, true>(a, w, st);
    if (a.b == 4) return launch<4, true>(a, w, st);
    if (a.b == 8) return launch<8, true>(a, w, st);
    if (a.b == 16) return launch<16, true>(a, w, st);
  } else {
    if (a.b == KVK_BITS_BF16) return launch<KVK_BITS_BF16, false>(a, w, st);
    if (a.b == 2) return launch<2, false>(a, w, st);
    if (a.b == 4) return launch<4, false>(a, w, st);
    if (a.b == 8) return launch<8, false>(a, w, st);
    if (a.b == 16) return launch<16, false>(a, w, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kvk
