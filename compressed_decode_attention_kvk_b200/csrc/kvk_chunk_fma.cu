// kvk_chunk_fma.cu -- CUDA-core (FFMA) attention of chunks of new tokens over a paged cache.
//
// Query row j of sequence i (position p = len - count + j) and head h:
//     z_t = sigma (q_lat . c_hat_t[:d] + q_rope . c_hat_t[d:]),  t <= p
//     out = sum_t softmax(z)_t c_hat_t[:d],   lse = log sum_t exp(z_t)
// (the absorbed MLA attention of kvk_decode_fma.cu with a causal limit per row and the rows
// found through the block table).  This kernel takes every shape and every query type; fp32
// queries always take it.
//
// Schedule: a cluster of S CTAs per query token and group of 8 heads (one warp per head): the
// token's heads share the dequantised tile of TT tokens in shared memory, CTA z takes tiles z,
// z + S, ...  Every lane scores one token, the warp runs the online softmax (base 2, fp32), lane j
// accumulates features j, j + 32, ...  The CTAs' partials are joined through distributed shared
// memory.  The host picks S (1 to 8) so that the grid fills the GPU: at 3 tokens, 8 heads and 256
// cached tokens the kernel takes 8.1 us with S = 8 and 44.8 us with S = 1.
//
// Bound by shared memory: a score reads two words for each FMA, an output one, and every query token
// unpacks the cache again, once per 8 heads.  5 to 7 TFLOP/s at sizes that fill the GPU: fp32 decode
// of 32 x 8192 tokens of 16 bits, 40 heads, d = 512, 4.6 ms (the tensor-core kernel under bf16
// queries 0.22); f16 queries over bf16 rows of that size 5.5 ms (bf16 queries 0.27); 8 x <= 128 fp32
// rows over 8192 tokens of 4-bit groups, d = 128, 23.6 ms (bf16 queries 0.32).
#include <float.h>

#include <math_constants.h>

#include "kvk_paged.cuh"

namespace kvk {
namespace {

constexpr int kHG = 8;   // heads per CTA = warps per block
constexpr size_t kSmemMax = 227 * 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float load_q(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_q(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_q(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ void store_o(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_o(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_o(__half* p, float v) { *p = __float2half_rn(v); }

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ float load_rank(const float* p, uint32_t rank) {
  uint32_t at;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// The elements of row word i (32 bits) as floats
template <int B>
__device__ __forceinline__ void unpack_word(uint32_t w, bool bf16_rows, float* out) {
  constexpr int kN = 32 / B;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const uint32_t u = (w >> (j * B)) & ((B == 32) ? 0xFFFFFFFFu : ((1u << B) - 1u));
    out[j] = (B == 16 && bf16_rows) ? __uint_as_float(u << 16) : (float)((int)u - (1 << (B - 1)));
  }
}
// One warp dequantises its tokens (i = warp, warp + 8, ...) of a tile into rows of shared memory:
// consecutive lanes take consecutive words of a row.
template <int TT, int B>
__device__ __forceinline__ void load_tile(const ChunkArgs& a, const int32_t* slot_s, float* cs,
                                          int ldc) {
  constexpr int kN = 32 / B;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int words = a.n / kN;            // n is a multiple of 8: exact but for b = 2, see below
  const bool bf16_rows = a.b == KVK_BITS_BF16;
  for (int x0 = 0; x0 < words; x0 += 32) {
    const int x = x0 + lane;
    uint32_t w[TT / kHG];
#pragma unroll
    for (int i = 0; i < TT / kHG; ++i) {
      const int t = slot_s[warp + kHG * i];
      if (t >= 0 && x < words)
        w[i] = __ldg(reinterpret_cast<const uint32_t*>(a.codes + (int64_t)t * a.row_bytes) + x);
    }
#pragma unroll
    for (int i = 0; i < TT / kHG; ++i) {
      const int t = slot_s[warp + kHG * i];
      if (x >= words) continue;
      float v[kN];
      if (t >= 0) {
        unpack_word<B>(w[i], bf16_rows, v);
        if (a.group) {                   // a word's elements share their scale (G >= 16)
          const float s = __half2float(a.scales[(int64_t)t * a.sg + x * kN / a.group]);
#pragma unroll
          for (int j = 0; j < kN; ++j) v[j] *= s;
        }
      } else {
#pragma unroll
        for (int j = 0; j < kN; ++j) v[j] = 0.0f;
      }
      float* dst = cs + (warp + kHG * i) * ldc + x * kN;
#pragma unroll
      for (int j = 0; j < kN; ++j) dst[j] = v[j];
    }
  }
  if (B == 2 && (a.n & 15)) {            // n = 8 (mod 16): the last half word
    for (int i = warp; i < TT; i += kHG) {
      const int t = slot_s[i], k = a.n - 8 + lane;
      if (lane < 8) {
        float v = 0.0f;
        if (t >= 0) {
          const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(
                                       a.codes + (int64_t)t * a.row_bytes) + words);
          v = (float)((int)((u >> (2 * lane)) & 3u) - 2);
          if (a.group) v *= __half2float(a.scales[(int64_t)t * a.sg + k / a.group]);
        }
        cs[i * ldc + k] = v;
      }
    }
  }
}

template <int TT, int R, typename Tq>
__global__ void __launch_bounds__(kHG * 32) chunk_fma_kernel(const __grid_constant__ ChunkArgs a) {
  extern __shared__ float4 smem4[];
  float* smem = reinterpret_cast<float*>(smem4);
  const int n = a.n, d = a.d;
  const int ldc = n + 1;
  float* qs = smem;                                        // [kHG][n]
  float* cs = qs + kHG * n;                                // [TT][n + 1]
  float* ss = cs + TT * ldc;                               // [TT]
  int32_t* slot_s = reinterpret_cast<int32_t*>(ss + TT);   // [TT]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  const int row = blockIdx.x, h = blockIdx.y * kHG + warp;
  const bool hv = h < a.H;

  // the sequence of this query row: the first whose rows end behind it.  Every CTA checks all
  // offsets (they are read for the search anyway): where any is wrong, the call writes nothing.
  int seq = 0;
  bool bad = false;
  for (int i0 = 0; i0 < a.batch; i0 += nt) {
    const int i = i0 + tid;
    bool before = false;
    if (i < a.batch) {
      const int s0 = __ldg(a.q_start + i), s1 = __ldg(a.q_start + i + 1);
      bad = bad || s0 < 0 || s1 < s0 || s1 > a.n_q;
      before = s1 <= row;
    }
    seq += __syncthreads_count(before);
  }
  const bool stop = __syncthreads_or(bad) != 0;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {   // one CTA reports
    for (int i = tid; i < a.batch; i += nt) {
      bool b1;
      chunk_seq(a, i, &b1);
      bad = bad || b1;
    }
    if (bad) atomicOr(a.flags, KVK_FLAG_SEQ_LEN);
  }
  if (stop) return;
  if (seq >= a.batch) return;                  // a row behind the last sequence: left alone
  const ChunkSeq s = chunk_seq(a, seq, &bad);
  if (row < s.row0 || row >= s.row0 + s.count) return;
  const int limit = min(s.len, max(0, s.len - s.count + (row - s.row0) + 1));   // tokens seen

  const Tq* qlat = static_cast<const Tq*>(a.q_lat) + (int64_t)row * a.ql_st;
  const Tq* qrope = static_cast<const Tq*>(a.q_rope) + (int64_t)row * a.qr_st;
  const int S = gridDim.z, z = blockIdx.z;
  const float zscale = a.sigma * kLog2e;
  for (int k = lane; k < n; k += 32) {
    float v = 0.0f;
    if (hv)
      v = (k < d) ? load_q(qlat + (int64_t)h * a.ql_sh + k)
                  : load_q(qrope + (int64_t)h * a.qr_sh + (k - d));
    qs[warp * n + k] = v;
  }
  float m = -INFINITY, l = 0.0f;
  float o[R];
#pragma unroll
  for (int r = 0; r < R; ++r) o[r] = 0.0f;

  for (int p = z * TT; p < limit; p += S * TT) {
    const int cnt = min(TT, limit - p);
    __syncthreads();
    if (tid < TT) {
      const int t = (tid < cnt) ? chunk_slot(a, seq, p + tid) : -1;
      slot_s[tid] = t;
      // a group-scaled cache carries its scales per element (below): unit token scale
      ss[tid] = (t >= 0) ? (a.group ? 1.0f : __half2float(a.scales[t])) : 0.0f;
    }
    __syncthreads();
    if (a.b == 8) load_tile<TT, 8>(a, slot_s, cs, ldc);
    else if (a.b == 4) load_tile<TT, 4>(a, slot_s, cs, ldc);
    else if (a.b == 2) load_tile<TT, 2>(a, slot_s, cs, ldc);
    else load_tile<TT, 16>(a, slot_s, cs, ldc);     // 16-bit codes and bf16 values
    __syncthreads();
    float z2 = -INFINITY;
    if (hv && lane < cnt && slot_s[lane] >= 0) {
      float acc = 0.0f;
      const float* qr = qs + warp * n;
      const float* cr = cs + lane * ldc;
      for (int k = 0; k < n; ++k) acc = fmaf(qr[k], cr[k], acc);
      z2 = acc * ss[lane] * zscale;
      // an element that is not finite leaves no finite score (finite x inf, 0 x inf, inf - inf);
      // as NaN it turns the whole row into NaN, a -inf included, as the tensor-core kernel does
      if (!isfinite(z2)) z2 = CUDART_NAN_F;
    }
    const float mn = fmaxf(m, warp_max(z2));
    const float alpha = (m == -INFINITY || mn == -INFINITY) ? 0.0f : exp2f(m - mn);
    const float pz = (z2 == -INFINITY) ? 0.0f : exp2f(z2 - mn);
    l = l * alpha + warp_sum(pz);
    const float wgt = pz * ss[lane];
#pragma unroll
    for (int r = 0; r < R; ++r) o[r] *= alpha;
    for (int i = 0; i < cnt; ++i) {
      const float wi = __shfl_sync(0xffffffffu, wgt, i);
      const float* cr = cs + i * ldc;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int j = lane + 32 * r;
        if (j < d) o[r] = fmaf(wi, cr[j], o[r]);
      }
    }
    m = mn;
  }
  if (S > 1) {
    // partials of the eight heads (the tile's memory holds them), joined by CTA 0
    __syncthreads();
    float* ml = qs;                      // [kHG][2]
    float* po = cs;                      // [kHG][32 R], kHG * 32 R <= TT (n + 1) for every R
    if (lane == 0) {
      ml[2 * warp] = m;
      ml[2 * warp + 1] = l;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (lane + 32 * r < d) po[warp * d + lane + 32 * r] = o[r];
    __syncthreads();
    cluster_sync();
    if (z == 0 && hv) {
      float M = -INFINITY;
      for (int c = 0; c < S; ++c) M = fmaxf(M, load_rank(ml + 2 * warp, c));
      const float ref = M == -INFINITY ? 0.0f : M;
      l = 0.0f;
#pragma unroll
      for (int r = 0; r < R; ++r) o[r] = 0.0f;
      for (int c = 0; c < S; ++c) {
        const float w = exp2f(load_rank(ml + 2 * warp, c) - ref);   // (-inf: 0)
        l += w * load_rank(ml + 2 * warp + 1, c);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int j = lane + 32 * r;
          if (j < d) o[r] = fmaf(w, load_rank(po + warp * d + j, c), o[r]);
        }
      }
      m = M;
    }
    __syncwarp();                        // (the barrier wants whole warps)
    cluster_sync();                      // nobody's shared memory goes while it is read
    if (z) return;
  }
  if (!hv) return;
  const float inv = (l > 0.0f || l != l) ? 1.0f / l : 0.0f;
  Tq* out = static_cast<Tq*>(a.out) + (int64_t)row * a.o_st + (int64_t)h * a.o_sh;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int j = lane + 32 * r;
    if (j < d) store_o(out + j, o[r] * inv);
  }
  if (a.lse && lane == 0)
    a.lse[(int64_t)row * a.H + h] = (l == 0.0f) ? -INFINITY : kLn2 * (m + log2f(l));
}

// CTAs that share a query token and head group: enough of them to fill the GPU about twice, no more
// than the tiles of the longest sequence, at most a portable cluster.
int split_of(const ChunkArgs& a, int tt) {
  const int64_t ctas = (int64_t)a.n_q * ((a.H + kHG - 1) / kHG);
  int s = 1;
  while (s < 8 && ctas * s < 2 * 148 && (int64_t)s * tt < a.cap) s *= 2;
  return s;
}

template <int TT, int R>
cudaError_t launch_tt_r(const ChunkArgs& a, int dtype, size_t smem, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  const int S = split_of(a, TT);
  cfg.gridDim = dim3((unsigned)a.n_q, (unsigned)((a.H + kHG - 1) / kHG), (unsigned)S);
  cfg.blockDim = dim3(kHG * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = (unsigned)S;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaSuccess;
#define KVK_LAUNCH(T)                                                                   \
  do {                                                                                  \
    auto k = chunk_fma_kernel<TT, R, T>;                                                \
    static std::atomic<uint64_t> done{0};                                               \
    e = once_per_device(done, [&] {                                                     \
      return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax); \
    });                                                                                 \
    if (e != cudaSuccess) return e;                                                     \
    e = cudaLaunchKernelEx(&cfg, k, a);                                                 \
    if (e != cudaSuccess) return e;                                                     \
  } while (0)
  if (dtype == KVK_F32) KVK_LAUNCH(float);
  else if (dtype == KVK_BF16) KVK_LAUNCH(__nv_bfloat16);
  else KVK_LAUNCH(__half);
#undef KVK_LAUNCH
  return cudaGetLastError();
}

template <int TT>
cudaError_t launch_tt(const ChunkArgs& a, int dtype, size_t smem, cudaStream_t st) {
  if (a.d <= 64) return launch_tt_r<TT, 2>(a, dtype, smem, st);
  if (a.d <= 128) return launch_tt_r<TT, 4>(a, dtype, smem, st);
  if (a.d <= 512) return launch_tt_r<TT, 16>(a, dtype, smem, st);
  return launch_tt_r<TT, 64>(a, dtype, smem, st);
}

size_t smem_bytes(int TT, int n) {
  return sizeof(float) * ((size_t)kHG * n + (size_t)TT * (n + 1) + TT) + sizeof(int32_t) * (size_t)TT;
}

}  // namespace

bool chunk_fma_fits(int n) { return smem_bytes(16, n) <= kSmemMax; }

cudaError_t launch_chunk_fma(const ChunkArgs& a, int dtype, cudaStream_t st) {
  const size_t s32 = smem_bytes(32, a.n);
  if (s32 <= kSmemMax) return launch_tt<32>(a, dtype, s32, st);
  const size_t s16 = smem_bytes(16, a.n);
  if (s16 <= kSmemMax) return launch_tt<16>(a, dtype, s16, st);
  return cudaErrorInvalidValue;
}

}  // namespace kvk
