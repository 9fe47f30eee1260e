// kvk_paged.cu -- the bookkeeping of a paged serving step, and quantise-on-write through its
// slot map.
//
// Plan.  With P tokens per page, a_i cached and f_i new tokens of sequence i: the sequence holds
// have_i = ceil(a_i / P) pages and needs need_i = ceil((a_i + f_i) / P); the pages it lacks come
// off the end of the free list in sequence order, so the k-th page taken (k counted over the
// whole batch) is free[count - 1 - k].  q_start is the exclusive prefix sum of the f_i, and the
// new token at position t of sequence i goes to slot table[i][t / P] P + t % P.  Where the batch has
// more new tokens than max_new, those behind it are none of the step's: no row, slot or page, and the
// lengths end with the ones before, so that the attention over the offsets and lengths sees every row
// at its token's position.
//
// One launch: every CTA computes both prefix sums itself (at most 4096 sequences, four a thread),
// then the CTAs share out the pages taken and the tokens.  A new token's page is computed from the
// prefix sums (the free list) or read from an entry that was there before the call, never from
// one that another CTA writes, so the CTAs need no order between them, except that a free count
// that is updated in place is read by all before it is written: such a call is one cluster.
// Bound by latency: 4 us on the device for 32 tokens of a decode step, and for 144,000 tokens of
// 32 prompts the two searches and loads a thread makes per four tokens.
#include "kvk_paged.cuh"
#include "kvk_quant_common.cuh"

namespace kvk {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 64, kPlanCluster = 8;   // most CTAs; most with the count updated in place

struct PlanSeq {
  int cached, fresh, kept;   // clamped counts; kept: new tokens that fit the table row and max_new
  int have, need;
  bool bad;
};
// Sequence i with room for at most `room` new tokens.
__device__ __forceinline__ PlanSeq plan_seq(const PlanArgs& a, int i, int64_t room) {
  const int c = __ldg(a.cached + i), f = __ldg(a.fresh + i);
  const int cap = (int)min((int64_t)a.table_pages << a.page_shift, (int64_t)0x7FFFFFFF);
  PlanSeq s;
  s.cached = min(max(c, 0), cap);
  s.fresh = max(f, 0);
  s.kept = min(s.fresh, cap - s.cached);
  s.bad = s.cached != c || s.kept != f;
  s.kept = (int)min((int64_t)s.kept, max(room, (int64_t)0));
  const int64_t r = (1 << a.page_shift) - 1;
  s.have = (int)((s.cached + r) >> a.page_shift);
  s.need = (int)((s.cached + (int64_t)s.kept + r) >> a.page_shift);
  return s;
}

// The page that is the k-th taken, or -1 (flagged) when the free list is short or names no page
// of the pool.
__device__ __forceinline__ int plan_page(const PlanArgs& a, int count, int64_t k) {
  if (k < count) {
    const int page = __ldg(a.free_pages + (count - 1 - (int)k));
    if (page >= 0 && page < a.pool_pages) return page;
  }
  atomicOr(a.flags, KVK_FLAG_PAGE);
  return -1;
}

// Inclusive prefix sums of x and y over the block; x_all[31] and y_all[31] become the totals.
__device__ __forceinline__ void plan_scan(int64_t& x, int64_t& y, int64_t* x_all, int64_t* y_all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    x_all[warp] = x;
    y_all[warp] = y;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t u = x_all[lane], v = y_all[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t p = __shfl_up_sync(0xffffffffu, u, o), q = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) {
        u += p;
        v += q;
      }
    }
    x_all[lane] = u;
    y_all[lane] = v;
  }
  __syncthreads();
  if (warp) {
    x += x_all[warp - 1];
    y += y_all[warp - 1];
  }
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  int32_t* start_s = plan_smem;                     // [batch + 1] first new token of each sequence
  int32_t* taken_s = start_s + a.batch + 1;         // [batch] pages taken before each sequence
  int32_t* cached_s = taken_s + a.batch;            // [batch] its cached and its kept new tokens
  int32_t* kept_s = cached_s + a.batch;
  __shared__ int64_t warp_new[32], warp_page[32];
  const int tid = threadIdx.x;
  const int count = min(max(__ldg(a.free_count), 0), a.free_capacity);

  // prefix sums over the sequences, a run of consecutive ones a thread: of the new tokens, and of the
  // pages taken, first as though max_new held all the tokens
  const int per = (a.batch + kPlanThreads - 1) / kPlanThreads;
  const int i0 = min(a.batch, tid * per), i1 = min(a.batch, i0 + per);
  const int64_t all = (int64_t)1 << 62;
  int64_t fresh = 0, pages = 0;
  bool bad = false;
  for (int i = i0; i < i1; ++i) {
    const PlanSeq s = plan_seq(a, i, all);
    fresh += s.fresh;
    pages += s.need - s.have;
    bad = bad || s.bad;
  }
  int64_t x = fresh, y = pages;
  plan_scan(x, y, warp_new, warp_page);
  const int64_t at0 = x - fresh;                    // new tokens before this thread's sequences
  const int64_t asked = warp_new[31], total = min(asked, (int64_t)a.max_new);
  if (asked > a.max_new) {                          // (the same in every thread)
    pages = 0;
    int64_t at = at0;
    for (int i = i0; i < i1; ++i) {
      const PlanSeq s = plan_seq(a, i, a.max_new - at);
      at += s.fresh;
      pages += s.need - s.have;
    }
    __syncthreads();                                // the sums have been read
    x = fresh, y = pages;
    plan_scan(x, y, warp_new, warp_page);
  }
  const int64_t taken = warp_page[31];
  int64_t at = at0, page_at = y - pages;
  for (int i = i0; i < i1; ++i) {
    const PlanSeq s = plan_seq(a, i, a.max_new - at);
    start_s[i] = (int32_t)min(at, (int64_t)a.max_new);
    taken_s[i] = (int32_t)min(page_at, (int64_t)0x7FFFFFFF);
    cached_s[i] = s.cached;
    kept_s[i] = s.kept;
    at += s.fresh;
    page_at += s.need - s.have;
  }
  if (tid == 0) start_s[a.batch] = (int32_t)total;
  __syncthreads();

  if (blockIdx.x == 0) {
    if (bad || (tid == 0 && asked > a.max_new)) atomicOr(a.flags, KVK_FLAG_SEQ_LEN);
    for (int i = tid; i <= a.batch; i += kPlanThreads) {
      a.q_start[i] = start_s[i];
      if (i < a.batch) a.seq_lens[i] = cached_s[i] + kept_s[i];
    }
  }
  // the pages taken, one a thread
  const int P = 1 << a.page_shift;
  for (int64_t k = (int64_t)blockIdx.x * kPlanThreads + tid; k < taken; k += gridDim.x * kPlanThreads) {
    int lo = 0, hi = a.batch - 1;   // the last sequence whose pages start at or before k
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (taken_s[mid] <= k) lo = mid; else hi = mid - 1;
    }
    const int have = (int)(((int64_t)cached_s[lo] + P - 1) >> a.page_shift);
    a.table[(int64_t)lo * a.table_stride + have + (k - taken_s[lo])] = plan_page(a, count, k);
  }
  // the new tokens, four consecutive ones a thread; entries behind the last one are marked as no
  // token's
  const bool wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0;
  for (int64_t j0 = ((int64_t)blockIdx.x * kPlanThreads + tid) * 4; j0 < a.max_new;
       j0 += 4 * gridDim.x * kPlanThreads) {
    int slot[4], pos[4];
    int lo = 0;
    if (j0 < total) {
      int hi = a.batch - 1;   // the last sequence that starts at or before j0
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start_s[mid] <= j0) lo = mid; else hi = mid - 1;
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int64_t j = j0 + x;
      slot[x] = -1;
      pos[x] = 0;
      if (j >= total) continue;
      while (lo + 1 < a.batch && start_s[lo + 1] <= j) ++lo;
      const int k = (int)j - start_s[lo];
      if (k >= kept_s[lo]) continue;
      const int held = cached_s[lo], have = (int)(((int64_t)held + P - 1) >> a.page_shift);
      pos[x] = held + k;
      const int pg = pos[x] >> a.page_shift;
      int page;
      if (pg >= have) {
        page = plan_page(a, count, (int64_t)taken_s[lo] + (pg - have));
      } else {   // the page that the cached tokens left unfinished
        page = a.table[(int64_t)lo * a.table_stride + pg];
        if (page < 0 || page >= a.pool_pages) {
          atomicOr(a.flags, KVK_FLAG_PAGE);
          page = -1;
        }
      }
      if (page >= 0) slot[x] = (page << a.page_shift) + (pos[x] & (P - 1));
    }
    if (wide && j0 + 4 <= a.max_new) {
      *reinterpret_cast<int4*>(a.slots + j0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      if (a.positions)
        *reinterpret_cast<int4*>(a.positions + j0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (j0 + x >= a.max_new) break;
        a.slots[j0 + x] = slot[x];
        if (a.positions) a.positions[j0 + x] = pos[x];
      }
    }
  }
  // every CTA has read the free count before it changes (one cluster, if it is updated in place);
  // the cluster's barrier wants whole warps, and the loops above leave theirs thread by thread
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
  if (blockIdx.x == 0 && tid == 0)
    *a.free_count_out = (int32_t)max((int64_t)count - taken, (int64_t)0);
}

// ---------------------------------------------------------------------------------------
// quantise-on-write through a slot map
// ---------------------------------------------------------------------------------------
// Rows of up to kFastElems elements: 8 lanes a token, four tokens a warp, lane i of a token holding
// groups i, i + 8, ... of 8 elements, so that every width of the layouts (192 to 576) keeps all
// lanes busy and a lane has all its loads in flight at once.  The codes are kvk_quant_write's bit
// for bit: round-half-even of the binary32 quotient v / s.  The quotient comes from the scale's
// reciprocal by Markstein's division (P. W. Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990): with r = RN(1 / s), q0 = RN(v r) and two steps
// q' = RN(q + r RN(v - s q)) the result is RN(v / s); it need not hold where the quotient is so
// small that the steps underflow, whose code is zero either way.  Longer rows take the two-pass
// form, one warp a token.  Bound by instruction issue: 52,500 tokens of 576 bf16 elements at 8 bits
// take 29 us (3.2 TB/s) with 0.72 instructions a cycle and scheduler, 2.9 of its 6.9 warps ready on
// average, and memory 28 % busy; the same tokens as bf16 rows, without quotients, 27 us (4.6 TB/s).
// One warp a token with a division per element took 57 us, and rows held as fp32 values (two blocks
// an SM instead of four) 56 us.  The two-pass form: rows of 1088 elements at 8 bits 92 us, as bf16
// rows 66 us.
constexpr int kWarpsPerBlock = 8;
constexpr int kFastRounds = 10, kFastElems = 64 * kFastRounds;

__device__ __forceinline__ float markstein(float v, float s, float r) {
  float q = v * r;
  q = fmaf(fmaf(-s, q, v), r, q);
  return fmaf(fmaf(-s, q, v), r, q);
}
// field of v: round-half-even of v / s, clamped to +-top, in offset binary.  Adding 1.5 2^23 to a
// number below 2^22 rounds it half to even into the sum's low bits.
template <int B>
__device__ __forceinline__ uint32_t field_of(float v, float s, float r) {
  constexpr float top = (float)((1 << (B - 1)) - 1);
  const float q = fminf(fmaxf(markstein(v, s, r), -top), top);
  return (__float_as_uint(q + 12582912.0f) + (1u << (B - 1))) & ((1u << B) - 1u);
}

// Eight elements as they were read (bf16: 4 registers, so that a row in flight leaves room for four
// blocks an SM), and their values.
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void read8(const T* p, Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
}
__device__ __forceinline__ void values8(const Raw8<float>& r, float (&v)[8]) {
  const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
}
__device__ __forceinline__ void values8(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {   // a bf16 is the high half of a binary32
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

template <typename T, int B, bool GROUP>
__global__ void __launch_bounds__(kWarpsPerBlock * 32, sizeof(T) == 2 ? 4 : 2)
paged_write_fast_kernel(uint8_t* __restrict__ codes, __half* __restrict__ scales, int row_bytes,
                        int d, int d_rope, int group, int sg, int pool_slots,
                        const T* __restrict__ c_kv, int64_t c_st, const T* __restrict__ k_rope,
                        int64_t kr_st, int n_tokens, const int32_t* __restrict__ slots,
                        uint32_t* __restrict__ flags) {
  constexpr bool kBf16 = B == KVK_BITS_BF16;
  constexpr int gb = kBf16 ? 16 : B;                  // bytes of 8 elements
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int64_t j = ((int64_t)blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5)) * 4 + (lane >> 3);
  const int slot = j < n_tokens ? __ldg(slots + j) : -1;
  const bool inside = slot >= 0 && slot < pool_slots;
  if (slot >= pool_slots && sub == 0) atomicOr(flags, KVK_FLAG_WRITE_RANGE);
  const int groups = (d + d_rope) >> 3, d_groups = d >> 3;
  const T* crow = c_kv + j * c_st;
  const T* krow = k_rope + j * kr_st;
  // (the rows are read whether or not their slot, itself still in flight, takes them)
  Raw8<T> in[kFastRounds];
  float amax = 0.0f;
  bool finite = true;
#pragma unroll
  for (int x = 0; x < kFastRounds; ++x) {
    const int g = 8 * x + sub;
    if (j >= n_tokens || g >= groups) continue;
    if (g < d_groups) read8<T>(crow + 8 * g, in[x]);
    else read8<T>(krow + 8 * (g - d_groups), in[x]);
  }
#pragma unroll
  for (int x = 0; x < kFastRounds; ++x) {
    if (j >= n_tokens || 8 * x + sub >= groups) continue;
    float v[8];
    values8(in[x], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float m = fabsf(v[k]);
      finite = finite && m <= 3.4028234663852886e38f;   // false for inf and NaN
      amax = fmaxf(amax, m);
    }
  }
  if constexpr (!GROUP) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  }
  uint8_t* row = codes + (int64_t)max(slot, 0) * row_bytes;
  __half* srow = scales + (int64_t)max(slot, 0) * sg;
  __half s16 = __float2half(1.0f);
  if constexpr (!GROUP && !kBf16) s16 = quant_scale(amax, B);
  float s = __half2float(s16), r = s > 0.0f ? __frcp_rn(s) : 0.0f;
  if (!GROUP && inside && sub == 0) *srow = s16;
  bool bad = !finite || (!GROUP && !kBf16 && isinf(s));
#pragma unroll
  for (int x = 0; x < kFastRounds; ++x) {
    if (8 * x >= groups) break;                       // the same in every lane
    const int g = 8 * x + sub;
    const bool mine = inside && g < groups;
    float v[8];
    if (mine) values8(in[x], v);
    if constexpr (GROUP) {
      float ga = 0.0f;
      if (mine) {
#pragma unroll
        for (int k = 0; k < 8; ++k) ga = fmaxf(ga, fabsf(v[k]));
      }
      const int lpg = group >> 3;
      for (int o = 1; o < lpg; o <<= 1) ga = fmaxf(ga, __shfl_xor_sync(0xffffffffu, ga, o));
      s16 = quant_scale(ga, B);
      s = __half2float(s16);
      r = s > 0.0f ? __frcp_rn(s) : 0.0f;
      bad = bad || (mine && isinf(s));
      if (mine && (sub & (lpg - 1)) == 0) srow[(8 * g) / group] = s16;
    }
    if (!mine) continue;
    uint8_t* dst = row + (int64_t)g * gb;
    if constexpr (kBf16) {
      store_bf16x8(dst, v);
    } else {
      uint32_t u[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = field_of<B>(v[k], s, r);   // (s = 0: r = 0, code 0)
      store_fields8(dst, u, B);
    }
  }
  // the row's padding (fewer than 16 bytes)
  const int used = groups * gb;
  if (inside)
    for (int k = used + sub; k < row_bytes; k += 8) row[k] = 0;
  if (bad && inside) atomicOr(flags, KVK_FLAG_NONFINITE);
}

// Longer rows: one warp per token, two passes over the inputs.
template <typename T>
__global__ void __launch_bounds__(kWarpsPerBlock * 32)
paged_write_kernel(uint8_t* __restrict__ codes, __half* __restrict__ scales, int row_bytes, int d,
                   int d_rope, int b, int group, int sg, int pool_slots,
                   const T* __restrict__ c_kv, int64_t c_st, const T* __restrict__ k_rope,
                   int64_t kr_st, int n_tokens, const int32_t* __restrict__ slots,
                   uint32_t* __restrict__ flags) {
  const int64_t j = (int64_t)blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5);
  if (j >= n_tokens) return;
  const int slot = __ldg(slots + j);
  if (slot < 0) return;                        // no token's
  const bool lead = (threadIdx.x & 31) == 0;
  if (slot >= pool_slots) {
    if (lead) atomicOr(flags, KVK_FLAG_WRITE_RANGE);
    return;
  }
  if (!write_token_two_pass<T>(c_kv + j * c_st, k_rope + j * kr_st, d, d_rope, b, group,
                               codes + (int64_t)slot * row_bytes, row_bytes,
                               scales + (int64_t)slot * sg) &&
      lead)
    atomicOr(flags, KVK_FLAG_NONFINITE);
}

template <typename T>
cudaError_t launch_write(const kvk_layout* L, const AnchorDesc& A, const T* c_kv, int64_t c_st,
                         const T* k_rope, int64_t kr_st, int n_tokens, const int32_t* slots,
                         cudaStream_t st) {
  uint8_t* codes = L->arena + A.codes_off;
  __half* scales = reinterpret_cast<__half*>(L->arena + A.scales_off);
  uint32_t* flags = reinterpret_cast<uint32_t*>(L->arena);
  const int pool = L->max_batch * L->max_tokens, group = anchor_group(L, A);
  const dim3 block(kWarpsPerBlock * 32);
  if (A.n <= kFastElems) {
    const int per = 4 * kWarpsPerBlock;
    const dim3 grid((unsigned)(((int64_t)n_tokens + per - 1) / per));
#define KVK_FAST(B, G)                                                                       \
  paged_write_fast_kernel<T, B, G><<<grid, block, 0, st>>>(codes, scales, A.row_bytes, A.d,   \
                                                           L->d_rope, group, A.sg, pool, c_kv, \
                                                           c_st, k_rope, kr_st, n_tokens, slots, \
                                                           flags)
    if (A.b == KVK_BITS_BF16) KVK_FAST(KVK_BITS_BF16, false);
    else if (A.b == 2 && group) KVK_FAST(2, true);
    else if (A.b == 4 && group) KVK_FAST(4, true);
    else if (A.b == 8 && group) KVK_FAST(8, true);
    else if (group) KVK_FAST(16, true);
    else if (A.b == 2) KVK_FAST(2, false);
    else if (A.b == 4) KVK_FAST(4, false);
    else if (A.b == 8) KVK_FAST(8, false);
    else KVK_FAST(16, false);
#undef KVK_FAST
  } else {
    const dim3 grid((unsigned)(((int64_t)n_tokens + kWarpsPerBlock - 1) / kWarpsPerBlock));
    paged_write_kernel<T><<<grid, block, 0, st>>>(codes, scales, A.row_bytes, A.d, L->d_rope, A.b,
                                                  group, A.sg, pool, c_kv, c_st, k_rope, kr_st,
                                                  n_tokens, slots, flags);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  // a CTA per 4096 tokens (four a thread)
  const bool in_place = a.free_count_out == a.free_count;
  const int want = (int)(((int64_t)a.max_new + 4 * kPlanThreads - 1) / (4 * kPlanThreads));
  int ctas = want < 1 ? 1 : want > kPlanCtas ? kPlanCtas : want;
  if (in_place && ctas > kPlanCluster) ctas = kPlanCluster;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = sizeof(int32_t) * (4 * (size_t)a.batch + 1);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)sizeof(int32_t) * (4 * kMaxPagedBatch + 1));
  });
  if (e != cudaSuccess) return e;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = in_place ? ctas : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, paged_plan_kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_paged_write(const kvk_layout* L, const AnchorDesc& A, const void* c_kv,
                               int dtype, int64_t c_st, const void* k_rope, int64_t kr_st,
                               int n_tokens, const int32_t* slots, cudaStream_t st) {
  if (dtype == KVK_BF16)
    return launch_write(L, A, static_cast<const __nv_bfloat16*>(c_kv), c_st,
                        static_cast<const __nv_bfloat16*>(k_rope), kr_st, n_tokens, slots, st);
  return launch_write(L, A, static_cast<const float*>(c_kv), c_st,
                      static_cast<const float*>(k_rope), kr_st, n_tokens, slots, st);
}

}  // namespace kvk
