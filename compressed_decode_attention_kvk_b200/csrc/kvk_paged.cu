// kvk_paged.cu -- the bookkeeping of a paged serving step, and quantise-on-write through its
// slot map.
//
// Plan.  With P tokens per page, a_i cached and f_i new tokens of sequence i: the sequence holds
// have_i = ceil(a_i / P) pages and needs need_i = ceil((a_i + f_i) / P); the pages it lacks come
// off the end of the free list in sequence order, so the k-th page taken (k counted over the
// whole batch) is free[count - 1 - k].  q_start is the exclusive prefix sum of the f_i, and the
// new token at position t of sequence i goes to slot table[i][t / P] P + t % P.
//
// One launch of one cluster: every CTA computes both prefix sums itself (at most 4096
// sequences, four a thread), then the CTAs share out the table rows and the tokens.  A new
// token's page is computed from the prefix sums (the free list) or read from an entry that was
// there before the call, never from one that another CTA writes, so the CTAs need no order
// between them except that the free count is read by all before it is written (it may be
// updated in place): the cluster barrier.
#include "kvk_paged.cuh"
#include "kvk_quant_common.cuh"

namespace kvk {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;   // one portable cluster
constexpr int kPlanPer = kMaxPagedBatch / kPlanThreads;

struct PlanSeq {
  int cached, fresh, kept;   // clamped counts; kept: new tokens that fit the table row
  int have, need;
  bool bad;
};
__device__ __forceinline__ PlanSeq plan_seq(const PlanArgs& a, int i) {
  const int c = __ldg(a.cached + i), f = __ldg(a.fresh + i);
  const int cap = (int)min((int64_t)a.table_pages << a.page_shift, (int64_t)0x7FFFFFFF);
  PlanSeq s;
  s.cached = min(max(c, 0), cap);
  s.fresh = max(f, 0);
  s.kept = min(s.fresh, cap - s.cached);
  s.bad = s.cached != c || s.kept != f;
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

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PlanArgs a) {
  __shared__ int32_t start_s[kMaxPagedBatch + 1];   // first new token of each sequence
  __shared__ int32_t taken_s[kMaxPagedBatch];       // pages taken before each sequence
  __shared__ int64_t warp_new[32], warp_page[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int count = min(max(__ldg(a.free_count), 0), a.free_capacity);

  // prefix sums over the sequences, kPlanPer consecutive ones a thread
  const int per = (a.batch + kPlanThreads - 1) / kPlanThreads;
  const int i0 = min(a.batch, tid * per), i1 = min(a.batch, i0 + per);
  int64_t fresh = 0, pages = 0;
  bool bad = false;
  for (int i = i0; i < i1; ++i) {
    const PlanSeq s = plan_seq(a, i);
    fresh += s.fresh;
    pages += s.need - s.have;
    bad = bad || s.bad;
  }
  int64_t x = fresh, y = pages;   // inclusive warp scans
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    warp_new[warp] = x;
    warp_page[warp] = y;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t u = warp_new[lane], v = warp_page[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t p = __shfl_up_sync(0xffffffffu, u, o), q = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) {
        u += p;
        v += q;
      }
    }
    warp_new[lane] = u;
    warp_page[lane] = v;
  }
  __syncthreads();
  int64_t at = x - fresh + (warp ? warp_new[warp - 1] : 0);
  int64_t page_at = y - pages + (warp ? warp_page[warp - 1] : 0);
  const int64_t total = min(warp_new[31], (int64_t)a.max_new);
  const int64_t taken = warp_page[31];
  for (int i = i0; i < i1; ++i) {
    const PlanSeq s = plan_seq(a, i);
    start_s[i] = (int32_t)min(at, (int64_t)a.max_new);
    taken_s[i] = (int32_t)min(page_at, (int64_t)0x7FFFFFFF);
    at += s.fresh;
    page_at += s.need - s.have;
  }
  if (tid == 0) start_s[a.batch] = (int32_t)total;
  __syncthreads();

  if (blockIdx.x == 0) {
    if (bad || (tid == 0 && warp_new[31] > a.max_new)) atomicOr(a.flags, KVK_FLAG_SEQ_LEN);
    for (int i = tid; i <= a.batch; i += kPlanThreads) {
      a.q_start[i] = start_s[i];
      if (i < a.batch) {
        const PlanSeq s = plan_seq(a, i);
        a.seq_lens[i] = s.cached + s.kept;
      }
    }
  }
  // the pages taken: one warp per sequence
  for (int i = blockIdx.x * 32 + warp; i < a.batch; i += kPlanCtas * 32) {
    const PlanSeq s = plan_seq(a, i);
    for (int k = s.have + lane; k < s.need; k += 32)
      a.table[(int64_t)i * a.table_stride + k] =
          plan_page(a, count, (int64_t)taken_s[i] + (k - s.have));
  }
  // the new tokens; entries behind the last one are marked as no token's
  const int P = 1 << a.page_shift;
  for (int64_t j64 = (int64_t)blockIdx.x * kPlanThreads + tid; j64 < a.max_new;
       j64 += kPlanCtas * kPlanThreads) {
    const int j = (int)j64;
    int slot = -1, pos = 0;
    if (j < total) {
      int lo = 0, hi = a.batch - 1;   // the last sequence that starts at or before j
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start_s[mid] <= j) lo = mid; else hi = mid - 1;
      }
      const PlanSeq s = plan_seq(a, lo);
      const int k = j - start_s[lo];
      if (k < s.kept) {
        pos = s.cached + k;
        const int pg = pos >> a.page_shift;
        int page;
        if (pg >= s.have) {
          page = plan_page(a, count, (int64_t)taken_s[lo] + (pg - s.have));
        } else {   // the page that the cached tokens left unfinished
          page = a.table[(int64_t)lo * a.table_stride + pg];
          if (page < 0 || page >= a.pool_pages) {
            atomicOr(a.flags, KVK_FLAG_PAGE);
            page = -1;
          }
        }
        if (page >= 0) slot = (page << a.page_shift) + (pos & (P - 1));
      }
    }
    a.slots[j] = slot;
    if (a.positions) a.positions[j] = pos;
  }
  // every CTA has read the free count before it changes
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
  if (blockIdx.x == 0 && tid == 0)
    *a.free_count_out = (int32_t)max((int64_t)count - taken, (int64_t)0);
}

// ---------------------------------------------------------------------------------------
// quantise-on-write through a slot map: one warp per token
// ---------------------------------------------------------------------------------------
constexpr int kWarpsPerBlock = 8;

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

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPlanCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, paged_plan_kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_paged_write(const kvk_layout* L, const AnchorDesc& A, const void* c_kv,
                               int dtype, int64_t c_st, const void* k_rope, int64_t kr_st,
                               int n_tokens, const int32_t* slots, cudaStream_t st) {
  uint8_t* codes = L->arena + A.codes_off;
  __half* scales = reinterpret_cast<__half*>(L->arena + A.scales_off);
  uint32_t* flags = reinterpret_cast<uint32_t*>(L->arena);
  const int pool = L->max_batch * L->max_tokens;
  dim3 grid((unsigned)((n_tokens + kWarpsPerBlock - 1) / kWarpsPerBlock)), block(kWarpsPerBlock * 32);
  if (dtype == KVK_BF16)
    paged_write_kernel<__nv_bfloat16><<<grid, block, 0, st>>>(
        codes, scales, A.row_bytes, A.d, L->d_rope, A.b, anchor_group(L, A), A.sg, pool,
        static_cast<const __nv_bfloat16*>(c_kv), c_st, static_cast<const __nv_bfloat16*>(k_rope),
        kr_st, n_tokens, slots, flags);
  else
    paged_write_kernel<float><<<grid, block, 0, st>>>(
        codes, scales, A.row_bytes, A.d, L->d_rope, A.b, anchor_group(L, A), A.sg, pool,
        static_cast<const float*>(c_kv), c_st, static_cast<const float*>(k_rope), kr_st, n_tokens,
        slots, flags);
  return cudaGetLastError();
}

}  // namespace kvk
