// kvk_paged.cuh -- types shared by the host layer and the kernels of the paged cache: the plan
// (kvk_paged.cu), the write through a slot map (kvk_paged.cu) and the attention of chunks of
// new tokens (kvk_chunk_fma.cu, kvk_chunk_tc.cu).
//
// A layout's planes used as a pool: slot s of an anchor is row s of its codes plane, 0 <= s <
// max_batch * max_tokens, and page p the slots [p P, (p + 1) P) with P tokens per page (a
// power of two).  Position t of sequence i lives in slot table[i][t / P] * P + t % P.
#pragma once

#include <atomic>

#include "kvk_internal.cuh"

namespace kvk {

// A kernel's attributes belong to a device: `set` runs once on each that launches it (and again
// after a failure).  `done` is the kernel's own, a bit per device.
template <typename F>
cudaError_t once_per_device(std::atomic<uint64_t>& done, F set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = set();
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

constexpr int kMaxPagedBatch = 4096;

struct PlanArgs {
  const int32_t* cached;       // [batch] tokens already in the cache
  const int32_t* fresh;        // [batch] new tokens
  int batch;
  const int32_t* free_pages;   // [free_capacity] page ids, taken from the end
  const int32_t* free_count;   // valid entries of free_pages
  int free_capacity;
  int page_shift;
  int pool_pages;              // pages of the pool: valid ids are [0, pool_pages)
  int32_t* table;
  int table_pages;             // entries per row
  int64_t table_stride;
  int max_new;                 // capacity of slots / positions
  int32_t* seq_lens;
  int32_t* q_start;            // [batch + 1]
  int32_t* slots;
  int32_t* positions;          // nullable
  int32_t* free_count_out;
  uint32_t* flags;
};
cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t st);

// Packed rows j < n_tokens of c_kv / k_rope quantised to slot slots[j] (negative: skipped).
cudaError_t launch_paged_write(const kvk_layout* L, const AnchorDesc& A, const void* c_kv,
                               int dtype, int64_t c_st, const void* k_rope, int64_t kr_st,
                               int n_tokens, const int32_t* slots, cudaStream_t st);

struct ChunkArgs {
  const uint8_t* codes;        // the anchor's pool
  const __half* scales;
  int row_bytes, d, d_rope, n, b;
  int group, sg;               // elements per scale (0: one per token), scales per token
  const void* q_lat;           // element (token, head, k) at token * ql_st + head * ql_sh + k
  const void* q_rope;
  int64_t ql_st, ql_sh, qr_st, qr_sh;
  int n_q, batch, H;
  const int32_t* q_start;      // [batch + 1] first query row of each sequence
  const int32_t* seq_lens;     // [batch] tokens in the cache, the new ones among them
  const int32_t* table;
  int table_pages;
  int64_t table_stride;
  int page_shift, pool_pages;
  int cap;                     // longest sequence a table row can hold: table_pages << shift
  float sigma;
  void* out;                   // the queries' type, element strides
  int64_t o_st, o_sh;
  float* lse;                  // nullable [n_q][H]
  uint32_t* flags;
  uint64_t limit_ns;
};

// The query rows and the tokens of sequence i, clamped to what the call's buffers hold; *bad
// reports a value that had to be clamped.  Query row j of the sequence sits at position
// len - count + j and sees the tokens up to its own.
struct ChunkSeq {
  int row0, count, len;
};
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkArgs& a, int i, bool* bad) {
  const int s0 = __ldg(a.q_start + i), s1 = __ldg(a.q_start + i + 1), l = __ldg(a.seq_lens + i);
  ChunkSeq s;
  s.row0 = min(max(s0, 0), a.n_q);
  s.count = min(max(s1, s.row0), a.n_q) - s.row0;
  s.len = min(max(l, 0), a.cap);
  *bad = s.row0 != s0 || s.row0 + s.count != s1 || s.len != l;
  return s;
}

// Slot of position t of sequence i, or -1 (flagged) where the table names no page of the pool.
__device__ __forceinline__ int chunk_slot(const ChunkArgs& a, int i, int t) {
  const int page = __ldg(a.table + (int64_t)i * a.table_stride + (t >> a.page_shift));
  if (page < 0 || page >= a.pool_pages) {
    atomicOr(a.flags, KVK_FLAG_PAGE);
    return -1;
  }
  return (page << a.page_shift) + (t & ((1 << a.page_shift) - 1));
}

cudaError_t launch_chunk_fma(const ChunkArgs& a, int dtype, cudaStream_t st);
bool chunk_fma_fits(int n);

}  // namespace kvk
