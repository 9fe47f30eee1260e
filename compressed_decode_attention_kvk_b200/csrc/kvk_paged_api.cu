// kvk_paged_api.cu -- host side of the paged entry points: argument checks and dispatch.  Every
// exported symbol is declared in include/kvk.h.
#include <string.h>

#include <algorithm>

#include "kvk_chunk_route.cuh"
#include "kvk_chunk_tc.cuh"

using kvk::AnchorDesc;

namespace {

bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// As for every call of a layout: its device has to be the current one.
kvk_status check_device(const kvk_layout* L) {
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) {
    cudaGetLastError();
    return KVK_ERR_CUDA;
  }
  return cur == L->device ? KVK_OK : KVK_ERR_INVALID_ARG;
}

// Tokens per page: a power of two up to 2^16.  Returns its logarithm, or -1.
int page_shift(int page_tokens) {
  if (page_tokens < 1 || page_tokens > 65536 || (page_tokens & (page_tokens - 1))) return -1;
  int s = 0;
  while ((1 << s) < page_tokens) ++s;
  return s;
}

int64_t pool_slots(const kvk_layout* L) { return (int64_t)L->max_batch * L->max_tokens; }

int chunk_clusters(const kvk_layout* L) {
  return std::max(1, (L->num_sms > 0 ? L->num_sms : 148) / 2);
}

// The kernel a chunk call takes, or -1 (bf16 and f16 queries may take the tensor-core kernel).
int chunk_path(const kvk_layout* L, const AnchorDesc& A, int dtype) {
  const bool tensor = kvk::chunk_tc_supported(L, A, dtype);
  const int regs = tensor && L->arena ? kvk::chunk_tc_regs(A.b, kvk::anchor_group(L, A)) : -1;
  return kvk::chunk_route(L->path, tensor, regs, kvk::chunk_fma_fits(A.n));
}

// Whether a call's rows are converted once ahead of the attention (kvk_chunk_expand.cu) instead
// of in every row tile: from two row tiles of 128 per sequence on, over the batch, or one where the
// rows are bf16 and nothing is converted but much is loaded.  8 sequences of 4096 tokens, 40 heads,
// d = 512, row tiles per sequence (us converting / expanded): 8 bits 1.9 (71 / 76), 2.5 (86 / 83);
// 16 bits 1.9 (87 / 93), 2.5 (109 / 107); bf16 0.6 (61 / 59), 1.2 (89 / 64).  The host knows the
// batch's average only, and every sequence with queries is expanded, those of one token too: 512 new
// tokens beside 63 decode sequences, all near 8192 tokens, 8 bits (967 / 685), 16 bits (1237 / 1071);
// but 512 new tokens of a fresh prompt beside 31 decode sequences of 16384, where the expanded rows
// are mostly read once, 8 bits (357 / 409), 16 bits (454 / 671), bf16 (538 / 418).
bool expand_pays(int b, int n_q, int batch, int n_heads) {
  const int tiles = b == KVK_BITS_BF16 ? 1 : 2;
  return (int64_t)n_q * n_heads >= (int64_t)tiles * 128 * batch;
}

size_t chunk_bytes(const kvk_layout* L, const AnchorDesc& A, bool expand, void* base,
                   kvk::ChunkWork* w) {
  return kvk::chunk_workspace(A, L->d_rope, kvk::anchor_group(L, A), pool_slots(L),
                              chunk_clusters(L), expand, base, w);
}

bool known_dtype(int t) { return t == KVK_F32 || t == KVK_BF16 || t == KVK_F16; }

}  // namespace

extern "C" {

kvk_status kvk_paged_plan(kvk_layout* L, const int32_t* dev_cached, const int32_t* dev_new,
                          int batch, const int32_t* dev_free_pages, const int32_t* dev_free_count,
                          int free_capacity, int page_tokens, int32_t* dev_block_table,
                          int table_pages, int64_t table_stride, int max_new,
                          int32_t* dev_seq_lens, int32_t* dev_q_start, int32_t* dev_slots,
                          int32_t* dev_positions, int32_t* dev_free_count_out,
                          kvk_stream_t stream) {
  if (!L || !L->arena) return KVK_ERR_INVALID_ARG;
  if (batch < 1 || batch > kvk::kMaxPagedBatch || free_capacity < 0 || table_pages < 1 ||
      table_stride < table_pages || max_new < 0)
    return KVK_ERR_INVALID_ARG;
  const int shift = page_shift(page_tokens);
  if (shift < 0) return KVK_ERR_INVALID_ARG;
  if (!dev_cached || !dev_new || !dev_free_count || !dev_block_table || !dev_seq_lens ||
      !dev_q_start || !dev_free_count_out || (free_capacity > 0 && !dev_free_pages) ||
      (max_new > 0 && !dev_slots))
    return KVK_ERR_INVALID_ARG;
  // the inputs are read while the results are written: no result overlaps an input or another
  // result (but the free count may be updated in place)
  struct Span {
    const int32_t* p;
    int64_t n;
  };
  const Span in[] = {{dev_cached, batch}, {dev_new, batch}, {dev_free_pages, free_capacity},
                     {dev_free_count, 1}};
  const Span res[] = {{dev_block_table, (batch - 1) * table_stride + table_pages},
                      {dev_seq_lens, batch}, {dev_q_start, batch + 1}, {dev_slots, max_new},
                      {dev_positions, dev_positions ? max_new : 0}, {dev_free_count_out, 1}};
  auto meet = [](const Span& x, const Span& y) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
    return x.n > 0 && y.n > 0 && a < b + 4 * (uintptr_t)y.n && b < a + 4 * (uintptr_t)x.n;
  };
  for (int i = 0; i < 6; ++i) {
    for (int j = i + 1; j < 6; ++j)
      if (meet(res[i], res[j])) return KVK_ERR_INVALID_ARG;
    for (const Span& x : in)
      if (meet(res[i], x) && !(i == 5 && x.p == dev_free_count && x.p == res[5].p))
        return KVK_ERR_INVALID_ARG;
  }
  for (const void* p : {(const void*)dev_cached, (const void*)dev_new, (const void*)dev_free_pages,
                        (const void*)dev_free_count, (const void*)dev_block_table,
                        (const void*)dev_seq_lens, (const void*)dev_q_start,
                        (const void*)dev_slots, (const void*)dev_positions,
                        (const void*)dev_free_count_out})
    if (!aligned(p, 4)) return KVK_ERR_ALIGNMENT;
  if (kvk_status ds = check_device(L)) return ds;
  kvk::PlanArgs a;
  memset(&a, 0, sizeof(a));
  a.cached = dev_cached;
  a.fresh = dev_new;
  a.batch = batch;
  a.free_pages = dev_free_pages;
  a.free_count = dev_free_count;
  a.free_capacity = free_capacity;
  a.page_shift = shift;
  a.pool_pages = (int)(pool_slots(L) >> shift);
  a.table = dev_block_table;
  a.table_pages = table_pages;
  a.table_stride = table_stride;
  a.max_new = max_new;
  a.seq_lens = dev_seq_lens;
  a.q_start = dev_q_start;
  a.slots = dev_slots;
  a.positions = dev_positions;
  a.free_count_out = dev_free_count_out;
  a.flags = reinterpret_cast<uint32_t*>(L->arena);
  const cudaError_t e = kvk::launch_paged_plan(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVK_OK : KVK_ERR_CUDA;
}

kvk_status kvk_paged_write(kvk_layout* L, int layer, const void* c_kv, int dtype,
                           int64_t c_stride_tok, const void* k_rope, int64_t kr_stride_tok,
                           int n_tokens, const int32_t* dev_slots, kvk_stream_t stream) {
  if (!L || layer < 0 || layer >= L->n_layers) return KVK_ERR_INVALID_ARG;
  if (L->anchor[layer] != layer) return KVK_ERR_INHERITING_LAYER;
  if (!L->arena) return KVK_ERR_INVALID_ARG;
  if (dtype != KVK_F32 && dtype != KVK_BF16) return KVK_ERR_INVALID_ARG;
  if (n_tokens < 0) return KVK_ERR_INVALID_ARG;
  if (n_tokens == 0) return KVK_OK;
  if (!c_kv || !dev_slots || (L->d_rope > 0 && !k_rope)) return KVK_ERR_INVALID_ARG;
  if (c_stride_tok < 0 || kr_stride_tok < 0) return KVK_ERR_INVALID_ARG;
  if (!aligned(c_kv, 16) || !aligned(k_rope, 16) || !aligned(dev_slots, 4) || c_stride_tok % 8 ||
      kr_stride_tok % 8)
    return KVK_ERR_ALIGNMENT;
  if (kvk_status ds = check_device(L)) return ds;
  const AnchorDesc& A = L->anchors[L->slot[layer]];
  const cudaError_t e =
      kvk::launch_paged_write(L, A, c_kv, dtype, c_stride_tok, k_rope, kr_stride_tok, n_tokens,
                              dev_slots, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVK_OK : KVK_ERR_CUDA;
}

kvk_status kvk_chunk_path_for(const kvk_layout* L, int layer, int dtype, int* path) {
  if (!L || !path || layer < 0 || layer >= L->n_layers || !known_dtype(dtype))
    return KVK_ERR_INVALID_ARG;
  const int p = chunk_path(L, L->anchors[L->slot[layer]], dtype);
  if (p < 0) return KVK_ERR_UNSUPPORTED;
  *path = p;
  return KVK_OK;
}

kvk_status kvk_chunk_workspace_bytes(const kvk_layout* L, int layer, int n_q, int batch,
                                     int n_heads, size_t* bytes) {
  if (!L || !bytes || layer < 0 || layer >= L->n_layers || n_q < 0 || batch < 1 ||
      batch > kvk::kMaxPagedBatch || n_heads < 1 || n_heads > 4096)
    return KVK_ERR_INVALID_ARG;
  const AnchorDesc& A = L->anchors[L->slot[layer]];
  // (bf16 queries take the tensor-core kernel wherever any do)
  const bool expand = kvk::chunk_tc_supported(L, A, KVK_BF16) && expand_pays(A.b, n_q, batch, n_heads);
  *bytes = chunk_bytes(L, A, expand, nullptr, nullptr);
  return KVK_OK;
}

kvk_status kvk_mla_chunk(kvk_layout* L, int layer, const void* q_lat, const void* q_rope,
                         int dtype, int64_t q_lat_stride_tok, int64_t q_lat_stride_head,
                         int64_t q_rope_stride_tok, int64_t q_rope_stride_head, int n_q, int batch,
                         int n_heads, const int32_t* dev_q_start, const int32_t* dev_seq_lens,
                         const int32_t* dev_block_table, int table_pages, int64_t table_stride,
                         int page_tokens, float softmax_scale, void* out, int64_t out_stride_tok,
                         int64_t out_stride_head, float* lse, void* workspace,
                         size_t workspace_bytes, kvk_stream_t stream) {
  if (!L || layer < 0 || layer >= L->n_layers || !L->arena) return KVK_ERR_INVALID_ARG;
  if (!known_dtype(dtype)) return KVK_ERR_INVALID_ARG;
  if (n_q < 0 || batch < 1 || batch > kvk::kMaxPagedBatch || n_heads < 1 || n_heads > 4096 ||
      (int64_t)n_q * n_heads > ((int64_t)1 << 31) - 256)   // row indexes of whole tiles are ints
    return KVK_ERR_INVALID_ARG;
  const int shift = page_shift(page_tokens);
  if (shift < 0 || table_pages < 1 || table_stride < table_pages) return KVK_ERR_INVALID_ARG;
  if (n_q == 0) return KVK_OK;
  if (!q_lat || (L->d_rope > 0 && !q_rope) || !dev_q_start || !dev_seq_lens || !dev_block_table ||
      !out || !workspace)
    return KVK_ERR_INVALID_ARG;
  for (int64_t s : {q_lat_stride_tok, q_lat_stride_head, q_rope_stride_tok, q_rope_stride_head,
                    out_stride_tok, out_stride_head}) {
    if (s < 0) return KVK_ERR_INVALID_ARG;
    if (s % 8) return KVK_ERR_ALIGNMENT;
  }
  for (const void* p : {(const void*)q_lat, (const void*)q_rope, (const void*)out,
                        (const void*)lse, (const void*)workspace})
    if (!aligned(p, 16)) return KVK_ERR_ALIGNMENT;
  for (const int32_t* p : {dev_q_start, dev_seq_lens, dev_block_table})
    if (!aligned(p, 4)) return KVK_ERR_ALIGNMENT;
  if (kvk_status ds = check_device(L)) return ds;
  const AnchorDesc& A = L->anchors[L->slot[layer]];
  const int path = chunk_path(L, A, dtype);
  if (path < 0) return KVK_ERR_UNSUPPORTED;

  kvk::ChunkArgs a;
  memset(&a, 0, sizeof(a));
  a.codes = L->arena + A.codes_off;
  a.scales = reinterpret_cast<const __half*>(L->arena + A.scales_off);
  a.row_bytes = A.row_bytes;
  a.d = A.d;
  a.d_rope = L->d_rope;
  a.n = A.n;
  a.b = A.b;
  a.group = kvk::anchor_group(L, A);
  a.sg = A.sg;
  a.q_lat = q_lat;
  a.q_rope = q_rope;
  a.ql_st = q_lat_stride_tok;
  a.ql_sh = q_lat_stride_head;
  a.qr_st = q_rope_stride_tok;
  a.qr_sh = q_rope_stride_head;
  a.n_q = n_q;
  a.batch = batch;
  a.H = n_heads;
  a.q_start = dev_q_start;
  a.seq_lens = dev_seq_lens;
  a.table = dev_block_table;
  a.table_pages = table_pages;
  a.table_stride = table_stride;
  a.page_shift = shift;
  a.pool_pages = (int)(pool_slots(L) >> shift);
  a.cap = (int)std::min<int64_t>((int64_t)table_pages << shift, (int64_t)1 << 30);
  a.sigma = softmax_scale;
  a.out = out;
  a.o_st = out_stride_tok;
  a.o_sh = out_stride_head;
  a.lse = lse;
  a.flags = reinterpret_cast<uint32_t*>(L->arena);
  a.limit_ns = L->wait_limit_ns ? L->wait_limit_ns : kvk::kDefaultWaitLimitNs;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (path == KVK_PATH_TENSOR) {
    kvk::ChunkWork w;
    memset(&w, 0, sizeof(w));
    // a box of expanded rows is 8 rows at least (the swizzle's period) and lies in one page
    const bool expand = expand_pays(A.b, n_q, batch, n_heads) && page_tokens >= 8 &&
                        workspace_bytes >= chunk_bytes(L, A, true, nullptr, nullptr);
    if (workspace_bytes < chunk_bytes(L, A, expand, workspace, &w)) return KVK_ERR_WORKSPACE;
    e = kvk::launch_chunk_tc(a, w, dtype, st);
  } else {
    e = kvk::launch_chunk_fma(a, dtype, st);
  }
  return e == cudaSuccess ? KVK_OK : KVK_ERR_CUDA;
}

}  // extern "C"
