// kvk_chunk_tc.cu -- tensor-core (tcgen05) attention of chunks of new tokens over a paged cache.
//
// The rows of a sequence are its (new token, head) pairs, row = token * H + head: all of them
// attend to the one latent stream, so 128 consecutive rows are one tile of
//     S[128 rows x 128 tokens] = Q . C^T,   O[128 x d] += P . C[:, :d]
// whatever the head count.  At d = 512 an O tile of 128 rows takes all of an SM's tensor memory,
// so a tile belongs to a pair of CTAs (a cluster, tcgen05 cta_group::2, M = 128): each CTA holds
// 64 rows of Q, S and O, supplies 64 of the 128 tokens to the score MMA and half the features to
// the output MMA (N = 256 a step).  Measured rate of this form on B200, operands walking through
// shared memory: 64 cycles per MMA at N = 256 (the full rate; one CTA alone reaches it only with
// 128 rows, and takes 80 cycles for 64 rows with .ws), 46 at N = 128 (ideal 32).
//
// Work.  A row tile costs its 128-token blocks plus kCost (query staging, output); every
// cluster takes an equal slice of the batch's cost.  A tile that falls into several slices is
// written as partials (running reference m, weight sum l, un-normalised o) and joined by
// chunk_merge_kernel; a cluster owns at most two partial tiles, its first and its last, so the
// workspace does not grow with the batch.
//
// Warps of a CTA (512 threads):
//   0-3    softmax: a row and 64 tokens a thread; S from TMEM, P (16 bit) to shared memory, O
//          rescaled when a row's reference grows by more than 2^8, outputs
//   4-7    K team: own 64 tokens, packed codes -> 16-bit operand atoms (64 tokens x 64 features,
//          128-byte swizzle) of a ring that the score MMA drains
//   8-11   V team: all 128 tokens, this CTA's half of the latent features, for the output MMA
//   12     score MMAs (the leader CTA's)
//   13     token warp: walks the cluster's pieces, resolves pages to slots, loads token scales,
//          warms L2 with the rows, ahead of the others by its ring (3 to 6 blocks, what memory
//          the other rings leave)
//   14     relay: passes the barriers of written operands on to the leader
//   15     output MMAs (the leader CTA's)
// Both teams stage the query rows at a piece's start.
//
// With expanded rows (kvk_chunk_expand.cu) nothing is converted here: warps 4-7 are a second set of
// softmax warps (32 tokens a thread), warp 15 loads K, two atoms a ring slot, warp 8 V (TMA, counted
// on the leader's barriers), warps 8-11 stage the query, and warp 14 issues the output MMAs in the
// relay's place.  What a block costs
// beside its MMAs is the hand-over at the barriers (a skeleton without MMAs, loads and softmax took
// 4200 cycles a block with a relay and single atoms), hence few and large steps.
//
// Numbers.  Codes enter the MMA exactly: a code of at most 8 bits is an f16 integer; a 16-bit
// code c and a group-scaled value c s are split into two f16 parts (hi = f16(x), lo = x - hi)
// whose score MMAs add up.  The output MMA takes the high part (at most 2^-11 of the value) and P
// in f16 (2^-11): with bf16 outputs (2^-8) neither shows, with f16 outputs (2^-11) the error against
// 64 bits is 2.3e-4 where rounding the output alone gives 2.1e-4.  bf16 rows stay bf16, since f16
// lacks their range and both operands of an MMA have one type; P is then bf16 too (2^-8, the outputs'
// and the rows' own rounding), where the contiguous decode converts such rows and keeps P in f16.  A
// weight's low part would take a second output MMA.  A bf16 query is
// scaled by a power of two of its row into f16's range: exact but for elements far below the
// row's largest, which f16's subnormals leave off by at most 2^-39 of it.
// Scores, references and sums are fp32.
//
// Softmax with token scales.  With z_t the score in log2 units and s_t the token's scale, the
// weight of code row t is s_t 2^(z_t): the kernel tracks w_t = z_t + log2 s_t, m >= max w_t - 8,
// P_t = 2^(w_t - m + 7) and l = sum P_t / s_t, so that P fits 16 bits whatever the scales: at most
// 2^15, the largest at least 2^7.  f16 holds weights down to 2^-25 of 1 (half its smallest step):
// 2^-32 of the largest, of which a sum of 2^20 such tokens loses 2^-12 at most; l, in fp32, counts
// them all.  A token that does not exist (behind the end, or on a page outside the pool) has
// log2 s_t = -inf.
//
// Measured on one B200 (us, with expansion and merge; of the measured bf16 rate or copy bandwidth):
// 1024 rows x 40 heads over 32768 bf16 tokens, d = 512: 2371 (0.73); 4 x 512 rows near 8192 tokens
// of 8 bits: 1357 (0.60); 16 ragged sequences with 4 to 301 new tokens, 16 bits, d = 384: 741
// (0.31, two score MMAs); 8 ragged chunks over 4-bit groups, d = 128: 320 (0.28, two score MMAs);
// decode of 32 x 8192 16-bit tokens, 40 heads: 221 (0.21 of the bandwidth).  Counters of the last
// four: tensor pipe active 57, 48, 40 and 25 %, 1.1 to 1.8 instructions a cycle, no pipe full: the
// hand-overs of a block (rows landed, scores done, weights written, output free) bound it.
#include <math_constants.h>
#include <string.h>

#include <algorithm>

#include "kvk_chunk_convert.cuh"
#include "kvk_chunk_route.cuh"
#include "kvk_chunk_stop.cuh"
#include "kvk_chunk_tc.cuh"
#include "kvk_decode_common.cuh"
#include "kvk_sm100.cuh"

namespace kvk {
namespace {

using namespace sm100;
using namespace chunk;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kKWarp0 = 4, kVWarp0 = 8, kMmaWarp = 12, kTokWarp = 13, kRelayWarp = 14, kLoadWarp = 15;   // (see below)
constexpr uint32_t kAtom = 8192;       // 64 rows x 128 bytes
constexpr int kMinTok = 3, kMaxTok = 6;   // token stages: as many as the memory left holds
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;        // S buffers at 256 and 320 (64 columns); O at 0
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazy = 8.0f;          // growth of a row's maximum that its reference lets pass
constexpr float kHead = 7.0f;          // weights are held times 2^7 (below)
static_assert(kLazy + kHead <= 15.0f, "a weight fits f16");
constexpr int kSmemLimit = 232448;
constexpr int kMaxK = 8;               // slots of the K ring, two atoms each
constexpr int kStep = 2;               // atoms of a K ring slot
constexpr uint64_t kDrainLimitNs = 2000000000ull;

constexpr uint32_t kLaunchRegs = kChunkLaunchRegs;
static_assert(kLaunchRegs * kThreads == 65536, "one block takes the SM's registers");
template <uint32_t N>
__device__ __forceinline__ void regs_set() {
  if constexpr (N > kLaunchRegs) regs_inc<N>();
  else if constexpr (N < kLaunchRegs) regs_dec<N>();
}

// One block of 128 tokens of a piece, published by the token warp.
struct alignas(16) TokStage {
  int32_t slot[128];
  float sc[128], lsc[128], isc[128];   // s_t, log2 s_t, 1 / s_t
  int32_t flags;                       // kEnd, kFirst, kLast
  int32_t row0, flat0, rows;           // the sequence's first query row; the tile's first row
                                       // within the sequence and the sequence's row count
  int32_t len, count, t0;              // tokens, query tokens; first token of the block
  int32_t piece;                       // running number of the piece
  int32_t dest;                        // partial slot (0, 1) or -1: whole tile
  int32_t seq, b1, nblk;               // for the partial's header
};
constexpr int kEnd = 1, kFirst = 2, kLast = 4;

struct Shared {
  int8_t qexp[4][64];                  // per row: e of its query's scaling 2^e
  float xch[2][256];                   // maxima (at a piece's end: sums) of a row's threads
  uint64_t tok_full[kMaxTok], tok_empty[kMaxTok];
  // operands: written (by this CTA's warps), passed on (to the leader, by both relays), free
  uint64_t k_full[kMaxK], k_ready[kMaxK], k_empty[kMaxK];
  uint64_t v_full[4], v_ready[4], v_empty[4];
  uint64_t q_full, q_ready, q_empty, q_local[4];
  uint64_t s_full[2], s_free[2], p_full, p_ready, pv_done, x_bar, drain[2];
  int64_t scan[kWarps + 1];
  int64_t start_base;
  int32_t start_seq, start_k;
  int32_t issued[2];                   // steps whose loads this CTA has issued: K, V
  uint32_t tmem_base, abort_word;
};

static_assert(sizeof(Shared) + kMinTok * sizeof(TokStage) <= 11264, "leaves 27 atoms of 8 KB");

// Position in the ring of token stages.
struct TokRing {
  int n, st = 0;
  uint32_t par = 0;
  __device__ __forceinline__ explicit TokRing(int stages) : n(stages) {}
  __device__ __forceinline__ void next() {
    if (++st == n) {
      st = 0;
      par ^= 1;
    }
  }
};

// The fields of a piece's first block that query staging reads.
struct QueryTile {
  int row0, flat0, rows, piece;
};

struct TcChunk {
  ChunkArgs a;
  ChunkWork w;
  int NL, NA, NV;          // latent atoms (padded to whole 128), all atoms, V atoms per CTA
  int NK, NVS, NT;         // K ring slots, V stages, token stages
  uint32_t off_k, off_v, off_p, off_misc, off_tok;
  uint32_t idesc_s, idesc_o2, idesc_o1;   // score; output with 128 / 64 features per CTA
  int q_bf16;
  // expanded rows (kExp)
  const float* mark;       // per slot: 0, or NaN for a row with non-finite elements
  int box;                 // rows of a tensor-map box: min(page tokens, 64)
  int pool_slots;
};

// At a kernel's end: waits, until the clock shows `end` at the latest, for a phase that operations
// in flight complete.
__device__ __forceinline__ void drain(uint64_t* b, uint32_t parity, uint64_t end) {
  while (!mbar_try_hint(b, parity, 20000u) && globaltimer() < end) {
  }
}
// Counts bytes as landed that no load brings (a stopped kernel's).
__device__ __forceinline__ void mbar_complete_tx(uint64_t* b, uint32_t tx) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)),
               "r"(tx)
               : "memory");
}

// ---- cluster-scope barriers -----------------------------------------------------------------
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
// Arrives on the barrier of the pair's CTA `rank`.  What it orders is this CTA's shared memory, read
// by this SM's tensor core, so CTA scope serves; at cluster scope the arrival waits for this
// SM's global accesses too (measured about 1000 cycles).
__device__ __forceinline__ void arrive_at(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(
                   map_rank(smem_u32(bar), rank))
               : "memory");
}
template <typename T>
__device__ __forceinline__ T uniform(T x) {
  return __shfl_sync(0xffffffffu, x, 0);
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Arrives on the barrier of both CTAs once the elected lane's MMAs so far are complete.
__device__ __forceinline__ void commit_both(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// Four MMAs of the pair, D (+)= A_k B_k, issued by the elected lane of a converged warp: with the
// descriptors in uniform registers the pattern of one block (36 score and 16 output MMAs) takes
// 2380 cycles with its commits (2176 at the full rate); a lone thread issuing them took 6500.
// a, b: low words of the descriptors, hi: their common high word.
__device__ __forceinline__ void mma2x4(uint32_t d, uint32_t a, uint32_t b, uint32_t b_step,
                                       uint32_t hi_a, uint32_t hi_b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 x0, x1, x2, x3, y0, y1, y2, y3;\n\t.reg .b32 t;\n\t"
      "mov.b64 x0, {%1, %4};\n\t"
      "add.u32 t, %1, 2;\n\tmov.b64 x1, {t, %4};\n\t"     // K steps of 16: 32 bytes
      "add.u32 t, %1, 4;\n\tmov.b64 x2, {t, %4};\n\t"
      "add.u32 t, %1, 6;\n\tmov.b64 x3, {t, %4};\n\t"
      "mov.b64 y0, {%2, %5};\n\t"
      "add.u32 t, %2, %3;\n\tmov.b64 y1, {t, %5};\n\t"
      "add.u32 t, t, %3;\n\tmov.b64 y2, {t, %5};\n\t"
      "add.u32 t, t, %3;\n\tmov.b64 y3, {t, %5};\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %7, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], x0, y0, %6, p;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], x1, y1, %6, 1;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], x2, y2, %6, 1;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], x3, y3, %6, 1;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(b_step), "r"(hi_a), "r"(hi_b), "r"(idesc), "r"(acc)
      : "memory");
}
// 32 lanes x 32 columns: thread i of the warp holds lane base + i
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]),
      "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]),
      "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]),
      "f"(v[29]), "f"(v[30]), "f"(v[31])
      : "memory");
}

// Loads a box into this CTA's shared memory, counted on the barrier at cluster address `bar` (the
// leader's: the MMA that reads the pair's operands waits for both CTAs' loads there).
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void* tmap, int x, int y,
                                              uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// A stopped kernel's loads (kvk_chunk_stop.cuh): the leader waits for those of both CTAs, which have
// left their loops.  One deadline for all of them.
template <bool kLo>
__device__ __forceinline__ void finish_loads(const TcChunk& P, Shared& S, int nch) {
  const uint64_t end = globaltimer() + kDrainLimitNs;
  const int atoms = P.NA * (kLo ? 2 : 1), steps = (atoms + kStep - 1) / kStep;   // of a block
#pragma unroll 1
  for (int ring = 0; ring < 2; ++ring) {
    const int slots = ring == 0 ? P.NK : P.NVS * nch, own = S.issued[ring];
    int peer;
    asm volatile("ld.volatile.shared::cluster.s32 %0, [%1];"
                 : "=r"(peer)
                 : "r"(map_rank(smem_u32(&S.issued[ring]), 1))
                 : "memory");
#pragma unroll 1
    for (int i = stop_first(slots, own, peer); i < max(own, peer); ++i) {
      const StopStep t = stop_step(i, slots, own, peer);
      const int ch = t.slot % nch;
      uint64_t* bar = ring == 0 ? &S.k_ready[t.slot] : &S.v_ready[t.slot / nch * 2 + ch];
      // a CTA's atoms of the step (V: for both halves of the block's tokens)
      const int n = ring == 0 ? min(kStep, atoms - kStep * (i % steps)) : 2 * min(2, P.NV - 2 * ch);
      if (t.arm) mbar_arrive_expect_tx(bar, (uint32_t)n * kAtom);
      if (t.complete) mbar_complete_tx(bar, (uint32_t)n * kAtom);
      drain(bar, t.parity, end);
    }
  }
}

// Bounded waits of one call: a wait that runs out stops both CTAs.
__device__ __forceinline__ bool wait_slow(uint64_t* b, uint32_t parity, uint32_t abort_saddr,
                                       uint64_t limit) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_hint(b, parity, 20000u)) {
    if (abort_read(abort_saddr)) return false;
    if (globaltimer() - t0 > limit) {
      for (uint32_t r = 0; r < 2; ++r)
        asm volatile("st.volatile.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(abort_saddr, r)),
                     "r"(1u)
                     : "memory");
      return false;
    }
  }
  return true;
}
struct Waiter {
  uint32_t abort_saddr;
  uint64_t limit;
  __device__ __forceinline__ bool operator()(uint64_t* b, uint32_t parity) const {
    return mbar_try(b, parity) || wait_slow(b, parity, abort_saddr, limit);
  }
};

// Store 16 converted elements of atom row t, columns 16 sub .. 16 sub + 15 (two 16-byte chunks
// under the 128-byte swizzle)
__device__ __forceinline__ void store_unit(uint32_t atom, int t, int sub, const uint32_t (&w)[8]) {
  const uint32_t row = atom + (uint32_t)t * 128u;
  sts128(row + (uint32_t)(((2 * sub) ^ (t & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
  sts128(row + (uint32_t)(((2 * sub + 1) ^ (t & 7)) << 4), make_uint4(w[4], w[5], w[6], w[7]));
}

// Element index of columns 16 sub.. of atom `at` (latent atoms, then RoPE atoms), -1: padding
__device__ __forceinline__ int unit_elem(const TcChunk& P, int at, int sub) {
  const int x = (at < P.NL ? at : at - P.NL) * 64 + 16 * sub;
  if (at < P.NL) return x < P.a.d ? x : -1;
  return x < P.a.d_rope ? P.a.d + x : -1;
}

__device__ __forceinline__ int blocks_of(int len, int count, int H, int flat0, int rows) {
  // tokens that the tile's last row sees, in blocks of 128; one block where it sees none (its
  // rows are written all the same)
  const int last = min(flat0 + 128, rows) - 1;
  const int64_t vis = (int64_t)len - count + last / H + 1;
  const int v = (int)max((int64_t)0, min(vis, (int64_t)len));
  return max(1, (v + 127) >> 7);
}

// Query rows [r0, r1) of this CTA's 64, by one warp: four rows' loads in flight.  A bf16 query for f16
// operands is scaled by the power of two that brings its row's largest element into
// [2^14, 2^15); other queries are copied.  A negative softmax scale flips the sign.
template <bool OP_BF16>
__device__ __forceinline__ void stage_query(const TcChunk& P, Shared& S, uint32_t q_saddr,
                                            const QueryTile& h, int rank, int r0, int r1) {
  const int lane = threadIdx.x & 31;
  const int chunks = P.NA * 8;                    // 16-byte chunks of 8 features
  const bool scale = !OP_BF16 && P.q_bf16;
  const uint32_t flip = P.a.sigma < 0.0f ? 0x80008000u : 0u;
  constexpr int kC = 3;                           // chunks a lane: up to 96 (768 features)
  constexpr int kR = 4;
  const uint16_t* qlat = static_cast<const uint16_t*>(P.a.q_lat);
  const uint16_t* qrope = static_cast<const uint16_t*>(P.a.q_rope);
#pragma unroll 1
  for (int r = r0; r < r1; r += kR) {
    uint4 v[kR][kC];
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int flat = h.flat0 + rank * 64 + r + i;
      const bool ok = flat < h.rows;
      const int j = ok ? flat / P.a.H : 0, hd = flat - j * P.a.H;
      const uint16_t* pl = qlat + (int64_t)(h.row0 + j) * P.a.ql_st + (int64_t)hd * P.a.ql_sh;
      const uint16_t* pr = qrope + (int64_t)(h.row0 + j) * P.a.qr_st + (int64_t)hd * P.a.qr_sh;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int ch = c * 32 + lane;
        const int x = ch * 8 - (ch * 8 >= P.NL * 64 ? P.NL * 64 : 0);
        v[i][c] = make_uint4(0u, 0u, 0u, 0u);
        if (ok && ch < chunks) {
          if (ch * 8 < P.NL * 64) {
            if (x < P.a.d) v[i][c] = __ldg(reinterpret_cast<const uint4*>(pl + x));
          } else if (x < P.a.d_rope) {
            v[i][c] = __ldg(reinterpret_cast<const uint4*>(pr + x));
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      int e = 0;
      float mul = 1.0f;
      if (scale) {
        uint32_t mx = 0;   // largest magnitude as bf16 bits (sign cleared: ordered as integers)
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const uint32_t w[4] = {v[i][c].x, v[i][c].y, v[i][c].z, v[i][c].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx = max(mx, max((w[k] & 0x7FFFu), ((w[k] >> 16) & 0x7FFFu)));
        }
        mx = __reduce_max_sync(0xffffffffu, mx);
        const int ex = (int)(mx >> 7);             // biased exponent of the largest
        if (ex > 0 && ex < 255) {
          // e = 14 - (ex - 127), kept where 2^e and 2^-e are normal numbers
          e = max(-126, min(126, 141 - ex));
          mul = __uint_as_float((uint32_t)(127 + e) << 23);
        }
      }
      const int t = r + i;
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int ch = c * 32 + lane;
        if (ch >= chunks) continue;
        uint32_t w[4] = {v[i][c].x, v[i][c].y, v[i][c].z, v[i][c].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (scale) {
            const __half2 x = __floats2half2_rn(__uint_as_float(w[k] << 16) * mul,
                                                __uint_as_float(w[k] & 0xFFFF0000u) * mul);
            w[k] = *reinterpret_cast<const uint32_t*>(&x);
          }
          w[k] ^= flip;
        }
        sts128(q_saddr + (uint32_t)(ch >> 3) * kAtom + (uint32_t)t * 128u +
                   (uint32_t)(((ch & 7) ^ (t & 7)) << 4),
               make_uint4(w[0], w[1], w[2], w[3]));
      }
      if (lane == 0) S.qexp[h.piece & 3][t] = (int8_t)e;
    }
  }
}

// The rarely taken parts of the softmax warps.
__device__ __forceinline__ void rescale_o(uint32_t obase, int cols, float alpha) {
#pragma unroll 1
  for (int c = 0; c < cols; c += 32) {
    float o[32];
    tmem_ld32(obase + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] *= alpha;
    tmem_st32(obase + c, o);
  }
  tmem_wait_st();
}
// Features f0 .. f0 + cols (those below d) of a row: fp32 sums (type < 0), or bf16 / f16 results.
__device__ __forceinline__ void write_o(uint32_t obase, int cols, int f0, int d, void* to, int type,
                                     float inv) {
#pragma unroll 1
  for (int c = 0; c < cols; c += 32) {
    float o[32];
    tmem_ld32(obase + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int q = 0; q < 4; ++q) {                // d is a multiple of 16
      const int f = f0 + c + 8 * q;
      if (f >= d) break;
      if (type < 0) {
        float* po = static_cast<float*>(to) + f;
        *reinterpret_cast<float4*>(po) =
            make_float4(o[8 * q], o[8 * q + 1], o[8 * q + 2], o[8 * q + 3]);
        *reinterpret_cast<float4*>(po + 4) =
            make_float4(o[8 * q + 4], o[8 * q + 5], o[8 * q + 6], o[8 * q + 7]);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = pack_out(type, o[8 * q + 2 * k] * inv, o[8 * q + 2 * k + 1] * inv);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(to) + f) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// Exclusive prefix of v over the block; *total gets the sum.  All threads call it.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* buf, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int64_t t = buf[w];
    if (w < warp) before += t;
    all += t;
  }
  *total = all;
  return before + x - v;
}

template <int BITS, bool GROUP, bool kExp>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
chunk_tc_kernel(const __grid_constant__ TcChunk P, const __grid_constant__ CUtensorMap map_hi,
                const __grid_constant__ CUtensorMap map_lo) {
  constexpr bool kBf16 = BITS == KVK_BITS_BF16;
  constexpr bool kTok = !GROUP && !kBf16;             // one scale per token
  constexpr bool kLo = kSplit<BITS, GROUP>;
  constexpr int kSoftWarps = kExp ? 8 : 4;
  // cost of a row tile beside its blocks, in blocks (a ragged batch of 16 over expanded rows: 951 us
  // with 2, 831 with 4, 822 with 6; decode of 32 sequences from packed rows: 230, 245, 250)
  constexpr int kCost = kExp ? 5 : 2;
  // the output MMAs' warp is the one that has no other work: the relay's with expanded rows, else
  // the loads'
  constexpr int kOutWarp = kExp ? kRelayWarp : kLoadWarp;
  extern __shared__ __align__(1024) uint8_t smem[];
  const ChunkArgs& a = P.a;
  TokStage* const toks = reinterpret_cast<TokStage*>(smem + P.off_tok);
  TokRing ring(P.NT);
  Shared& S = *reinterpret_cast<Shared*>(smem + P.off_misc);
  const uint32_t q_s = smem_u32(smem), k_s = q_s + P.off_k, v_s = q_s + P.off_v, p_s = q_s + P.off_p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cta_rank();
  const int cluster = blockIdx.x >> 1;
  const int G = P.w.G;

  if (tid == 0) {
    S.abort_word = 0;
    S.issued[0] = S.issued[1] = 0;
    for (int i = 0; i < kMaxTok; ++i) {
      mbar_init(&S.tok_full[i], 1);
      // softmax warps, loading or converting warps and relay, the leader's MMA warps
      mbar_init(&S.tok_empty[i], kSoftWarps + (kExp ? 5 : 9) + (rank == 0 ? 2 : 0));
    }
    for (int i = 0; i < kMaxK; ++i) {
      mbar_init(&S.k_full[i], 4);
      mbar_init(&S.k_ready[i], kExp ? 1 : 2);      // loads: one arming for both CTAs' bytes
      mbar_init(&S.k_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&S.v_full[i], 4);
      mbar_init(&S.v_ready[i], kExp ? 1 : 2);
      mbar_init(&S.v_empty[i], 1);
      mbar_init(&S.q_local[i], kExp ? 4 : 8);
    }
    mbar_init(&S.q_full, 8);
    mbar_init(&S.q_ready, kExp ? 8 : 2);
    mbar_init(&S.q_empty, 1);
    mbar_init(&S.s_full[0], 1);
    mbar_init(&S.s_full[1], 1);
    mbar_init(&S.s_free[0], 2 * kSoftWarps);
    mbar_init(&S.s_free[1], 2 * kSoftWarps);
    mbar_init(&S.p_full, kSoftWarps);
    mbar_init(&S.p_ready, kExp ? 2 * kSoftWarps : 2);
    mbar_init(&S.pv_done, 1);
    mbar_init(&S.x_bar, kSoftWarps);
    mbar_init(&S.drain[0], 1);
    mbar_init(&S.drain[1], 1);
    fence_mbar_init();
    // no partials of this cluster yet
    if (rank == 0) {
      P.w.head[cluster * 2].valid = 0;
      P.w.head[cluster * 2 + 1].valid = 0;
    }
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&S.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }

  // ---- this cluster's slice of the work -------------------------------------------------------
  // tiles of every sequence (prefix sums in the ring's memory, not yet in use), then their costs
  int32_t* pre = reinterpret_cast<int32_t*>(smem);
  int64_t u0 = 0, u1 = 0;
  {
    const int per = (a.batch + kThreads - 1) / kThreads;
    const int i0 = min(a.batch, tid * per), i1 = min(a.batch, i0 + per);
    int64_t tiles = 0, total_tiles = 0, total = 0;
    bool bad_rows = false, bad_len = false;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const int s0 = __ldg(a.q_start + i), s1 = __ldg(a.q_start + i + 1), l = __ldg(a.seq_lens + i);
      bad_rows = bad_rows || s0 < 0 || s1 < s0 || s1 > a.n_q;
      bad_len = bad_len || l < 0 || l > a.cap;
      tiles += ((int64_t)max(0, s1 - s0) * a.H + 127) >> 7;
    }
    const bool stop = __syncthreads_or(bad_rows) != 0;
    if ((bad_rows || bad_len) && blockIdx.x == 0) atomicOr(a.flags, KVK_FLAG_SEQ_LEN);
    int64_t at = block_scan(stop ? 0 : tiles, S.scan, &total_tiles);
    if (!stop) {
#pragma unroll 1
      for (int i = i0; i < i1; ++i) {
        const int s0 = __ldg(a.q_start + i), s1 = __ldg(a.q_start + i + 1);
        pre[i] = (int32_t)at;
        at += ((int64_t)(s1 - s0) * a.H + 127) >> 7;
      }
      if (tid == 0) pre[a.batch] = (int32_t)total_tiles;
    }
    __syncthreads();
    // costs of a run of consecutive tiles a thread
    const int nt = (int)total_tiles;
    const int tper = (nt + kThreads - 1) / kThreads;
    const int f0 = min(nt, tid * tper), f1 = min(nt, f0 + tper);
    int seq0 = 0;
    if (f0 < f1) {
      int lo = 0, hi = a.batch - 1;   // the last sequence whose tiles start at or before f0
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= f0) lo = mid; else hi = mid - 1;
      }
      seq0 = lo;
    }
    int64_t cost = 0, base = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      int seq = seq0, loaded = -1;
      ChunkSeq s = {0, 0, 0};
#pragma unroll 1
      for (int f = f0; f < f1; ++f) {
        while (pre[seq + 1] <= f) ++seq;
        if (loaded != seq) {
          bool b;
          s = chunk_seq(a, seq, &b);
          loaded = seq;
        }
        const int k = f - pre[seq];
        const int c = kCost + blocks_of(s.len, s.count, a.H, k * 128, s.count * a.H);
        if (pass == 0) {
          cost += c;
        } else {
          if (base <= u0 && u0 < base + c) {
            S.start_seq = seq;
            S.start_k = k;
            S.start_base = base;
          }
          base += c;
        }
      }
      if (pass == 0) {
        base = block_scan(cost, S.scan, &total);
        u0 = split_cost(cluster, total, G);
        u1 = split_cost(cluster + 1, total, G);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers are initialised, both have allocated
  tc_fence_after();
  const uint32_t tmem = S.tmem_base;
  const Waiter wait{smem_u32(&S.abort_word), a.limit_ns};
  // Registers: the block is launched with kLaunchRegs a thread (the host checks it); the last
  // warpgroup gives some of its to the others, whose spills would go to L2 (shared memory takes
  // the cache's place).
  constexpr uint32_t kRegs0 = kExp ? 152 : 144, kRegs1 = 152, kRegs2 = kExp ? 128 : 144,
                     kRegs3 = kExp ? 80 : 72;
  static_assert(kRegs0 + kRegs1 + kRegs2 + kRegs3 <= 4 * kLaunchRegs, "register split");
  const int nch = (P.NV + 1) >> 1;       // output MMA steps over the features: 2 atoms, or the last 1

  // The warp index, and what a warp reads from shared memory to steer its MMAs, go through a
  // shuffle: known to be the same in every lane, they and all that follows from them stay in
  // uniform registers, where the MMA's operands have to be.  (A block's MMAs with their waits and
  // commits: 2264 cycles issued so, 4545 from per-lane registers.)
  if (uniform(warp) == kMmaWarp || uniform(warp) == kOutWarp) {
    regs_set<kRegs3>();
    // ======================= MMA issuers: scores, outputs =======================================
    // Two warps, each converged: what one spends between its MMAs (a wait, a commit: about 280
    // cycles a step) the tensor cores spend on the other's.
    if (rank == 0) {
      auto all = [&](uint64_t* b, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, wait(b, parity));
      };
      const uint64_t q0 = sdesc(q_s, 16u, 1024u, kLayoutSw128);
      const uint64_t vb0 = sdesc(v_s, kAtom, 1024u, kLayoutSw128);
      const uint32_t hk = (uint32_t)(q0 >> 32), hv = (uint32_t)(vb0 >> 32);
      const uint32_t ql = (uint32_t)q0, vl = (uint32_t)vb0;
      const uint32_t kl = ql + (P.off_k >> 4), pl = ql + (P.off_p >> 4);
      constexpr uint32_t kA = kAtom >> 4;             // an atom in descriptor units
      const uint32_t tmem = uniform(S.tmem_base);
      const bool scores = uniform(warp) == kMmaWarp;
      int kslot = 0, pieces = 0;
      uint32_t kpar = 0;
      bool ok = true;
      for (int g = 0;; ++g) {
        const int st = ring.st;
        ok = all(&S.tok_full[st], ring.par);
        ring.next();
        if (!ok) break;
        const int now = uniform(*const_cast<volatile int32_t*>(&toks[st].flags));
        if (lane == 0) mbar_arrive(&S.tok_empty[st]);
        if (now & kEnd) break;
        if (scores) {
          if (now & kFirst) ok = all(&S.q_ready, pieces & 1);
          ok = ok && all(&S.s_free[g & 1], ((g >> 1) & 1) ^ 1);
          if (!ok) break;
          tc_fence_after();   // the softmax's reads of this S buffer
          const uint32_t scol = tmem + kSCol + 64u * (g & 1);
          const int atoms = P.NA * (kLo ? 2 : 1);
          uint32_t acc = 0, qa = ql;
#pragma unroll 1
          for (int i = 0; i < atoms; i += kStep) {
            ok = all(&S.k_ready[kslot], kpar);
            if (!ok) break;
            const uint32_t kb = kl + (uint32_t)(kslot * kStep) * kA;
            mma2x4(scol, qa, kb, 2u, hk, hk, P.idesc_s, acc);
            if (!kLo) qa += kA;      // the next atom, or the low part of the same elements
            if (i + 1 < atoms) mma2x4(scol, qa, kb + kA, 2u, hk, hk, P.idesc_s, 1u);
            qa += kA;
            commit_both(&S.k_empty[kslot]);
            acc = 1;
            if (++kslot == P.NK) {
              kslot = 0;
              kpar ^= 1;
            }
          }
          if (!ok) break;
          commit_both(&S.s_full[g & 1]);
          if (now & kLast) {
            commit_both(&S.q_empty);
            ++pieces;
          }
        } else {
          ok = all(&S.p_ready, g & 1);
          if (!ok) break;
          tc_fence_after();   // the softmax's stores to O
          const int vs = g % P.NVS;
          const uint32_t vpar = (g / P.NVS) & 1;
          const uint32_t acc = (now & kFirst) ? 0u : 1u;   // a piece starts the sums anew
          uint32_t vb = vl + (uint32_t)(vs * 2 * P.NV) * kA;
#pragma unroll 1
          for (int ch = 0; ch < nch; ++ch, vb += 4 * kA) {
            ok = all(&S.v_ready[vs * 2 + ch], vpar);
            if (!ok) break;
            const bool two = 2 * ch + 2 <= P.NV;
            const uint32_t idesc = two ? P.idesc_o2 : P.idesc_o1;
            mma2x4(tmem + 128u * ch, pl, vb, 128u, hk, hv, idesc, acc);
            mma2x4(tmem + 128u * ch, pl + kA, vb + (two ? 2 * kA : kA), 128u, hk, hv, idesc, 1u);
            commit_both(&S.v_empty[vs * 2 + ch]);
          }
          if (!ok) break;
          commit_both(&S.pv_done);
        }
      }
      // every MMA is done before either CTA leaves
      __syncwarp();
      commit_both(&S.drain[scores ? 0 : 1]);
      drain(&S.drain[scores ? 0 : 1], 0u, globaltimer() + kDrainLimitNs);
    }
  } else if (warp == kTokWarp) {
    regs_set<kRegs3>();
    // ======================= token warp: pieces, slots, scales ==================================
    int seq = S.start_seq, k = S.start_k;
    int64_t base = S.start_base;
    int g = 0, piece = 0;
    bool ok = true;
    if (u0 < u1) {
      bool b;
      ChunkSeq s = chunk_seq(a, seq, &b);
      while (ok && base < u1) {
        const int rows = s.count * a.H;
        const int nblk = blocks_of(s.len, s.count, a.H, k * 128, rows);
        const int64_t x0 = u0 - base - kCost, x1 = u1 - base - kCost;
        const int b0 = (int)max((int64_t)0, min(x0, (int64_t)nblk));
        const int b1 = (int)max((int64_t)0, min(x1, (int64_t)nblk));
        auto slots_of = [&](int t0, int (&sl)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = t0 + 32 * i + lane;
            sl[i] = t < s.len ? chunk_slot(a, seq, t) : -1;
          }
        };
        // scales and marks; the rows that this CTA converts for the scores are fetched into L2
        auto scales_of = [&](const int (&sl)[4], float (&sc)[4], float (&mk)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[i] = (kTok && sl[i] >= 0) ? __half2float(a.scales[sl[i]]) : 1.0f;
            mk[i] = (kExp && sl[i] >= 0) ? __ldg(P.mark + sl[i]) : 0.0f;
          }
#pragma unroll
          for (int i = 0; !kExp && i < 2; ++i) {
            const int my = rank ? sl[2 + i] : sl[i];
            if (my >= 0) {
              const uint8_t* p = a.codes + (int64_t)my * a.row_bytes;
#pragma unroll 1
              for (int x = 0; x < a.row_bytes; x += 128) prefetch_l2(p + x);
            }
          }
        };
        int sl[4];
        float sc[4], mk[4];
        if (b0 < b1) {
          slots_of(b0 << 7, sl);
          scales_of(sl, sc, mk);
        }
#pragma unroll 1
        for (int blk = b0; ok && blk < b1; ++blk, ++g) {
          const int st = ring.st;
          ok = wait(&S.tok_empty[st], ring.par ^ 1);
          ring.next();
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          TokStage& T = toks[st];
          const int t0 = blk << 7;
          // the next block's slots are on their way while this one's entries are written
          int sn[4];
          if (blk + 1 < b1) slots_of(t0 + 128, sn);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            T.slot[32 * i + lane] = sl[i];
            if constexpr (kTok) T.sc[32 * i + lane] = sc[i];
            T.lsc[32 * i + lane] = sl[i] >= 0 ? mk[i] : -CUDART_INF_F;
          }
          if constexpr (kTok) {
            // (the lane's own entries again, rolled: little code)
#pragma unroll 1
            for (int x = lane; x < 128; x += 32) {
              const bool real = T.slot[x] >= 0;
              const float v = T.sc[x];
              // an all-zero token (scale 0) keeps its score 0; its weight multiplies zeros, so
              // any positive scale serves
              const float w = v == 0.0f ? 5.9604644775390625e-8f : v;
              T.sc[x] = real ? v : 0.0f;
              // (a scale that is not finite shows in the weight of those who see the token; here
              // it would reach, times a weight of 0, those who do not)
              T.isc[x] = real && isfinite(w) ? __frcp_rn(w) : 0.0f;
              T.lsc[x] += log2f(w);
            }
          }
          if (lane == 0) {
            T.flags = (blk == b0 ? kFirst : 0) | (blk == b1 - 1 ? kLast : 0);
            T.row0 = s.row0;
            T.flat0 = k * 128;
            T.rows = rows;
            T.len = s.len;
            T.count = s.count;
            T.t0 = t0;
            T.piece = piece;
            T.dest = (b0 == 0 && b1 == nblk) ? -1 : (b0 > 0 ? 0 : 1);
            T.seq = seq;
            T.b1 = b1;
            T.nblk = nblk;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.tok_full[st]);
          if (blk + 1 < b1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sl[i] = sn[i];
            scales_of(sl, sc, mk);
          }
        }
        if (b1 > b0) ++piece;
        base += kCost + nblk;
        ++k;
        if (base < u1 && k * 128 >= rows) {   // the next sequence that has query rows
          k = 0;
          ++seq;
          while (seq < a.batch) {
            const int i = seq + lane;
            const bool has = i < a.batch && __ldg(a.q_start + i + 1) > __ldg(a.q_start + i);
            const unsigned m = __ballot_sync(0xffffffffu, has);
            if (m) {
              seq += __ffs(m) - 1;
              break;
            }
            seq += 32;
          }
          if (seq >= a.batch) break;
          s = chunk_seq(a, seq, &b);
        }
      }
    }
    if (ok) {
      const int st = ring.st;
      ok = __all_sync(0xffffffffu, wait(&S.tok_empty[st], ring.par ^ 1));
      if (ok && lane == 0) {
        toks[st].flags = kEnd;
        mbar_arrive(&S.tok_full[st]);
      }
    }
  } else if (warp == kRelayWarp) {
    regs_set<kRegs3>();
    // ======================= relay (converted rows) =============================================
    // One thread passes this CTA's full barriers on to the leader: query and K in the order of the
    // score MMAs, P and V in that of the output MMAs, whichever comes first.  It makes the proxy
    // fence for the threads that wrote the operands, whose own would wait for all their loads in
    // flight (measured 1600 cycles per atom of the K team).
    if (!kExp && lane == 0) {
      const int steps = (P.NA * (kLo ? 2 : 1) + kStep - 1) / kStep;
      // score side: block gk, its barrier ik (-1: not entered, 0: query, 1 + step); output side: gp,
      // ip (0: P, 1 + step)
      int gk = 0, ik = -1, kslot = 0, pieces = 0, gp = 0, ip = 0, end = 0x7FFFFFFF;
      uint32_t kpar = 0;
      uint64_t t0 = globaltimer();
      int idle = 0;
      auto pass = [&](uint64_t* b, uint64_t* ready, uint32_t parity) -> bool {
        if (!mbar_test(b, parity)) return false;
        fence_proxy_async_smem();
        arrive_at(ready, 0);
        return true;
      };
      while (gk < end || gp < end) {
        bool moved = false;
        if (gk < end) {
          if (ik < 0) {
            const int st = ring.st;
            if (mbar_test(&S.tok_full[st], ring.par)) {
              ring.next();
              const int fl = *const_cast<volatile int32_t*>(&toks[st].flags);
              mbar_arrive(&S.tok_empty[st]);
              moved = true;
              if (fl & kEnd) end = gk;
              else ik = (fl & kFirst) ? 0 : 1;
            }
          } else if (ik == 0) {
            if (pass(&S.q_full, &S.q_ready, pieces & 1)) {
              ++pieces;
              ik = 1;
              moved = true;
            }
          } else if (pass(&S.k_full[kslot], &S.k_ready[kslot], kpar)) {
            moved = true;
            if (++kslot == P.NK) {
              kslot = 0;
              kpar ^= 1;
            }
            if (++ik > steps) {
              ik = -1;
              ++gk;
            }
          }
        }
        if (gp < end) {
          const int vs = gp % P.NVS * 2 + ip - 1;
          if (ip == 0 ? pass(&S.p_full, &S.p_ready, gp & 1)
                      : pass(&S.v_full[vs], &S.v_ready[vs], (gp / P.NVS) & 1)) {
            moved = true;
            if (++ip > nch) {
              ip = 0;
              ++gp;
            }
          }
        }
        if (moved) {
          idle = 0;
        } else if ((++idle & 63) == 0) {
          if (abort_read(smem_u32(&S.abort_word))) break;
          if (idle == 64) t0 = globaltimer();
          else if (globaltimer() - t0 > a.limit_ns) {
            wait_slow(&S.drain[0], 0u, smem_u32(&S.abort_word), 0ull);   // (stops both CTAs)
            break;
          }
        }
      }
    }
  } else if (warp == kLoadWarp) {
    regs_set<kRegs3>();
    // ======================= K loads (expanded rows) ============================================
    int kslot = 0, issued = 0;
    uint32_t kpar = 1;
    bool ok = kExp;
    while (ok) {
      const int st = ring.st;
      ok = __all_sync(0xffffffffu, wait(&S.tok_full[st], ring.par));
      ring.next();
      if (!ok || (toks[st].flags & kEnd)) break;
      // a lane per box: slots of the block's boxes, atoms of the step
      const int per = 64 / P.box, lg = 31 - __clz(per);
      int sl = P.pool_slots;                          // reads as zero
      if (lane < 2 * per) {
        const int x = toks[st].slot[64 * (int)rank + (lane & (per - 1)) * P.box];
        if (x >= 0) sl = x;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.tok_empty[st]);
      const int atoms = P.NA * (kLo ? 2 : 1), j = lane >> lg;
      const uint32_t to = q_s + P.off_k + (uint32_t)j * kAtom + (uint32_t)((lane & (per - 1)) * P.box) * 128u;
      const void* map = kLo && j ? &map_lo : &map_hi;
#pragma unroll 1
      for (int i = 0; i < atoms; i += kStep) {
        ok = __all_sync(0xffffffffu, wait(&S.k_empty[kslot], kpar));
        if (!ok) break;
        const int n = min(kStep, atoms - i);
        if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&S.k_ready[kslot], 2u * n * kAtom);
        if (j < n)
          tma_load_pair(to + (uint32_t)(kslot * kStep) * kAtom, map, (kLo ? i >> 1 : i + j) * 64, sl,
                        map_rank(smem_u32(&S.k_ready[kslot]), 0));
        __syncwarp();
        ++issued;
        if (++kslot == P.NK) {
          kslot = 0;
          kpar ^= 1;
        }
      }
    }
    if (lane == 0) S.issued[0] = issued;
  } else if (kExp && warp >= kVWarp0) {
    regs_set<kRegs2>();
    // ======================= V loads (expanded rows), query rows ================================
    const int vw = warp - kVWarp0;
    int issued = 0;
    bool ok = true;
    for (int g = 0;; ++g) {
      const int st = ring.st;
      ok = __all_sync(0xffffffffu, wait(&S.tok_full[st], ring.par));
      ring.next();
      if (!ok) break;
      const TokStage& T = toks[st];
      const int fl = T.flags;
      if (fl & kEnd) break;
      if (fl & kFirst) {
        const QueryTile head = {T.row0, T.flat0, T.rows, T.piece};
        if (head.piece > 0) ok = wait(&S.q_empty, (head.piece - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        stage_query<kBf16>(P, S, q_s, head, (int)rank, vw * 16, vw * 16 + 16);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.q_local[head.piece & 3]);
          arrive_at(&S.q_ready, 0);
        }
      }
      if (vw == 0) {
        const int vs = g % P.NVS;
        const uint32_t vpar = (g / P.NVS) & 1;
        const uint32_t stage = q_s + P.off_v + (uint32_t)(vs * 2 * P.NV) * kAtom;
        // a lane per box: slots of the block's boxes, atoms of the step
        const int per = 128 / P.box;
#pragma unroll 1
        for (int ch = 0; ch < nch; ++ch) {
          const int nj = min(2, P.NV - 2 * ch);
          uint64_t* bar = &S.v_ready[vs * 2 + ch];
          ok = __all_sync(0xffffffffu, wait(&S.v_empty[vs * 2 + ch], vpar ^ 1));
          if (!ok) break;
          if (rank == 0 && lane == 0) mbar_arrive_expect_tx(bar, 2u * 2u * nj * kAtom);
#pragma unroll 1
          for (int i = lane; i < per * nj; i += 32) {
            const int jj = i >= per, t = (i - jj * per) * P.box;
            const int sl = T.slot[t];
            tma_load_pair(stage + (uint32_t)(4 * ch + (t >> 6) * nj + jj) * kAtom +
                              (uint32_t)(t & 63) * 128u,
                          &map_hi, ((int)rank * P.NV + 2 * ch + jj) * 64,
                          sl < 0 ? P.pool_slots : sl, map_rank(smem_u32(bar), 0));
          }
          __syncwarp();
          ++issued;
        }
        if (!ok) break;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.tok_empty[st]);
    }
    if (vw == 0 && lane == 0) S.issued[1] = issued;
  } else if (!kExp && warp >= kVWarp0) {
    regs_set<kRegs2>();
    // ======================= V team =============================================================
    const int vt = tid - kVWarp0 * 32, tq = vt >> 2, sub = vt & 3;
    const int vw = warp - kVWarp0;
    bool ok = true;
    for (int g = 0;; ++g) {
      const int st = ring.st;
      ok = __all_sync(0xffffffffu, wait(&S.tok_full[st], ring.par));
      ring.next();
      if (!ok) break;
      const TokStage& T = toks[st];
      const int fl = T.flags;
      if (fl & kEnd) break;
      Row<GROUP> row[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) row[u] = row_of<GROUP>(a, T.slot[tq + 32 * u]);
      Unit<BITS, GROUP> cur[4], nxt[4];
      auto load = [&](int j, Unit<BITS, GROUP> (&to)[4]) {
        const int e = unit_elem(P, (int)rank * P.NV + j, sub);
        if (e >= 0) {
#pragma unroll
          for (int u = 0; u < 4; ++u) load_unit<BITS, GROUP>(a, row[u], e, to[u]);
        }
      };
      load(0, cur);
      if (fl & kFirst) {
        if (T.piece > 0) ok = wait(&S.q_empty, (T.piece - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const QueryTile head = {T.row0, T.flat0, T.rows, T.piece};
        stage_query<kBf16>(P, S, q_s, head, (int)rank, 32 + vw * 8, 32 + vw * 8 + 8);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.q_local[T.piece & 3]);
          mbar_arrive(&S.q_full);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.tok_empty[st]);
      const int vs = g % P.NVS;
      const uint32_t vpar = ((g / P.NVS) & 1) ^ 1;
      const uint32_t stage = v_s + (uint32_t)(vs * 2 * P.NV) * kAtom;
#pragma unroll 1
      for (int j = 0; j < P.NV; ++j) {
        const int ch = j >> 1, jj = j & 1, nj = min(2, P.NV - 2 * ch);
        if (j + 1 < P.NV) load(j + 1, nxt);
        if (jj == 0) {
          ok = __all_sync(0xffffffffu, wait(&S.v_empty[vs * 2 + ch], vpar));
          if (!ok) break;
        }
        const int e = unit_elem(P, (int)rank * P.NV + j, sub);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t hi[8], lo[8];
          operand16<BITS, GROUP, false>(cur[u], e >= 0 && (kTok || row[u].real), 0u, hi, lo);
          // [token half][atom of the step][64 tokens]
          store_unit(stage + (uint32_t)(4 * ch + (u >> 1) * nj + jj) * kAtom, tq + 32 * (u & 1), sub, hi);
        }
        if (jj + 1 == nj) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&S.v_full[vs * 2 + ch]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) cur[u] = nxt[u];
      }
      if (!ok) break;
    }
  } else if (!kExp && warp >= kKWarp0) {
    regs_set<kRegs1>();
    // ======================= K team =============================================================
    // A ring slot is two atoms: two of the row's, or the high and the low part of one.  The next
    // slot's rows are loaded while this one's are converted.
    constexpr int kPer = kLo ? 1 : 2;             // atoms of the row in a slot
    const int kt = tid - kKWarp0 * 32, tq = kt >> 2, sub = kt & 3;
    const int kw = warp - kKWarp0;
    const int steps = (P.NA + kPer - 1) / kPer;
    int kslot = 0;
    uint32_t kpar = 1;
    bool ok = true, last = false;
    Row<GROUP> row[2];     // of the block whose rows are loaded next
    Unit<BITS, GROUP> cur[kPer][2], nxt[kPer][2];
    bool real[2], next_real[2];
    auto take = [&]() -> bool {
      const int s1 = ring.st;
      if (!__all_sync(0xffffffffu, wait(&S.tok_full[s1], ring.par))) return false;
      ring.next();
      const TokStage& T = toks[s1];
      last = (T.flags & kLast) != 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        row[u] = row_of<GROUP>(a, T.slot[64 * (int)rank + tq + 32 * u]);
        next_real[u] = row[u].real;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.tok_empty[s1]);
      return true;
    };
    auto load = [&](int step, Unit<BITS, GROUP> (&to)[kPer][2]) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int at = step * kPer + j;
        const int e = at < P.NA ? unit_elem(P, at, sub) : -1;
        if (e >= 0) {
#pragma unroll
          for (int u = 0; u < 2; ++u) load_unit<BITS, GROUP>(a, row[u], e, to[j][u]);
        }
      }
    };
    for (;;) {             // one piece
      const int st = ring.st;
      ok = __all_sync(0xffffffffu, wait(&S.tok_full[st], ring.par));
      if (!ok) break;
      if (toks[st].flags & kEnd) break;
      const QueryTile head = {toks[st].row0, toks[st].flat0, toks[st].rows, toks[st].piece};
      ok = take();
      if (!ok) break;
      load(0, cur);
      real[0] = next_real[0], real[1] = next_real[1];
      if (head.piece > 0) ok = __all_sync(0xffffffffu, wait(&S.q_empty, (head.piece - 1) & 1));
      if (!ok) break;
      stage_query<kBf16>(P, S, q_s, head, (int)rank, kw * 8, kw * 8 + 8);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&S.q_local[head.piece & 3]);
        mbar_arrive(&S.q_full);
      }
      int step = 0;
      for (bool more = true; more;) {
        // the rows after these
        int next = step + 1;
        if (next < steps) {
          load(next, nxt);
        } else if (last) {
          more = false;
        } else {
          next = 0;
          ok = take();
          if (!ok) break;
          load(0, nxt);
        }
        ok = __all_sync(0xffffffffu, wait(&S.k_empty[kslot], kpar));
        if (!ok) break;
        const uint32_t slot = k_s + (uint32_t)(2 * kslot) * kAtom;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int at = step * kPer + j;
          if (at >= P.NA) break;
          const int e = unit_elem(P, at, sub);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t hi[8], lo[8];
            operand16<BITS, GROUP, kLo>(cur[j][u], e >= 0 && (kTok || real[u]), 0x7FFFu, hi, lo);
            store_unit(slot + (uint32_t)j * kAtom, tq + 32 * u, sub, hi);
            if constexpr (kLo) store_unit(slot + kAtom, tq + 32 * u, sub, lo);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.k_full[kslot]);
        if (++kslot == P.NK) {
          kslot = 0;
          kpar ^= 1;
        }
        step = next;
        if (next == 0) real[0] = next_real[0], real[1] = next_real[1];
#pragma unroll
        for (int j = 0; j < kPer; ++j)
#pragma unroll
          for (int u = 0; u < 2; ++u) cur[j][u] = nxt[j][u];
      }
      if (!ok) break;
    }
  } else {
    // ======================= softmax ============================================================
    regs_set<kRegs0>();
    // A row belongs to one thread per token half and, with expanded rows, column group: the
    // converting warps' place is then taken by a second set of softmax warps.
    constexpr int kCols = kExp ? 32 : 64;            // S columns (tokens) of a thread
    const int r = tid & 63, hh = (tid >> 6) & 1, cg = tid >> 7;
    const int col0 = 64 * hh + kCols * cg;           // first token of the block
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const int oc = P.NV * 64;                        // O columns (features of one half)
    const int ocg = kExp ? oc / 2 : oc;              // and those of this thread
    const uint32_t obase = tmem + (uint32_t)(ocg * cg) + lanes;
    float m = -CUDART_INF_F, l = 0.0f, rc = 0.0f;
    int lim = 0, row_q = 0, row_h = 0;
    bool row_ok = false;
    bool ok = true;
    uint32_t met = 0;
    auto meet = [&]() -> bool {                      // the softmax warps, bounded like every wait
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.x_bar);
      return __all_sync(0xffffffffu, wait(&S.x_bar, met++ & 1));
    };
    for (int g = 0;; ++g) {
      const int st = ring.st;
      ok = __all_sync(0xffffffffu, wait(&S.tok_full[st], ring.par));
      ring.next();
      if (!ok) break;
      const TokStage& T = toks[st];
      const int fl = T.flags;
      if (fl & kEnd) break;
      if (fl & kFirst) {
        const int piece = T.piece;
        const int flat = T.flat0 + (int)rank * 64 + r;
        row_ok = flat < T.rows;
        const int j = row_ok ? flat / a.H : 0;
        row_h = flat - j * a.H;
        row_q = T.row0 + j;
        lim = row_ok ? min(T.len, max(0, T.len - T.count + j + 1)) : 0;
        ok = __all_sync(0xffffffffu, wait(&S.q_local[piece & 3], (piece >> 2) & 1));
        if (!ok) break;
        rc = fabsf(a.sigma) * kLog2e *
             __uint_as_float((uint32_t)(127 - S.qexp[piece & 3][r]) << 23);   // 2^-e
        m = -CUDART_INF_F;
        l = 0.0f;
      }
      ok = __all_sync(0xffffffffu, wait(&S.s_full[g & 1], (g >> 1) & 1));
      if (!ok) break;
      tc_fence_after();
      // w_t = z_t + log2 s_t of 32 columns from c0 on (the S columns are read again for the second
      // pass: the loops over a thread's columns stay rolled, since the steady loops of all roles
      // share an instruction cache that they overfill)
      const uint32_t sb = tmem + kSCol + 64u * (g & 1) + (uint32_t)(kCols * cg) + lanes;
      const int vis = lim - T.t0 - col0;             // columns that the row sees
      const bool partly = __any_sync(0xffffffffu, vis < kCols);
      auto weights = [&](int c0, float (&w)[32]) {
        tmem_ld32(sb + c0, w);
        tmem_wait_ld();
        const float4* lsc4 = reinterpret_cast<const float4*>(T.lsc + col0 + c0);
        const float4* sc4 = reinterpret_cast<const float4*>(T.sc + col0 + c0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 b = lsc4[i];
          float4 c = make_float4(1.f, 1.f, 1.f, 1.f);
          if constexpr (kTok) c = sc4[i];
          const float bb[4] = {b.x, b.y, b.z, b.w}, cc[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float z = w[4 * i + k];
            if constexpr (kTok) z *= cc[k];
            w[4 * i + k] = fmaf(z, rc, bb[k]);
          }
        }
        if (partly) {
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = c0 + i < vis ? w[i] : -CUDART_INF_F;
        }
      };
      float s[32];
      float mx = -CUDART_INF_F;
#pragma unroll 1
      for (int c0 = 0; c0 < kCols; c0 += 32) {
        weights(c0, s);
#pragma unroll
        for (int i = 0; i < 32; ++i) mx = fmaxf(mx, s[i]);
      }
      S.xch[g & 1][tid] = mx;
      ok = meet();
      if (!ok) break;
      mx = fmaxf(mx, S.xch[g & 1][tid ^ 64]);
      if constexpr (kExp)
        mx = fmaxf(mx, fmaxf(S.xch[g & 1][tid ^ 128], S.xch[g & 1][tid ^ 192]));
      float alpha = 1.0f;
      if (mx > m + kLazy) {
        alpha = exp2f(m - mx);   // m = -inf: 0
        l *= alpha;
        m = mx;
      }
      const float mref = m == -CUDART_INF_F ? 0.0f : m - kHead;
      // The previous output MMA has to have read P and left O before this block's P is written.
      // Waited for ahead of the exponentials, but over bf16 rows (one score MMA a block, softmax
      // the longer side) behind the first of them; us ahead / behind, expanded rows, d = 512: 8
      // bits (1.35 TFLOP) 1140 / 1152, groups of 32 (0.15) 318 / 330, bf16 (2.9) 2570 / 2355.
      auto pv_before = [&]() {
        if (g == 0) return true;
        if (!__all_sync(0xffffffffu, wait(&S.pv_done, (g - 1) & 1))) return false;
        tc_fence_after();
        return true;
      };
      if (!kBf16) ok = pv_before();
      if (!ok) break;
#pragma unroll 1
      for (int c0 = 0; c0 < kCols; c0 += 32) {
        if (kCols > 32) weights(c0, s);
        if (c0 + 32 == kCols) {                       // S has been read for the last time
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(&S.s_free[g & 1], 0);
        }
        const float4* isc4 = reinterpret_cast<const float4*>(T.isc + col0 + c0);
        uint32_t pk[16];
        float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float4 c = make_float4(1.f, 1.f, 1.f, 1.f);
          if constexpr (kTok) c = isc4[i];
          const float cc[4] = {c.x, c.y, c.z, c.w};
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e[k] = ex2_approx(s[4 * i + k] - mref);
            if (k & 1) l1 = fmaf(e[k], cc[k], l1); else l0 = fmaf(e[k], cc[k], l0);
          }
          pk[2 * i] = pack_out(kBf16, e[0], e[1]);
          pk[2 * i + 1] = pack_out(kBf16, e[2], e[3]);
        }
        l += l0 + l1;
        if (kBf16 && c0 == 0) ok = pv_before();
        if (!ok) break;
        const uint32_t row = p_s + (uint32_t)hh * kAtom + (uint32_t)r * 128u;
        const int c1 = (kCols * cg + c0) >> 3;        // first 16-byte chunk of the row
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sts128(row + (uint32_t)(((c + c1) ^ (r & 7)) << 4),
                 make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]));
      }
      if (!ok) break;
      // the scales and this block's header have been read
      const int last = fl & kLast, dest = T.dest, t_seq = T.seq, t_b1 = T.b1, t_nblk = T.nblk;
      const int t_flat0 = T.flat0, t_row0 = T.row0, t_rows = T.rows;
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.tok_empty[st]);
      if (!(fl & kFirst) && __any_sync(0xffffffffu, alpha != 1.0f)) {
        rescale_o(obase, ocg, alpha);
      }
      if constexpr (kExp) fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kExp) arrive_at(&S.p_ready, 0);
        else mbar_arrive(&S.p_full);
      }
      if (!last) continue;

      // ---- the piece's output ----
      // (the buffer of the last block's neighbours: free again once all have met twice)
      float* xl = S.xch[(g + 1) & 1];
      xl[tid] = l;
      ok = meet();
      if (!ok) break;
      float lt = xl[r] + xl[r + 64];
      if constexpr (kExp) lt += xl[r + 128] + xl[r + 192];
      ok = meet();
      if (!ok) break;
      ok = __all_sync(0xffffffffu, wait(&S.pv_done, g & 1));
      if (!ok) break;
      tc_fence_after();
      const int f0 = hh * oc + cg * ocg;             // first feature of this thread
      const int part = (cluster * 2 + dest) * 128 + (int)rank * 64 + r;
      // a sum of zero: no token seen (or none that exists)
      const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
      void* to = dest >= 0 ? static_cast<void*>(P.w.o + (int64_t)part * a.d)
                           : static_cast<void*>(static_cast<uint16_t*>(a.out) +
                                                (int64_t)row_q * a.o_st + (int64_t)row_h * a.o_sh);
      write_o(obase, ocg, f0, row_ok ? a.d : 0, to, dest >= 0 ? -1 : P.q_bf16, inv);
      if (hh == 0 && cg == 0 && row_ok) {
        if (dest >= 0) {
          P.w.ml[2 * (int64_t)part] = m - kHead;
          P.w.ml[2 * (int64_t)part + 1] = lt;
        } else if (a.lse) {
          a.lse[(int64_t)row_q * a.H + row_h] =
              lt == 0.0f ? -CUDART_INF_F : kLn2 * (m - kHead + log2f(lt));
        }
      }
      if (dest >= 0 && rank == 0 && tid == 0) {
        ChunkPartial& h = P.w.head[cluster * 2 + dest];
        h.seq = t_seq;
        h.flat0 = t_flat0;
        h.row0 = t_row0;
        h.rows = t_rows;
        h.b1 = t_b1;
        h.nblk = t_nblk;
        h.valid = 1;
      }
      tc_fence_before();
    }
  }
  // Every role of both CTAs is through.  A wait that ran out anywhere has stopped both: then loads
  // may be in flight, into either CTA's memory, and both stay until the leader has seen them land.
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (abort_read(smem_u32(&S.abort_word))) {           // (the same in both CTAs)
    if (tid == 0) atomicOr(a.flags, KVK_FLAG_TIMEOUT);
    if constexpr (kExp) {
      if (rank == 0 && tid == 0) finish_loads<kLo>(P, S, nch);
      __syncthreads();
      cluster_sync();
    }
  }
  // the leader's last commits arrive here too: nothing is on its way to this memory any more
  if (rank == 1 && tid == 0) {
    const uint64_t end = globaltimer() + kDrainLimitNs;
    drain(&S.drain[0], 0u, end);
    drain(&S.drain[1], 0u, end);
  }
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
}

// ---------------------------------------------------------------------------------------
// join of the row tiles that several clusters worked on
// ---------------------------------------------------------------------------------------
constexpr int kMergeWarps = 8;
constexpr int kMergeRounds = 4;   // pieces of a tile in rounds of 32 lanes: up to 127 clusters

// CTA (g, y, z): if the last piece of cluster g began a tile it did not finish, rows 8 y .. 8 y + 7
// (one a warp) of that tile and kF x 128 of its features, whose further pieces are the first ones
// of clusters g + 1, ... up to the one that ends it.  A lane holds reference and sum of one piece a
// round; the outputs are then added up piece by piece, their loads independent of one another.
// kF = 4 takes all features in one warp; kF = 1 spreads them over d / 128 CTAs, for tiles of many
// pieces, at the price of the CTAs that find no work (decode calls, kF = 4 / 1, us: one sequence of
// 8192 tokens 66.0 / 56.8, of 32768 93.5 / 82.5, of 64 25.0 / 26.5; 4 of 8192 50.5 / 50.4; 8 of 4096
// 46.8 / 47.3).
template <int kF>
__global__ void __launch_bounds__(kMergeWarps * 32)
chunk_merge_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ ChunkWork w,
                   int q_bf16) {
  griddep_wait();                        // the partials are complete and visible
  const int g = blockIdx.x, lane = threadIdx.x & 31;
  const ChunkPartial h = w.head[2 * g + 1];
  if (!h.valid) return;
  const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const int flat = h.flat0 + row;
  if (flat >= h.rows) return;
  // piece i of the tile: cluster g + i, its first slot (cluster g: its second)
  auto slot = [&](int i) { return (int64_t)(2 * (g + i) + (i == 0 ? 1 : 0)) * 128 + row; };
  float m[kMergeRounds], l[kMergeRounds];
  int n = 0;                             // pieces, those of clusters without one among them
  bool open = true;
#pragma unroll
  for (int r = 0; r < kMergeRounds; ++r) {
    m[r] = -CUDART_INF_F;
    l[r] = 0.0f;
    if (!open) continue;
    const int i = 32 * r + lane, c = g + i;
    bool in = i == 0, stop = c >= w.G, ends = false;
    if (i > 0 && !stop) {
      const ChunkPartial& x = w.head[2 * c];
      in = x.valid != 0;
      stop = in && (x.seq != h.seq || x.flat0 != h.flat0);
      ends = in && !stop && x.b1 == x.nblk;
    }
    const unsigned before = __ballot_sync(0xffffffffu, stop), fin = __ballot_sync(0xffffffffu, ends);
    int take = 32;                       // lanes of this round that belong to the tile
    if (fin) take = __ffs(fin);
    if (before) take = min(take, __ffs(before) - 1);
    open = take == 32 && !(fin >> 31);
    n = 32 * r + take;
    if (in && lane < take) {
      const float2 v = *reinterpret_cast<const float2*>(w.ml + 2 * slot(i));
      m[r] = v.x;
      l[r] = v.y;
    }
  }
  float M = -CUDART_INF_F;
#pragma unroll
  for (int r = 0; r < kMergeRounds; ++r) M = fmaxf(M, m[r]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.0f;
#pragma unroll
  for (int r = 0; r < kMergeRounds; ++r) {
    m[r] = m[r] == -CUDART_INF_F ? 0.0f : exp2f(m[r] - M);   // (NaN stays NaN)
    L += m[r] * l[r];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  const int f0 = 128 * kF * blockIdx.z + 4 * lane;
  float4 acc[kF];
#pragma unroll
  for (int k = 0; k < kF; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int r = 0; r < kMergeRounds; ++r) {
    const int top = min(32, n - 32 * r);
#pragma unroll (kF == 1 ? 8 : 4)
    for (int i = 0; i < top; ++i) {
      const float x = __shfl_sync(0xffffffffu, m[r], i);
      if (kF > 1 && x == 0.0f) continue;
      const float* o = w.o + slot(32 * r + i) * a.d;
#pragma unroll
      for (int k = 0; k < kF; ++k) {
        const int f = 128 * k + f0;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);   // x = 0: no piece, or no weight
        if (x != 0.0f && f < a.d) v = *reinterpret_cast<const float4*>(o + f);
        acc[k].x = fmaf(x, v.x, acc[k].x);
        acc[k].y = fmaf(x, v.y, acc[k].y);
        acc[k].z = fmaf(x, v.z, acc[k].z);
        acc[k].w = fmaf(x, v.w, acc[k].w);
      }
    }
  }
  const int j = flat / a.H, hd = flat - j * a.H;
  uint16_t* out = static_cast<uint16_t*>(a.out) + (int64_t)(h.row0 + j) * a.o_st +
                  (int64_t)hd * a.o_sh;
#pragma unroll
  for (int k = 0; k < kF; ++k) {
    const int f = 128 * k + f0;
    if (f < a.d)
      *reinterpret_cast<uint2*>(out + f) =
          make_uint2(pack_out(q_bf16, acc[k].x * inv, acc[k].y * inv),
                     pack_out(q_bf16, acc[k].z * inv, acc[k].w * inv));
  }
  if (a.lse && lane == 0 && blockIdx.z == 0)
    a.lse[(int64_t)(h.row0 + j) * a.H + hd] = L == 0.0f ? -CUDART_INF_F : kLn2 * (M + log2f(L));
}

__host__ constexpr uint32_t idesc_of(bool bf16, int N, bool b_mn) {
  return idesc_f16(128, N, false, b_mn) | (bf16 ? (1u << 7) | (1u << 10) : 0u);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The expanded rows as a 2D tensor [slots][64 NA] of 16-bit elements; box = one atom's 64
// features x `rows` slots, 128-byte swizzle.  Rows behind the pool read as zero.
bool expanded_map(CUtensorMap* m, void* base, int NA, int64_t slots, int rows) {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)NA * 64, (cuuint64_t)slots};
  const cuuint64_t strides[1] = {(cuuint64_t)NA * 128};
  const cuuint32_t box[2] = {64, (cuuint32_t)rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, base, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Registers a thread of an instance (0 where the device does not tell; asked again then).
template <int BITS, bool GROUP, bool kExp>
int instance_regs() {
  static std::atomic<int> regs{0};
  int r = regs.load(std::memory_order_relaxed);
  if (r) return r;
  cudaFuncAttributes at;
  if (cudaFuncGetAttributes(&at, chunk_tc_kernel<BITS, GROUP, kExp>) == cudaSuccess) r = at.numRegs;
  else cudaGetLastError();
  regs.store(r, std::memory_order_relaxed);
  return r;
}
// Of the converting instance for rows of BITS and the expanded one that they share with others.
template <int BITS, int EXP_BITS, bool GROUP>
int both_regs() {
  const int r = instance_regs<BITS, GROUP, false>();
  return r == instance_regs<EXP_BITS, GROUP, true>() ? r : 0;
}

template <int BITS, bool GROUP, bool kExp>
cudaError_t launch(const TcChunk& P, const CUtensorMap& hi, const CUtensorMap& lo, size_t smem,
                   cudaStream_t st) {
  auto k = chunk_tc_kernel<BITS, GROUP, kExp>;
  // the kernel hands registers from warpgroup to warpgroup: their number at launch is part of it
  // (the caller has chosen its path by it)
  if (instance_regs<BITS, GROUP, kExp>() != (int)kLaunchRegs) return cudaErrorNotSupported;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  });
  if (e != cudaSuccess) return e;
  k<<<dim3(2 * P.w.G), dim3(kThreads), smem, st>>>(P, hi, lo);
  return cudaGetLastError();
}

}  // namespace

bool chunk_tc_supported(const kvk_layout* L, const AnchorDesc& A, int dtype) {
  if (dtype != KVK_BF16 && dtype != KVK_F16) return false;
  // bf16 rows stay bf16 in the MMA, whose two operands have one type
  if (A.b == KVK_BITS_BF16 && dtype != KVK_BF16) return false;
  return A.d <= 512 && L->d_rope <= 64 && L->d_rope % 16 == 0;
}

int chunk_tc_regs(int b, int group) {
  if (group) {
    if (b == 2) return both_regs<2, 8, true>();
    if (b == 4) return both_regs<4, 8, true>();
    if (b == 8) return both_regs<8, 8, true>();
    return both_regs<16, 8, true>();
  }
  if (b == KVK_BITS_BF16) return both_regs<KVK_BITS_BF16, KVK_BITS_BF16, false>();
  if (b == 2) return both_regs<2, 8, false>();
  if (b == 4) return both_regs<4, 8, false>();
  if (b == 8) return both_regs<8, 8, false>();
  return both_regs<16, 16, false>();
}

cudaError_t launch_chunk_tc(const ChunkArgs& a, const ChunkWork& w, int dtype, cudaStream_t st) {
  TcChunk P;
  memset(&P, 0, sizeof(P));
  P.a = a;
  P.w = w;
  P.NL = latent_atoms(a.d);
  P.NA = row_atoms(a.d, a.d_rope);
  P.NV = P.NL / 2;
  P.NVS = P.NV <= 2 ? 2 : 1;
  const int room = (kSmemLimit - (int)(sizeof(Shared) + kMinTok * sizeof(TokStage))) / (int)kAtom - P.NA - 2 * P.NV * P.NVS - 2;
  P.NK = std::min(kMaxK, room / 2);   // slots of two atoms
  P.off_k = (uint32_t)P.NA * kAtom;
  P.off_v = P.off_k + (uint32_t)(2 * P.NK) * kAtom;
  P.off_p = P.off_v + (uint32_t)(2 * P.NV * P.NVS) * kAtom;
  P.off_misc = P.off_p + 2 * kAtom;
  P.off_tok = (uint32_t)align_up_sz(P.off_misc + sizeof(Shared), 16);
  P.NT = std::min(kMaxTok, (kSmemLimit - (int)P.off_tok) / (int)sizeof(TokStage));
  const bool bf = a.b == KVK_BITS_BF16;
  P.idesc_s = idesc_of(bf, 128, false);
  P.idesc_o2 = idesc_of(bf, 256, true);
  P.idesc_o1 = idesc_of(bf, 128, true);
  P.q_bf16 = dtype == KVK_BF16;
  const size_t smem = P.off_tok + (size_t)P.NT * sizeof(TokStage);
  // the prologue's prefix sums use the rings' memory
  if (w.G >= 32 * kMergeRounds || P.NT < kMinTok || P.NK < 2 || smem > (size_t)kSmemLimit || (size_t)(a.batch + 1) * 4 > P.off_misc)
    return cudaErrorInvalidValue;
  CUtensorMap hi, lo;
  memset(&hi, 0, sizeof(hi));
  memset(&lo, 0, sizeof(lo));
  cudaError_t e = cudaErrorInvalidValue;
  if (w.hi) {
    const bool split = chunk_split(a.b, a.group);
    P.mark = w.mark;
    P.box = std::min(1 << a.page_shift, 64);
    P.pool_slots = w.pool_slots;
    if (!expanded_map(&hi, w.hi, P.NA, w.pool_slots, P.box) ||
        (split && !expanded_map(&lo, w.lo, P.NA, w.pool_slots, P.box)))
      return cudaErrorInvalidValue;
    e = launch_chunk_expand(a, w, st);
    if (e != cudaSuccess) return e;
    // (the operands' form does not depend on the width of the codes any more)
    if (bf) e = launch<KVK_BITS_BF16, false, true>(P, hi, lo, smem, st);
    else if (a.group) e = launch<8, true, true>(P, hi, lo, smem, st);
    else if (split) e = launch<16, false, true>(P, hi, lo, smem, st);
    else e = launch<8, false, true>(P, hi, lo, smem, st);
  } else if (a.group) {
    if (a.b == 2) e = launch<2, true, false>(P, hi, lo, smem, st);
    else if (a.b == 4) e = launch<4, true, false>(P, hi, lo, smem, st);
    else if (a.b == 8) e = launch<8, true, false>(P, hi, lo, smem, st);
    else if (a.b == 16) e = launch<16, true, false>(P, hi, lo, smem, st);
  } else {
    if (bf) e = launch<KVK_BITS_BF16, false, false>(P, hi, lo, smem, st);
    else if (a.b == 2) e = launch<2, false, false>(P, hi, lo, smem, st);
    else if (a.b == 4) e = launch<4, false, false>(P, hi, lo, smem, st);
    else if (a.b == 8) e = launch<8, false, false>(P, hi, lo, smem, st);
    else if (a.b == 16) e = launch<16, false, false>(P, hi, lo, smem, st);
  }
  if (e != cudaSuccess) return e;
  // a programmatic dependent: its CTAs are in place when the partials are
  // features spread where a tile may have sixteen pieces or more, were each sequence one tile
  if (a.batch <= w.G / 16 && a.cap >= 16 * 128)
    e = launch_pdl(chunk_merge_kernel<1>, dim3(w.G, 128 / kMergeWarps, (a.d + 127) / 128),
                   dim3(kMergeWarps * 32), 0, st, a, w, P.q_bf16);
  else
    e = launch_pdl(chunk_merge_kernel<4>, dim3(w.G, 128 / kMergeWarps), dim3(kMergeWarps * 32), 0, st, a,
                   w, P.q_bf16);
  return e != cudaSuccess ? e : cudaGetLastError();
}

size_t chunk_workspace(const AnchorDesc& A, int d_rope, int group, int64_t slots, int G, bool expand,
                       void* base, ChunkWork* w) {
  size_t off = 0;
  const size_t o_head = off;
  off = align_up_sz(off + sizeof(ChunkPartial) * 2 * (size_t)G, 256);
  const size_t o_ml = off;
  off = align_up_sz(off + sizeof(float) * 2 * 128 * 2 * (size_t)G, 256);
  const size_t o_o = off;
  off = align_up_sz(off + sizeof(float) * (size_t)A.d * 128 * 2 * (size_t)G, 256);
  const size_t plane = (size_t)slots * row_atoms(A.d, d_rope) * 128;
  const bool split = chunk_split(A.b, group);
  size_t o_mark = off, o_hi = off, o_lo = off;
  if (expand) {
    off = align_up_sz(off + sizeof(float) * (size_t)slots, 256);
    o_hi = off;
    off = align_up_sz(off + plane, 256);
    o_lo = off;
    if (split) off = align_up_sz(off + plane, 256);
  }
  if (base && w) {
    uint8_t* p = static_cast<uint8_t*>(base);
    w->head = reinterpret_cast<ChunkPartial*>(p + o_head);
    w->ml = reinterpret_cast<float*>(p + o_ml);
    w->o = reinterpret_cast<float*>(p + o_o);
    w->G = G;
    w->mark = expand ? reinterpret_cast<float*>(p + o_mark) : nullptr;
    w->hi = expand ? p + o_hi : nullptr;
    w->lo = expand && split ? p + o_lo : nullptr;
    w->pool_slots = (int)slots;
  }
  return off;
}

}  // namespace kvk
