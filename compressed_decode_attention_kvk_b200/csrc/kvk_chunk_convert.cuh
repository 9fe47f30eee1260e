// kvk_chunk_convert.cuh -- cached rows as 16-bit tensor-core operands: 16 elements at a time, read
// from the packed pool and turned into f16 (codes exact; 16-bit and group-scaled values as a high
// and a low part) or bf16 (uncompressed rows).
#pragma once

#include "kvk_paged.cuh"

namespace kvk {
namespace chunk {

// ---- conversion of 16 consecutive elements --------------------------------------------------
template <int BITS>
constexpr int kRaw = BITS == 2 ? 1 : BITS == 4 ? 2 : BITS == 8 ? 4 : 8;   // 32-bit words
template <int BITS, bool GROUP>
constexpr bool kSplit = BITS == 16 || GROUP;   // two f16 parts in the score MMA
template <int BITS>
constexpr int kElemBits = BITS == KVK_BITS_BF16 ? 16 : BITS;

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) {
  return __byte_perm(a, b, s);
}
__device__ __forceinline__ uint32_t h2add(uint32_t a, uint32_t b) {
  const __half2 r = __hadd2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t h2fma(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b),
                            *reinterpret_cast<__half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t h2neg(uint32_t a) { return a ^ 0x80008000u; }
constexpr uint32_t kH1024 = 0x64006400u;   // f16 1024: 0x6400 | u is the integer 1024 + u

// four bytes, one field each, to f16 integers field - bias (bias as the f16 pair -(1024 + bias))
__device__ __forceinline__ void bytes_to_f16(uint32_t w, uint32_t bias, uint32_t* out) {
  out[0] = h2add(prmt(w, kH1024, 0x7170), bias);
  out[1] = h2add(prmt(w, kH1024, 0x7372), bias);
}

// The 16 elements of `raw` as two-element words: hi (the operand, or its high part) and, when
// LO, the low part lo = x - hi.  s: the unit's group scale (f16 bits).
template <int BITS, bool GROUP, bool LO>
__device__ __forceinline__ void convert16(const uint32_t (&raw)[kRaw<BITS>], uint32_t s,
                                          uint32_t (&hi)[8], uint32_t (&lo)[8]) {
  if constexpr (BITS == KVK_BITS_BF16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) hi[i] = raw[i];
  } else if constexpr (BITS == 16) {
    // field u = 256 a + b, code c = 256 (a - 128) + b: A and b are exact f16 integers, one fused
    // multiply-add rounds c to f16, and c - hi is exact (|256 A| >= b, or A = 0 and hi = b)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t A = h2add(prmt(raw[i], kH1024, 0x7371), 0xE480E480u);   // - 1152
      const uint32_t B = h2add(prmt(raw[i], kH1024, 0x7270), 0xE400E400u);   // - 1024
      const uint32_t h = h2fma(A, 0x5C005C00u, B);                           // 256 A + b
      if constexpr (!GROUP) {
        hi[i] = h;
        if constexpr (LO) lo[i] = h2add(B, h2neg(h2fma(A, 0xDC00DC00u, h)));   // b - (h - 256 A)
      } else {
        // the product in fp32 (24 of its 27 bits), split into two f16 parts
        const float sf = __half2float(__ushort_as_half((unsigned short)s));
        const uint32_t r = raw[i] ^ 0x80008000u;
        const float x0 = (float)(int)(short)(r & 0xFFFFu) * sf;
        const float x1 = (float)(int)(short)(r >> 16) * sf;
        const __half2 hh = __floats2half2_rn(x0, x1);
        hi[i] = *reinterpret_cast<const uint32_t*>(&hh);
        if constexpr (LO) {
          const __half2 ll = __floats2half2_rn(x0 - __low2float(hh), x1 - __high2float(hh));
          lo[i] = *reinterpret_cast<const uint32_t*>(&ll);
        }
      }
    }
  } else {
    uint32_t c[8];
    if constexpr (BITS == 8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) bytes_to_f16(raw[i], 0xE480E480u, c + 2 * i);   // -(1024 + 128)
    } else if constexpr (BITS == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t x = raw[i] & 0x0F0F0F0Fu, y = (raw[i] >> 4) & 0x0F0F0F0Fu;
        bytes_to_f16(prmt(x, y, 0x5140), 0xE408E408u, c + 4 * i);       // -(1024 + 8)
        bytes_to_f16(prmt(x, y, 0x7362), 0xE408E408u, c + 4 * i + 2);
      }
    } else {
      const uint32_t x0 = raw[0] & 0x03030303u, x1 = (raw[0] >> 2) & 0x03030303u,
                     x2 = (raw[0] >> 4) & 0x03030303u, x3 = (raw[0] >> 6) & 0x03030303u;
      const uint32_t p = prmt(x0, x1, 0x5140), q = prmt(x2, x3, 0x5140);
      const uint32_t r = prmt(x0, x1, 0x7362), t = prmt(x2, x3, 0x7362);
      bytes_to_f16(prmt(p, q, 0x5410), 0xE402E402u, c);                 // -(1024 + 2)
      bytes_to_f16(prmt(p, q, 0x7632), 0xE402E402u, c + 2);
      bytes_to_f16(prmt(r, t, 0x5410), 0xE402E402u, c + 4);
      bytes_to_f16(prmt(r, t, 0x7632), 0xE402E402u, c + 6);
    }
    if constexpr (!GROUP) {
#pragma unroll
      for (int i = 0; i < 8; ++i) hi[i] = c[i];
    } else {
      const uint32_t s2 = s | (s << 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        hi[i] = h2mul(c[i], s2);
        if constexpr (LO) lo[i] = h2fma(c[i], s2, h2neg(hi[i]));   // exact but for f16 subnormals
      }
    }
  }
}

// Non-finite elements of a row.  A token whose row holds one must not reach the queries that do
// not see it, although its zero weight multiplies it there: it goes into the score operand as
// NaN (every query that sees it becomes NaN) and into the output operand as zero.
template <bool BF16>
__device__ __forceinline__ bool nonfinite16(const uint32_t (&w)[8]) {
  const uint32_t e = BF16 ? 0x7F807F80u : 0x7C007C00u;
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t x = w[i] & e;   // a half equal to its exponent mask is inf or NaN
    any |= ((x & 0xFFFFu) == (e & 0xFFFFu)) | ((x >> 16) == (e >> 16));
  }
  return any != 0;
}
template <bool BF16>
__device__ __forceinline__ void replace_nonfinite(uint32_t (&w)[8], uint32_t with) {
  const uint32_t e = BF16 ? 0x7F80u : 0x7C00u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if ((w[i] & e) == e) w[i] = (w[i] & 0xFFFF0000u) | with;
    if (((w[i] >> 16) & e) == e) w[i] = (w[i] & 0xFFFFu) | (with << 16);
  }
}

template <int BITS, bool GROUP>
struct Unit {
  uint32_t w[kRaw<BITS>];
  uint32_t s;
};

// A token's packed row and, with group scales, its scales; a slot that does not exist (negative)
// points at the pool's first row, whose values nothing may depend on.
template <bool GROUP>
struct Row {
  const uint8_t* codes;
  const unsigned short* scales;
  bool real;
};
template <bool GROUP>
__device__ __forceinline__ Row<GROUP> row_of(const ChunkArgs& a, int slot) {
  Row<GROUP> r;
  r.real = slot >= 0;
  const int64_t at = max(slot, 0);
  r.codes = a.codes + at * a.row_bytes;
  r.scales = GROUP ? reinterpret_cast<const unsigned short*>(a.scales) + at * a.sg : nullptr;
  return r;
}

// 16 elements of a row from element e (a multiple of 16) on
template <int BITS, bool GROUP>
__device__ __forceinline__ void load_unit(const ChunkArgs& a, const Row<GROUP>& r, int e,
                                          Unit<BITS, GROUP>& u) {
  constexpr int RW = kRaw<BITS>;
  const uint8_t* p = r.codes + e * kElemBits<BITS> / 8;
  if constexpr (RW == 1) {
    u.w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (RW == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    u.w[0] = v.x;
    u.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < RW / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
      u.w[4 * i] = v.x;
      u.w[4 * i + 1] = v.y;
      u.w[4 * i + 2] = v.z;
      u.w[4 * i + 3] = v.w;
    }
  }
  if constexpr (GROUP) u.s = __ldg(r.scales + e / a.group);
}

// The unit as operand words (hi, and lo where LO), zero unless `real`; a non-finite element becomes
// `odd` (0x7FFF: NaN in either type) in the high part and zero in the low one.
template <int BITS, bool GROUP, bool LO>
__device__ __forceinline__ void operand16(const Unit<BITS, GROUP>& u, bool real, uint32_t odd,
                                          uint32_t (&hi)[8], uint32_t (&lo)[8]) {
  constexpr bool kBf16 = BITS == KVK_BITS_BF16;
  convert16<BITS, GROUP, LO>(u.w, u.s, hi, lo);
  if (!real) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi[i] = 0u;
      if constexpr (LO) lo[i] = 0u;
    }
  } else if constexpr (kBf16 || GROUP) {
    if (nonfinite16<kBf16>(hi)) {
      replace_nonfinite<kBf16>(hi, odd);
      if constexpr (LO) replace_nonfinite<kBf16>(lo, 0u);
    }
  }
}

}  // namespace chunk
}  // namespace kvk
