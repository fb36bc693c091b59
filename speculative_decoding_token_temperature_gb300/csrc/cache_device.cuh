// Device-side pieces shared by the cache operators: lengths, page lookups, 16-bit types, and
// the 4-bit and 8-bit values.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_ops.h"

namespace specdec {

template <typename T> struct Half16;
template <> struct Half16<__nv_bfloat16> {
  static __device__ __forceinline__ float2 to_f32(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {  // round to nearest even
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
  }
};
template <> struct Half16<__half> {
  static __device__ __forceinline__ float2 to_f32(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {  // round to nearest even
    uint32_t w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
  }
};

// The lengths of one sequence.  ok is false where they do not fit the table: a negative
// length, more new tokens than n or than the length, or slots past the table.
struct SeqLen {
  int len, nq, first;  // tokens in the cache, new ones among them, slot of the first new one
  bool ok;
};
__device__ __forceinline__ SeqLen seq_len(const int32_t* context_len, const int32_t* query_len, int b, int n,
                                          int64_t slots) {
  SeqLen s;
  s.len = __ldg(context_len + b);
  s.nq = query_len ? __ldg(query_len + b) : n;
  s.ok = s.len >= 0 && s.nq >= 0 && s.nq <= n && s.nq <= s.len && s.len <= slots;
  s.first = s.len - s.nq;
  return s;
}

// The page of a slot: slot / page_size as the high half of a product (exact for slots below 2^31).
__device__ __forceinline__ int page_of(const Pages& pg, int slot) {
  return pg.page_magic == 0 ? slot : static_cast<int>(__umul64hi(static_cast<uint64_t>(slot), pg.page_magic));
}

// Whether sequence b's lengths and the pages of its slots [first, len) are in range; every
// thread of the CTA calls it, and gets the same answer.
__device__ __forceinline__ bool sequence_fits(const SeqLen& S, const Pages& pg, int b) {
  int bad = S.ok ? 0 : 1;
  if (S.ok && S.nq > 0) {
    const int32_t* table = pg.table + static_cast<int64_t>(b) * pg.max_pages;
    const int p0 = page_of(pg, S.first), p1 = page_of(pg, S.len - 1);
    for (int p = p0 + threadIdx.x; p <= p1; p += blockDim.x)
      bad |= static_cast<unsigned>(__ldg(table + p)) >= static_cast<unsigned>(pg.num_pages);
  }
  return !__syncthreads_or(bad);
}

// Eight 4-bit values (E2M1, the low nibble first) of a word as four fp16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm("{\n.reg .b8 x0, x1, x2, x3;\n"
      "mov.b32 {x0, x1, x2, x3}, %4;\n"
      "cvt.rn.f16x2.e2m1x2 %0, x0;\n"
      "cvt.rn.f16x2.e2m1x2 %1, x1;\n"
      "cvt.rn.f16x2.e2m1x2 %2, x2;\n"
      "cvt.rn.f16x2.e2m1x2 %3, x3;\n}"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
      : "r"(w));
}
// Two E4M3 values as an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t r;
  const uint16_t t = static_cast<uint16_t>(two);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(t));
  return r;
}
// The four E4M3 values of a word as two fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& a, uint32_t& b) {
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.rn.f16x2.e4m3x2 %0, lo;\ncvt.rn.f16x2.e4m3x2 %1, hi;\n}"
      : "=r"(a), "=r"(b)
      : "r"(w));
}
// Two values as E4M3 codes, the first in the low byte: nearest, ties to the even code, saturated.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}


// ---- the blocks of 8-bit pages ------------------------------------------------------------

constexpr int kLeastExponent = -15, kMostExponent = 7;  // of a block's scale
// The exponent that a scale byte holds.  (Clamped: bytes of blocks that nobody wrote may hold anything, and what is
// made of them is finite then.)
__device__ __forceinline__ int scale_exponent(uint32_t byte) {
  return min(max(static_cast<int>(byte) - 127, kLeastExponent), kMostExponent);
}
__device__ __forceinline__ float power_f32(int e) { return __int_as_float((e + 127) << 23); }
// 2^e twice in fp16; 2^-15 is subnormal there.
__device__ __forceinline__ uint32_t power_f16x2(int e) { return 0x00010001u * (e < -14 ? 0x0200u : static_cast<uint32_t>(e + 15) << 10); }
// The block of a page's slot.
__device__ __forceinline__ int block_of(const Pages& pg, int in_page) {
  return static_cast<int>(__umul64hi(static_cast<uint64_t>(in_page), pg.block_magic));
}

}  // namespace specdec
