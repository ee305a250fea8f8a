// lsc_kv_batch.cuh -- device helpers shared by the K/V step kernels: reading the
// batch description (include/lsc_kv.h, lsc_kv_batch) and the E4M3 and E2M1 row formats.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lsc_internal.h"

namespace lsc {
namespace kv {

static __device__ __noinline__ void report(int32_t *status, int32_t code) {
  if (status) atomicCAS(status, 0, code);
}

// A sequence's lengths as the kernels use them: kv outside what its table holds
// counts as an empty cache (and is recorded).
__device__ __forceinline__ int32_t checked_kv(const KvLayer &L, const KvBatch &b, int32_t kv) {
  if ((uint32_t)kv > (uint32_t)b.held) {
    report(L.status, LSC_ERR_INVALID_ARG);
    return 0;
  }
  return kv;
}

// The sequence that row t of the dense arrays belongs to, -1 for none.
__device__ __forceinline__ int32_t seq_of_row(const KvBatch &b, int32_t t) {
  int32_t lo = -1, hi = b.n_seq + 1;  // the last entry <= t
  while (hi - lo > 1) {
    const int32_t m = lo + ((hi - lo) >> 1);
    if (b.cu[m] <= t) lo = m;
    else hi = m;
  }
  return lo >= 0 && lo < b.n_seq && b.cu[lo] <= t && t < b.cu[lo + 1] ? lo : -1;
}

// A sequence as attend sees it: its first dense row, its new tokens and its
// cached tokens.  Lengths outside the host's bounds are recorded: too many
// cached tokens count as none (its rows see nothing), and a sequence of too many
// new ones has no rows (they stay as they are).
struct Seq {
  int32_t row0, n, kv;
};
__device__ __forceinline__ Seq attend_seq(const KvLayer &L, const KvBatch &b, int32_t i, int32_t max_seq,
                                          int32_t max_kv) {
  Seq s;
  const int32_t c0 = b.cu[i], c1 = b.cu[i + 1], kv = b.kv[i];
  s.row0 = c0;
  s.n = c0 >= 0 && c1 >= c0 && c1 <= b.total_tokens ? c1 - c0 : 0;  // else: recorded by check_cu
  s.kv = kv;
  if ((uint32_t)kv > (uint32_t)max_kv || s.n > max_seq) {
    report(L.status, LSC_ERR_INVALID_ARG);
    if ((uint32_t)kv > (uint32_t)max_kv) s.kv = 0;
    if (s.n > max_seq) s.n = 0;
  }
  return s;
}

// Positions that new token j (< n) of the sequence sees: [0, result), result <= kv.
__device__ __forceinline__ int32_t visible(const Seq &s, int32_t j, int32_t causal) {
  if (!causal) return s.kv;
  const int32_t v = s.kv - s.n + j + 1;  // both lengths are below 2^31 and j < n
  return v < 0 ? 0 : v;
}

// Record a cu_seqlens that is not what the batch promises; one CTA looks at all
// of it (every kernel stays inside its arrays whatever it holds).
__device__ __forceinline__ void check_cu(const KvLayer &L, const KvBatch &b) {
  for (int64_t i = threadIdx.x; i <= b.n_seq; i += blockDim.x) {
    const int32_t c = b.cu[i];
    if ((i == 0 && c != 0) || (i == b.n_seq ? c > b.total_tokens : b.cu[i + 1] < c))
      report(L.status, LSC_ERR_INVALID_ARG);
  }
}

// ---- E4M3 rows ---------------------------------------------------------------
// 2^(byte - 127) of a scale byte: the byte is the exponent field of that fp32
// value, but for 0 (2^-127, below the normal range) and 255 (NaN).
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

// The exponent e of V's scale as attend's reference m counts it, at least -76:
// weights 2^(s + e - m) are 2^15 at most, so a position adds 2^(15 + 76) at most to
// the sum of 2^(s - m), and 2^31 of them stay finite.  Rows of a smaller scale come
// out with weights smaller by the difference; their error is 2^-93 (half an e5m2
// step, 2^-17, times 448 over a sum of 2^(9 + 76)).  At the other end the heaviest
// position adds 2^(7 - e) at least, and what is below 2^-126 is lost: positions
// lighter than 2^(e - 133) of it.  A row of NaN (255) counts as 1: the sum, and lse,
// do not depend on what v holds.
__device__ __forceinline__ float v_exponent(uint32_t byte) {
  return byte < 51 ? -76.f : byte == 255 ? 0.f : (float)((int)byte - 127);
}

// The scale byte of a row whose largest magnitude has these fp32 bits (as an
// unsigned number, so NaN counts as the largest): the smallest power of two
// that brings m * 2^k (1 <= m < 2) to 448 = 1.75 * 2^8 is 2^(k - 8), or
// 2^(k - 7) when m > 1.75.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255;
  const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < 0 ? 0 : (uint32_t)e;
}

// 2^(127 - byte): what an element is multiplied by before its rounding (exact
// unless the product is far below the smallest code).
__device__ __forceinline__ float inv_scale_of(uint32_t byte) {
  return __uint_as_float(byte >= 254 ? 0x00400000u : (254 - byte) << 23);
}

// Two floats -> two codes (lo in the low byte), to nearest even.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two codes -> two halves, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// ---- E2M1 rows: groups of 16 elements ------------------------------------------
constexpr uint32_t kE2M1Top = 226;  // scale byte of 10240: six times it is the largest magnitude that f16 holds

// The group's scale byte for its largest magnitude, as fp32 bits (NaN counts as the
// largest): the smallest scale s with 6 s >= top.  u = top / 1.5 is the scale it would
// need, four times; its fp32 mantissa rounded up to 3 bits is the scale's.  Where top is
// 6 s itself u comes out as 4 s: the factor is off by 2^-25, half an fp32 step at 4 s's
// four bits is more.
__device__ __forceinline__ uint32_t e2m1_scale_byte(uint32_t top_bits) {
  const float u = __uint_as_float(top_bits) * (2.f / 3.f);
  const int32_t x = (int32_t)((__float_as_uint(u) + 0xfffffu) >> 20) - ((127 + 2 - 15) << 3);
  const int32_t b = min(x < 8 ? (int32_t)ceilf(u * 32768.f) : x, (int32_t)kE2M1Top);  // below 2^-14: multiples of 2^-17
  return top_bits >= 0x7f800000u ? 255 : (uint32_t)b;
}

// Two magnitudes over their scale -> codes (lo in the low nibble), to nearest even, 6 at most.
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u32.u8 %0, t;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// What elements x over their scale s are rounded from: x / s rounded once to 32 bits, as x r + x rest with r just below
// 1 / s and rest = (1 - s r) r, what it is off by (positive, so a zero keeps its sign).  An element of a 16-bit type has
// 11 bits and a scale 4, so a quotient that is no tie between codes is 2^-11 or more of a tie away from it, and one that
// is (three bits) comes out as it is.
__device__ __forceinline__ uint64_t f32x2(float x, float y) {
  return (uint64_t)__float_as_uint(x) | (uint64_t)__float_as_uint(y) << 32;
}
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi, float r, float rest) {
  uint64_t t;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(f32x2(lo, hi)), "l"(f32x2(rest, rest)));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(t) : "l"(f32x2(lo, hi)), "l"(f32x2(r, r)));
  return to_e2m1x2(__uint_as_float((uint32_t)t), __uint_as_float((uint32_t)(t >> 32)));
}
// With 32 bits a quotient may be nearer to a tie than x r is exact: rounded to 20 bits it is that tie, and the sign of
// x - tie s, exact in one fma, moves it to the right side.
__device__ __forceinline__ float e2m1_quotient32(float x, float s, float r) {
  const float a = fabsf(x);
  uint32_t t = (__float_as_uint(a * r) + 4) & ~7u;
  const float d = __fmaf_rn(-__uint_as_float(t), s, a);
  t += (d > 0.f ? 1 : 0) - (d < 0.f ? 1 : 0);
  return __uint_as_float(t | (__float_as_uint(x) & 0x80000000u));
}

// A group's scale as its elements meet it.
struct E2m1Scale {
  float s, r, low, rest;
  bool none;  // codes of 0: a group of zeros, or one that holds a NaN or an infinity
};
__device__ __forceinline__ E2m1Scale e2m1_scale(uint32_t byte) {
  E2m1Scale g;
  g.s = __half2float(__ushort_as_half((uint16_t)(byte << 7)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(g.r) : "f"(g.s));  // off by 2^-23 at most
  g.low = __uint_as_float(__float_as_uint(g.r) - 2);
  g.rest = __fmaf_rn(-g.s, g.low, 1.f) * g.low;
  g.none = byte == 0 || byte == 255;
  return g;
}

// Eight elements -> their codes.  FULL: they may have more than 11 bits.
template <bool FULL>
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&x)[8], const E2m1Scale &g) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = FULL ? to_e2m1x2(e2m1_quotient32(x[2 * i], g.s, g.r), e2m1_quotient32(x[2 * i + 1], g.s, g.r))
                : to_e2m1x2(x[2 * i], x[2 * i + 1], g.low, g.rest);
  const uint32_t w = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  return g.none ? 0 : w;
}

// Eight codes -> four pairs of halves, exactly.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// A scale byte as both halves of a pair.
__device__ __forceinline__ __half2 e2m1_scale2(uint32_t byte) {
  const uint32_t x = (byte | byte << 16) << 7;
  return *reinterpret_cast<const __half2 *>(&x);
}

// Eight codes times their scale as four pairs of halves: 6 bits at most, exact.
__device__ __forceinline__ void e2m1x8_times(uint32_t w, __half2 scale, uint32_t (&h)[4]) {
  e2m1x8_to_f16(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&h[i]), scale);
    h[i] = *reinterpret_cast<const uint32_t *>(&y);
  }
}

// Element i of a block (its rows' elements in order), in 32 bits.
__device__ __forceinline__ float e2m1_element(const uint8_t *page, int32_t scale_off, int64_t i) {
  uint32_t h[4];
  e2m1x8_times((uint32_t)page[i >> 1] >> (4 * (i & 1)), e2m1_scale2(page[scale_off + (i >> 4)]), h);
  return __low2float(*reinterpret_cast<const __half2 *>(&h[0]));
}

}  // namespace kv
}  // namespace lsc
