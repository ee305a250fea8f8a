// lsc_kv_batch.cuh -- device helpers shared by the K/V step kernels: reading the
// batch description (include/lsc_kv.h, lsc_kv_batch) and the E4M3 row format.
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

}  // namespace kv
}  // namespace lsc
