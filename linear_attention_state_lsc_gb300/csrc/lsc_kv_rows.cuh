// lsc_kv_rows.cuh -- what the kernels that write and read rows of the K/V block pool
// share: where a run of tokens sits in the blocks, and eight elements of a dense row.
#pragma once

#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_batch.cuh"

namespace lsc {
namespace kv {
namespace row {

constexpr int kThreads = 256;
constexpr int kMaxTok = 16;  // tokens of a CTA's run

struct E4M3 {};
struct E2M1 {};

// Where the tokens [t0, t0 + n) sit: page[i] = byte offset of the token's block
// in a lane, row[i] its row there; row -1: no row in the cache, -2: the token
// belongs to no sequence.
struct Places {
  int64_t page[kMaxTok];
  int32_t row[kMaxTok];
  int32_t cu[kThreads];
};

__device__ __forceinline__ void find_places(const KvLayer &L, const KvBatch &b, int32_t t0, int n, Places &s) {
  // samples of cu_seqlens, a step of `step` apart: one load per thread
  const int step = b.n_seq / kThreads + 1;
  {
    const int64_t i = (int64_t)threadIdx.x * step;
    s.cu[threadIdx.x] = b.cu[i < b.n_seq ? i : b.n_seq];
  }
  __syncthreads();
  if ((int)threadIdx.x < n) {
    const int32_t t = t0 + threadIdx.x;
    int lo = -1, hi = kThreads;  // the last sample <= t
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (s.cu[m] <= t) lo = m;
      else hi = m;
    }
    int32_t row = -2;
    int64_t page = 0;
    if (lo >= 0) {
      int64_t a = (int64_t)lo * step, z = a + step;  // the last entry <= t is in [a, z)
      if (a > b.n_seq) a = b.n_seq;
      if (z > (int64_t)b.n_seq + 1) z = (int64_t)b.n_seq + 1;
      while (z - a > 1) {
        const int64_t m = (a + z) >> 1;
        if (b.cu[m] <= t) a = m;
        else z = m;
      }
      if (a < b.n_seq) {
        const int32_t c0 = b.cu[a], c1 = b.cu[a + 1];
        row = -1;
        if (c0 <= t && t < c1) {
          const int32_t kv = checked_kv(L, b, b.kv[a]);
          const int64_t pos = (int64_t)kv - ((int64_t)c1 - c0) + (t - c0);
          if (pos >= 0) {
            const int32_t q = L.by_block.div((int32_t)pos);
            const int32_t blk = b.table[a * b.max_blocks + q];
            if (blk >= 0 && blk < L.num_blocks) {
              row = (int32_t)pos - q * L.block_tokens;
              page = (int64_t)blk * L.page;
            } else {
              report(L.status, LSC_ERR_OUT_OF_RANGE);
            }
          }
        }
      }
    }
    s.row[threadIdx.x] = row;
    s.page[threadIdx.x] = page;
  }
  __syncthreads();
}

// ---- eight elements of a row ---------------------------------------------------
template <typename T>
struct Eight;  // raw vector of 8 elements, and its floats
template <>
struct Eight<float> {
  uint4 a, b;
  __device__ void load(const void *p) { a = __ldcs((const uint4 *)p), b = __ldcs((const uint4 *)p + 1); }
  __device__ void store(void *p) const { ((uint4 *)p)[0] = a, ((uint4 *)p)[1] = b; }
  __device__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ void get(float (&x)[8]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
  // the largest magnitude as a whole number that orders like it (NaN above infinity), and that as fp32 bits
  __device__ uint32_t top() const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7fffffffu);
    return m;
  }
  static __device__ uint32_t bits(uint32_t m) { return m; }
  __device__ uint32_t top_with(const Eight &y) const { return max(top(), y.top()); }
  __device__ void put(const float (&x)[8]) {
    a = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    b = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
  }
};
template <typename H2>
struct Eight16 {
  uint4 a;
  __device__ void load(const void *p) { a = __ldcs((const uint4 *)p); }
  __device__ void store(void *p) const { *(uint4 *)p = a; }
  __device__ void zero() { a = make_uint4(0, 0, 0, 0); }
  static __device__ float2 two(uint32_t w);
  __device__ uint32_t top() const {  // two magnitudes a word
    const uint32_t k = 0x7fff7fffu, m = __vmaxu2(__vmaxu2(a.x & k, a.y & k), __vmaxu2(a.z & k, a.w & k));
    return max(m & 0xffffu, m >> 16);
  }
  __device__ uint32_t top_with(const Eight16 &y) const {  // of 16 elements, on the floats' own maximum
    const auto most = [](H2 p, H2 q) { return __hmax2_nan(__habs2(p), __habs2(q)); };
    const auto h = [](uint32_t w) { return *reinterpret_cast<const H2 *>(&w); };
    const H2 m = most(most(most(h(a.x), h(a.y)), most(h(a.z), h(a.w))), most(most(h(y.a.x), h(y.a.y)), most(h(y.a.z), h(y.a.w))));
    const uint32_t w = *reinterpret_cast<const uint32_t *>(&m);
    return max(w & 0xffffu, w >> 16);
  }
  static __device__ uint32_t bits(uint32_t m) { return __float_as_uint(two(m).x); }
  static __device__ uint32_t pack(float x, float y);
  __device__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = two(w[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  __device__ void put(const float (&x)[8]) {
    a = make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7]));
  }
};
template <>
__device__ __forceinline__ float2 Eight16<__nv_bfloat162>::two(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ uint32_t Eight16<__nv_bfloat162>::pack(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
__device__ __forceinline__ float2 Eight16<__half2>::two(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <>
__device__ __forceinline__ uint32_t Eight16<__half2>::pack(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}
template <>
struct Eight<__nv_bfloat16> : Eight16<__nv_bfloat162> {};
template <>
struct Eight<__half> : Eight16<__half2> {};

template <typename T>
constexpr int kSize = (int)sizeof(T);
template <>
constexpr int kSize<E4M3> = 1;
template <typename A, typename B>
struct Same {
  static constexpr bool value = false;
};
template <typename A>
struct Same<A, A> {
  static constexpr bool value = true;
};

// Eight codes times their scale as elements of the dense type.
template <typename D>
__device__ __forceinline__ void e2m1_to(uint32_t w, __half2 scale, Eight<D> &x) {
  uint32_t h[4];
  e2m1x8_times(w, scale, h);
  if constexpr (Same<D, __half>::value) {
    x.a = make_uint4(h[0], h[1], h[2], h[3]);
  } else {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
      f[2 * i] = y.x, f[2 * i + 1] = y.y;
    }
    x.put(f);
  }
}

__device__ __forceinline__ float load_any(const void *p, int64_t i, int dtype) {
  if (dtype == LSC_F32) return ((const float *)p)[i];
  if (dtype == LSC_BF16) return __bfloat162float(((const __nv_bfloat16 *)p)[i]);
  return __half2float(((const __half *)p)[i]);
}
__device__ __forceinline__ void store_any(void *p, int64_t i, int dtype, float x) {
  if (dtype == LSC_F32) ((float *)p)[i] = x;
  else if (dtype == LSC_BF16) ((__nv_bfloat16 *)p)[i] = __float2bfloat16_rn(x);
  else ((__half *)p)[i] = __float2half_rn(x);
}
// The same type on both sides moves as bits (a NaN keeps its payload).
__device__ __forceinline__ void move_any(void *d, int64_t i, const void *s, int64_t j, int dtype) {
  if (dtype == LSC_F32) ((uint32_t *)d)[i] = ((const uint32_t *)s)[j];
  else ((uint16_t *)d)[i] = ((const uint16_t *)s)[j];
}

}  // namespace row
}  // namespace kv
}  // namespace lsc
