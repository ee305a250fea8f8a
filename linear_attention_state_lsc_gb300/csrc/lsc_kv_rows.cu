// lsc_kv_rows.cu -- append and gather over a layer of the K/V block pool
// (include/lsc_kv.h): dense rows of the new tokens -> rows of the sequences'
// blocks, and back, with the E4M3 quantisation in the same pass.
//
// Both only move bytes: each dense element is read (written) once and each
// element of a block written (read) once, so HBM bounds a large call and the
// launch a small one.  A CTA takes a run of consecutive tokens, finds the
// block row of each once (one thread per token: the sequence by a search of
// cu_seqlens samples in shared memory, then the block table), then streams the
// K and V rows of the run, kUnroll 16-byte loads in flight per thread; append's
// first loads, whose addresses need no search, are issued before it.  A
// (token, head) row is handled by one group of a warp's lanes, 8 elements each
// (16 to and from E4M3: append issued 195 instructions a row and 256 elements with
// 8, most of them addresses, and that bounded it),
// so an E4M3 row's largest magnitude is a shuffle reduction and the row is
// never read twice.  Measured: bf16 to E4M3, 64 chunks of 64 to 2048 tokens, 2
// heads of 256, 209 MB in 47.6 us (4.4 TB/s, 66 % of a copy's rate; 62 % of the issue
// slots); back from E4M3, 24 contexts, 8 heads of 128, 1088 MB in 176 us (6.2 TB/s, 93 %).
#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_batch.cuh"
#include "lsc_ptx.h"

namespace lsc {
namespace {

using namespace kv;

constexpr int kThreads = 256;
constexpr int kMaxTok = 16;  // tokens of a CTA's run
constexpr int kStagedHeads = 64;
// Rows in flight per lane group, and CTAs per SM.  Append computes (the quantisation) and wants few address steps,
// gather waits for memory and wants threads: from E4M3, 24 contexts, 8 heads of 128: 4 rows and 4 CTAs 224 us, 2 and 6
// 179 us.
template <bool APPEND, int NV>
constexpr int kUnroll = (APPEND ? 4 : 2) / (APPEND ? NV : 1);
template <bool APPEND, int NV>
constexpr int kOcc = APPEND ? 4 : NV == 1 ? 8 : 6;

struct E4M3 {};

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

// ---- vector kernel: head_dim a multiple of 8 and at most 256 --------------------
// APPEND: dense -> pool; else pool -> dense.  A lane has NV vectors of 8 elements,
// lanes = lanes of a row's group (a power of two >= head_dim / (8 NV)).
template <bool APPEND, typename D, typename P, int NV>
__global__ void __launch_bounds__(kThreads, (kOcc<APPEND, NV>)) rows_kernel(const __grid_constant__ KvRowsParams p, int tok, int lanes) {
  __shared__ Places s;
  // scale bytes on their way out, [lane][token][head]: a byte a store would touch a sector each
  __shared__ uint8_t s_scale[APPEND && Same<P, E4M3>::value ? 2 * kMaxTok * kStagedHeads : 1];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const KvLayer &L = p.L;
  if (blockIdx.x == 0) check_cu(L, p.b);
  const int32_t t0 = (int32_t)blockIdx.x * tok;
  const int n = p.b.total_tokens - t0 < tok ? p.b.total_tokens - t0 : tok;
  const bool staged = L.heads <= kStagedHeads;
  constexpr int kUnroll = lsc::kUnroll<APPEND, NV>, EV = 8 * NV;
  const int groups = kThreads / lanes, g = threadIdx.x / lanes, sub = threadIdx.x & (lanes - 1);
  const bool on = sub * EV < L.head_dim;
  const int rows = n * 2 * L.heads;
  const int64_t head_bytes = (int64_t)L.head_dim * kSize<P>;
  // Row r of the run is head r % heads of lane (r / heads) % 2 (K, V) of token r / (2 heads); a group's rows are `groups`
  // apart, so its walk steps by a whole number of tokens and a rest.
  const int per = 2 * L.heads, step_i = groups / per, step_w = groups - step_i * per;
  struct Walk {
    int i, w;  // token of the run; row of the token
  };
  auto next = [&](Walk &x) {
    x.w += step_w;
    x.i += step_i;
    if (x.w >= per) x.w -= per, ++x.i;
  };
  auto dense_at = [&](const Walk &x) {
    const int lane = x.w >= L.heads;
    return (uint8_t *)(lane ? p.v : p.k) + ((int64_t)(t0 + x.i) * (lane ? p.v_stride : p.k_stride) +
                                            (x.w - lane * L.heads) * L.head_dim + sub * EV) *
                                               kSize<D>;
  };
  Walk ahead, at;
  ahead.i = g / per;
  ahead.w = g - ahead.i * per;
  at = ahead;
  Eight<D> x[kUnroll][NV];
  auto load_dense = [&]() {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint8_t *src = dense_at(ahead);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        x[u][v].zero();
        if (ahead.i < n && on) x[u][v].load(src + v * 8 * kSize<D>);
      }
      next(ahead);
    }
  };
  if (APPEND) load_dense();
  find_places(L, p.b, t0, n, s);
  for (int r0 = 0; r0 < rows; r0 += groups * kUnroll) {  // the same trips in every thread: the groups shuffle
    uint2 code[kUnroll][NV];
    uint32_t byte[kUnroll];
    int32_t row[kUnroll];
    uint8_t *page[kUnroll];
    int head[kUnroll], where[kUnroll];
    uint8_t *dense[kUnroll];
    if (APPEND && r0 > 0) load_dense();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u, next(at)) {
      const int i = at.i, lane = at.w >= L.heads;
      head[u] = at.w - lane * L.heads;
      where[u] = lane * n + i;
      if (!APPEND) dense[u] = dense_at(at);
      row[u] = i < n ? s.row[i] : -2;
#pragma unroll
      for (int v = 0; v < NV; ++v) code[u][v] = make_uint2(0, 0);
      byte[u] = 0;
      if (row[u] == -2) continue;
      page[u] = (lane ? L.v : L.k) + s.page[i];
      if constexpr (!APPEND) {
#pragma unroll
        for (int v = 0; v < NV; ++v) x[u][v].zero();
        if (row[u] == -1 || !on) continue;
        const uint8_t *src = page[u] + ((int64_t)row[u] * L.heads + head[u]) * head_bytes + sub * EV * kSize<P>;
        if constexpr (Same<P, E4M3>::value) {
          if constexpr (NV == 2) {
            const uint4 c = __ldcs((const uint4 *)src);
            code[u][0] = make_uint2(c.x, c.y), code[u][1] = make_uint2(c.z, c.w);
          } else {
            code[u][0] = __ldcs((const uint2 *)src);
          }
          byte[u] = __ldcs(page[u] + L.scale_off + (int64_t)row[u] * L.heads + head[u]);
        } else if constexpr (Same<P, D>::value) {
          x[u][0].load(src);
        } else {
          Eight<P> y;
          float f[8];
          y.load(src);
          y.get(f);
          x[u][0].put(f);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if constexpr (APPEND) {
        uint8_t *dst = row[u] < 0 ? nullptr : page[u] + ((int64_t)row[u] * L.heads + head[u]) * head_bytes +
                                                  sub * EV * kSize<P>;
        if constexpr (Same<P, E4M3>::value) {
          uint32_t m = x[u][0].top();
          if constexpr (NV == 2) m = max(m, x[u][1].top());
          if (lanes == 32) m = __reduce_max_sync(0xffffffffu, m);
          else
            for (int o = lanes >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          const uint32_t sb = scale_byte(x[u][0].bits(m));
          const float inv = inv_scale_of(sb);
          uint2 c[NV];
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            float f[8];
            x[u][v].get(f);
            c[v].x = __byte_perm(to_e4m3x2(f[0] * inv, f[1] * inv), to_e4m3x2(f[2] * inv, f[3] * inv), 0x5410);
            c[v].y = __byte_perm(to_e4m3x2(f[4] * inv, f[5] * inv), to_e4m3x2(f[6] * inv, f[7] * inv), 0x5410);
            if (sb == 255) c[v] = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
          }
          if (dst && on) {
            if constexpr (NV == 2) *(uint4 *)dst = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
            else *(uint2 *)dst = c[0];
          }
          if (dst && sub == 0) {
            if (staged) s_scale[where[u] * L.heads + head[u]] = (uint8_t)sb;
            else page[u][L.scale_off + (int64_t)row[u] * L.heads + head[u]] = (uint8_t)sb;
          }
        } else if (dst && on) {
          if constexpr (Same<P, D>::value) {
            x[u][0].store(dst);
          } else {
            Eight<P> y;
            float f[8];
            x[u][0].get(f);
            y.put(f);
            y.store(dst);
          }
        }
      } else {
        if (row[u] == -2 || !on) continue;
        if constexpr (Same<P, E4M3>::value) {
          if (row[u] >= 0) {
            const float k = scale_of(byte[u]);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
              const uint32_t w[4] = {code[u][v].x & 0xffffu, code[u][v].x >> 16, code[u][v].y & 0xffffu, code[u][v].y >> 16};
              float f[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 y = e4m3x2_to_float2(w[e]);
                f[2 * e] = y.x * k, f[2 * e + 1] = y.y * k;
              }
              x[u][v].put(f);
            }
          }
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) x[u][v].store(dense[u] + v * 8 * kSize<D>);
      }
    }
  }
  if constexpr (APPEND && Same<P, E4M3>::value) {
    if (!staged) return;
    __syncthreads();
    for (int j = threadIdx.x; j < 2 * n * L.heads; j += kThreads) {
      const int w = p.by_heads.div(j), lane = w >= n, i = w - lane * n;
      if (s.row[i] >= 0)
        ((lane ? L.v : L.k) + s.page[i])[L.scale_off + (int64_t)s.row[i] * L.heads + (j - w * L.heads)] = s_scale[j];
    }
  }
}

// ---- element kernel: any head_dim, types and alignment -------------------------
// A warp takes a (token, lane, head) row, its lanes stride over the elements.
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

template <bool APPEND>
__global__ void __launch_bounds__(kThreads) rows_any_kernel(const __grid_constant__ KvRowsParams p, int tok) {
  __shared__ Places s;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const KvLayer &L = p.L;
  if (blockIdx.x == 0) check_cu(L, p.b);
  const int32_t t0 = (int32_t)blockIdx.x * tok;
  const int n = p.b.total_tokens - t0 < tok ? p.b.total_tokens - t0 : tok;
  find_places(L, p.b, t0, n, s);
  const int warp = threadIdx.x >> 5, ln = threadIdx.x & 31;
  const int rows = n * 2 * L.heads, D = L.head_dim;
  for (int r = warp; r < rows; r += kThreads / 32) {
    const int i = r / (2 * L.heads), lane = (r / L.heads) & 1, head = r - (r / L.heads) * L.heads;
    const int32_t row = s.row[i];
    if (row == -2 || (APPEND && row == -1)) continue;
    uint8_t *page = (lane ? L.v : L.k) + s.page[i];
    const int64_t in = ((int64_t)row * L.heads + head) * D;  // first element within the block
    void *dense = lane ? p.v : p.k;
    const int64_t at = (int64_t)(t0 + i) * (lane ? p.v_stride : p.k_stride) + (int64_t)head * D;
    uint8_t *scale = page + L.scale_off + (int64_t)row * L.heads + head;
    if (row == -1) {
      for (int d = ln; d < D; d += 32) store_any(dense, at + d, p.dtype, 0.f);
    } else if (L.dtype == LSC_E4M3 && APPEND) {
      uint32_t m = 0;
      for (int d = ln; d < D; d += 32) m = max(m, __float_as_uint(load_any(dense, at + d, p.dtype)) & 0x7fffffffu);
      m = __reduce_max_sync(0xffffffffu, m);
      const uint32_t sb = scale_byte(m);
      const float inv = inv_scale_of(sb);
      for (int d = ln; d < D; d += 32)
        page[in + d] = sb == 255 ? 0x7f : (uint8_t)to_e4m3x2(load_any(dense, at + d, p.dtype) * inv, 0.f);
      if (ln == 0) *scale = (uint8_t)sb;
    } else if (L.dtype == LSC_E4M3) {
      const float k = scale_of(*scale);
      for (int d = ln; d < D; d += 32) store_any(dense, at + d, p.dtype, e4m3x2_to_float2(page[in + d]).x * k);
    } else if (L.dtype == p.dtype) {
      for (int d = ln; d < D; d += 32) {
        if (APPEND) move_any(page, in + d, dense, at + d, p.dtype);
        else move_any(dense, at + d, page, in + d, p.dtype);
      }
    } else {
      for (int d = ln; d < D; d += 32) {
        if (APPEND) store_any(page, in + d, L.dtype, load_any(dense, at + d, p.dtype));
        else store_any(dense, at + d, p.dtype, load_any(page, in + d, L.dtype));
      }
    }
  }
}

template <bool APPEND, typename D, typename P, int NV>
cudaError_t launch_typed(const KvRowsParams &p, int grid, int tok, cudaStream_t stream) {
  int lanes = 1;
  while (lanes * 8 * NV < p.L.head_dim) lanes <<= 1;
  return launch_pdl(rows_kernel<APPEND, D, P, NV>, grid, kThreads, 0, stream, p, tok, lanes);
}

template <bool APPEND, typename D>
cudaError_t launch_dense(const KvRowsParams &p, int grid, int tok, cudaStream_t stream) {
  switch (p.L.dtype) {
    case LSC_F32: return launch_typed<APPEND, D, float, 1>(p, grid, tok, stream);
    case LSC_BF16: return launch_typed<APPEND, D, __nv_bfloat16, 1>(p, grid, tok, stream);
    case LSC_F16: return launch_typed<APPEND, D, __half, 1>(p, grid, tok, stream);
    default:
      return p.L.head_dim % 16 == 0 ? launch_typed<APPEND, D, E4M3, 2>(p, grid, tok, stream)
                                    : launch_typed<APPEND, D, E4M3, 1>(p, grid, tok, stream);
  }
}

template <bool APPEND>
cudaError_t launch_rows(const KvRowsParams &p, int num_sms, cudaStream_t stream) {
  const KvLayer &L = p.L;
  const int64_t T = p.b.total_tokens;
  // A run of kMaxTok tokens per CTA, shorter while the grid would leave SMs idle.
  int tok = kMaxTok;
  while (tok > 1 && (T + tok - 1) / tok < 2 * (int64_t)num_sms) tok >>= 1;
  const int grid = (int)((T + tok - 1) / tok);
  const int es = p.dtype == LSC_F32 ? 4 : 2;
  const bool vec = L.head_dim % 8 == 0 && L.head_dim <= 256 &&
                   (((uintptr_t)p.k | (uintptr_t)p.v | (uintptr_t)(p.k_stride * es) | (uintptr_t)(p.v_stride * es)) & 15) == 0;
  cudaError_t e;
  if (!vec) {
    e = launch_pdl(rows_any_kernel<APPEND>, grid, kThreads, 0, stream, p, tok);
  } else {
    e = p.dtype == LSC_F32    ? launch_dense<APPEND, float>(p, grid, tok, stream)
        : p.dtype == LSC_BF16 ? launch_dense<APPEND, __nv_bfloat16>(p, grid, tok, stream)
                              : launch_dense<APPEND, __half>(p, grid, tok, stream);
  }
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

cudaError_t launch_kv_append(const KvRowsParams &p, int num_sms, cudaStream_t stream) {
  return launch_rows<true>(p, num_sms, stream);
}

cudaError_t launch_kv_gather(const KvRowsParams &p, int num_sms, cudaStream_t stream) {
  return launch_rows<false>(p, num_sms, stream);
}

}  // namespace lsc
