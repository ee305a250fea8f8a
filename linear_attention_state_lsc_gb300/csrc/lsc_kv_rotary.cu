// lsc_kv_rotary.cu -- rotary positions (include/lsc_kv.h): rows of heads turned by
// their tokens' positions, dense to dense (lsc_rotate), and with the append of a
// step in the same pass (lsc_kv_append_rotated): q dense to dense, k turned on its
// way into the pool's blocks, v beside it.
//
// Pair i of a head is turned by positions[axis(i)] * inv_freq[i].  An angle counts
// modulo a whole turn only, so the host passes inv_freq / (2 pi) as a 64-bit fraction
// of a turn: position times it in whole numbers keeps the low 64 bits, which is the
// exact fraction for every position of 32 bits (the fraction is within 2^-63 or so of
// inv_freq's, 2^-32 turns at position 2^31), where a product in fp32 would have lost the
// angle at a few thousand.  Its upper 32 bits, as a signed number of half turns in
// fp32, go to sincospif.
//
// Each element is read once and written once: HBM bounds a large call, the launch a
// small one.  A CTA takes a run of tokens and forms their cosines and sines in shared
// memory once for all heads (a head's pairs are the same for each), then streams the
// rows; a row is one group of a warp's lanes with 8 elements each (16 where the pool is
// E2M1: a group of one scale), its pairs' other halves come from the lane that has
// them by shuffles, so a row is read once and may be turned in place.
#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_batch.cuh"
#include "lsc_kv_rows.cuh"
#include "lsc_ptx.h"

namespace lsc {
namespace {

using namespace kv;
using namespace kv::row;

struct NoPool {};

constexpr int kUnroll = 2;  // rows in flight per lane group

// The run's cosines and sines times the factor, [token][pair]; a token of no sequence has none.  A thread has one pair:
// its frequency and axis come from the constant bank, one address a lane.
template <bool POOL>
__device__ __forceinline__ void fill_turns(const KvRotaryParams &p, int32_t t0, int n, const Places &s, float2 *cs) {
  const Rotary &r = p.r;
  const int at_once = kThreads / r.half, first = p.by_half.div(threadIdx.x), pair = threadIdx.x - first * r.half;
  if (first < at_once) {
    const uint64_t turns = r.turns[pair];
    const int32_t *positions = r.positions + r.axis[pair] * r.axis_stride + t0;
    for (int i = first; i < n; i += at_once) {
      if (POOL && s.row[i] == -2) continue;
      const int64_t pos = positions[i];
      const int32_t half_turns = (int32_t)(((uint64_t)pos * turns) >> 32);  // in units of 2^-31
      float sn, cn;
      sincospif((float)half_turns * 0x1p-31f, &sn, &cn);
      cs[i * r.half + pair] = make_float2(cn * r.scale, sn * r.scale);
    }
  }
  __syncthreads();
}

__device__ __forceinline__ uint4 shfl4(uint4 x, int from) {
  return make_uint4(__shfl_sync(0xffffffffu, x.x, from), __shfl_sync(0xffffffffu, x.y, from),
                    __shfl_sync(0xffffffffu, x.z, from), __shfl_sync(0xffffffffu, x.w, from));
}
__device__ __forceinline__ void shfl8(const Eight<float> &x, int from, Eight<float> &y) {
  y.a = shfl4(x.a, from);
  y.b = shfl4(x.b, from);
}
template <typename T>
__device__ __forceinline__ void shfl8(const Eight<T> &x, int from, Eight<T> &y) {
  y.a = shfl4(x.a, from);
}

// ---- vector kernel: head_dim a multiple of 8 and at most 256, pairs that lanes do not split ---------
// A lane has NV vectors of 8 elements; lanes: of a row's group (a power of two >= head_dim / (8 NV)).
template <typename D, typename P, int NV>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ KvRotaryParams p, int tok, int lanes) {
  constexpr bool POOL = !Same<P, NoPool>::value;
  constexpr int EV = 8 * NV, U = kUnroll;
  __shared__ Places s;
  extern __shared__ float4 cs4[];
  float2 *cs = reinterpret_cast<float2 *>(cs4);
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const KvLayer &L = p.L;
  const int32_t t0 = (int32_t)blockIdx.x * tok;
  const int n = p.b.total_tokens - t0 < tok ? p.b.total_tokens - t0 : tok;
  const int groups = kThreads / lanes, g = threadIdx.x / lanes, sub = threadIdx.x & (lanes - 1);
  const int ln = threadIdx.x & 31;
  const bool on = sub * EV < p.head_dim;
  const int half = p.r.half, hl = half / EV;
  const bool turned = sub * EV < 2 * half, upper = sub >= hl;  // halves: this lane has second elements of pairs
  // the lane with the other elements of this one's pairs; its first pair (its own, when neighbours are the pairs)
  const int from = (ln & ~(lanes - 1)) | (!turned ? sub : upper ? sub - hl : sub + hl);
  const int pair0 = !turned ? 0 : p.r.interleaved ? sub * (EV / 2) : (upper ? sub - hl : sub) * EV;
  // Row r of the run is row r % per of token r / per: q's heads, then k's, then v's; a group's rows are `groups` apart.
  const int kh = POOL ? L.heads : 0, per = p.heads + 2 * kh, rows = n * per, step_i = groups / per, step_w = groups - step_i * per;
  struct Walk {
    int i, w;
  };
  auto next = [&](Walk &x) {
    x.w += step_w;
    x.i += step_i;
    if (x.w >= per) x.w -= per, ++x.i;
  };
  Walk ahead, at;
  ahead.i = g / per;
  ahead.w = g - ahead.i * per;
  at = ahead;
  Eight<D> x[U][NV];
  auto load_rows = [&]() {
#pragma unroll
    for (int u = 0; u < U; ++u, next(ahead)) {
      const bool q = ahead.w < p.heads, v = ahead.w >= p.heads + kh;
      const int head = q ? ahead.w : ahead.w - p.heads - (v ? kh : 0);
      const uint8_t *src = (const uint8_t *)(q ? p.x : v ? p.v : p.k) +
                           ((int64_t)(t0 + ahead.i) * (q ? p.x_stride : v ? p.v_stride : p.k_stride) +
                            (int64_t)head * p.head_dim + sub * EV) * kSize<D>;
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        x[u][e].zero();
        if (ahead.i < n && on) x[u][e].load(src + e * 8 * kSize<D>);
      }
    }
  };
  load_rows();
  if constexpr (POOL) {
    if (blockIdx.x == 0) check_cu(L, p.b);
    find_places(L, p.b, t0, n, s);
  }
  fill_turns<POOL>(p, t0, n, s, cs);
  for (int r0 = 0; r0 < rows; r0 += groups * U) {  // the same trips in every thread: the groups shuffle
    if (r0 > 0) load_rows();
#pragma unroll
    for (int u = 0; u < U; ++u, next(at)) {
      const bool q = at.w < p.heads, v = at.w >= p.heads + kh, turn = turned && !v;
      const int head = q ? at.w : at.w - p.heads - (v ? kh : 0);
      int32_t row = at.i < n ? 0 : -2;
      if constexpr (POOL)
        if (row == 0) row = s.row[at.i];
      float y[EV];
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        float f[8], o[8];
        x[u][e].get(f);
        const float2 *c = cs + (row == -2 ? 0 : at.i) * half + pair0;
        if (!p.r.interleaved) {
          Eight<D> other;
          shfl8(x[u][e], from, other);
          other.get(o);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float4 z = *(const float4 *)(c + e * 8 + i);
            const float o0 = upper ? o[i] : -o[i], o1 = upper ? o[i + 1] : -o[i + 1];
            y[8 * e + i] = turn ? fmaf(f[i], z.x, o0 * z.y) : f[i];
            y[8 * e + i + 1] = turn ? fmaf(f[i + 1], z.z, o1 * z.w) : f[i + 1];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 z = c[e * 4 + i / 2];
            y[8 * e + i] = turn ? fmaf(f[i], z.x, -f[i + 1] * z.y) : f[i];
            y[8 * e + i + 1] = turn ? fmaf(f[i + 1], z.x, f[i] * z.y) : f[i + 1];
          }
        }
      }
      auto as_eight = [&](int e) -> const float(&)[8] { return *reinterpret_cast<const float(*)[8]>(&y[8 * e]); };
      // what is not turned keeps its bits where its type stays
      auto store_same = [&](uint8_t *dst) {
#pragma unroll
        for (int e = 0; e < NV; ++e) {
          if (turn) x[u][e].put(as_eight(e));
          x[u][e].store(dst + e * 8 * kSize<D>);
        }
      };
      if (q && row != -2 && on && (turned || p.out != p.x))
        store_same((uint8_t *)p.out + ((int64_t)(t0 + at.i) * p.out_stride + (int64_t)head * p.head_dim + sub * EV) * kSize<D>);
      if constexpr (POOL) {
        uint8_t *page = (v ? L.v : L.k) + (row < 0 ? 0 : s.page[at.i]);
        const bool put = !q && row >= 0 && on;
        uint8_t *dst = page + ((int64_t)row * L.heads + head) * held<P>(p.head_dim) + held<P>(sub * EV);
        if constexpr (Same<P, E4M3>::value) {
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < EV; ++i) m = max(m, __float_as_uint(y[i]) & 0x7fffffffu);
          for (int o = lanes >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          const uint32_t sb = scale_byte(m);
          const float inv = inv_scale_of(sb);
          uint2 c = make_uint2(
              __byte_perm(to_e4m3x2(y[0] * inv, y[1] * inv), to_e4m3x2(y[2] * inv, y[3] * inv), 0x5410),
              __byte_perm(to_e4m3x2(y[4] * inv, y[5] * inv), to_e4m3x2(y[6] * inv, y[7] * inv), 0x5410));
          if (sb == 255) c = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
          if (put) *(uint2 *)dst = c;
          if (put && sub == 0) page[L.scale_off + (int64_t)row * L.heads + head] = (uint8_t)sb;
        } else if constexpr (Same<P, E2M1>::value) {
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < EV; ++i) m = max(m, __float_as_uint(y[i]) & 0x7fffffffu);
          const uint32_t sb = e2m1_scale_byte(m);
          if (put) {
            *(uint2 *)dst = to_e2m1x16<true>(y, sb);  // a turned element has 24 bits
            page[L.scale_off + ((int64_t)row * L.heads + head) * (p.head_dim / 16) + sub] = (uint8_t)sb;
          }
        } else if (put) {
          if constexpr (Same<P, D>::value) {
            store_same(dst);
          } else {
            Eight<P> z;
            z.put(as_eight(0));
            z.store(dst);
          }
        }
      }
    }
  }
}

// ---- element kernel: any head_dim, rotary_dim, types and alignment ------------------------------
// A warp takes a row.
template <bool POOL>
__global__ void __launch_bounds__(kThreads) rotary_any_kernel(const __grid_constant__ KvRotaryParams p, int tok) {
  __shared__ Places s;
  extern __shared__ float4 cs4[];
  float2 *cs = reinterpret_cast<float2 *>(cs4);
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const KvLayer &L = p.L;
  const int32_t t0 = (int32_t)blockIdx.x * tok;
  const int n = p.b.total_tokens - t0 < tok ? p.b.total_tokens - t0 : tok;
  if constexpr (POOL) {
    if (blockIdx.x == 0) check_cu(L, p.b);
    find_places(L, p.b, t0, n, s);
  }
  fill_turns<POOL>(p, t0, n, s, cs);
  const int warp = threadIdx.x >> 5, ln = threadIdx.x & 31, D = p.head_dim, half = p.r.half;
  const int kh = POOL ? L.heads : 0, per = p.heads + 2 * kh;
  for (int r = warp; r < n * per; r += kThreads / 32) {
    const int i = r / per, w = r - i * per;
    const bool q = w < p.heads, v = w >= p.heads + kh;
    const int head = q ? w : w - p.heads - (v ? kh : 0);
    const int32_t row = POOL ? s.row[i] : 0;
    if (row == -2 || (!q && row < 0)) continue;
    const void *src = q ? p.x : v ? p.v : p.k;
    const int64_t at = (int64_t)(t0 + i) * (q ? p.x_stride : v ? p.v_stride : p.k_stride) + (int64_t)head * D;
    const float2 *c = cs + i * half;
    auto first_of = [&](int j) { return p.r.interleaved ? 2 * j : j; };
    auto second_of = [&](int j) { return p.r.interleaved ? 2 * j + 1 : j + half; };
    // element d after the turn
    auto value = [&](int d) {
      const float x = load_any(src, at + d, p.dtype);
      if (v || d >= 2 * half) return x;
      const int j = p.r.interleaved ? d >> 1 : d < half ? d : d - half;
      const bool second = d == second_of(j);
      const float o = load_any(src, at + (second ? first_of(j) : second_of(j)), p.dtype);
      return fmaf(x, c[j].x, (second ? o : -o) * c[j].y);
    };
    if (q) {
      const int64_t to = (int64_t)(t0 + i) * p.out_stride + (int64_t)head * D;
      for (int j = ln; j < half; j += 32) {  // both of a pair are read before either is written: out may be x
        const float a = load_any(src, at + first_of(j), p.dtype), b = load_any(src, at + second_of(j), p.dtype);
        store_any(p.out, to + first_of(j), p.dtype, fmaf(a, c[j].x, -b * c[j].y));
        store_any(p.out, to + second_of(j), p.dtype, fmaf(b, c[j].x, a * c[j].y));
      }
      if (p.out != p.x)
        for (int d = 2 * half + ln; d < D; d += 32) move_any(p.out, to + d, src, at + d, p.dtype);
      continue;
    }
    if constexpr (POOL) {
      uint8_t *page = (v ? L.v : L.k) + s.page[i];
      const int64_t in = ((int64_t)row * L.heads + head) * D;  // first element within the block
      if (L.dtype == LSC_E2M1) {
        for (int j = ln; j < D / 16; j += 32) {  // a lane has a group
          float x[16];
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[e] = value(16 * j + e);
            m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
          }
          const uint32_t sb = e2m1_scale_byte(m);
          *(uint2 *)(page + (in >> 1) + 8 * j) = to_e2m1x16<true>(x, sb);
          page[L.scale_off + (in >> 4) + j] = (uint8_t)sb;
        }
      } else if (L.dtype == LSC_E4M3) {
        uint32_t m = 0;
        for (int d = ln; d < D; d += 32) m = max(m, __float_as_uint(value(d)) & 0x7fffffffu);
        m = __reduce_max_sync(0xffffffffu, m);
        const uint32_t sb = scale_byte(m);
        const float inv = inv_scale_of(sb);
        for (int d = ln; d < D; d += 32) page[in + d] = sb == 255 ? 0x7f : (uint8_t)to_e4m3x2(value(d) * inv, 0.f);
        if (ln == 0) page[L.scale_off + (int64_t)row * L.heads + head] = (uint8_t)sb;
      } else {
        for (int d = ln; d < D; d += 32) {
          if (L.dtype == p.dtype && (v || d >= 2 * half)) move_any(page, in + d, src, at + d, p.dtype);
          else store_any(page, in + d, L.dtype, value(d));
        }
      }
    }
  }
}

template <typename D, typename P, int NV>
cudaError_t launch_typed(const KvRotaryParams &p, int grid, int tok, size_t smem, cudaStream_t stream) {
  int lanes = 1;
  while (lanes * 8 * NV < p.head_dim) lanes <<= 1;
  return launch_pdl(rotary_kernel<D, P, NV>, grid, kThreads, smem, stream, p, tok, lanes);
}

template <typename D>
cudaError_t launch_dense(const KvRotaryParams &p, int grid, int tok, size_t smem, cudaStream_t stream) {
  if (!p.L.k) return launch_typed<D, NoPool, 1>(p, grid, tok, smem, stream);
  switch (p.L.dtype) {
    case LSC_F32: return launch_typed<D, float, 1>(p, grid, tok, smem, stream);
    case LSC_BF16: return launch_typed<D, __nv_bfloat16, 1>(p, grid, tok, smem, stream);
    case LSC_F16: return launch_typed<D, __half, 1>(p, grid, tok, smem, stream);
    case LSC_E4M3: return launch_typed<D, E4M3, 1>(p, grid, tok, smem, stream);
    default: return launch_typed<D, E2M1, 2>(p, grid, tok, smem, stream);
  }
}

}  // namespace

cudaError_t launch_kv_rotary(const KvRotaryParams &p, int num_sms, cudaStream_t stream) {
  const int64_t T = p.b.total_tokens;
  // A run of kMaxTok tokens per CTA, shorter while the grid would leave SMs idle.
  int tok = kMaxTok;
  while (tok > 1 && (T + tok - 1) / tok < 2 * (int64_t)num_sms) tok >>= 1;
  const int grid = (int)((T + tok - 1) / tok);
  const int es = p.dtype == LSC_F32 ? 4 : 2, ev = p.L.k && p.L.dtype == LSC_E2M1 ? 16 : 8;
  const size_t smem = (size_t)tok * p.r.half * sizeof(float2);
  uintptr_t mis = (uintptr_t)p.x | (uintptr_t)p.out | (uintptr_t)(p.x_stride * es) | (uintptr_t)(p.out_stride * es);
  if (p.L.k) mis |= (uintptr_t)p.k | (uintptr_t)p.v | (uintptr_t)(p.k_stride * es) | (uintptr_t)(p.v_stride * es);
  const bool vec = p.head_dim % 8 == 0 && p.head_dim <= 256 && (p.r.interleaved ? 2 : 1) * p.r.half % ev == 0 && (mis & 15) == 0;
  cudaError_t e;
  if (!vec) {
    e = p.L.k ? launch_pdl(rotary_any_kernel<true>, grid, kThreads, smem, stream, p, tok)
              : launch_pdl(rotary_any_kernel<false>, grid, kThreads, smem, stream, p, tok);
  } else {
    e = p.dtype == LSC_F32    ? launch_dense<float>(p, grid, tok, smem, stream)
        : p.dtype == LSC_BF16 ? launch_dense<__nv_bfloat16>(p, grid, tok, smem, stream)
                              : launch_dense<__half>(p, grid, tok, smem, stream);
  }
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace lsc
