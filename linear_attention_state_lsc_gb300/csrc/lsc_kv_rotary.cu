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
// fp32 (24 bits: off by 2^-26 turns at most), go to sincospif.
//
// Each element is read once and written once: HBM bounds a large call, the launch a
// small one.  All rows of all tokens are cut into equal runs, one a warp
// (lsc_kv_walk.cuh).  A warp forms a token's cosines and sines once, in shared memory,
// for all its heads, and then takes its rows 512 elements at a time: a lane has 16, the
// 8 first and the 8 second elements of 8 pairs (of neighbouring pairs: 4 and 4 pairs half
// the turned elements apart; likewise of the elements that are not turned), so no
// element is needed by another lane, rows may be turned in place, loads and stores of
// neighbouring lanes lie side by side, and so do their cosines.  A first form, CTAs of 16
// tokens whose lanes had 8 elements and fetched their pairs' others by shuffles, had the
// shared memory 94 % busy.  Measured, bf16: 30011 tokens, 40 heads of 128 turned whole, 615 MB in
// 101 us (6.1 TB/s, 91 % of a copy's rate; the first form 170 us); with the append, 64 chunks of 64 to
// 2048 tokens, 16 q heads and 2 kv heads of 256, a quarter turned, 1.39 GB in 228 us (91 %; 286).  CTAs
// of 256 threads an SM and rows a warp has on the way: 4 and 2; 3 and 3 104 and 224 us, 4 and 1 104 and 229, 3 and 2 111 and
// 244, 2 and 4 116 and 261.
#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_batch.cuh"
#include "lsc_kv_rows.cuh"
#include "lsc_kv_walk.cuh"
#include "lsc_ptx.h"

namespace lsc {
namespace {

using namespace kv;
using namespace kv::row;

struct NoPool {};

// ---- vector kernel: head_dim and rotary_dim multiples of 16, head_dim at most 512 ---------
constexpr int kOcc = 4;  // CTAs per SM

// Lane `ln`'s places of its item: slot 32 rest + ln of the token, head_dim / 16 slots a head.
struct Slot {
  int32_t head, s;
  int32_t v0, v1;  // first elements of its two eights
  bool turned;
};

template <typename D, typename P>
__global__ void __launch_bounds__(kWalkThreads, kOcc) rotary_kernel(const __grid_constant__ KvRotaryParams p, int per, FastDiv by_slots) {
  constexpr bool POOL = !Same<P, NoPool>::value;
  constexpr int U = sizeof(D) == 4 ? 1 : 2;  // items on the way, a warp
  __shared__ uint64_t s_turns[kRotaryPairs];
  __shared__ uint8_t s_axis[kRotaryPairs];
  __shared__ float4 s_cs[kWalkWarps][4][kRotaryPairs / 8];  // of two pairs; a slot's eight pairs are [0 .. 3][slot]
  if ((int)threadIdx.x < p.r.half) s_turns[threadIdx.x] = p.r.turns[threadIdx.x], s_axis[threadIdx.x] = p.r.axis[threadIdx.x];
  __syncthreads();
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const KvLayer &L = p.L;
  const int ln = threadIdx.x & 31, half = p.r.half, sr = half / 8, rest_dim = p.head_dim - 2 * half;
  const int kh = POOL ? L.heads : 0, heads = p.heads + 2 * kh;
  float4(&cs)[4][kRotaryPairs / 8] = s_cs[threadIdx.x >> 5];
  const WarpRun run = warp_run((int64_t)p.b.total_tokens * per);
  int32_t t = (int32_t)(run.begin / per), rest = (int32_t)(run.begin - (int64_t)t * per), left = (int32_t)(run.end - run.begin);
  int32_t t_ahead = t, rest_ahead = rest, left_ahead = left;
  auto slot_of = [&](int32_t rest) {
    Slot z;
    const int32_t i = rest * 32 + ln;
    z.head = by_slots.div(i);
    z.s = i - z.head * (int32_t)by_slots.d;
    z.turned = z.s < sr;
    z.v0 = z.turned ? 8 * z.s : 2 * half + 8 * (z.s - sr);
    z.v1 = z.v0 + (z.turned ? half : rest_dim / 2);
    return z;
  };
  Eight<D> x[U][2];
  auto load = [&](int u) {
    const Slot z = slot_of(rest_ahead);
    const bool q = z.head < p.heads, v = z.head >= p.heads + kh;
    const uint8_t *src = (const uint8_t *)(q ? p.x : v ? p.v : p.k) +
                         ((int64_t)t_ahead * (q ? p.x_stride : v ? p.v_stride : p.k_stride) +
                          (int64_t)(z.head - (q ? 0 : v ? p.heads + kh : p.heads)) * p.head_dim) * kSize<D>;
    x[u][0].zero(), x[u][1].zero();
    if (left_ahead > 0 && z.head < heads) x[u][0].load(src + z.v0 * kSize<D>), x[u][1].load(src + z.v1 * kSize<D>);
    --left_ahead;
    if (++rest_ahead == per) rest_ahead = 0, ++t_ahead;
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u);
  if constexpr (POOL)
    if (blockIdx.x == 0) check_cu(L, p.b);
  PlaceWalk place;
  int32_t row = 0;
  bool fresh = true;
  while (left > 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u > 0 && left <= 0) break;
      if (fresh) {
        if constexpr (POOL) row = place.at(L, p.b, t);
        __syncwarp();  // the last token's have been read
        if (row != -2) {
          for (int j = ln; j < half; j += 32) {
            const int64_t pos = p.r.positions[s_axis[j] * p.r.axis_stride + t];
            const int32_t half_turns = (int32_t)(((uint64_t)pos * s_turns[j]) >> 32);  // in units of 2^-31
            float sn, cn;
            sincospif((float)half_turns * 0x1p-31f, &sn, &cn);
            const int up = p.r.interleaved && j >= half / 2, i = j - (up ? half / 2 : 0);
            const int slot = p.r.interleaved ? i >> 2 : i >> 3, at = p.r.interleaved ? 2 * up + (i >> 1 & 1) : i >> 1 & 3;
            *((float2 *)&cs[at][slot] + (i & 1)) = make_float2(cn * p.r.scale, sn * p.r.scale);
          }
        }
        __syncwarp();
      }
      const Slot z = slot_of(rest);
      const bool on = z.head < heads, q = z.head < p.heads, v = z.head >= p.heads + kh, turn = z.turned && !v;
      const int head = z.head - (q ? 0 : v ? p.heads + kh : p.heads);
      Eight<D> raw[2] = {x[u][0], x[u][1]};
      load(u);
      float f[2][8];
      raw[0].get(f[0]);
      raw[1].get(f[1]);
      if (turn && on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 c = cs[i][z.s];
          if (!p.r.interleaved) {
            const float a0 = f[0][2 * i], b0 = f[1][2 * i], a1 = f[0][2 * i + 1], b1 = f[1][2 * i + 1];
            f[0][2 * i] = fmaf(a0, c.x, -b0 * c.y), f[1][2 * i] = fmaf(b0, c.x, a0 * c.y);
            f[0][2 * i + 1] = fmaf(a1, c.z, -b1 * c.w), f[1][2 * i + 1] = fmaf(b1, c.z, a1 * c.w);
          } else {
            float(&g)[8] = f[i >> 1];
            const int e = 4 * (i & 1);
            const float a0 = g[e], b0 = g[e + 1], a1 = g[e + 2], b1 = g[e + 3];
            g[e] = fmaf(a0, c.x, -b0 * c.y), g[e + 1] = fmaf(b0, c.x, a0 * c.y);
            g[e + 2] = fmaf(a1, c.z, -b1 * c.w), g[e + 3] = fmaf(b1, c.z, a1 * c.w);
          }
        }
        raw[0].put(f[0]);  // what is not turned keeps its bits where its type stays
        raw[1].put(f[1]);
      }
      if (q && on && row != -2 && (z.turned || p.out != p.x)) {
        uint8_t *dst = (uint8_t *)p.out + ((int64_t)t * p.out_stride + (int64_t)head * p.head_dim) * kSize<D>;
        raw[0].store(dst + z.v0 * kSize<D>);
        raw[1].store(dst + z.v1 * kSize<D>);
      }
      if constexpr (POOL) {
        const bool put = !q && on && row >= 0;
        uint8_t *const page = L.k + (v ? L.v - L.k : 0) + (row >= 0 ? place.page : 0);
        const int64_t first = ((int64_t)row * L.heads + head) * p.head_dim;  // element of the block
        if constexpr (Same<P, E4M3>::value) {
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(f[i >> 3][i & 7]) & 0x7fffffffu);
          for (int o = (int)by_slots.d >> 1; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          const uint32_t sb = scale_byte(m);
          const float inv = inv_scale_of(sb);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float(&y)[8] = f[e];
            uint2 c = make_uint2(
                __byte_perm(to_e4m3x2(y[0] * inv, y[1] * inv), to_e4m3x2(y[2] * inv, y[3] * inv), 0x5410),
                __byte_perm(to_e4m3x2(y[4] * inv, y[5] * inv), to_e4m3x2(y[6] * inv, y[7] * inv), 0x5410));
            if (sb == 255) c = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
            if (put) *(uint2 *)(page + first + (e ? z.v1 : z.v0)) = c;
          }
          if (put && z.s == 0) page[L.scale_off + (int64_t)row * L.heads + head] = (uint8_t)sb;
        } else if constexpr (Same<P, E2M1>::value) {  // a group of 16 is the same eight of two neighbouring lanes
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[e][i]) & 0x7fffffffu);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            const uint32_t sb = e2m1_scale_byte(m), el = (uint32_t)first + (e ? z.v1 : z.v0);  // 2^32 a block at most
            const uint32_t c = to_e2m1x8<true>(f[e], e2m1_scale(sb));  // a turned element has 24 bits
            if (put) *(uint32_t *)(page + (el >> 1)) = c;
            if (put && (ln & 1) == 0) page[L.scale_off + (el >> 4)] = (uint8_t)sb;
          }
        } else if (put) {
          uint8_t *dst = page + first * kSize<P>;
          if constexpr (Same<P, D>::value) {
            raw[0].store(dst + z.v0 * kSize<P>);
            raw[1].store(dst + z.v1 * kSize<P>);
          } else {
            Eight<P> y;
            y.put(f[0]);
            y.store(dst + z.v0 * kSize<P>);
            y.put(f[1]);
            y.store(dst + z.v1 * kSize<P>);
          }
        }
      }
      --left;
      fresh = ++rest == per;
      if (fresh) rest = 0, ++t;
    }
  }
}

// ---- element kernel: any head_dim, rotary_dim, types and alignment ------------------------------
// A warp takes a row.
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
      const int32_t half_turns = (int32_t)(((uint64_t)pos * turns) >> 32);
      float sn, cn;
      sincospif((float)half_turns * 0x1p-31f, &sn, &cn);
      cs[i * r.half + pair] = make_float2(cn * r.scale, sn * r.scale);
    }
  }
  __syncthreads();
}

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
          float x[2][8];
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[e >> 3][e & 7] = value(16 * j + e);
            m = max(m, __float_as_uint(x[e >> 3][e & 7]) & 0x7fffffffu);
          }
          const uint32_t sb = e2m1_scale_byte(m);
          const E2m1Scale scale = e2m1_scale(sb);
          *(uint2 *)(page + (in >> 1) + 8 * j) = make_uint2(to_e2m1x8<true>(x[0], scale), to_e2m1x8<true>(x[1], scale));
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

template <typename D, typename P>
cudaError_t launch_typed(const KvRotaryParams &p, int num_sms, cudaStream_t stream) {
  FastDiv by_slots;
  by_slots.set((uint32_t)p.head_dim / 16);
  const int64_t slots = ((int64_t)p.heads + (p.L.k ? 2 * p.L.heads : 0)) * (p.head_dim / 16);
  const int per = (int)((slots + 31) / 32);
  const int grid = walk_grid((int64_t)p.b.total_tokens * per, num_sms, kOcc);
  return launch_pdl(rotary_kernel<D, P>, grid, kWalkThreads, 0, stream, p, per, by_slots);
}

template <typename D>
cudaError_t launch_dense(const KvRotaryParams &p, int num_sms, cudaStream_t stream) {
  if (!p.L.k) return launch_typed<D, NoPool>(p, num_sms, stream);
  switch (p.L.dtype) {
    case LSC_F32: return launch_typed<D, float>(p, num_sms, stream);
    case LSC_BF16: return launch_typed<D, __nv_bfloat16>(p, num_sms, stream);
    case LSC_F16: return launch_typed<D, __half>(p, num_sms, stream);
    case LSC_E4M3: return launch_typed<D, E4M3>(p, num_sms, stream);
    default: return launch_typed<D, E2M1>(p, num_sms, stream);
  }
}

cudaError_t launch_any(const KvRotaryParams &p, int num_sms, cudaStream_t stream) {
  const int64_t T = p.b.total_tokens;
  // A run of kMaxTok tokens per CTA, shorter while the grid would leave SMs idle.
  int tok = kMaxTok;
  while (tok > 1 && (T + tok - 1) / tok < 2 * (int64_t)num_sms) tok >>= 1;
  const int grid = (int)((T + tok - 1) / tok);
  const size_t smem = (size_t)tok * p.r.half * sizeof(float2);
  return p.L.k ? launch_pdl(rotary_any_kernel<true>, grid, kThreads, smem, stream, p, tok)
               : launch_pdl(rotary_any_kernel<false>, grid, kThreads, smem, stream, p, tok);
}

}  // namespace

cudaError_t launch_kv_rotary(const KvRotaryParams &p, int num_sms, cudaStream_t stream) {
  const int es = p.dtype == LSC_F32 ? 4 : 2, slots = p.head_dim / 16;
  uintptr_t mis = (uintptr_t)p.x | (uintptr_t)p.out | (uintptr_t)(p.x_stride * es) | (uintptr_t)(p.out_stride * es);
  if (p.L.k) mis |= (uintptr_t)p.k | (uintptr_t)p.v | (uintptr_t)(p.k_stride * es) | (uintptr_t)(p.v_stride * es);
  bool vec = p.head_dim % 16 == 0 && p.head_dim <= 512 && p.r.half % 8 == 0 && (mis & 15) == 0;
  if (p.L.k && p.L.dtype == LSC_E4M3) vec = vec && 32 % slots == 0;  // a head's largest magnitude: its lanes, by shuffles
  if (p.L.k && p.L.dtype == LSC_E2M1) vec = vec && slots % 2 == 0 && p.r.half % 16 == 0;  // groups are pairs of lanes
  const cudaError_t e = !vec                   ? launch_any(p, num_sms, stream)
                        : p.dtype == LSC_F32  ? launch_dense<float>(p, num_sms, stream)
                        : p.dtype == LSC_BF16 ? launch_dense<__nv_bfloat16>(p, num_sms, stream)
                                              : launch_dense<__half>(p, num_sms, stream);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace lsc
