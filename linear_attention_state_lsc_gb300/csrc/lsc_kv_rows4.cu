// lsc_kv_rows4.cu -- append and gather over an E2M1 layer of the K/V block pool
// (include/lsc_kv.h), and a batch's cached rows as f16 in a workspace for prefill
// chunks (lsc_kv_attend).
//
// Both directions move 2 bytes a dense element (16-bit types) and 9/16 of a byte in
// the pool, once: HBM bounds a large call, the launch a small one.  A token's K row of
// all heads is one stretch of codes, one of scales and one dense row, and its V row the
// same at constant distances, so a warp takes stretches of both at once and what is left
// per element is the arithmetic.  (With a group of lanes a head, as the other types have
// it in lsc_kv_rows.cu, finding addresses took more of the issue slots than the codes did.)
//   * append: a lane has a group of 16 elements of K and of V (two 16-byte loads each)
//     and stores their 8 bytes of codes and scale byte; runs of tokens are a warp's
//     (lsc_kv_walk.cuh) and the next stretches are loaded while one is worked on.
//     64 chunks of 64 to 2048 tokens, 2 heads of 256, bf16: 178 MB in 31.2 us (5.7 TB/s, 85 %
//     of a copy's rate; 51 us by head groups; 41 with runs of 16 tokens a CTA, which wait for
//     their places).  The quantisation, some 125 issue slots for 16 elements, shares the rest.
//   * gather: a lane has 8 elements of each stretch, so that its 16-byte stores are side
//     by side; a CTA has a run of 16 tokens.  24 contexts of 900 to 16000, 8 heads of 128:
//     927 MB in 142 us (6.5 TB/s, 98 %; 180 us by head groups, 167 a row at a time).
// Rows that are not aligned to 16 bytes are left to the element kernel of lsc_kv_rows.cu.
// None of them lets what follows in before its end, whose waiting CTAs took the room of those to come (64 chunks' append
// and gather 63.9 us in place of 62.8, 1000 tokens' gather in a captured graph 3.6 in place of 3.2).
//
// Expanded rows: blocks of kExpandTokens positions, sequence i's from block i *
// blocks_of_a_sequence on, with a block table of their own, so the f16 chunk kernels
// read them as they read a pool.  The chunk kernel for E2M1 pools makes the codes f16 for
// each row block anew; with many row blocks a sequence doing it once is cheaper.
#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_attend.cuh"
#include "lsc_kv_batch.cuh"
#include "lsc_kv_rows.cuh"
#include "lsc_kv_walk.cuh"
#include "lsc_ptx.h"

namespace lsc {
namespace {

using namespace kv;
using namespace kv::row;

constexpr int kWarps = kThreads / 32;

// Tokens of a CTA's run: at most kMaxTok, and CTAs for whole turns of the SMs (of `occ` CTAs each).
int run_tokens(int64_t T, int num_sms, int occ) {
  const int64_t slots = (int64_t)num_sms * occ, turns = (T + slots * kMaxTok - 1) / (slots * kMaxTok);
  return (int)((T + slots * turns - 1) / (slots * turns));
}

// ---- append --------------------------------------------------------------------
constexpr int kAppendOcc = 3;

// An item is a stretch of 512 elements of a token's K and V rows, `per` of them a row; the warps' runs of items are those of
// lsc_kv_walk.cuh (with runs of 16 tokens a CTA, as gather has them, finding a run's places took as long as its rows).
template <typename D>
__global__ void __launch_bounds__(kWalkThreads, kAppendOcc) append4_kernel(const __grid_constant__ KvRowsParams p, int per) {
  constexpr int U = sizeof(D) == 4 ? 1 : 2;  // items on the way, a warp
  griddep_wait();
  const KvLayer &L = p.L;
  const int ln = threadIdx.x & 31, row_el = L.heads * L.head_dim;
  const WarpRun run = warp_run((int64_t)p.b.total_tokens * per);
  int32_t t = (int32_t)(run.begin / per), rest = (int32_t)(run.begin - (int64_t)t * per), left = (int32_t)(run.end - run.begin);
  int32_t t_ahead = t, rest_ahead = rest, left_ahead = left;
  Eight<D> x[U][2][2];  // K's and V's
  auto load = [&](int u) {
    const int el = rest_ahead * 512 + ln * 16;
    const bool on = left_ahead > 0 && el < row_el;
    const uint8_t *k = (const uint8_t *)p.k + ((int64_t)t_ahead * p.k_stride + el) * kSize<D>;
    const uint8_t *v = (const uint8_t *)p.v + ((int64_t)t_ahead * p.v_stride + el) * kSize<D>;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      x[u][0][e].zero(), x[u][1][e].zero();
      if (on) x[u][0][e].load(k + e * 8 * kSize<D>), x[u][1][e].load(v + e * 8 * kSize<D>);
    }
    --left_ahead;
    if (++rest_ahead == per) rest_ahead = 0, ++t_ahead;
  };
#pragma unroll
  for (int u = 0; u < U; ++u) load(u);
  if (blockIdx.x == 0) check_cu(L, p.b);
  const int64_t lane_off = L.v - L.k;
  PlaceWalk place;
  int32_t row = -1;
  bool fresh = true;
  while (left > 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u > 0 && left <= 0) break;
      if (fresh) row = place.at(L, p.b, t);
      uint2 code[2];
      uint32_t sb[2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        sb[v] = e2m1_scale_byte(Eight<D>::bits(x[u][v][0].top_with(x[u][v][1])));
        const E2m1Scale scale = e2m1_scale(sb[v]);
        float f[2][8];
        x[u][v][0].get(f[0]);
        x[u][v][1].get(f[1]);
        code[v] = make_uint2(to_e2m1x8<sizeof(D) == 4>(f[0], scale), to_e2m1x8<sizeof(D) == 4>(f[1], scale));
      }
      load(u);
      const int el = rest * 512 + ln * 16;
      if (row >= 0 && el < row_el) {
        const uint32_t at = (uint32_t)row * row_el + el;  // a block has 2^32 elements at most
        uint8_t *c = L.k + place.page + (at >> 1), *b = L.k + place.page + L.scale_off + (at >> 4);
        *(uint2 *)c = code[0];
        *(uint2 *)(c + lane_off) = code[1];
        *b = (uint8_t)sb[0];
        b[lane_off] = (uint8_t)sb[1];
      }
      --left;
      fresh = ++rest == per;
      if (fresh) rest = 0, ++t;
    }
  }
}

// ---- gather --------------------------------------------------------------------
// An item: NS stretches of 256 elements of a token's K and V rows, whose addresses differ by constants.
template <typename D, int NS>
struct Item {
  uint32_t code[NS][2], byte[NS][2];
  // page: K's block, element `at` of it (row < 0: zeros); `left` elements of the row from this lane's first on
  __device__ __forceinline__ void load(const uint8_t *page, int64_t lane_off, int32_t scale_off, int32_t row, uint32_t at, int left) {
    const uint8_t *c = page + (at >> 1), *b = page + scale_off + (at >> 4);
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        code[n][v] = byte[n][v] = 0;
        if (row >= 0 && n * 256 < left) {
          code[n][v] = __ldcs((const uint32_t *)(c + (v ? lane_off : 0)) + n * 32);
          byte[n][v] = __ldcs(b + (v ? lane_off : 0) + n * 16);
        }
      }
  }
  __device__ __forceinline__ void store(uint8_t *k, uint8_t *v, int left) const {
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      if (n * 256 >= left) break;
#pragma unroll
      for (int l = 0; l < 2; ++l) {
        Eight<D> y;
        e2m1_to<D>(code[n][l], e2m1_scale2(byte[n][l]), y);
        y.store((l ? v : k) + n * 256 * kSize<D>);
      }
    }
  }
};

constexpr int kGatherOcc = 6;

// U items on the way, a warp
template <typename D, int NS, int U>
__global__ void __launch_bounds__(kThreads, kGatherOcc) gather4_kernel(const __grid_constant__ KvRowsParams p, int tok, int per, FastDiv by_per) {
  __shared__ Places s;
  griddep_wait();
  const KvLayer &L = p.L;
  if (blockIdx.x == 0) check_cu(L, p.b);
  const int32_t t0 = (int32_t)blockIdx.x * tok;
  const int n = p.b.total_tokens - t0 < tok ? p.b.total_tokens - t0 : tok;
  find_places(L, p.b, t0, n, s);
  const int ln = threadIdx.x & 31, row_el = L.heads * L.head_dim, all = n * per;
  const int64_t lane_off = L.v - L.k;
  for (int i0 = threadIdx.x >> 5; i0 < all; i0 += kWarps * U) {
    Item<D, NS> x[U];
    int at[U], el[U];  // token of the run, -1: none
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int item = i0 + u * kWarps;
      at[u] = by_per.div(item);
      el[u] = (item - at[u] * per) * (256 * NS) + ln * 8;
      const int32_t row = item < all ? s.row[at[u]] : -2;
      x[u].load(L.k + (row < 0 ? 0 : s.page[at[u]]), lane_off, L.scale_off, row, (uint32_t)row * row_el + el[u], row_el - el[u]);
      if (row == -2) el[u] = row_el;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + at[u];
      x[u].store((uint8_t *)p.k + (t * p.k_stride + el[u]) * kSize<D>, (uint8_t *)p.v + (t * p.v_stride + el[u]) * kSize<D>,
                 row_el - el[u]);
    }
  }
}

// ---- expanded rows ---------------------------------------------------------------
constexpr int kExpandRows = 32;  // positions of a CTA

template <int NS, int U>
__global__ void __launch_bounds__(kThreads, kGatherOcc) expand_kernel(const __grid_constant__ KvAttendParams p, const __grid_constant__ KvExpand x,
                                                                      int per, FastDiv by_per) {
  __shared__ int64_t s_page[kExpandRows];
  __shared__ int32_t s_row[kExpandRows];
  griddep_wait();
  const KvLayer &L = p.L;
  const int32_t i = x.by_chunks.div(blockIdx.x), pos0 = (blockIdx.x - i * x.chunks) * kExpandRows;
  const int32_t kv = p.b.kv[i];
  if ((uint32_t)kv > (uint32_t)p.max_kv || pos0 >= kv) return;  // too many are recorded by the kernel behind
  const int n = kv - pos0 < kExpandRows ? kv - pos0 : kExpandRows;
  if ((int)threadIdx.x < n) {
    const int32_t pos = pos0 + threadIdx.x, b = L.by_block.div(pos), blk = p.b.table[(int64_t)i * p.b.max_blocks + b];
    const bool in = (uint32_t)blk < (uint32_t)L.num_blocks;
    if (!in) report(L.status, LSC_ERR_OUT_OF_RANGE);
    s_page[threadIdx.x] = in ? (int64_t)blk * L.page : 0;
    s_row[threadIdx.x] = in ? pos - b * L.block_tokens : -1;
  }
  const int32_t block0 = i * x.blocks + pos0 / kExpandTokens;
  if (threadIdx.x == 0 && pos0 % kExpandTokens == 0) x.table[block0] = block0;
  __syncthreads();
  const int ln = threadIdx.x & 31, row_el = L.heads * L.head_dim, all = n * per;
  const int64_t row0 = (int64_t)block0 * kExpandTokens + pos0 % kExpandTokens, lane_off = L.v - L.k;
  for (int i0 = threadIdx.x >> 5; i0 < all; i0 += kWarps * U) {
    Item<__half, NS> y[U];
    int at[U], el[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int item = i0 + u * kWarps;
      at[u] = by_per.div(item);
      el[u] = (item - at[u] * per) * (256 * NS) + ln * 8;
      if (item >= all) el[u] = row_el;
      const int32_t row = item < all ? s_row[at[u]] : -1;
      y[u].load(L.k + (row < 0 ? 0 : s_page[at[u]]), lane_off, L.scale_off, row, (uint32_t)row * row_el + el[u], row_el - el[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t to = ((row0 + at[u]) * row_el + el[u]) * kSize<__half>;
      y[u].store((uint8_t *)x.k + to, (uint8_t *)x.v + to, row_el - el[u]);
    }
  }
}

int stretches(const KvLayer &L, int el) { return (L.heads * L.head_dim + el - 1) / el; }

FastDiv by(int n) {
  FastDiv d;
  d.set((uint32_t)n);
  return d;
}

// Stretches of 256 elements of an item: as many as fill rows without a rest, so that no lane idles.
int stretches_of_item(const KvLayer &L) {
  const int row = L.heads * L.head_dim;
  return row % 1024 == 0 ? 4 : row % 512 == 0 ? 2 : 1;
}

template <typename D>
cudaError_t gather_typed(const KvRowsParams &p, int grid, int tok, cudaStream_t stream) {
  const int ns = stretches_of_item(p.L), per = stretches(p.L, 256 * ns);
  return ns == 4   ? launch_pdl(gather4_kernel<D, 4, 1>, grid, kThreads, 0, stream, p, tok, per, by(per))
         : ns == 2 ? launch_pdl(gather4_kernel<D, 2, 2>, grid, kThreads, 0, stream, p, tok, per, by(per))
                   : launch_pdl(gather4_kernel<D, 1, 4>, grid, kThreads, 0, stream, p, tok, per, by(per));
}

cudaError_t expand_typed(const KvAttendParams &p, const KvExpand &x, int grid, cudaStream_t stream) {
  const int ns = stretches_of_item(p.L), per = stretches(p.L, 256 * ns);
  return ns == 4   ? launch_pdl(expand_kernel<4, 1>, grid, kThreads, 0, stream, p, x, per, by(per))
         : ns == 2 ? launch_pdl(expand_kernel<2, 2>, grid, kThreads, 0, stream, p, x, per, by(per))
                   : launch_pdl(expand_kernel<1, 4>, grid, kThreads, 0, stream, p, x, per, by(per));
}

}  // namespace

cudaError_t launch_kv_append4(const KvRowsParams &p, int num_sms, cudaStream_t stream) {
  const int per = stretches(p.L, 512), grid = walk_grid((int64_t)p.b.total_tokens * per, num_sms, kAppendOcc);
  return p.dtype == LSC_F32    ? launch_pdl(append4_kernel<float>, grid, kWalkThreads, 0, stream, p, per)
         : p.dtype == LSC_BF16 ? launch_pdl(append4_kernel<__nv_bfloat16>, grid, kWalkThreads, 0, stream, p, per)
                               : launch_pdl(append4_kernel<__half>, grid, kWalkThreads, 0, stream, p, per);
}

cudaError_t launch_kv_gather4(const KvRowsParams &p, int num_sms, cudaStream_t stream) {
  const int tok = run_tokens(p.b.total_tokens, num_sms, kGatherOcc), grid = (int)(((int64_t)p.b.total_tokens + tok - 1) / tok);
  return p.dtype == LSC_F32    ? gather_typed<float>(p, grid, tok, stream)
         : p.dtype == LSC_BF16 ? gather_typed<__nv_bfloat16>(p, grid, tok, stream)
                               : gather_typed<__half>(p, grid, tok, stream);
}

cudaError_t launch_kv_expand(const KvAttendParams &p, KvExpand x, cudaStream_t stream) {
  x.chunks = (p.max_kv + kExpandRows - 1) / kExpandRows;
  x.by_chunks.set((uint32_t)x.chunks);
  const int grid = p.b.n_seq * x.chunks;
  const cudaError_t e = expand_typed(p, x, grid, stream);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace lsc
