// lsc_kv_rows4.cu -- append and gather over an E2M1 layer of the K/V block pool
// (include/lsc_kv.h), and a batch's cached rows at 16 bits in a workspace for prefill
// chunks (lsc_kv_attend).
//
// Both directions move 2 bytes a dense element (16-bit types) and 9/16 of a byte in
// the pool, once: HBM bounds a large call, the launch a small one.  A (token, lane) row
// of all heads is one stretch of codes, one of scales and one dense row, so a warp takes
// a stretch of such a row at a time, and what is left per element is the arithmetic: with
// a group of lanes a head, as the other types have it (lsc_kv_rows.cu), finding each
// head's addresses cost as much as the codes.
//   * append: a lane has a group of 16 elements (two 16-byte loads) and stores its 8 bytes
//     of codes and its scale byte; a warp's next stretches are loaded while one is
//     worked on.
//   * gather: a lane has 8 elements, so that its 16-byte stores are side by side.
// Rows that are not aligned to 16 bytes are left to the element kernel of lsc_kv_rows.cu.
//
// Expanded rows: blocks of kExpandTokens positions, sequence i's from block i *
// blocks_of_a_sequence on, with a block table of their own, so the 16-bit chunk kernels
// read them as they read a pool.  The chunk kernel for E2M1 pools makes the codes f16 for
// each row block anew; with many row blocks a sequence doing it once is cheaper.
#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_attend.cuh"
#include "lsc_kv_batch.cuh"
#include "lsc_kv_rows.cuh"
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
constexpr int kAppendOcc = 4;

// items: stretches of 512 elements of a row
template <typename D>
__global__ void __launch_bounds__(kThreads, kAppendOcc) append4_kernel(const __grid_constant__ KvRowsParams p, int tok, FastDiv by_items) {
  constexpr int U = sizeof(D) == 4 ? 1 : 2;  // stretches on the way, a warp
  __shared__ Places s;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const KvLayer &L = p.L;
  const int32_t t0 = (int32_t)blockIdx.x * tok;
  const int n = p.b.total_tokens - t0 < tok ? p.b.total_tokens - t0 : tok;
  const int ln = threadIdx.x & 31, row_el = L.heads * L.head_dim, items = by_items.d, all = 2 * n * items;
  Eight<D> x[U][2];
  auto load = [&](int u, int item) {
    x[u][0].zero(), x[u][1].zero();
    const int r2 = by_items.div(item), el = (item - r2 * items) * 512 + ln * 16;
    if (item >= all || el >= row_el) return;
    const uint8_t *src = (const uint8_t *)(r2 & 1 ? p.v : p.k) +
                         ((int64_t)(t0 + (r2 >> 1)) * (r2 & 1 ? p.v_stride : p.k_stride) + el) * kSize<D>;
    x[u][0].load(src);
    x[u][1].load(src + 8 * kSize<D>);
  };
  int ahead = threadIdx.x >> 5;
#pragma unroll
  for (int u = 0; u < U; ++u, ahead += kWarps) load(u, ahead);
  if (blockIdx.x == 0) check_cu(L, p.b);
  find_places(L, p.b, t0, n, s);
  for (int i0 = threadIdx.x >> 5; i0 < all; i0 += kWarps * U) {
#pragma unroll
    for (int u = 0; u < U; ++u, ahead += kWarps) {
      const int item = i0 + u * kWarps, r2 = by_items.div(item), el = (item - r2 * items) * 512 + ln * 16;
      const uint32_t sb = e2m1_scale_byte(x[u][0].bits(max(x[u][0].top(), x[u][1].top())));
      float lo[8], hi[8], f[16];
      x[u][0].get(lo);
      x[u][1].get(hi);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = lo[e], f[8 + e] = hi[e];
      load(u, ahead);
      const uint2 code = to_e2m1x16<sizeof(D) == 4>(f, sb);
      if (item >= all || el >= row_el) continue;
      const int32_t row = s.row[r2 >> 1];
      if (row < 0) continue;
      const uint32_t at = (uint32_t)row * row_el + el;  // a block has 2^32 elements at most
      uint8_t *page = (r2 & 1 ? L.v : L.k) + s.page[r2 >> 1];
      *(uint2 *)(page + (at >> 1)) = code;
      page[L.scale_off + (at >> 4)] = (uint8_t)sb;
    }
  }
}

// ---- gather --------------------------------------------------------------------
// A warp's stretches of 256 elements of the run's rows: rows(r2, page, row, dst) says where row r2 (K and V of a token
// in turn) is, and is false for one that is not written; row < 0: zeros.
template <typename D, typename F>
__device__ __forceinline__ void read_rows(const KvLayer &L, int n, const FastDiv &by_items, const F &rows) {
  constexpr int U = 4;
  const int ln = threadIdx.x & 31, row_el = L.heads * L.head_dim, items = by_items.d, all = 2 * n * items;
  for (int i0 = threadIdx.x >> 5; i0 < all; i0 += kWarps * U) {
    uint32_t code[U], byte[U];
    uint8_t *dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int item = i0 + u * kWarps, r2 = by_items.div(item), el = (item - r2 * items) * 256 + ln * 8;
      dst[u] = nullptr;
      code[u] = byte[u] = 0;
      if (item >= all || el >= row_el) continue;
      const uint8_t *page;
      int32_t row;
      if (!rows(r2, page, row, dst[u])) continue;
      dst[u] += (int64_t)el * kSize<D>;
      if (row < 0) continue;
      const uint32_t at = (uint32_t)row * row_el + el;
      code[u] = __ldcs((const uint32_t *)(page + (at >> 1)));
      byte[u] = __ldcs(page + L.scale_off + (at >> 4));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Eight<D> y;
      e2m1_to<D>(code[u], e2m1_scale2(byte[u]), y);
      if (dst[u]) y.store(dst[u]);
    }
  }
}

constexpr int kGatherOcc = 6;

template <typename D>
__global__ void __launch_bounds__(kThreads, kGatherOcc) gather4_kernel(const __grid_constant__ KvRowsParams p, int tok, FastDiv by_items) {
  __shared__ Places s;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const KvLayer &L = p.L;
  if (blockIdx.x == 0) check_cu(L, p.b);
  const int32_t t0 = (int32_t)blockIdx.x * tok;
  const int n = p.b.total_tokens - t0 < tok ? p.b.total_tokens - t0 : tok;
  find_places(L, p.b, t0, n, s);
  read_rows<D>(L, n, by_items, [&](int r2, const uint8_t *&page, int32_t &row, uint8_t *&dst) {
    const int i = r2 >> 1, v = r2 & 1;
    row = s.row[i];
    if (row == -2) return false;
    page = (v ? L.v : L.k) + s.page[i];
    dst = (uint8_t *)(v ? p.v : p.k) + (int64_t)(t0 + i) * (v ? p.v_stride : p.k_stride) * kSize<D>;
    return true;
  });
}

// ---- expanded rows ---------------------------------------------------------------
constexpr int kExpandRows = 32;  // positions of a CTA

template <typename D>
__global__ void __launch_bounds__(kThreads, kGatherOcc) expand_kernel(const __grid_constant__ KvAttendParams p, const __grid_constant__ KvExpand x,
                                                                      FastDiv by_items) {
  __shared__ int64_t s_page[kExpandRows];
  __shared__ int32_t s_row[kExpandRows];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
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
  const int64_t row_bytes = (int64_t)L.heads * L.head_dim * kSize<D>;
  const int64_t out0 = ((int64_t)block0 * kExpandTokens + pos0 % kExpandTokens) * row_bytes;
  read_rows<D>(L, n, by_items, [&](int r2, const uint8_t *&page, int32_t &row, uint8_t *&dst) {
    const int j = r2 >> 1, v = r2 & 1;
    row = s_row[j];
    page = (v ? L.v : L.k) + s_page[j];
    dst = (uint8_t *)(v ? x.v : x.k) + out0 + j * row_bytes;
    return true;
  });
}

FastDiv items_of(const KvLayer &L, int el) {
  FastDiv d;
  d.set((uint32_t)((L.heads * L.head_dim + el - 1) / el));
  return d;
}

}  // namespace

cudaError_t launch_kv_append4(const KvRowsParams &p, int num_sms, cudaStream_t stream) {
  const int tok = run_tokens(p.b.total_tokens, num_sms, kAppendOcc), grid = (int)(((int64_t)p.b.total_tokens + tok - 1) / tok);
  const FastDiv d = items_of(p.L, 512);
  return p.dtype == LSC_F32    ? launch_pdl(append4_kernel<float>, grid, kThreads, 0, stream, p, tok, d)
         : p.dtype == LSC_BF16 ? launch_pdl(append4_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, p, tok, d)
                               : launch_pdl(append4_kernel<__half>, grid, kThreads, 0, stream, p, tok, d);
}

cudaError_t launch_kv_gather4(const KvRowsParams &p, int num_sms, cudaStream_t stream) {
  const int tok = run_tokens(p.b.total_tokens, num_sms, kGatherOcc), grid = (int)(((int64_t)p.b.total_tokens + tok - 1) / tok);
  const FastDiv d = items_of(p.L, 256);
  return p.dtype == LSC_F32    ? launch_pdl(gather4_kernel<float>, grid, kThreads, 0, stream, p, tok, d)
         : p.dtype == LSC_BF16 ? launch_pdl(gather4_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, p, tok, d)
                               : launch_pdl(gather4_kernel<__half>, grid, kThreads, 0, stream, p, tok, d);
}

cudaError_t launch_kv_expand(const KvAttendParams &p, KvExpand x, cudaStream_t stream) {
  x.chunks = (p.max_kv + kExpandRows - 1) / kExpandRows;
  x.by_chunks.set((uint32_t)x.chunks);
  const int grid = p.b.n_seq * x.chunks;
  const FastDiv d = items_of(p.L, 256);
  const cudaError_t e = p.dtype == LSC_BF16 ? launch_pdl(expand_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, p, x, d)
                                            : launch_pdl(expand_kernel<__half>, grid, kThreads, 0, stream, p, x, d);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace lsc
