// lsc_kv_expand.cu -- an E2M1 layer's cached rows of a batch as 16-bit rows in a
// workspace, for prefill chunks (lsc_kv_attend): blocks of kExpandTokens positions,
// sequence i's from i * blocks_of_a_sequence on, with a block table of their own, so
// the 16-bit chunk kernels read them as they read a pool.
//
// The chunk kernel for E2M1 pools makes the codes f16 for each row block anew; with
// many row blocks a sequence doing it once is cheaper.  An element is exact in f16 and
// bf16 alike (6 bits).  HBM bounds it: 9/16 of a byte read and 2 bytes written an element,
// a thread 8 elements at a time, so that both sides are coalesced.
#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_attend.cuh"
#include "lsc_kv_batch.cuh"
#include "lsc_ptx.h"

namespace lsc {
namespace {

using namespace kv;

constexpr int kThreads = 256, kRows = 64, kUnroll = 4;

__global__ void __launch_bounds__(kThreads) expand_kernel(const __grid_constant__ KvAttendParams p, const __grid_constant__ KvExpand x) {
  __shared__ int64_t s_at[kRows];  // byte of a row's block in a lane, -1: none
  __shared__ int32_t s_row[kRows];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const KvLayer &L = p.L;
  const int32_t i = x.by_chunks.div(blockIdx.x), pos0 = (blockIdx.x - i * x.chunks) * kRows;
  const int32_t kv = p.b.kv[i];
  if ((uint32_t)kv > (uint32_t)p.max_kv || pos0 >= kv) return;  // too many are recorded by the kernel behind
  const int n = kv - pos0 < kRows ? kv - pos0 : kRows;
  if ((int)threadIdx.x < n) {
    const int32_t pos = pos0 + threadIdx.x, b = L.by_block.div(pos), blk = p.b.table[(int64_t)i * p.b.max_blocks + b];
    const bool in = (uint32_t)blk < (uint32_t)L.num_blocks;
    if (!in) report(L.status, LSC_ERR_OUT_OF_RANGE);
    s_at[threadIdx.x] = in ? (int64_t)blk * L.page : -1;
    s_row[threadIdx.x] = pos - b * L.block_tokens;
  }
  const int32_t block0 = i * x.blocks + pos0 / kExpandTokens;
  if (threadIdx.x == 0 && pos0 % kExpandTokens == 0) x.table[block0] = block0;
  __syncthreads();
  const int32_t units = L.heads * L.head_dim / 8, all = 2 * n * units;  // of a row; of 8 elements
  const int64_t out0 = ((int64_t)block0 * kExpandTokens + pos0 % kExpandTokens) * units;
  for (int32_t j0 = threadIdx.x; j0 < all; j0 += kThreads * kUnroll) {
    uint32_t codes[kUnroll], byte[kUnroll];
    uint4 *dst[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int32_t j = j0 + u * kThreads;
      dst[u] = nullptr;
      codes[u] = byte[u] = 0;
      if (j >= all) continue;
      const int32_t r2 = x.by_units.div(j), e = j - r2 * units, r = r2 >= n ? r2 - n : r2;  // K's rows, then V's
      const int64_t at = s_at[r];
      const uint8_t *page = (r2 >= n ? L.v : L.k) + at;
      dst[u] = (uint4 *)(r2 >= n ? x.v : x.k) + out0 + (int64_t)r * units + e;
      if (at < 0) continue;
      codes[u] = __ldcs((const uint32_t *)(page + (int64_t)s_row[r] * (units * 4)) + e);
      byte[u] = __ldcs(page + L.scale_off + (int64_t)s_row[r] * (units / 2) + (e >> 1));
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (!dst[u]) continue;
      uint32_t h[4];
      e2m1x8_times(codes[u], e2m1_scale2(byte[u]), h);
      if (x.bf16) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[c]));
          h[c] = pack2(f.x, f.y, 1);
        }
      }
      *dst[u] = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}

}  // namespace

cudaError_t launch_kv_expand(const KvAttendParams &p, KvExpand x, cudaStream_t stream) {
  x.chunks = (p.max_kv + kRows - 1) / kRows;
  x.by_chunks.set((uint32_t)x.chunks);
  x.by_units.set((uint32_t)(p.L.heads * p.L.head_dim / 8));
  const cudaError_t e = launch_pdl(expand_kernel, p.b.n_seq * x.chunks, kThreads, 0, stream, p, x);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace lsc
