// lsc_kv_attend_any.cu -- attention over a layer of the K/V block pool on the
// CUDA cores: the form of lsc_kv_attend (include/lsc_kv.h) for the types, head
// sizes and alignments that the tensor-core kernels do not take.
//
// A CTA takes one (token, q head) row.  Its warps take the visible positions in
// groups of kKeys in turn; a warp's lanes hold the row of q and their share of
// the weighted sum, d = lane + 32 i, and a score is a shuffle sum.  Each warp
// keeps the running maximum m and the sum l of 2^(s - m) of the positions it
// has seen (s already times log2 e); at the end the warps' parts are joined in
// warp order.  fp32 throughout.  K and V are read once a q head, mostly from L2; the
// shuffles bound it: 16 bf16 tokens behind 64 to 16384, 16 q heads, 2 heads of 80, take
// 4.3 ms.
#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_batch.cuh"
#include "lsc_ptx.h"

namespace lsc {
namespace {

using namespace kv;

constexpr int kWarps = 4;
constexpr int kKeys = 4;   // positions a warp works on at once
constexpr int kMaxD = 512;

__device__ __forceinline__ float load_el(const void *p, int64_t i, int dtype) {
  switch (dtype) {
    case LSC_F32: return ((const float *)p)[i];
    case LSC_BF16: return __bfloat162float(((const __nv_bfloat16 *)p)[i]);
    case LSC_F16: return __half2float(((const __half *)p)[i]);
    default: return e4m3x2_to_float2(((const uint8_t *)p)[i]).x;
  }
}
// Element i of a pool block; E4M3 without its scale.
__device__ __forceinline__ float load_row(const KvLayer &L, const uint8_t *page, int64_t i) {
  return L.dtype == LSC_E2M1 ? e2m1_element(page, L.scale_off, i) : load_el(page, i, L.dtype);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// NE = elements of a row per lane, head_dim <= 32 * NE
template <int NE>
__global__ void __launch_bounds__(kWarps * 32) attend_any_kernel(const __grid_constant__ KvAttendParams p) {
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][32 * NE];
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const KvLayer &L = p.L;
  if (blockIdx.x == 0) check_cu(L, p.b);
  const int warp = threadIdx.x >> 5, ln = threadIdx.x & 31, D = L.head_dim;
  const int64_t units = (int64_t)p.b.total_tokens * p.heads;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int32_t t = (int32_t)(u / p.heads), h = (int32_t)(u - (int64_t)t * p.heads);
    const int32_t i = seq_of_row(p.b, t);
    if (i < 0) continue;  // the whole CTA
    const Seq s = attend_seq(L, p.b, i, p.max_seq, p.max_kv);
    if (t - s.row0 >= s.n) continue;  // a sequence with lengths that were recorded: its rows stay as they are
    const int32_t vis = visible(s, t - s.row0, p.causal), kh = p.by_group.div(h);
    const int32_t *table = p.b.table + (int64_t)i * p.b.max_blocks;
    float q[NE], o[NE], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < NE; ++e) {
      const int d = ln + 32 * e;
      q[e] = d < D ? load_el(p.q, (int64_t)t * p.q_stride + (int64_t)h * D + d, p.dtype) * p.scale_log2 : 0.f;
      o[e] = 0.f;
    }
    for (int32_t j0 = warp * kKeys; j0 < vis; j0 += kWarps * kKeys) {
      int64_t at[kKeys];
      float sc[kKeys], vs[kKeys];
#pragma unroll
      for (int c = 0; c < kKeys; ++c) {
        at[c] = -1;
        sc[c] = 0.f;
        vs[c] = 1.f;
        const int32_t j = j0 + c;
        if (j < vis) {
          const int32_t jb = L.by_block.div(j), blk = table[jb], row = j - jb * L.block_tokens;
          if (blk >= 0 && blk < L.num_blocks) {
            const uint8_t *page = L.k + (int64_t)blk * L.page;
            at[c] = (int64_t)blk * L.page;
#pragma unroll
            for (int e = 0; e < NE; ++e)
              if (ln + 32 * e < D)
                sc[c] += q[e] * load_row(L, page, ((int64_t)row * L.heads + kh) * D + ln + 32 * e);
            if (L.dtype == LSC_E4M3) {
              const int64_t so = L.scale_off + (int64_t)row * L.heads + kh;
              sc[c] *= scale_of(page[so]);
              vs[c] = scale_of(L.v[at[c] + so]);
            }
          } else {
            report(L.status, LSC_ERR_OUT_OF_RANGE);
          }
        }
      }
      float top = m;
#pragma unroll
      for (int c = 0; c < kKeys; ++c) {
        sc[c] = warp_sum(sc[c]);
        if (at[c] < 0) sc[c] = -INFINITY;
        top = fmaxf(top, sc[c]);
      }
      const float ref = top == -INFINITY ? 0.f : top, keep = exp2f(m - ref);
      m = top;
      l *= keep;
#pragma unroll
      for (int e = 0; e < NE; ++e) o[e] *= keep;
#pragma unroll
      for (int c = 0; c < kKeys; ++c) {
        if (at[c] < 0) continue;
        const float w = exp2f(sc[c] - ref);
        l += w;
        const int32_t j = j0 + c, row = j - L.by_block.div(j) * L.block_tokens;
#pragma unroll
        for (int e = 0; e < NE; ++e)
          if (ln + 32 * e < D)
            o[e] += w * vs[c] * load_row(L, L.v + at[c], ((int64_t)row * L.heads + kh) * D + ln + 32 * e);
      }
    }
    __syncthreads();  // the last row's parts have been read
    if (ln == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int e = 0; e < NE; ++e) s_o[warp][ln + 32 * e] = o[e];
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += s_l[w] * exp2f(s_m[w] - ref);
    const bool empty = vis == 0;
    const float inv = empty ? 0.f : 1.f / sum;
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) x += s_o[w][d] * exp2f(s_m[w] - ref);
      x = empty ? 0.f : x * inv;
      const int64_t y = (int64_t)t * p.out_stride + (int64_t)h * D + d;
      if (p.dtype == LSC_F32) ((float *)p.out)[y] = x;
      else if (p.dtype == LSC_BF16) ((__nv_bfloat16 *)p.out)[y] = __float2bfloat16_rn(x);
      else ((__half *)p.out)[y] = __float2half_rn(x);
    }
    if (p.lse && threadIdx.x == 0)
      p.lse[(int64_t)t * p.heads + h] = empty ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
  }
}

}  // namespace

cudaError_t launch_kv_attend_any(const KvAttendParams &p, cudaStream_t stream) {
  const int64_t units = (int64_t)p.b.total_tokens * p.heads;
  const int64_t most = (int64_t)p.num_sms * 16;  // kWarps-warp CTAs an SM can hold
  const int grid = (int)(units < most ? units : most);
  const int ne = (p.L.head_dim + 31) / 32;
  cudaError_t e;
  if (ne <= 2) e = launch_pdl(attend_any_kernel<2>, grid, kWarps * 32, 0, stream, p);
  else if (ne <= 4) e = launch_pdl(attend_any_kernel<4>, grid, kWarps * 32, 0, stream, p);
  else if (ne <= 8) e = launch_pdl(attend_any_kernel<8>, grid, kWarps * 32, 0, stream, p);
  else e = launch_pdl(attend_any_kernel<kMaxD / 32>, grid, kWarps * 32, 0, stream, p);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace lsc
