// lsc_kv_attend_join.cu -- joins the parts of cut units (lsc_kv_attend.cuh).
//
// For each run whose last unit goes on in other runs, a warp takes a row: its
// parts i have maximum m_i, sum l_i and unnormalised row o_i, and
//   m = max m_i,  l = sum 2^(m_i - m) l_i,  out = sum 2^(m_i - m) o_i / l,
// in the order of the tiles, so the result does not depend on timing.  It reads
// what the parts wrote (at most 2 M rows of D floats per run) once: a few us
// even for 152 runs of 256 rows.
#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_attend.cuh"
#include "lsc_kv_attend_chunk.cuh"
#include "lsc_kv_attend_decode.cuh"
#include "lsc_kv_attend_rows.cuh"
#include "lsc_ptx.h"

namespace lsc {
namespace {

using namespace kv;

constexpr int kWarps = 8;

// NV = float4 vectors of a row per lane, head_dim = 128 * NV (64: half the lanes)
template <int NV>
__global__ void __launch_bounds__(kWarps * 32) join_kernel(const __grid_constant__ KvAttendParams p, int ctas, int M, int together) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const Workspace w = workspace_at(p.ws, ctas, M);
  const int c = blockIdx.x, D = p.L.head_dim, ln = threadIdx.x & 31;
  const Cut cut = w.cut[c];
  if (cut.more == 0) return;
  const Seq s = attend_seq(p.L, p.b, cut.seq, p.max_seq, p.max_kv);
  const int r = blockIdx.y * kWarps + (threadIdx.x >> 5);
  const int MR = M / together, hr = r / MR;  // rows of a head; which head of the unit
  const int32_t R = cut.block * MR + r - hr * MR;
  if (r >= M || R >= s.n * p.group) return;
  auto part = [&](int i) { return i == 0 ? 2 * c + 1 : 2 * (c + i); };
  float m = -INFINITY;
  for (int i = ln; i <= cut.more; i += 32) m = fmaxf(m, w.ml[(int64_t)part(i) * M + r].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 acc[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i <= cut.more; ++i) {
    const int64_t at = (int64_t)part(i) * M + r;
    const float2 ml = w.ml[at];
    const float k = exp2f(ml.x - ref);
    l += ml.y * k;
    const float4 *src = (const float4 *)(w.o + at * D);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if ((ln + 32 * v) * 4 >= D) continue;
      const float4 x = src[ln + 32 * v];
      acc[v].x += k * x.x, acc[v].y += k * x.y, acc[v].z += k * x.z, acc[v].w += k * x.w;
    }
  }
  const int32_t tok = p.by_group.div(R);
  const bool empty = visible(s, tok, p.causal) == 0;
  const float inv = empty ? 0.f : 1.f / l;
  const int64_t t = s.row0 + tok, h = (int64_t)(cut.head * together + hr) * p.group + (R - tok * p.group);
  uint2 *dst = (uint2 *)((uint16_t *)p.out + t * p.out_stride + h * D);
  const int bf16 = p.dtype == LSC_BF16;
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if ((ln + 32 * v) * 4 < D)
      dst[ln + 32 * v] = make_uint2(pack2(acc[v].x * inv, acc[v].y * inv, bf16), pack2(acc[v].z * inv, acc[v].w * inv, bf16));
  if (p.lse && ln == 0) p.lse[t * p.heads + h] = empty ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

}  // namespace

cudaError_t launch_kv_attend_join(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  const dim3 grid(plan.ctas, (plan.M + kWarps - 1) / kWarps);
  const cudaError_t e = p.L.head_dim <= 128
                            ? launch_pdl(join_kernel<1>, grid, kWarps * 32, 0, stream, p, plan.ctas, plan.M, plan.together)
                            : launch_pdl(join_kernel<2>, grid, kWarps * 32, 0, stream, p, plan.ctas, plan.M, plan.together);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

AttendPlan plan_kv_attend_rows(const KvAttendParams &p) {
  using namespace kv::rows;
  const int D = p.L.head_dim, q8 = p.L.dtype == LSC_E4M3;
  AttendPlan plan{};
  plan.together = 1;
  plan.TK = kTK;
  plan.M = (int64_t)p.max_seq * p.group <= 16 ? 16 : 64;
  const int occ = q8 ? (D == 64 ? occ_of<1, 64>(plan.M) : D == 128 ? occ_of<1, 128>(plan.M) : occ_of<1, 256>(plan.M))
                     : (D == 64 ? occ_of<2, 64>(plan.M) : D == 128 ? occ_of<2, 128>(plan.M) : occ_of<2, 256>(plan.M));
  const int64_t tiles = ((int64_t)p.max_kv + kTK - 1) / kTK;
  const int64_t units = (int64_t)p.b.n_seq * p.L.heads, most = units * (tiles < 1 ? 1 : tiles);
  plan.may_cut = tiles > 1;
  plan.min_run = 1;
  plan.ctas = (int)(most < (int64_t)p.num_sms * occ ? most : (int64_t)p.num_sms * occ);
  plan.ws_bytes = plan.may_cut ? kv::workspace_size(plan.ctas, plan.M, D) : 0;
  return plan;
}

AttendPlan plan_kv_attend_decode(const KvAttendParams &p, bool side_by_side) {
  using namespace kv::decode;
  const int D = p.L.head_dim, q8 = p.L.dtype == LSC_E4M3;
  AttendPlan plan{};
  plan.TK = kTK;
  // Heads that lie side by side in a row are read side by side, up to 1 KB of them: 128 bytes at a time left the memory
  // at 61 % of the copy rate.  Not where that would leave CTAs without a tile: one sequence of 1001 tokens over 2 heads
  // took 17 us on 32 CTAs and 22 on 16.
  const int row = D * (q8 ? 1 : 2), H = p.L.heads;
  plan.together = !side_by_side ? 1 : H % 4 == 0 && row <= 256 ? 4 : H % 2 == 0 && row <= 512 ? 2 : 1;
  if ((int64_t)p.b.n_seq * (H / plan.together) * p.max_kv < (int64_t)p.num_sms * 4 * kTK) plan.together = 1;
  plan.M = ((int64_t)p.max_seq * p.group <= 8 ? 8 : 16) * plan.together;
  const int occ = q8 ? (D == 64 ? Conf<1, 64>::occ : D == 128 ? Conf<1, 128>::occ : Conf<1, 256>::occ)
                     : (D == 64 ? Conf<2, 64>::occ : D == 128 ? Conf<2, 128>::occ : Conf<2, 256>::occ);
  const int64_t tiles = ((int64_t)p.max_kv + kTK - 1) / kTK;
  const int64_t units = (int64_t)p.b.n_seq * (H / plan.together), most = units * (tiles < 1 ? 1 : tiles);
  plan.may_cut = tiles > 1;
  plan.min_run = 1;
  plan.ctas = (int)(most < (int64_t)p.num_sms * occ ? most : (int64_t)p.num_sms * occ);
  plan.ws_bytes = plan.may_cut ? kv::workspace_size(plan.ctas, plan.M, D) : 0;
  return plan;
}

cudaError_t launch_kv_attend_decode(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  const cudaError_t e = p.L.dtype == LSC_E4M3   ? launch_kv_attend_decode_e4m3(p, plan, stream)
                        : p.L.dtype == LSC_BF16 ? launch_kv_attend_decode_bf16(p, plan, stream)
                                                : launch_kv_attend_decode_f16(p, plan, stream);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_kv_attend_rows(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  const cudaError_t e = p.L.dtype == LSC_E4M3   ? launch_kv_attend_rows_e4m3(p, plan, stream)
                        : p.L.dtype == LSC_BF16 ? launch_kv_attend_rows_bf16(p, plan, stream)
                                                : launch_kv_attend_rows_f16(p, plan, stream);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

constexpr int kWhole = 8, kMinRun = 4, kLead = 4;  // in tiles of 128 positions

AttendPlan plan_kv_attend_chunk(const KvAttendParams &p) {
  using namespace kv::chunk;
  const int D = p.L.head_dim, TK = D == 256 ? Conf<256, false>::TK : Conf<128, false>::TK;
  AttendPlan plan{};
  plan.together = 1;
  plan.TK = TK;
  plan.M = D == 256 ? Conf<256, false>::M : Conf<128, false>::M;
  const int64_t tiles = ((int64_t)p.max_kv + TK - 1) / TK;
  const int64_t units = (((int64_t)p.b.total_tokens * p.group + plan.M - 1) / plan.M + p.b.n_seq) * p.L.heads;
  // Uncut up to kWhole tiles of 128 positions: at 5 tiles a unit, 256 rows of 128, cutting each over 5 CTAs took 33 us
  // and leaving them whole 25.
  plan.may_cut = tiles > kWhole * 128 / TK;
  plan.min_run = plan.may_cut ? kMinRun * 128 / TK : 1;
  // A unit's queries, its first tile on the way through empty pipes, its clearing of v and its result took 15000 cycles,
  // ten tiles of 64 at head_dim 256: with tiles alone counted, runs of many short units took up to twice the time of the
  // others.  Counted as 0, 256, 512 and 1024 positions: bf16, 24 sequences of 1 to 2048 tokens behind up to 8192, 818,
  // 740, 690 and 684 us; E4M3, 8 of 64 to 2048 behind up to 16384, 1515, 1177, 1004 and 1045.
  plan.lead = plan.may_cut ? kLead * 128 / TK : 0;
  const int64_t most = plan.may_cut ? units * tiles / plan.min_run + 1 : units;
  plan.ctas = (int)(most < p.num_sms ? most : p.num_sms);
  plan.ws_bytes = plan.may_cut ? kv::workspace_size(plan.ctas, plan.M, D) : 0;
  return plan;
}

cudaError_t launch_kv_attend_chunk(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  const cudaError_t e = p.L.dtype == LSC_E4M3   ? launch_kv_attend_chunk_e4m3(p, plan, stream)
                        : p.L.dtype == LSC_BF16 ? launch_kv_attend_chunk_bf16(p, plan, stream)
                                                : launch_kv_attend_chunk_f16(p, plan, stream);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace lsc
