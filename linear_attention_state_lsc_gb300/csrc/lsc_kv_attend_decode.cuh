// lsc_kv_attend_decode.cuh -- attention over a layer of the K/V block pool for
// sequences of up to 16 packed rows (lsc_kv_attend.cuh): decode steps.
//
// K and V are read once, so HBM bounds it.  The products run transposed, S^T = K Q^T
// and O^T = V^T P^T, as m16n8k16 tiles of mma.sync with positions and columns in the
// 16 and the packed rows in the 8: the usual 8 or fewer rows fill a tile (with rows
// in the 16, half of each product went to padding and 64 products a sub-tile were
// what bounded it), and scores, weights and sums stay in registers.  tcgen05 would
// want 128 rows and a trip through TMEM each way.  What matters is that nothing
// holds up the stream: a first version with block-wide tiles and cp.async spent
// 1420 of a tile's 3300 cycles in the copies' issue and another 700 in barriers
// (75 % of the copy rate).  So each of the four warps works alone: it takes one of
// the unit's 4, 2 or 1 kv heads and every 1st, 2nd or 4th sub-tile of KEYS
// positions of the CTA's run, loads it with tiled TMA
// into a ring of its own (boxes through the block table, swizzled rows, so
// ldmatrix meets no bank twice), and keeps its own running maximum, sum and
// weighted rows of all columns; scores become the weights' operand without leaving
// the registers (a transposition of 8 x 8 each).  The warps meet at the end of a piece, where a head's parts are
// joined in order.  The maximum is a reference that moves only when a row's
// maximum rose by more than 2^8 (bf16 weights are 2^8 at most; f16 ones, whose smallest
// is 2^-24, take the room up to 2^15), so the weighted rows are rarely rescaled.  Measured, 16 q heads, 64 tokens behind 64 to 16384, bf16, 2 heads of 256:
// 1018 MB in 160 us (6.4 TB/s, 95 % of a copy's rate); E4M3, 32 q heads, 128 tokens
// behind 500 to 8000, 8 heads of 128: 1060 MB in 178 us (6.0 TB/s, 89 %).
//
// E4M3 pools: codes go to f16 exactly (one conversion per two codes), so the
// products run in f16; K's scale multiplies the scores.  V's scale 2^e joins the
// weight: the reference is that of s + e, the weight 2^(s + e - m) is rounded to
// f16 relative to the largest contribution, and the sum takes 2^(s - m).  q's rows
// are brought to [1, 2) by a power of two that the scores take back, so bf16 q
// loses nothing that counts in f16.
//
// Positions that only some rows see: see lsc_kv_attend_rows.cuh.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_attend.cuh"
#include "lsc_kv_attend_rows.cuh"
#include "lsc_ptx.h"

namespace lsc {
namespace kv {
namespace decode {

using rows::ldsm4;
using rows::ldsm4t;
using rows::mma;

constexpr int kTK = 64;       // positions of a tile, what runs are cut in
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

template <int ES, int D>
struct Conf {
  static constexpr int RB = D * ES;                    // bytes of a row
  static constexpr int KEYS = kv_decode_keys(D, ES);   // positions of a sub-tile
  static constexpr int half = KEYS * RB;               // bytes of its K or V rows
  static constexpr int ST = half >= 4096 ? 3 : 6;      // sub-tiles in flight per warp
  static constexpr int occ = half >= 8192 ? 1 : 2;     // CTAs per SM: 192 KB of rings
};

template <int ES, int D>
struct Smem {
  using C = Conf<ES, D>;
  alignas(1024) uint8_t ring[kWarps][C::ST][2][C::half];  // at a piece's end: the warps' weighted rows
  float2 ml[kWarps][16];
  int32_t vis[16];
  int32_t bad[ES == 1 ? 1 : kWarps][ES == 1 ? 1 : 3][ES == 1 ? 1 : D];  // by head of the unit
  int32_t any_bad;
  uint64_t full[kWarps][C::ST];
  RunScratch run;
};

// An 8 x 8 matrix of 16-bit values over the lanes (row g, columns 2 tq, 2 tq + 1), transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <bool BF16, int ES, int D, int NR>
__global__ void __launch_bounds__(kThreads, (Conf<ES, D>::occ))
decode_attend_kernel(const __grid_constant__ KvAttendParams p, const __grid_constant__ CUtensorMap map, int together) {
  using C = Conf<ES, D>;
  constexpr bool Q8 = ES == 1;
  constexpr int M = 8 * NR;         // rows of a head, NR tiles of 8
  constexpr int KEYS = C::KEYS, ST = C::ST, RB = C::RB, LINE = RB < 128 ? RB : 128;
  constexpr int KS = D / 16;        // k steps of a score, output tiles of 16 columns
  constexpr int NK = KEYS / 16;     // score tiles of 16 positions
  constexpr float lift = BF16 ? 0.f : 7.f;  // powers of two that the reference lies below the maximum that set it
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<ES, D> &sm = *reinterpret_cast<Smem<ES, D> *>(smem_raw);
  const int tid = threadIdx.x, w = tid >> 5, ln = tid & 31, g = ln >> 2, tq = ln & 3;
  if (tid < kWarps * ST) mbar_init(&sm.full[tid / ST][tid % ST], 1);
  fence_mbar_init();
  griddep_wait();
  if (tid == 0) griddep_launch_dependents();
  const KvLayer &L = p.L;
  const int ctas = gridDim.x, cta = blockIdx.x;
  if (cta == 0) check_cu(L, p.b);
  const int MU = M * together, splits = kWarps / together;  // rows of a unit; warps of a head
  const int wh = w & (together - 1), wsp = w / together;    // this warp's head of the unit, its share of the sub-tiles
  const Workspace ws = workspace_at(p.ws, ctas, MU);
  if (tid == 0) sm.any_bad = 0;
  if (!Q8)
    for (int i = tid; i < kWarps * 3 * D; i += kThreads) (&sm.bad[0][0][0])[i] = INT32_MAX;
  Run run = find_run<kThreads, M, kTK>(p, cta, ctas, sm.run);
  Piece pc;
  Cut cut = {0, 0, 0, 0};
  bool ok = true;
  // TMA boxes: `box` rows and all columns of 128 bytes when that is a sub-tile, else one column; K's on lanes 0-15, V's
  // on 16-31
  const int box = p.box_decode, per = box == KEYS ? 1 : (RB + 127) / 128, boxes = KEYS / box * per;
  const int bi = ln & 15, bc = bi % per, br = bi < boxes ? bi / per * box : 0;
  uint8_t *const ring = sm.ring[w][0][0];
  int slot = 0;
  uint32_t phase = 0;
  __syncthreads();
  while (ok && next_piece<M, kTK>(p, run, pc)) {
    const int R = pc.s.n * p.group < M ? pc.s.n * p.group : M;  // this launch's units have one block
    const int32_t kv = pc.s.kv, lo = pc.t0 * kTK, hi = kv < pc.t1 * kTK ? kv : pc.t1 * kTK;
    const int32_t *table = p.b.table + (int64_t)pc.seq * p.b.max_blocks;
    const int nsub = hi > lo ? (hi - lo + KEYS - 1) / KEYS : 0, mine = nsub > wsp ? (nsub - wsp + splits - 1) / splits : 0, head = pc.head * together + wh;
    // Block of a position, 0 behind the last one.  Looked up a sub-tile ahead and checked only where it is used (a bad
    // one is recorded and read as 0): a look at it any earlier would wait for the load.
    auto block_at = [&](int32_t pos) { return pos < kv ? __ldg(table + L.by_block.div(pos)) : 0; };
    auto checked = [&](int32_t blk) {
      if ((uint32_t)blk < (uint32_t)L.num_blocks) return blk;
      report(L.status, LSC_ERR_OUT_OF_RANGE);
      return 0;
    };
    auto first_of = [&](int i) { return lo + (i * splits + wsp) * KEYS; };  // first position of this warp's sub-tile i
    auto issue = [&](int i, int st, int32_t blk) {
      const int32_t pos = first_of(i) + br;
      blk = checked(blk);
      if (ln == 0) mbar_arrive_expect_tx(&sm.full[w][st], 2 * C::half);
      __syncwarp();
      if (bi < boxes)
        tma_box(ring + (st * 2 + (ln >> 4)) * C::half + bc * (KEYS * 128) + br * (RB < 128 ? RB : 128), &map,
                pos - L.by_block.div(pos) * L.block_tokens, bc, head, blk + (ln < 16 ? 0 : L.num_blocks),
                &sm.full[w][st]);
    };
    // E4M3: lane i's scale bytes of position i of a sub-tile, 127 behind the last one
    auto scales = [&](int i, int32_t blk, uint32_t &kb, uint32_t &vb) {
      const int32_t pos = first_of(i) + ln;
      kb = vb = 127;
      if (Q8 && i < mine && pos < hi) {
        const int64_t at = (int64_t)checked(blk) * L.page + L.scale_off +
                           (int64_t)(pos - L.by_block.div(pos) * L.block_tokens) * L.heads + head;
        kb = __ldg(L.k + at);
        vb = __ldg(L.v + at);
      }
    };
    int st_in = slot;
#pragma unroll
    for (int i = 0; i < ST; ++i)
      if (i < mine) {
        issue(i, st_in, block_at(first_of(i) + br));
        if (++st_in == ST) st_in = 0;
      }
    int32_t next_blk = ST < mine ? block_at(first_of(ST) + br) : 0;
    uint32_t kb_next, vb_next;
    int32_t blk_scale = 0;
    scales(0, Q8 && mine > 0 ? block_at(first_of(0) + ln) : 0, kb_next, vb_next);
    if (Q8 && mine > 1) blk_scale = block_at(first_of(1) + ln);

    if (tid < M) sm.vis[tid] = tid < R ? visible(pc.s, p.by_group.div(tid), p.causal) : 0;
    // q as operand registers: row g of each 8.  16 bits: elements 2 tq, 2 tq + 1 and 8 further of each 16.  E4M3: a lane
    // meets 4 consecutive codes, so it holds elements 4 tq .. 4 tq + 3, as f16 times a power of two.
    uint32_t qf[NR][KS][2];
    float q_up[NR];  // of row g: scale * log2 e, times that power
#pragma unroll
    for (int h = 0; h < NR; ++h) {
      const int r = 8 * h + g, tok = p.by_group.div(r);
      const uint16_t *src = (const uint16_t *)p.q + (int64_t)(pc.s.row0 + tok) * p.q_stride +
                            (int64_t)(head * p.group + (r - tok * p.group)) * D;
      q_up[h] = p.scale_log2;
      if constexpr (!Q8) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qf[h][k][0] = r < R ? *(const uint32_t *)(src + k * 16 + 2 * tq) : 0;
          qf[h][k][1] = r < R ? *(const uint32_t *)(src + k * 16 + 8 + 2 * tq) : 0;
        }
      } else {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const uint2 x = r < R ? *(const uint2 *)(src + k * 16 + 4 * tq) : make_uint2(0, 0);
          qf[h][k][0] = x.x, qf[h][k][1] = x.y;
          // magnitudes of 16-bit floats order as whole numbers
          top = __vmaxu2(top, __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu));
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const bool bf = p.dtype == LSC_BF16;
        const uint32_t f = __float_as_uint(bf ? __uint_as_float(top << 16) : __half2float(__ushort_as_half((uint16_t)top)));
        const uint32_t ex = f >> 23;  // 2^k <= the largest magnitude < 2^(k + 1), where that is a normal number
        const bool plain = ex == 0 || ex == 255;
        const float down = plain ? 1.f : inv_scale_of(ex);
        if (!plain) q_up[h] *= __uint_as_float(ex << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t b = qf[h][k][e];
            const float lo16 = bf ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((uint16_t)b));
            const float hi16 = bf ? __uint_as_float(b & 0xffff0000u) : __half2float(__ushort_as_half((uint16_t)(b >> 16)));
            qf[h][k][e] = pack2(lo16 * down, hi16 * down, 0);
          }
      }
    }
    // scores come with rows 2 tq, 2 tq + 1 of each 8
    float qsc[NR][2];
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) qsc[h][e] = __shfl_sync(0xffffffffu, q_up[h], (2 * tq + e) * 4);
    __syncthreads();  // vis; and the last piece's shared memory is free
    const int32_t sure = visible(pc.s, 0, p.causal);  // every row sees positions below this
    int32_t vis[NR][2];
    float m[NR][2], l[NR][2], o[NR][KS][4];
#pragma unroll
    for (int h = 0; h < NR; ++h) {
#pragma unroll
      for (int e = 0; e < 2; ++e) vis[h][e] = sm.vis[8 * h + 2 * tq + e], m[h][e] = -INFINITY, l[h][e] = 0.f;
#pragma unroll
      for (int n = 0; n < KS; ++n) o[h][n][0] = o[h][n][1] = o[h][n][2] = o[h][n][3] = 0.f;
    }

    int i = 0;
#pragma unroll 1
    for (; i < mine; ++i) {
      const int32_t first = first_of(i);
      const uint32_t kb_now = kb_next;
      uint32_t vb_now = vb_next;
      if constexpr (Q8) {
        scales(i + 1, blk_scale, kb_next, vb_next);
        blk_scale = i + 2 < mine ? block_at(first_of(i + 2) + ln) : 0;
      }
      if (!(ok = wait_warp(&sm.full[w][slot], phase, p.wait_limit_ns))) break;
      uint8_t *ks = ring + slot * 2 * C::half, *vs = ks + C::half;
      const uint32_t ka = smem_u32(ks), va = smem_u32(vs);
      if (first + KEYS > hi || first + KEYS > sure) {  // (some of) V's rows need a look before they meet a weight of 0
        const int past = hi - first < KEYS ? hi - first : KEYS, from = sure > first ? sure - first : 0;
        for (int x = past * (RB / 16) + ln; x < KEYS * (RB / 16); x += 32)
          *(uint4 *)(vs + chunk_at<LINE>(KEYS, x / (RB / 16), x % (RB / 16))) = make_uint4(0, 0, 0, 0);
        if constexpr (Q8) {
          bool nan = false;
          if (ln >= from && ln < past)
            for (int c = 0; c < RB / 16; ++c) {
              uint32_t *v = (uint32_t *)(vs + chunk_at<LINE>(KEYS, ln, c));
              for (int y = 0; y < 4; ++y)
                for (int z = 0; z < 32; z += 8)
                  if ((v[y] >> z & 0x7f) == 0x7f) nan = true, v[y] &= ~(0xffu << z);
            }
          if (nan) vb_now = 255;
        } else {
          constexpr uint32_t E = BF16 ? 0x7f80 : 0x7c00;
          for (int x = from * D + ln; x < past * D; x += 32) {
            const int key = x / D, d = x % D;
            uint16_t *v = (uint16_t *)(vs + chunk_at<LINE>(KEYS, key, d >> 3) + (d & 7) * 2);
            const uint32_t u = *v;
            if ((u & E) != E) continue;
            atomicMin(&sm.bad[wh][(u & (E ^ 0x7fff)) ? 0 : (u & 0x8000) ? 2 : 1][d], first + key);
            sm.any_bad = 1;
            *v = 0;
          }
        }
        fence_proxy_async_smem();  // before the box that lands here next
        __syncwarp();
      }
      // ---- scores: lane (g, tq) gets positions g, g + 8 of each 16 and rows 2 tq, 2 tq + 1 of each 8
      // (two sums a tile, all tiles in turn: a product waits some 30 cycles for the one before it in its sum)
      float s[NK][NR][4], s2[NK][NR][4];
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int h = 0; h < NR; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][h][e] = s2[n][h][e] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; k += 2)
#pragma unroll
        for (int n = 0; n < NK; ++n) {
          uint32_t x[2][4];
          if constexpr (Q8) {  // a chunk is a k step
            uint32_t b[4];
            ldsm4(b, ka + chunk_at<LINE>(KEYS, 16 * n + (ln & 15), k + (ln >> 4)));
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              x[y][0] = e4m3x2_to_f16x2(b[2 * y] & 0xffffu), x[y][1] = e4m3x2_to_f16x2(b[2 * y + 1] & 0xffffu);
              x[y][2] = e4m3x2_to_f16x2(b[2 * y] >> 16), x[y][3] = e4m3x2_to_f16x2(b[2 * y + 1] >> 16);
            }
          } else {
            ldsm4(x[0], ka + chunk_at<LINE>(KEYS, 16 * n + (ln & 15), 2 * k + (ln >> 4)));
            ldsm4(x[1], ka + chunk_at<LINE>(KEYS, 16 * n + (ln & 15), 2 * k + 2 + (ln >> 4)));
          }
#pragma unroll
          for (int h = 0; h < NR; ++h) {
            mma<BF16>(s[n][h], x[0], qf[h][k][0], qf[h][k][1]);
            mma<BF16>(s2[n][h], x[1], qf[h][k + 1][0], qf[h][k + 1][1]);
          }
        }
      // ---- weights
      float vx[NK][2];
      const float k_up = Q8 ? scale_of(kb_now) : 1.f, v_up = Q8 ? scale_of(vb_now) : 1.f;  // of position `lane`
      const float v_ex = Q8 ? v_exponent(vb_now) : 0.f;
      float top[NR][2];
#pragma unroll
      for (int h = 0; h < NR; ++h) top[h][0] = top[h][1] = -INFINITY;
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int key = 16 * n + 8 * y + g;
          float kx = 1.f, ve = 0.f;
          vx[n][y] = 1.f;
          if constexpr (Q8) {
            kx = __shfl_sync(0xffffffffu, k_up, key);
            vx[n][y] = __shfl_sync(0xffffffffu, v_up, key);
            ve = __shfl_sync(0xffffffffu, v_ex, key);
          }
#pragma unroll
          for (int h = 0; h < NR; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = (s[n][h][2 * y + e] + s2[n][h][2 * y + e]) * qsc[h][e];
              if constexpr (Q8) x *= kx;
              x = first + key < vis[h][e] ? x : -INFINITY;
              s[n][h][2 * y + e] = x;
              top[h][e] = fmaxf(top[h][e], x + ve);
            }
        }
      bool rise = false;
#pragma unroll
      for (int h = 0; h < NR; ++h) rise |= top[h][0] > m[h][0] + (8.f + lift) || top[h][1] > m[h][1] + (8.f + lift);
      if (__any_sync(0xffffffffu, rise)) {  // also the first one's (m is -inf)
#pragma unroll
        for (int h = 0; h < NR; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = top[h][e];
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            const float to = fmaxf(m[h][e], t - lift), f = ex2(m[h][e] - (to == -INFINITY ? 0.f : to));
            m[h][e] = to;
            l[h][e] *= f;
#pragma unroll
            for (int n = 0; n < KS; ++n) o[h][n][e] *= f, o[h][n][2 + e] *= f;
          }
      }
      uint32_t a[NK][NR][2];
#pragma unroll
      for (int h = 0; h < NR; ++h) {
        const float r0 = m[h][0] == -INFINITY ? 0.f : m[h][0], r1 = m[h][1] == -INFINITY ? 0.f : m[h][1];
#pragma unroll
        for (int n = 0; n < NK; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float p0 = ex2(s[n][h][2 * y] - r0), p1 = ex2(s[n][h][2 * y + 1] - r1);
            l[h][0] += p0;
            l[h][1] += p1;
            if constexpr (Q8) {  // a position that the row does not see has weight 0 whatever its scale
              const int key = first + 16 * n + 8 * y + g;
              p0 = key < vis[h][0] ? p0 * vx[n][y] : 0.f;
              p1 = key < vis[h][1] ? p1 * vx[n][y] : 0.f;
            }
            a[n][h][y] = transposed(pack2(p0, p1, BF16));
          }
      }
      // ---- V^T times weights
#pragma unroll
      for (int c = 0; c < KS; ++c) {  // 16 columns
        if constexpr (Q8) {  // a chunk of 32 positions; m index g: column 2 g, m index g + 8: column 2 g + 1
          uint32_t b[4];
          ldsm4t(b, va + chunk_at<LINE>(KEYS, ln, c));
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t x[4] = {e4m3x2_to_f16x2(__byte_perm(b[2 * n], 0, 0x20) & 0xffffu),
                                   e4m3x2_to_f16x2(__byte_perm(b[2 * n], 0, 0x31) & 0xffffu),
                                   e4m3x2_to_f16x2(__byte_perm(b[2 * n + 1], 0, 0x20) & 0xffffu),
                                   e4m3x2_to_f16x2(__byte_perm(b[2 * n + 1], 0, 0x31) & 0xffffu)};
#pragma unroll
            for (int h = 0; h < NR; ++h) mma<false>(o[h][c], x, a[n][h][0], a[n][h][1]);
          }
        } else {
#pragma unroll
          for (int n = 0; n < NK; ++n) {
            uint32_t x[4];
            ldsm4t(x, va + chunk_at<LINE>(KEYS, 16 * n + ((ln >> 4) << 3) + (ln & 7), 2 * c + ((ln >> 3) & 1)));
#pragma unroll
            for (int h = 0; h < NR; ++h) mma<BF16>(o[h][c], x, a[n][h][0], a[n][h][1]);
          }
        }
      }
      // ---- the slot's next sub-tile
      if (i + ST < mine) {
        __syncwarp();
        issue(i + ST, slot, next_blk);
        next_blk = i + ST + 1 < mine ? block_at(first_of(i + ST + 1) + br) : 0;
      }
      if (++slot == ST) slot = 0, phase ^= 1;
    }
    if (!ok) {  // nothing may be in flight when the CTA leaves: every slot that was filled
      for (int x = i; x < mine && x < i + ST; ++x) {
        wait_warp(&sm.full[w][slot], phase, p.drain_limit_ns);
        if (++slot == ST) slot = 0, phase ^= 1;
      }
      if (ln == 0) report(L.status, LSC_ERR_DEV_TIMEOUT);
    }
    // ---- the piece's end: the warps' parts through shared memory, then rows out or to the workspace
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[h][e] += __shfl_xor_sync(0xffffffffu, l[h][e], 4);
        l[h][e] += __shfl_xor_sync(0xffffffffu, l[h][e], 8);
        l[h][e] += __shfl_xor_sync(0xffffffffu, l[h][e], 16);
        if (g == 0) sm.ml[w][8 * h + 2 * tq + e] = make_float2(m[h][e], l[h][e]);
      }
    ok = __syncthreads_and(ok);
    if (!ok) break;
    // [row][column] of 32 bits, rows padded by 4 (D + 4: no bank twice in what follows); the rings are empty
    constexpr int PS = D + 4;
    static_assert(sizeof(sm.ring) >= (size_t)kWarps * 16 * PS * 4, "the parts fit");
    float *parts = (float *)sm.ring;
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * h + 2 * tq + e;
        if (r < R) {
          float *row = parts + (w * M + r) * PS;
#pragma unroll
          for (int n = 0; n < KS; ++n) {
            if constexpr (Q8) *(float2 *)(row + n * 16 + 2 * g) = make_float2(o[h][n][e], o[h][n][2 + e]);
            else row[n * 16 + g] = o[h][n][e], row[n * 16 + 8 + g] = o[h][n][2 + e];
          }
        }
      }
    __syncthreads();
    const bool whole = pc.t0 == 0 && pc.t1 == pc.tiles;
    const int64_t slot0 = (int64_t)(2 * cta + (pc.t0 == 0 ? 1 : 0)) * MU;
    const bool look = !Q8 && sm.any_bad != 0;
#pragma unroll 1
    for (int x = tid; x < together * M * (D / 4); x += kThreads) {
      const int hr = x / (D / 4), d = x % (D / 4) * 4, r = hr & (M - 1), hw = hr / M, tok = p.by_group.div(r);
      if (r >= R) continue;
      float mm = -INFINITY, sum = 0.f;
      for (int i = hw; i < kWarps; i += together) mm = fmaxf(mm, sm.ml[i][r].x);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = hw; i < kWarps; i += together) {
        const float2 ml = sm.ml[i][r];
        const float k = exp2f(ml.x - ref);
        const float4 z = *(const float4 *)(parts + (i * M + r) * PS + d);
        sum += ml.y * k;
        y.x += z.x * k, y.y += z.y * k, y.z += z.z * k, y.w += z.w * k;
      }
      const bool empty = sm.vis[r] == 0;
      const float inv = whole ? (empty ? 0.f : 1.f / sum) : 1.f;
      y.x *= inv, y.y *= inv, y.z *= inv, y.w *= inv;
      if constexpr (!Q8) {
        if (look) {
          float *v = &y.x;
          for (int e = 0; e < 4; ++e) {
            if (sm.bad[hw][1][d + e] < sm.vis[r]) v[e] += INFINITY;
            if (sm.bad[hw][2][d + e] < sm.vis[r]) v[e] -= INFINITY;
            if (sm.bad[hw][0][d + e] < sm.vis[r]) v[e] = __uint_as_float(0x7fc00000u);
          }
        }
      }
      const int64_t t = pc.s.row0 + tok, hd = (int64_t)(pc.head * together + hw) * p.group + (r - tok * p.group);
      if (whole) {
        const int bf = p.dtype == LSC_BF16;
        *(uint2 *)((uint16_t *)p.out + t * p.out_stride + hd * D + d) = make_uint2(pack2(y.x, y.y, bf), pack2(y.z, y.w, bf));
        if (d == 0 && p.lse) p.lse[t * p.heads + hd] = empty ? -INFINITY : (mm + log2f(sum)) * 0.693147180559945309f;
      } else {
        *(float4 *)(ws.o + (slot0 + hr) * D + d) = y;
        if (d == 0) ws.ml[slot0 + hr] = make_float2(mm, sum);
      }
    }
    cut = cut_of(run, pc, cta);
    fence_proxy_async_smem();  // the parts were written where the next piece's boxes land
    __syncthreads();
    if (look) {
      for (int i = tid; i < kWarps * 3 * D; i += kThreads) (&sm.bad[0][0][0])[i] = INT32_MAX;
      if (tid == 0) sm.any_bad = 0;
      __syncthreads();
    }
  }
  if (tid == 0 && p.ws) ws.cut[cta] = cut;
}

template <bool BF16, int ES, int D, int NR>
cudaError_t launch_one(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  static SmemLimit limit;
  const int smem = (int)sizeof(Smem<ES, D>);
  auto *k = decode_attend_kernel<BF16, ES, D, NR>;
  const cudaError_t e = limit.ensure((const void *)k, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, plan.ctas, kThreads, smem, stream, p, *p.map_decode, plan.together);
}

template <bool BF16, int ES, int D>
cudaError_t launch_rows(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  return plan.M == 8 * plan.together ? launch_one<BF16, ES, D, 1>(p, plan, stream)
                                     : launch_one<BF16, ES, D, 2>(p, plan, stream);
}

template <bool BF16, int ES>
cudaError_t launch_type(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  switch (p.L.head_dim) {
    case 64: return launch_rows<BF16, ES, 64>(p, plan, stream);
    case 128: return launch_rows<BF16, ES, 128>(p, plan, stream);
    default: return launch_rows<BF16, ES, 256>(p, plan, stream);
  }
}

}  // namespace decode
}  // namespace kv

cudaError_t launch_kv_attend_decode_bf16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
cudaError_t launch_kv_attend_decode_f16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
cudaError_t launch_kv_attend_decode_e4m3(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);

}  // namespace lsc
