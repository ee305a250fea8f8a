// lsc_kv_attend_decode.cuh -- attention over a layer of the K/V block pool for
// sequences of up to 16 packed rows (lsc_kv_attend.cuh): decode steps.
//
// K and V are read once, so HBM bounds it; 16 rows are one m16n8k16 tile of
// mma.sync, which keeps scores, weights and sums in registers, where tcgen05 would
// want 128 rows and a trip through TMEM each way.  What matters is that nothing
// holds up the stream: a first version with block-wide tiles and cp.async spent
// 1420 of a tile's 3300 cycles in the copies' issue and another 700 in barriers
// (75 % of the copy rate).  So each of the four warps works alone: it takes one of
// the unit's 4, 2 or 1 kv heads and every 1st, 2nd or 4th sub-tile of KEYS
// positions of the CTA's run, loads it with tiled TMA
// into a ring of its own (boxes through the block table, swizzled rows, so
// ldmatrix meets no bank twice), and keeps its own running maximum, sum and
// weighted rows of all columns; scores become the weights' operand without leaving
// the registers.  The warps meet at the end of a piece, where a head's parts are
// joined in order.  The maximum is a reference that moves only when a row's
// maximum rose by more than 2^8 (weights are 2^8 at most), so the weighted rows are
// rarely rescaled.
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
  float qs[16];
  int32_t vis[16];
  int32_t bad[ES == 1 ? 1 : kWarps][ES == 1 ? 1 : 3][ES == 1 ? 1 : D];  // by head of the unit
  int32_t any_bad;
  uint64_t full[kWarps][C::ST];
  RunScratch run;
};

// Byte of 16-byte chunk c of row r in a swizzled sub-tile of KEYS rows: columns of 128 bytes, chunks xor the row's low
// bits (rows of 64 bytes: pairs of rows share 128).
template <int RB, int KEYS>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (RB == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else return (c >> 3) * (KEYS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void tma_box(void *dst, const CUtensorMap *map, int row, int col, int head, int block,
                                        uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(0), "r"(row), "r"(col), "r"(head), "r"(block), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The first tries do without the clock (reading %globaltimer is slow); one answer for the whole warp.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t phase, uint64_t limit) {
  bool ok = limit != 0;
  if (ok) {
    ok = false;
    for (int i = 0; i < 16 && !ok; ++i) ok = mbar_try_wait(bar, phase & 1);
    if (!ok) ok = mbar_wait_bounded(bar, phase & 1, limit);
  }
  return __all_sync(0xffffffffu, ok);
}

template <bool BF16, int ES, int D>
__global__ void __launch_bounds__(kThreads, (Conf<ES, D>::occ))
decode_attend_kernel(const __grid_constant__ KvAttendParams p, const __grid_constant__ CUtensorMap map, int together) {
  using C = Conf<ES, D>;
  constexpr bool Q8 = ES == 1;
  constexpr int M = 16, KEYS = C::KEYS, ST = C::ST, RB = C::RB;
  constexpr int KS = D / 16;        // k steps of a score
  constexpr int NK = KEYS / 8;      // score tiles of 8 positions
  constexpr int NT = D / 8;         // output tiles of 8 columns
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
    // q as operand registers: rows g and g + 8.  16 bits: elements 2 tq, 2 tq + 1 and 8 further of each 16.  E4M3: a lane
    // meets 4 consecutive codes, so it holds elements 4 tq .. 4 tq + 3, as f16 times a power of two.
    uint32_t qf[KS][4];
    float qsc[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 8 * h + g, tok = p.by_group.div(r);
      const uint16_t *src = (const uint16_t *)p.q + (int64_t)(pc.s.row0 + tok) * p.q_stride +
                            (int64_t)(head * p.group + (r - tok * p.group)) * D;
      qsc[h] = p.scale_log2;
      if constexpr (!Q8) {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qf[k][h] = r < R ? *(const uint32_t *)(src + k * 16 + 2 * tq) : 0;
          qf[k][h + 2] = r < R ? *(const uint32_t *)(src + k * 16 + 8 + 2 * tq) : 0;
        }
      } else {
        uint2 x[KS];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          x[k] = r < R ? *(const uint2 *)(src + k * 16 + 4 * tq) : make_uint2(0, 0);
          // magnitudes of 16-bit floats order as whole numbers
          top = __vmaxu2(top, __vmaxu2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu));
        }
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const bool bf = p.dtype == LSC_BF16;
        const uint32_t f = __float_as_uint(bf ? __uint_as_float(top << 16) : __half2float(__ushort_as_half((uint16_t)top)));
        const uint32_t ex = f >> 23;  // 2^k <= the largest magnitude < 2^(k + 1), where that is a normal number
        const bool plain = ex == 0 || ex == 255;
        const float down = plain ? 1.f : inv_scale_of(ex);
        if (!plain) qsc[h] *= __uint_as_float(ex << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t b = (e < 2 ? x[k].x : x[k].y) >> (16 * (e & 1)) & 0xffffu;
            y[e] = (bf ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((uint16_t)b))) * down;
          }
          qf[k][h] = pack2(y[0], y[1], 0);
          qf[k][h + 2] = pack2(y[2], y[3], 0);
        }
      }
    }
    __syncthreads();  // vis; and the last piece's shared memory is free
    int32_t vis[2] = {sm.vis[g], sm.vis[g + 8]};
    const int32_t sure = visible(pc.s, 0, p.causal);  // every row sees positions below this
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

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
          *(uint4 *)(vs + chunk_at<RB, KEYS>(x / (RB / 16), x % (RB / 16))) = make_uint4(0, 0, 0, 0);
        if constexpr (Q8) {
          bool nan = false;
          if (ln >= from && ln < past)
            for (int c = 0; c < RB / 16; ++c) {
              uint32_t *v = (uint32_t *)(vs + chunk_at<RB, KEYS>(ln, c));
              for (int y = 0; y < 4; ++y)
                for (int z = 0; z < 32; z += 8)
                  if ((v[y] >> z & 0x7f) == 0x7f) nan = true, v[y] &= ~(0xffu << z);
            }
          if (nan) vb_now = 255;
        } else {
          constexpr uint32_t E = BF16 ? 0x7f80 : 0x7c00;
          for (int x = from * D + ln; x < past * D; x += 32) {
            const int key = x / D, d = x % D;
            uint16_t *v = (uint16_t *)(vs + chunk_at<RB, KEYS>(key, d >> 3) + (d & 7) * 2);
            const uint32_t u = *v;
            if ((u & E) != E) continue;
            atomicMin(&sm.bad[wh][(u & (E ^ 0x7fff)) ? 0 : (u & 0x8000) ? 2 : 1][d], first + key);
            sm.any_bad = 1;
            *v = 0;
          }
        }
        __syncwarp();
      }
      // ---- scores: lane (g, tq) gets rows g, g + 8 and positions 2 tq, 2 tq + 1 of each 8
      // (two sums a tile, all tiles in turn: a product waits some 30 cycles for the one before it in its sum)
      float s[NK][4], s2[NK][4];
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = s2[n][e] = 0.f;
      constexpr int PER = Q8 ? 4 : 2;  // k steps per ldmatrix.x4
#pragma unroll
      for (int k0 = 0; k0 < KS; k0 += PER)
#pragma unroll
        for (int n = 0; n < NK; ++n) {
          uint32_t b[4];
          ldsm4(b, ka + chunk_at<RB, KEYS>(8 * n + (ln & 7), k0 * 2 / (Q8 ? 2 : 1) + (ln >> 3)));
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            float(&c)[4] = k & 1 ? s2[n] : s[n];
            if constexpr (Q8) mma<false>(c, qf[k0 + k], e4m3x2_to_f16x2(b[k] & 0xffffu), e4m3x2_to_f16x2(b[k] >> 16));
            else mma<BF16>(c, qf[k0 + k], b[2 * k], b[2 * k + 1]);
          }
        }
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] += s2[n][e];
      // ---- weights
      float vx[Q8 ? NK : 1][2];
      const float k_up = Q8 ? scale_of(kb_now) : 1.f, v_up = Q8 ? scale_of(vb_now) : 1.f;  // of position `lane`
      // bounds keep the sum of 2^(s - m) a normal number
      const float v_ex = Q8 ? (float)(vb_now < 87 ? -40 : vb_now > 227 ? 100 : (int)vb_now - 127) : 0.f;
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = 8 * n + 2 * tq + e;
          float kx = 1.f, ve = 0.f;
          if constexpr (Q8) {
            kx = __shfl_sync(0xffffffffu, k_up, key);
            vx[n][e] = __shfl_sync(0xffffffffu, v_up, key);
            ve = __shfl_sync(0xffffffffu, v_ex, key);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = s[n][2 * h + e] * qsc[h];
            if constexpr (Q8) x *= kx;
            x = first + key < vis[h] ? x : -INFINITY;
            s[n][2 * h + e] = x;
            top[h] = fmaxf(top[h], x + ve);
          }
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
      }
      if (__any_sync(0xffffffffu, top[0] > m[0] + 8.f || top[1] > m[1] + 8.f)) {  // also the first one's (m is -inf)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float to = fmaxf(m[h], top[h]), f = ex2(m[h] - (to == -INFINITY ? 0.f : to));
          m[h] = to;
          l[h] *= f;
#pragma unroll
          for (int n = 0; n < NT; ++n) o[n][2 * h] *= f, o[n][2 * h + 1] *= f;
        }
      }
      uint32_t a[NK / 2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ref = m[h] == -INFINITY ? 0.f : m[h];
#pragma unroll
        for (int n = 0; n < NK; ++n) {
          const float p0 = ex2(s[n][2 * h] - ref), p1 = ex2(s[n][2 * h + 1] - ref);
          l[h] += p0 + p1;
          // a position that the row does not see has weight 0 whatever its scale
          const int key = first + 8 * n + 2 * tq;
          const float w0 = Q8 ? (key < vis[h] ? p0 * vx[Q8 ? n : 0][0] : 0.f) : p0;
          const float w1 = Q8 ? (key + 1 < vis[h] ? p1 * vx[Q8 ? n : 0][1] : 0.f) : p1;
          a[n >> 1][h + 2 * (n & 1)] = pack2(w0, w1, BF16);
        }
      }
      // ---- weights times V
#pragma unroll
      for (int y = 0; y < NK / 2; y += Q8 ? 2 : 1) {
        if constexpr (Q8) {  // 32 positions; 16 columns a chunk, the even ones in one output tile, the odd ones in the next
#pragma unroll
          for (int c = 0; c < RB / 16; ++c) {
            uint32_t b[4];
            ldsm4t(b, va + chunk_at<RB, KEYS>(y * 16 + ln, c));
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
              for (int odd = 0; odd < 2; ++odd) {
                const uint32_t sel = odd ? 0x31 : 0x20;
                mma<false>(o[2 * c + odd], a[y + z], e4m3x2_to_f16x2(__byte_perm(b[2 * z], 0, sel) & 0xffffu),
                           e4m3x2_to_f16x2(__byte_perm(b[2 * z + 1], 0, sel) & 0xffffu));
              }
          }
        } else {  // 16 positions, two chunks of 8 columns a load
#pragma unroll
          for (int c = 0; c < RB / 16; c += 2) {
            uint32_t b[4];
            ldsm4t(b, va + chunk_at<RB, KEYS>(y * 16 + (ln & 15), c + (ln >> 4)));
            mma<BF16>(o[c], a[y], b[0], b[1]);
            mma<BF16>(o[c + 1], a[y], b[2], b[3]);
          }
        }
      }
      // ---- the slot's next sub-tile
      if (i + ST < mine) {
        fence_proxy_async_smem();
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
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (tq == 0) sm.ml[w][8 * h + g] = make_float2(m[h], l[h]);
    }
    ok = __syncthreads_and(ok);
    if (!ok) break;
    // [row][column] of 32 bits, rows padded by 4 (D + 4: no bank twice in what follows); the rings are empty
    constexpr int PS = D + 4;
    static_assert(sizeof(sm.ring) >= (size_t)kWarps * M * PS * 4, "the parts fit");
    float *parts = (float *)sm.ring;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 8 * h + g;
      if (r < R) {
        float *row = parts + (w * M + r) * PS;
#pragma unroll
        for (int n = 0; n < NT; n += Q8 ? 2 : 1) {
          if constexpr (Q8) *(float4 *)(row + n * 8 + 4 * tq) = make_float4(o[n][2 * h], o[n + 1][2 * h], o[n][2 * h + 1], o[n + 1][2 * h + 1]);
          else *(float2 *)(row + n * 8 + 2 * tq) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
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
      const bool empty = sum == 0.f;
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

template <bool BF16, int ES, int D>
cudaError_t launch_one(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  static SmemLimit limit;
  const int smem = (int)sizeof(Smem<ES, D>);
  auto *k = decode_attend_kernel<BF16, ES, D>;
  const cudaError_t e = limit.ensure((const void *)k, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, plan.ctas, kThreads, smem, stream, p, *p.map_decode, plan.together);
}

template <bool BF16, int ES>
cudaError_t launch_type(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  switch (p.L.head_dim) {
    case 64: return launch_one<BF16, ES, 64>(p, plan, stream);
    case 128: return launch_one<BF16, ES, 128>(p, plan, stream);
    default: return launch_one<BF16, ES, 256>(p, plan, stream);
  }
}

}  // namespace decode
}  // namespace kv

cudaError_t launch_kv_attend_decode_bf16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
cudaError_t launch_kv_attend_decode_f16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
cudaError_t launch_kv_attend_decode_e4m3(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);

}  // namespace lsc
