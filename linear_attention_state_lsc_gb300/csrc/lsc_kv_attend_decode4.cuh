// lsc_kv_attend_decode4.cuh -- attention over an E2M1 layer of the K/V block pool for
// sequences of up to 16 packed rows (lsc_kv_attend.cuh): decode steps.
//
// The plan is that of lsc_kv_attend_decode.cuh: warps that work alone, each with a
// ring of TMA sub-tiles, transposed products S^T = K Q^T and O^T = V^T P^T on
// mma.sync, a reference instead of a maximum, joined at a piece's end.  A quarter of
// the bytes of 16 bits come in, so what is done to them counts for four times as much:
//   * K: a 32-bit word of a lane is 8 codes of one position and one scale.  Four
//     conversions give four pairs of halves, four products with the scale leave K's
//     exact values (6 bits), and they are the operands of two products as they are: which
//     element of a head a product's place holds does not matter as long as q has the same.
//   * V: ldmatrix transposes pairs of bytes, so a word is 4 columns of two neighbouring
//     positions; the conversions pair columns where a product wants pairs of positions.
//     Up to 4 rows: a product of 8 positions and 32 columns runs over (position, column's
//     parity), so that v's operands are the conversions' outputs times their scales, and the
//     weights stand twice, for the even columns with a zero behind each and for the odd ones
//     with a zero before it: half the product's places, which 4 rows leave empty anyhow.
//     More rows: a byte permutation for each pair of columns makes two pairs of positions.
//   * scales come with 4- to 16-byte cp.async, a position a lane, into a ring beside the codes'; V's go
//     through shared memory once more as f16, pairs of positions side by side as the products want them.
// What bounds it: nothing that is full; the latency of chains of instructions on few warps.  The ALU does a conversion, a
// permutation, a logic or a shift every second cycle (measured, each alone): 8 cycles a word of codes for conversions, 8 more for V's permutations where there are any.  Up
// to 4 rows it is 43 % busy and the issue 54 %, with 12 warps an SM waiting for one another's results; behind the
// permutations 60 and 63 %.  Rows that lie in L2 take 9 % less.  Measured, one token of 128 sequences behind 500 to 8000,
// 32 q heads, 8 heads of 128: 593 MB in 124 us (4.8 TB/s, 72 % of a copy's rate; with the permutations 139 us, the same
// rows as E4M3 176); 64 behind 64 to 16384, 16 q heads, 2 of 256: 75 us, 57 %.
// The weights that stand twice cost 8 and 16 rows more products than the permutations they save: two tokens, 32 q heads, 4
// heads of 128 71 us beside 63, 16 q heads, 2 of 256 84 beside 68; the one token of 64 sequences above (8 rows) 81 beside 75.
// Tried and not kept: V's pairs made by two products with a zero beside each scale (141 us beside 141), sub-tiles of 32
// positions (133 us beside 125), two sums a score tile and both halves of a sub-tile unrolled (the same); at 8 and 16
// rows nibbles paired by shifts and selections in front of the conversions (82 us beside 75, 65 beside 63), three CTAs an
// SM with sub-tiles of 32 (69 beside 63).
//
// q goes to f16: bf16 rows are brought to [2^14, 2^15) by a power of two that the scores
// take back, so what bf16 holds down to 2^-28 of a row's largest is exact.
//
// Positions that only some rows see, or none (what a block holds behind the last one):
// the code of a hidden position is finite whatever it is, so clearing the scale clears
// the element; a scale that may make it infinite or NaN is noted and added again, as
// NaN, to the rows that see the position.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_attend.cuh"
#include "lsc_kv_attend_decode.cuh"
#include "lsc_ptx.h"

namespace lsc {
namespace kv {
namespace decode4 {

using decode::transposed;
using rows::ldsm4;
using rows::ldsm4t;
using rows::mma;

constexpr int kTK = decode::kTK;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// M: packed rows of a head, up to 4, 8 or 16.
template <int D, int M>
struct Conf {
  static constexpr int KEYS = kv_decode_keys(D, 4), HALVES = KEYS / 32;  // positions of a sub-tile; a lane has one of each 32
  static constexpr int RB = D / 2, SB = D / 16;  // bytes of a row's codes and scales
  static constexpr int half = KEYS * RB;         // bytes of a sub-tile's K or V codes
  static constexpr int ST = D == 64 ? 3 : 2;     // sub-tiles in flight per warp
  static constexpr int occ = D == 256 ? 2 : D == 128 ? (M < 16 ? 3 : 2) : (M < 16 ? 4 : 3);  // CTAs per SM
  static constexpr bool QS = M == 16;            // q's rows in shared memory: else in registers
};

template <int D>
constexpr int occ_of(int rows) {
  return rows < 16 ? Conf<D, 8>::occ : Conf<D, 16>::occ;
}

template <int D, int M>
struct Smem {
  using C = Conf<D, M>;
  static constexpr int PS = D + 4;  // 32-bit columns of a weighted row at a piece's end (no bank twice in what follows)
  static constexpr int rings = kWarps * C::ST * 2 * C::half, parts = kWarps * M * PS * 4;
  alignas(1024) uint8_t ring[rings > parts ? rings : parts];  // [warp][sub-tile][K, V]; at a piece's end: the warps' weighted rows
  alignas(16) uint8_t scale[kWarps][C::ST][2][C::KEYS][C::SB];
  // V's scales of 32 positions as f16, by group: positions 2 tq, 2 tq + 1 of each 8 side by side for lane tq
  alignas(16) uint16_t v_scale[kWarps][C::SB][32];
  alignas(16) uint4 q[C::QS ? kWarps : 1][C::QS ? M : 1][C::QS ? D / 8 : 1];  // neighbouring rows' chunks xor 4: no bank twice
  float2 ml[kWarps][16];
  int32_t vis[16];
  int32_t bad[kWarps][C::SB];  // by head of the unit and group: the first position whose v is NaN
  int32_t any_bad;
  uint64_t full[kWarps][C::ST];
  RunScratch run;
};

// N bytes global -> shared, or zeros when `on` is false (nothing is read then).
template <int N>
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(on ? N : 0) : "memory");
}

__device__ __forceinline__ uint32_t times(uint32_t h, __half2 s) {
  const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&h), s);
  return *reinterpret_cast<const uint32_t *>(&y);
}

template <int D, int M>
__global__ void __launch_bounds__(kThreads, (Conf<D, M>::occ))
decode4_attend_kernel(const __grid_constant__ KvAttendParams p, const __grid_constant__ CUtensorMap map, int together) {
  using C = Conf<D, M>;
  constexpr bool few = M == 4;
  // Score tiles of 8 columns: 8 rows, or each of 4 rows twice, so that a lane has one row's scores alone and finds the
  // weights that the second product wants of it without asking another lane.
  constexpr int NR = M == 16 ? 2 : 1, E = few ? 1 : 2;
  constexpr int KEYS = C::KEYS, HALVES = C::HALVES, ST = C::ST, RB = C::RB, SB = C::SB, NC = D / 32;  // NC: 16-byte chunks of a row, 32 elements each
  constexpr float lift = 7.f;       // powers of two that the reference lies below the maximum that set it
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D, M> &sm = *reinterpret_cast<Smem<D, M> *>(smem_raw);
  const int tid = threadIdx.x, w = tid >> 5, ln = tid & 31, g = ln >> 2, tq = ln & 3;
  if (tid < kWarps * ST) mbar_init(&sm.full[tid / ST][tid % ST], 1);
  fence_mbar_init();
  // What follows is not let in before the end: the join's CTAs, and the next step's behind them, came in between this
  // grid's, three or four an SM, and cost 64 sequences behind 500 to 8000, 8 heads of 128, 85 us in place of 71 and 128 at
  // 8 heads of 64 91 in place of 81; no measured step gained by it.
  griddep_wait();
  const KvLayer &L = p.L;
  const int ctas = gridDim.x, cta = blockIdx.x;
  if (cta == 0) check_cu(L, p.b);
  const int MU = M * together, splits = kWarps / together;  // rows of a unit; warps of a head
  const int wh = w & (together - 1), wsp = w / together;    // this warp's head of the unit, its share of the sub-tiles
  const Workspace ws = workspace_at(p.ws, ctas, MU);
  if (tid == 0) sm.any_bad = 0;
  for (int i = tid; i < kWarps * SB; i += kThreads) (&sm.bad[0][0])[i] = INT32_MAX;
  Run run = find_run<kThreads, M, kTK>(p, cta, ctas, sm.run);
  Piece pc;
  Cut cut = {0, 0, 0, 0};
  bool ok = true;
  // TMA boxes of `box` rows: K's on lanes 0-15, V's on 16-31
  const int box = p.box_decode, boxes = KEYS / box;
  const int bi = ln & 15, br = bi < boxes ? bi * box : 0;
  uint8_t *const ring = sm.ring + w * ST * 2 * C::half;
  // ldmatrix rows: chunk c of K (c even) and V is the offset of chunk 0 xor 16 c
  const uint32_t koff = chunk_at<RB>(KEYS, ln & 15, ln >> 4), voff = chunk_at<RB>(KEYS, ln, 0);
  // where a lane's K scale bytes are in a word: its group of an even chunk and of the odd one behind it
  const uint32_t kh = tq >> 1, ksel = 0x4040u | kh | (kh + 2) << 8;
  // few: the weights of positions 2 tq, 2 tq + 1 -> the operand for each: the weight, and a zero behind it where this
  // lane's column of the product (g) is for v's even columns, before it where it is for the odd ones
  const uint32_t wsel[2] = {g & 1 ? 0x1044u : 0x4410u, g & 1 ? 0x3244u : 0x4432u};
  int slot = 0;
  uint32_t phase = 0;
  __syncthreads();
  while (ok && next_piece<M, kTK>(p, run, pc)) {
    const int R = pc.s.n * p.group < M ? pc.s.n * p.group : M;  // this launch's units have one block
    const int32_t kv = pc.s.kv, lo = pc.t0 * kTK, hi = kv < pc.t1 * kTK ? kv : pc.t1 * kTK;
    const int32_t *table = p.b.table + (int64_t)pc.seq * p.b.max_blocks;
    const int nsub = hi > lo ? (hi - lo + KEYS - 1) / KEYS : 0, mine = nsub > wsp ? (nsub - wsp + splits - 1) / splits : 0, head = pc.head * together + wh;
    auto first_of = [&](int i) { return lo + (i * splits + wsp) * KEYS; };  // first position of this warp's sub-tile i
    // Blocks of this lane's positions of sub-tile i, 0 behind the last one.  Looked up a sub-tile ahead and checked only
    // where they are used (a bad one is recorded and read as 0): a look at them any earlier would wait for the loads.
    int32_t blk[HALVES];
    auto look_up = [&](int i) {
#pragma unroll
      for (int u = 0; u < HALVES; ++u) {
        const int32_t pos = first_of(i) + 32 * u + ln;
        blk[u] = i < mine && pos < kv ? __ldg(table + L.by_block.div(pos)) : 0;
      }
    };
    const int64_t lane_off = L.v - L.k;
    auto issue = [&](int i, int st) {
      const int32_t first = first_of(i);
      int32_t row[HALVES];
      if (ln == 0) mbar_arrive_expect_tx(&sm.full[w][st], 2 * C::half);
      __syncwarp();
#pragma unroll
      for (int u = 0; u < HALVES; ++u) {
        if ((uint32_t)blk[u] >= (uint32_t)L.num_blocks) {
          report(L.status, LSC_ERR_OUT_OF_RANGE);
          blk[u] = 0;
        }
        const int32_t pos = first + 32 * u + ln;
        row[u] = pos - L.by_block.div(pos) * L.block_tokens;
        const bool on = pos < kv;
        const uint8_t *k = L.k + (on ? (int64_t)blk[u] * L.page + L.scale_off + ((int64_t)row[u] * L.heads + head) * SB : 0);
        cp_async_or_zero<SB>(smem_u32(sm.scale[w][st][0][32 * u + ln]), k, on);
        cp_async_or_zero<SB>(smem_u32(sm.scale[w][st][1][32 * u + ln]), k + lane_off, on);
      }
      int32_t box_blk = __shfl_sync(0xffffffffu, blk[0], br & 31), box_row = __shfl_sync(0xffffffffu, row[0], br & 31);
      if constexpr (HALVES == 2) {
        const int32_t b1 = __shfl_sync(0xffffffffu, blk[1], br & 31), r1 = __shfl_sync(0xffffffffu, row[1], br & 31);
        if (br >= 32) box_blk = b1, box_row = r1;
      }
      if (bi < boxes)
        tma_box(ring + (st * 2 + (ln >> 4)) * C::half + br * RB, &map, box_row, 0, head,
                box_blk + (ln < 16 ? 0 : L.num_blocks), &sm.full[w][st]);
    };
    int st_in = slot;
#pragma unroll
    for (int i = 0; i < ST; ++i) {
      if (i < mine) {
        look_up(i);
        issue(i, st_in);
        if (++st_in == ST) st_in = 0;
      }
      cp_async_commit();
    }
    look_up(ST);

    if (tid < M) sm.vis[tid] = tid < R ? visible(pc.s, p.by_group.div(tid), p.causal) : 0;
    // q as operands: row g of each 8, elements 8 tq .. 8 tq + 7 of each 32, as f16
    uint32_t qf[C::QS ? 1 : NR][C::QS ? 1 : NC][4];
    float q_up[NR];  // of row g: scale * log2 e, times the power of two that bf16 rows were brought down by
#pragma unroll
    for (int h = 0; h < NR; ++h) {
      const int r = few ? g >> 1 : 8 * h + g, tok = p.by_group.div(r);
      const uint16_t *src = (const uint16_t *)p.q + (int64_t)(pc.s.row0 + tok) * p.q_stride +
                            (int64_t)(head * p.group + (r - tok * p.group)) * D;
      uint32_t x[NC][4];
      q_up[h] = p.scale_log2;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint4 y = r < R ? *(const uint4 *)(src + c * 32 + 8 * tq) : make_uint4(0, 0, 0, 0);
        x[c][0] = y.x, x[c][1] = y.y, x[c][2] = y.z, x[c][3] = y.w;
      }
      if (p.dtype == LSC_BF16) {
        uint32_t top = 0;  // magnitudes of 16-bit floats order as whole numbers
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = __vmaxu2(top, x[c][e] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t ex = top >> 7;  // 2^k <= the largest magnitude < 2^(k + 1), where that is a normal number
        const bool plain = ex == 0 || ex == 255;
        const float down = plain ? 1.f : inv_scale_of(ex), more = plain ? 1.f : 16384.f;
        // (a hidden score is -infinity times this, so it may not be 0; products of q and k are below 2^39; the power by
        // itself first, 2^-140 to 2^113: with the scale in it 2^127 is too much before its 2^14 are taken back)
        if (!plain) q_up[h] = fmaxf(q_up[h] * (__uint_as_float(ex << 23) * (1.f / 16384.f)), 0x1p-120f);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t b = x[c][e];
            x[c][e] = pack2(__uint_as_float(b << 16) * down * more, __uint_as_float(b & 0xffff0000u) * down * more, 0);
          }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if constexpr (C::QS) {
          sm.q[w][r][(c * 4 + tq) ^ (r & 1) * 4] = make_uint4(x[c][0], x[c][1], x[c][2], x[c][3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) qf[h][c][e] = x[c][e];
        }
      }
    }
    // scores come with rows 2 tq, 2 tq + 1 of each 8 (few: row tq)
    float qsc[NR][E];
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int e = 0; e < E; ++e) qsc[h][e] = __shfl_sync(0xffffffffu, q_up[h], (2 * tq + e) * 4);
    __syncthreads();  // vis; and the last piece's shared memory is free
    const int32_t sure = visible(pc.s, 0, p.causal);  // every row sees positions below this
    int32_t vis[NR][E];
    float m[NR][E], ref[NR][E], l[NR][E];  // ref: m, 0 while no position has been seen
    float o[NR][few ? NC : 2 * NC][4];     // few: of row tq, columns 4 g .. 4 g + 3 of each 32
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int e = 0; e < E; ++e) vis[h][e] = sm.vis[few ? tq : 8 * h + 2 * tq + e], m[h][e] = -INFINITY, ref[h][e] = l[h][e] = 0.f;
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (auto &x : o[h]) x[0] = x[1] = x[2] = x[3] = 0.f;

    int i = 0;
#pragma unroll 1
    for (; i < mine; ++i) {
      const int32_t first = first_of(i);
      cp_async_wait<ST - 1>();
      if (!(ok = wait_warp(&sm.full[w][slot], phase, p.wait_limit_ns))) break;
      __syncwarp();  // every lane's scales are there
      const uint32_t ka = smem_u32(ring + slot * 2 * C::half), va = ka + C::half;
      const uint8_t *kscale = sm.scale[w][slot][0][0];
#pragma unroll 1
      for (int u = 0; u < HALVES && (u == 0 || first + 32 * u < hi); ++u) {  // 32 positions at a time
        const int32_t first32 = first + 32 * u;
        {
          // V's scales to f16, a position a lane.  Where some row does not see the position they need a look before they
          // meet a weight of 0.
          const int32_t pos = first32 + ln;
          uint32_t b[SB / 4];
#pragma unroll
          for (int x = 0; x < SB / 4; ++x) b[x] = *(const uint32_t *)&sm.scale[w][slot][1][32 * u + ln][4 * x];
          if (first32 + 32 > sure && pos >= sure && pos < hi) {
#pragma unroll
            for (int x = 0; x < SB; ++x)
              if ((b[x / 4] >> (x % 4 * 8) & 0xff) > kE2M1Top) {
                atomicMin(&sm.bad[wh][x], pos);
                sm.any_bad = 1;
                b[x / 4] &= ~(0xffu << (x % 4 * 8));
              }
          }
          uint16_t *to = sm.v_scale[w][0] + (ln >> 1 & 3) * 8 + (ln >> 3) * 2 + (ln & 1);
          __syncwarp();  // the last ones have been read
#pragma unroll
          for (int x = 0; x < SB / 4; ++x) {
            const uint32_t even = (b[x] & 0x00ff00ffu) << 7, odd = (b[x] & 0xff00ff00u) >> 1;  // bytes 0 and 2, 1 and 3
            to[(4 * x) * 32] = (uint16_t)even, to[(4 * x + 1) * 32] = (uint16_t)odd;
            to[(4 * x + 2) * 32] = (uint16_t)(even >> 16), to[(4 * x + 3) * 32] = (uint16_t)(odd >> 16);
          }
          __syncwarp();
        }
      // ---- scores: lane (g, tq) gets positions g, g + 8 of each 16 and rows 2 tq, 2 tq + 1 of each 8
      float s[2][NR][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < NR; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][h][e] = 0.f;
#pragma unroll
      for (int c = 0; c < NC; c += 2) {
        uint32_t ks[4];  // chunk c's and c + 1's scales (f16) of positions g + 8 y
#pragma unroll
        for (int y = 0; y < 4; ++y) ks[y] = __byte_perm(*(const uint32_t *)(kscale + (32 * u + g + 8 * y) * SB + 2 * c), 0, ksel) << 7;
        uint32_t qs[NR][2][4];  // QS: both chunks' q
        if constexpr (C::QS) {
#pragma unroll
          for (int h = 0; h < NR; ++h)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint4 x = sm.q[w][8 * h + g][((c + y) * 4 + tq) ^ (g & 1) * 4];
              qs[h][y][0] = x.x, qs[h][y][1] = x.y, qs[h][y][2] = x.z, qs[h][y][3] = x.w;
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          uint32_t b[4];
          ldsm4(b, ka + u * (32 * RB) + (koff ^ c << 4) + n * (16 * RB));
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // chunk c + y
            auto q_of = [&](int h, int e) { return C::QS ? qs[h][y][e] : qf[C::QS ? 0 : h][C::QS ? 0 : c + y][e]; };
            uint32_t x[2][4];
#pragma unroll
            for (int z = 0; z < 2; ++z) {  // positions g, g + 8
              const __half2 sc = *reinterpret_cast<const __half2 *>(&ks[2 * n + z]);
              e2m1x8_times(b[2 * y + z], y ? __high2half2(sc) : __low2half2(sc), x[z]);
            }
            const uint32_t a0[4] = {x[0][0], x[1][0], x[0][1], x[1][1]}, a1[4] = {x[0][2], x[1][2], x[0][3], x[1][3]};
#pragma unroll
            for (int h = 0; h < NR; ++h) {
              mma<false>(s[n][h], a0, q_of(h, 0), q_of(h, 1));
              mma<false>(s[n][h], a1, q_of(h, 2), q_of(h, 3));
            }
          }
        }
      }
      // ---- weights
      if (first32 + 32 > sure) {  // positions that some row does not see
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int h = 0; h < NR; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (first32 + 16 * n + 8 * (e >> 1) + g >= vis[h][(e & 1) % E]) s[n][h][e] = -INFINITY;
      }
      bool rise = false;
      float top[NR][E];
#pragma unroll
      for (int h = 0; h < NR; ++h)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          top[h][e] = fmaxf(fmaxf(s[0][h][e], s[0][h][2 + e]), fmaxf(s[1][h][e], s[1][h][2 + e])) * qsc[h][e];
          rise |= top[h][e] > m[h][e] + (8.f + lift);
        }
      if (__any_sync(0xffffffffu, rise)) {  // also the first one's (m is -inf)
#pragma unroll
        for (int h = 0; h < NR; ++h)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            float t = top[h][e];
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
            const float to = fmaxf(m[h][e], t - lift);
            ref[h][e] = to == -INFINITY ? 0.f : to;
            const float f = ex2(m[h][e] - ref[h][e]);
            m[h][e] = to;
            l[h][e] *= f;
#pragma unroll
            for (auto &x : o[h]) {
              x[e] *= f, x[2 + e] *= f;
              if constexpr (few) x[1] *= f, x[3] *= f;
            }
          }
      }
      uint32_t a[2][NR][2];  // of row g (few: g / 2): the weights of positions 2 tq, 2 tq + 1 of each 8
#pragma unroll
      for (int h = 0; h < NR; ++h) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float x[2];
#pragma unroll
            for (int e = 0; e < E; ++e) {
              x[e] = ex2(fmaf(s[n][h][2 * y + e], qsc[h][e], -ref[h][e]));
              l[h][e] += x[e];
            }
            a[n][h][y] = transposed(pack2(x[0], x[E - 1], 0));
          }
      }
      // ---- V^T times weights
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        uint32_t b[4];
        ldsm4t(b, va + u * (32 * RB) + (voff ^ c << 4));
        const uint4 sv4 = *(const uint4 *)&sm.v_scale[w][2 * c + (g >> 2)][tq * 8];  // of positions 2 tq, 2 tq + 1 of each 8
        const uint32_t sv[4] = {sv4.x, sv4.y, sv4.z, sv4.w};
        if constexpr (few) {  // m index g is columns 4 g, 4 g + 1 of 32, m index g + 8 the two behind them
#pragma unroll
          for (int y = 0; y < 4; ++y) {  // 8 positions
            const __half2 sc = *reinterpret_cast<const __half2 *>(&sv[y]);
            uint32_t x[4];
            e2m1x8_to_f16(b[y], x);
#pragma unroll
            for (int z = 0; z < 4; ++z) x[z] = times(x[z], z < 2 ? __low2half2(sc) : __high2half2(sc));
            const uint32_t pair = a[y / 2][0][y % 2];
            mma<false>(o[0][c], x, __byte_perm(pair, 0, wsel[0]), __byte_perm(pair, 0, wsel[1]));
          }
        } else {  // m index g is column 4 g (+ 2), m index g + 8 the one behind it
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            uint32_t x[2][4];  // columns 4 g .. 4 g + 3 of positions 2 tq, 2 tq + 1 and 8 further
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const __half2 sc = *reinterpret_cast<const __half2 *>(&sv[2 * n + y]);
              uint32_t h[4];
              e2m1x8_to_f16(b[2 * n + y], h);
              x[y][0] = times(__byte_perm(h[0], h[2], 0x5410), sc);
              x[y][1] = times(__byte_perm(h[0], h[2], 0x7632), sc);
              x[y][2] = times(__byte_perm(h[1], h[3], 0x5410), sc);
              x[y][3] = times(__byte_perm(h[1], h[3], 0x7632), sc);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t v[4] = {x[0][2 * z], x[0][2 * z + 1], x[1][2 * z], x[1][2 * z + 1]};
#pragma unroll
              for (int h = 0; h < NR; ++h) mma<false>(o[h][2 * c + z], v, a[n][h][0], a[n][h][1]);
            }
          }
        }
      }
      }
      // ---- the slot's next sub-tile
      __syncwarp();
      if (i + ST < mine) {
        issue(i + ST, slot);
        look_up(i + ST + 1);
      }
      cp_async_commit();
      if (++slot == ST) slot = 0, phase ^= 1;
    }
    if (!ok) {  // nothing may be in flight when the CTA leaves: every slot that was filled
      for (int x = i; x < mine && x < i + ST; ++x) {
        wait_warp(&sm.full[w][slot], phase, p.drain_limit_ns);
        if (++slot == ST) slot = 0, phase ^= 1;
      }
      cp_async_wait<0>();
      if (ln == 0) report(L.status, LSC_ERR_DEV_TIMEOUT);
    }
    // ---- the piece's end: the warps' parts through shared memory, then rows out or to the workspace
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        l[h][e] += __shfl_xor_sync(0xffffffffu, l[h][e], 4);
        l[h][e] += __shfl_xor_sync(0xffffffffu, l[h][e], 8);
        l[h][e] += __shfl_xor_sync(0xffffffffu, l[h][e], 16);
        if (g == 0) sm.ml[w][few ? tq : 8 * h + 2 * tq + e] = make_float2(m[h][e], l[h][e]);
      }
    ok = __syncthreads_and(ok);
    if (!ok) break;
    constexpr int PS = Smem<D, M>::PS;  // the rings are empty
    float *parts = (float *)sm.ring;
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int r = few ? tq : 8 * h + 2 * tq + e;
        if (r < R) {
          float *row = parts + (w * M + r) * PS;
#pragma unroll
          for (int c = 0; c < NC; ++c)  // columns 4 g .. 4 g + 3 of 32
            *(float4 *)(row + c * 32 + 4 * g) =
                few ? make_float4(o[h][c][0], o[h][c][1], o[h][c][2], o[h][c][3])
                    : make_float4(o[h][2 * c][e], o[h][2 * c][2 + e], o[h][2 * c + 1][e], o[h][2 * c + 1][2 + e]);
        }
      }
    __syncthreads();
    const bool whole = pc.t0 == 0 && pc.t1 == pc.tiles;
    const int64_t slot0 = (int64_t)(2 * cta + (pc.t0 == 0 ? 1 : 0)) * MU;
    const bool look = sm.any_bad != 0;
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
      if (look && sm.bad[hw][d / 16] < sm.vis[r]) y.x = y.y = y.z = y.w = __uint_as_float(0x7fc00000u);
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
      for (int i = tid; i < kWarps * SB; i += kThreads) (&sm.bad[0][0])[i] = INT32_MAX;
      if (tid == 0) sm.any_bad = 0;
      __syncthreads();
    }
  }
  if (tid == 0 && p.ws) ws.cut[cta] = cut;
}

template <int D, int M>
cudaError_t launch_one(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  static SmemLimit limit;
  const int smem = (int)sizeof(Smem<D, M>);
  static_assert(Conf<D, M>::occ * (sizeof(Smem<D, M>) + 1024) <= 228 * 1024, "CTAs that an SM holds at once");
  auto *k = decode4_attend_kernel<D, M>;
  const cudaError_t e = limit.ensure((const void *)k, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, plan.ctas, kThreads, smem, stream, p, *p.map_decode, plan.together);
}

template <int D>
cudaError_t launch_rows(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  const int rows = plan.M / plan.together;
  return rows == 4   ? launch_one<D, 4>(p, plan, stream)
         : rows == 8 ? launch_one<D, 8>(p, plan, stream)
                     : launch_one<D, 16>(p, plan, stream);
}

}  // namespace decode4
}  // namespace kv

cudaError_t launch_kv_attend_decode_e2m1(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);

}  // namespace lsc
