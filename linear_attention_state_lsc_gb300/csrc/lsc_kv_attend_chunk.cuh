// lsc_kv_attend_chunk.cuh -- attention over a layer of the K/V block pool for
// sequences with many packed rows (lsc_kv_attend.cuh): prefill chunks.
//
// 4 * head_dim operations a (row, position) pair, and K/V tiles that serve 128 or
// 256 rows: the 5th-generation tensor cores bound it.  One CTA per SM walks its
// run of tiles of TK positions with the warps in roles:
//   * softmax warps, one thread a row: wait for the scores S = Q K^T of a tile in
//     TMEM, weights 2^(s - m) to 16 bits back into the same TMEM columns, sum in a
//     register.  m is a reference, not the exact maximum: O is rescaled (in TMEM,
//     by these threads) only when a row's maximum rose by more than 2^8, so a
//     weight is at most 2^8 and the rescale is rare after the first tiles.
//   * one MMA warp: S = Q K^T, O += P V with P as the TMEM operand, issued so that
//     the products of one tile run while the softmax of another does.
//   * producer warps: K and V rows through the block table into a shared-memory
//     ring in the 128-byte-swizzled layout.  16-bit pools whose blocks are a
//     multiple of 8 tokens: tiled TMA boxes of rows x 64 elements (x head_dim /
//     64 when a block holds the tile: then one box a tile; coordinates
//     (element, row, column of 64, head, block) of the layer, element always
//     0); a tile that is not full, and other block sizes: 16-byte cp.async.
//     E4M3 pools: codes
//     through a staging ring of each thread, then bf16 with their scale
//     (exact above bf16's smallest normal).  Rows behind the last position
//     are zeros.
// head_dim 64 and 128: two row blocks of 128, each with its own S and O (S 2 x
// 128, O 2 x head_dim columns of TMEM), Q in shared memory, tiles of 128: one
// block's softmax runs under the other's products, and a K/V tile is
// fetched once for 256 rows.
// head_dim 256: O takes 256 columns, so one row block, tiles of 64 and two S
// buffers in turn; Q is a TMEM operand (128 columns), which leaves shared
// memory to K and V and halves what the score products read from it.
//
// Positions that only some rows of a unit see may hold infinities and NaN: see
// lsc_kv_attend_rows.cuh; here the softmax threads search such a tile's v.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_attend.cuh"
#include "lsc_ptx.h"
#include "lsc_tc.h"

namespace lsc {
namespace kv {
namespace chunk {

constexpr int kThreads = 512;  // four warpgroups; the last one has the MMA warp and three idle ones

template <int D, bool Q8>
struct Conf {
  static constexpr int NQ = D == 256 ? 1 : 2;   // row blocks of 128
  static constexpr int M = 128 * NQ;
  static constexpr int TK = D == 256 ? 64 : 128;
  static constexpr bool QT = D == 256;          // Q in TMEM
  static constexpr int slot = TK * D * 2;       // bytes of a K or V tile
  static constexpr int NS = Q8 ? (D == 64 ? 6 : D == 128 ? 4 : 5) : (D == 64 ? 8 : D == 128 ? 5 : 6);
  static constexpr int SD = D == 128 ? 2 : 3;   // E4M3: stages of codes
  static constexpr int SW = 4 * NQ;             // softmax warps
  static constexpr int PW = D == 256 ? 8 : 4;   // producer warps
  // registers a thread of a softmax, producer and MMA warpgroup keeps of the 128 at launch: 4 * (SW / 4 * soft +
  // PW / 4 * prod + mma) <= 16 * 128
  static constexpr int soft = D == 256 ? 200 : 160, prod = D == 256 ? 104 : 96, mma = D == 256 ? 104 : 96;
  static_assert(SW / 4 * soft + PW / 4 * prod + mma <= 4 * 128, "more registers than the block has");
  static_assert(SW + PW == 12, "three warpgroups beside the one of the MMA warp");
  // TMEM columns
  static constexpr int S0 = 0, SN = TK;         // S buffer b at S0 + b * SN; P in its first half
  static constexpr int Q0 = 128;                // QT only
  static constexpr int O0 = 256;                // O of row block b at O0 + b * D
};

template <int D, bool Q8>
struct Smem {
  using C = Conf<D, Q8>;
  alignas(1024) uint8_t ring[C::NS][C::slot];
  alignas(1024) uint8_t q[C::QT ? 16 : C::M * D * 2];
  alignas(16) uint4 stage[Q8 ? C::SD : 1][Q8 ? C::TK * D / 16 / (32 * C::PW) : 1][Q8 ? 32 * C::PW : 1];  // E4M3: codes by thread
  int32_t bad[3][D];      // first position whose v is NaN, +inf, -inf
  uint64_t full[C::NS], empty[C::NS], sfull[2], pfull[2], qfull[2], odone[2], fin[2], met[2], drain;
  uint32_t tmem;
  int32_t any_bad;
  RunScratch run;
};

// Shared-memory matrix descriptor, 128-byte swizzle (bits 61-63 = 2), version 1.
__device__ __forceinline__ uint64_t desc128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// Instruction descriptor of kind::f16 with an fp32 accumulator: both operands f16 (0) or bf16 (1).
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool bf16, bool b_mn_major) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_ss16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values as the operand of the packed instructions, which do two lanes' worth a cycle.
__device__ __forceinline__ uint64_t two(float x, float y) {
  return (uint64_t)__float_as_uint(x) | (uint64_t)__float_as_uint(y) << 32;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Wait for this thread's TMEM loads; v is tied to it, so nothing reads v earlier.
__device__ __forceinline__ void wait_ld(uint32_t (&v)[32]) {
#define LSC_R8(i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), \
                  "+r"(v[i + 6]), "+r"(v[i + 7])
  asm volatile("tcgen05.wait::ld.sync.aligned;" : LSC_R8(0), LSC_R8(8), LSC_R8(16), LSC_R8(24)::"memory");
#undef LSC_R8
}

// Scores of columns at and behind `seen` become -infinity.
__device__ __forceinline__ void hide(uint32_t (&s)[32], int32_t seen) {
#pragma unroll
  for (int y = 0; y < 32; ++y)
    if (y >= seen) s[y] = 0xff800000u;
}

__device__ __forceinline__ float top_of(const uint32_t (&s)[32]) {
  float t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = __uint_as_float(s[8 * i]);
#pragma unroll
    for (int y = 1; y < 8; ++y) t[i] = fmaxf(t[i], __uint_as_float(s[8 * i + y]));
  }
  return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
}

// 2^(s c + r) of 32 scores: added to l in 32 bits, rounded to 16 bits in q.
template <bool BF16>
__device__ __forceinline__ void weights(const uint32_t (&s)[32], uint64_t c, uint64_t r, uint64_t &l, uint32_t (&q)[16]) {
  uint64_t a[2] = {0, 0};
#pragma unroll
  for (int y = 0; y < 16; ++y) {
    const uint64_t x = fma2((uint64_t)s[2 * y] | (uint64_t)s[2 * y + 1] << 32, c, r);
    const float p0 = ex2(__uint_as_float((uint32_t)x)), p1 = ex2(__uint_as_float((uint32_t)(x >> 32)));
    a[y & 1] = add2(a[y & 1], two(p0, p1));
    q[y] = pack2(p0, p1, BF16);
  }
  l = add2(l, add2(a[0], a[1]));
}

// Tiled TMA load of one box (this CTA's shared memory), completing on `bar`.
__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, int c4,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar))
      : "memory");
}

// A bounded wait.  The first tries do without the clock: reading %globaltimer costs about a microsecond, several
// tiles' worth of waits.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t phase, uint64_t limit) {
  if (limit == 0) return false;
  for (int i = 0; i < 16; ++i)
    if (mbar_try_wait(bar, phase & 1)) return true;
  return mbar_wait_bounded(bar, phase & 1, limit);
}
// The same with one answer for the whole (converged) warp, so that a wait that gave up never splits it.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t phase, uint64_t limit) {
  return __all_sync(0xffffffffu, wait_bar(bar, phase, limit));
}

// A walk over the ring's slots.  Counting modulo a number that is no power of two, or dividing by a block size, costs a
// lone warp a hundred cycles and more each time, so the roles step instead.
template <int NS>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++slot == NS) slot = 0, phase ^= 1;
  }
};

// Place of V(j) of a piece of nt tiles in the order in which the ring is filled and used: K(0), V(0), K(1), V(1) ...
// with two row blocks, K(0), K(1), V(0), K(2), V(1) ... with one.
template <int NQ>
__device__ __forceinline__ int v_index(int j, int nt) {
  return NQ == 2 ? 2 * j + 1 : j < nt - 1 ? 2 * j + 2 : 2 * j + 1;
}

template <bool BF16, bool Q8, int D>
__global__ void __launch_bounds__(kThreads, 1)
chunk_attend_kernel(const __grid_constant__ KvAttendParams p, const __grid_constant__ CUtensorMap map) {
  using C = Conf<D, Q8>;
  constexpr int NQ = C::NQ, M = C::M, TK = C::TK, NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D, Q8> &sm = *reinterpret_cast<Smem<D, Q8> *>(smem_raw);
  const int tid = threadIdx.x, w = tid >> 5, ln = tid & 31;
  const KvLayer &L = p.L;
  if (w == C::SW + C::PW) {
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&sm.full[i], C::PW), mbar_init(&sm.empty[i], 1);
    for (int i = 0; i < 2; ++i)
      mbar_init(&sm.sfull[i], 1), mbar_init(&sm.pfull[i], 4), mbar_init(&sm.qfull[i], 4), mbar_init(&sm.odone[i], 1), mbar_init(&sm.fin[i], 1),
          mbar_init(&sm.met[i], 4);
    mbar_init(&sm.drain, 1);
    fence_mbar_init();
    sm.any_bad = 0;
  }
  for (int i = tid; i < 3 * D; i += kThreads) (&sm.bad[0][0])[i] = INT32_MAX;
  griddep_wait();
  if (tid == 0) griddep_launch_dependents();
  const int ctas = gridDim.x, cta = blockIdx.x;
  if (cta == 0) check_cu(L, p.b);
  tc::fence_before_sync();
  Run run = find_run<kThreads, M, TK>(p, cta, ctas, sm.run);
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = sm.tmem;
  const uint64_t limit = p.wait_limit_ns;
  bool ok = true;
  Cut cut = {0, 0, 0, 0};
  Piece pc;

  if (w < C::SW) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::soft));
    // ---------------------------------------------------------------- softmax
    const int b = w >> 2, row = (w & 3) * 32 + ln;  // row block, row in it
    const uint32_t lane = (uint32_t)((w & 3) * 32) << 16;
    const Workspace ws = workspace_at(p.ws, ctas, M);
    const float c = p.scale_log2;
    auto rows_of = [&](const Piece &q) {  // packed rows of the unit
      const int64_t r = (int64_t)q.s.n * p.group - (int64_t)q.block * M;
      return r < M ? (int)r : M;
    };
    auto load_q = [&](const Piece &q) {
      const int r = b * 128 + row;
      const bool on = r < rows_of(q);
      const int64_t R = (int64_t)q.block * M + r;
      const uint4 *src = on ? (const uint4 *)((const uint16_t *)p.q + row_token(q.s, p.group, R) * p.q_stride +
                                              ((int64_t)q.head * p.group + R % p.group) * D)
                            : nullptr;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      if constexpr (C::QT) {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          uint32_t v[32];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const uint4 y = on ? src[i * 8 + x] : zero;
            v[4 * x] = y.x, v[4 * x + 1] = y.y, v[4 * x + 2] = y.z, v[4 * x + 3] = y.w;
          }
          tc::tmem_st32(tm + lane + C::Q0 + 32 * i, v);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
      } else {
        uint8_t *dst = sm.q + b * 128 * D * 2 + row * 128;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint4 y = on ? src[i] : zero;
          *(uint4 *)(dst + (i >> 3) * 16384 + (((i & 7) ^ (row & 7)) << 4)) = y;
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (ln == 0) mbar_arrive(&sm.qfull[b]);
    };
    bool have = next_piece<M, TK>(p, run, pc);
    if (have && b * 128 < rows_of(pc)) load_q(pc);
    uint32_t it = 0;     // tiles this row block has been through
    uint32_t slots = 0;  // ring slots of the pieces before this one, modulo 2 NS
    uint32_t meets = 0, done = 0;
    while (have && ok) {
      const int nt = pc.t1 - pc.t0, rows = rows_of(pc);
      const bool mine = b * 128 < rows;
      const int r = b * 128 + row;
      const int64_t R = (int64_t)pc.block * M + r;
      const int32_t vis = r < rows ? visible(pc.s, (int32_t)(R / p.group), p.causal) : 0;
      const int32_t sure = visible(pc.s, (int32_t)((int64_t)pc.block * M / p.group), p.causal);
      const int32_t full_to = C::NQ == 2 && b == 1 && mine
                                  ? visible(pc.s, (int32_t)(((int64_t)pc.block * M + 128) / p.group), p.causal)
                                  : sure;  // every row of this block sees positions below it
      const bool rows_all = (b + 1) * 128 <= rows;
      float m = -INFINITY, l = 0.f;
      // does the piece reach positions that some row of the unit does not see
      const bool mixed = (pc.s.kv < (int64_t)pc.t1 * TK ? pc.s.kv : pc.t1 * TK) > sure;
      for (int j = 0; j < nt && mine; ++j, ++it) {
        const int sb = NQ == 2 ? b : (int)(it & 1);
        const uint32_t ph = NQ == 2 ? it : it >> 1;
        const uint32_t sa = tm + lane + C::S0 + sb * C::SN;
        const int32_t first = (pc.t0 + j) * TK;
        if (!(ok = wait_warp(&sm.sfull[sb], ph, limit))) break;
        tc::fence_after_sync();
        // a column is seen when first + column < vis
        const bool mask = first + TK > full_to || !rows_all;
        const int32_t seen = vis - first;
        constexpr int HELD = TK == 64 ? 64 : 32;  // columns in registers at a time
        uint32_t s[HELD], s2[HELD == 64 ? 1 : 32];
        float top = -INFINITY;
        // the next 32 columns are on their way while these are looked at
        auto &sa32 = *reinterpret_cast<uint32_t(*)[32]>(&s[0]);
        auto &sb32 = *reinterpret_cast<uint32_t(*)[32]>(HELD == 64 ? &s[HELD - 32] : &s2[0]);
        tc::tmem_ld32(sa, sa32);
        wait_ld(sa32);
#pragma unroll
        for (int x = 0; x < TK; x += 64) {
          tc::tmem_ld32(sa + x + 32, sb32);
          if (mask) hide(sa32, seen - x);
          top = fmaxf(top, top_of(sa32));
          wait_ld(sb32);
          if (x + 64 < TK) tc::tmem_ld32(sa + x + 64, sa32);
          if (mask) hide(sb32, seen - x - 32);
          top = fmaxf(top, top_of(sb32));
          if (x + 64 < TK) wait_ld(sa32);
        }
        const float mt = top * c;  // c > 0
        if (__any_sync(0xffffffffu, mt > m + 8.f)) {  // also the first tile's (m is -inf)
          const float to = fmaxf(m, mt), f = ex2(m - (to == -INFINITY ? 0.f : to));
          m = to;
          l *= f;
          if (j > 0) {
            if (!(ok = wait_warp(&sm.odone[NQ == 2 ? b : 0], it - 1, limit))) break;
            tc::fence_after_sync();
            const uint32_t oa = tm + lane + C::O0 + b * D;
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
              uint32_t o[32];
              tc::tmem_ld32(oa + x, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tc::tmem_st32(oa + x, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t c2 = two(c, c), r2 = two(-ref, -ref);
        uint64_t l2 = two(0.f, 0.f);
        uint32_t q[16];
        if constexpr (HELD == 64) {
          weights<BF16>(sa32, c2, r2, l2, q);
          tc::tmem_st16(sa, q);
          weights<BF16>(sb32, c2, r2, l2, q);
          tc::tmem_st16(sa + 16, q);
        } else {
          tc::tmem_ld32(sa, sa32);
          wait_ld(sa32);
#pragma unroll
          for (int x = 0; x < TK; x += 64) {
            tc::tmem_ld32(sa + x + 32, sb32);
            if (mask) hide(sa32, seen - x);
            weights<BF16>(sa32, c2, r2, l2, q);
            wait_ld(sb32);
            tc::tmem_st16(sa + x / 2, q);  // over columns that have been read
            if (x + 64 < TK) tc::tmem_ld32(sa + x + 64, sa32);
            if (mask) hide(sb32, seen - x - 32);
            weights<BF16>(sb32, c2, r2, l2, q);
            if (x + 64 < TK) wait_ld(sa32);
            tc::tmem_st16(sa + x / 2 + 16, q);
          }
        }
        const float2 lf = *reinterpret_cast<const float2 *>(&l2);
        l += lf.x + lf.y;
        const int32_t last = first + TK < pc.s.kv ? first + TK : pc.s.kv;
        if (last > sure) {  // positions [max(first, sure), last): some row of the unit does not see them
          const uint32_t vi = slots + v_index<NQ>(j, nt);
          const int slot = (int)(vi % NS);
          if (!(ok = wait_warp(&sm.full[slot], vi / NS, limit))) break;
          const int lo = (sure > first ? sure : first) - first, cnt = last - first - lo;
          constexpr uint32_t E = BF16 ? 0x7f80 : 0x7c00;
          for (int i = row; i < cnt * (D / 8); i += 128) {
            const int key = lo + i / (D / 8), ch = i % (D / 8);
            uint4 *at = (uint4 *)(sm.ring[slot] + (ch >> 3) * (TK * 128) + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
            uint4 v = *at;
            uint32_t e[4] = {v.x, v.y, v.z, v.w};
            bool hit = false;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t u = (e[x] >> (16 * h)) & 0xffffu;
                if ((u & E) == E) {
                  hit = true;
                  atomicMin(&sm.bad[(u & (E ^ 0x7fff)) ? 0 : (u & 0x8000) ? 2 : 1][ch * 8 + 2 * x + h], first + key);
                  e[x] &= ~(0xffffu << (16 * h));
                }
              }
            if (hit) {
              sm.any_bad = 1;
              *at = make_uint4(e[0], e[1], e[2], e[3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (ln == 0) mbar_arrive(&sm.pfull[sb]);
      }
      if (!ok) break;
      const Piece q = pc;
      const bool ends_here = mine;
      cut = cut_of(run, q, cta);
      slots = (slots + 2 * (uint32_t)nt) % (2 * NS);
      have = next_piece<M, TK>(p, run, pc);
      if (have && b * 128 < rows_of(pc)) load_q(pc);  // this piece's score products are done
      if (ends_here) {
        // a barrier of its own: odone may be up to two phases behind here, and a parity tells two apart, not three
        if (!(ok = wait_warp(&sm.fin[b], done++, limit))) break;
        tc::fence_after_sync();
        const bool whole = q.t0 == 0 && q.t1 == q.tiles;
        const bool empty = l == 0.f;
        const float inv = whole ? (empty ? 0.f : 1.f / l) : 1.f;
        const int64_t h = (int64_t)q.head * p.group + R % p.group, t = row_token(q.s, p.group, R);
        const int64_t slot = (int64_t)(2 * cta + (q.t0 == 0 ? 1 : 0)) * M + r;
        const bool on = r < rows;
        const bool look = mixed && *(volatile int32_t *)&sm.any_bad != 0;
        uint16_t *out = (uint16_t *)p.out + t * p.out_stride + h * D;
        float *part = ws.o + slot * D;
        const uint32_t oa = tm + lane + C::O0 + b * D;
#pragma unroll 1
        for (int x = 0; x < D; x += 32) {
          uint32_t o[32];
          tc::tmem_ld32(oa + x, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * inv);
          if (look) {
#pragma unroll
            for (int y = 0; y < 32; ++y) {
              float v = __uint_as_float(o[y]);
              if (sm.bad[1][x + y] < vis) v += INFINITY;
              if (sm.bad[2][x + y] < vis) v -= INFINITY;
              if (sm.bad[0][x + y] < vis) v = __uint_as_float(0x7fc00000u);
              o[y] = __float_as_uint(v);
            }
          }
          if (on && whole) {
#pragma unroll
            for (int y = 0; y < 32; y += 8) {
              uint4 v;
              v.x = pack2(__uint_as_float(o[y]), __uint_as_float(o[y + 1]), BF16);
              v.y = pack2(__uint_as_float(o[y + 2]), __uint_as_float(o[y + 3]), BF16);
              v.z = pack2(__uint_as_float(o[y + 4]), __uint_as_float(o[y + 5]), BF16);
              v.w = pack2(__uint_as_float(o[y + 6]), __uint_as_float(o[y + 7]), BF16);
              *(uint4 *)(out + x + y) = v;
            }
          } else if (on) {
#pragma unroll
            for (int y = 0; y < 32; y += 4) *(uint4 *)(part + x + y) = make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]);
          }
          __syncwarp();
        }
        if (on) {
          if (!whole) ws.ml[slot] = make_float2(m, l);
          else if (p.lse) p.lse[t * p.heads + h] = empty ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
        }
        tc::fence_before_sync();  // these reads before the next piece's products, through pfull
      }
      if (mixed) {  // the next unit starts with a clean list: all softmax warps meet before and after it is cleared
        for (int round = 0; round < 2 && ok; ++round, ++meets) {
          if (round == 1 && *(volatile int32_t *)&sm.any_bad)
            for (int i = b * 128 + row; i < 3 * D; i += M) (&sm.bad[0][0])[i] = INT32_MAX;
          __syncwarp();
          if (ln == 0) mbar_arrive(&sm.met[b]);
          for (int x = 0; x < NQ && ok; ++x) ok = wait_warp(&sm.met[x], meets, limit);
        }
      }
      if (!ok) break;
    }
  } else if (w < C::SW + C::PW) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::prod));
    // ---------------------------------------------------------------- producers
    const int pw = w - C::SW;
    constexpr int RPW = TK / C::PW;  // rows of a tile per warp
    static_assert(RPW <= 32, "a lane finds at most one row");
    Ring<NS> at_n, at_h;             // the next tile to issue, to hand on
    int pending = 0;                 // issued with cp.async, not handed on yet
    bool first = true;               // the ring's first turn: every slot is empty
    int nt = 0, kj = 0, vj = 0;
    const int64_t row_bytes = (int64_t)L.heads * D * (Q8 ? 1 : 2);
    // Block i of the piece's sequence, 0 behind its last position; a bad one is recorded and read as block 0.
    auto load_block = [&](int32_t i) {
      if ((int64_t)i * L.block_tokens >= pc.s.kv) return 0;
      int32_t blk = __ldg(p.b.table + (int64_t)pc.seq * p.b.max_blocks + i);
      if (blk < 0 || blk >= L.num_blocks) {
        report(L.status, LSC_ERR_OUT_OF_RANGE);
        blk = 0;
      }
      return blk;
    };
    // Table entries [base, base + 64) of the piece in the lanes' registers, the second half fetched a window ahead: a
    // lookup per tile would cost an L2 round trip, about a third of a tile's time (1000 of 3600 cycles measured).
    // Tiles reach at most 17 entries past V's first one, so two halves of 32 do; smaller blocks look up directly.
    const bool window = L.block_tokens >= 8;
    int32_t base_i = 0, near = 0, far = 0;
    auto block_of = [&](int32_t i) {  // converged; i may differ between lanes
      if (!window) return load_block(i);
      const int32_t o = i - base_i;
      const int32_t x = __shfl_sync(0xffffffffu, near, o & 31), y = __shfl_sync(0xffffffffu, far, o & 31);
      return o < 32 ? x : y;
    };
    // Block and row of a tile's first position (K's and V's walk), stepped by a tile; a lane adds its own offset.
    const int32_t tk_q = TK / L.block_tokens, tk_r = TK - tk_q * L.block_tokens;
    int32_t tq[2] = {0, 0}, tr[2] = {0, 0}, q0 = 0, r0 = 0;
    auto offset = [&](int32_t oq, int32_t orr, int32_t &q, int32_t &r) {
      q = q0 + oq;
      r = r0 + orr;
      if (r >= L.block_tokens) r -= L.block_tokens, ++q;
    };
    const int32_t my = pw * RPW + (ln < RPW ? ln : 0), my_q = my / L.block_tokens, my_r = my - my_q * L.block_tokens;
    // the next tile of the run, in the order of v_index
    auto next_tile = [&](bool &is_k, int &j) {
      while (vj >= nt) {
        if (!next_piece<M, TK>(p, run, pc)) return false;
        nt = pc.t1 - pc.t0;
        kj = vj = 0;
        tq[0] = tq[1] = (int32_t)((int64_t)pc.t0 * TK / L.block_tokens);
        tr[0] = tr[1] = (int32_t)((int64_t)pc.t0 * TK - (int64_t)tq[0] * L.block_tokens);
        if (window) {
          base_i = tq[0];
          near = load_block(base_i + ln);
          far = load_block(base_i + 32 + ln);
        }
      }
      is_k = NQ == 2 ? kj == vj : kj < nt && kj <= vj + 1;
      j = is_k ? kj++ : vj++;
      q0 = is_k ? tq[0] : tq[1];
      r0 = is_k ? tr[0] : tr[1];
      int32_t nq = q0 + tk_q, nr = r0 + tk_r;
      if (nr >= L.block_tokens) nr -= L.block_tokens, ++nq;
      if (is_k) tq[0] = nq, tr[0] = nr;
      else tq[1] = nq, tr[1] = nr;
      if (window && !is_k && q0 - base_i >= 32) {
        base_i += 32;
        near = far;
        far = load_block(base_i + 32 + ln);
      }
      return true;
    };
    // lane i's row of this warp's RPW rows of tile j: its byte offset in a lane, -1 behind the last position
    auto place = [&](int j, uint32_t *sb, bool is_k) {
      const int32_t pos = (pc.t0 + j) * TK + my;
      int32_t q, rr;
      offset(my_q, my_r, q, rr);
      const int64_t page = (int64_t)block_of(q) * L.page;
      if (ln >= RPW || pos >= pc.s.kv) return (int64_t)-1;
      if (Q8) *sb = __ldg((is_k ? L.k : L.v) + page + L.scale_off + (int64_t)rr * L.heads + pc.head);
      return page + (int64_t)rr * row_bytes + (int64_t)pc.head * D * (Q8 ? 1 : 2);
    };
    auto hand_on = [&]() {
      fence_proxy_async_smem();
      __syncwarp();
      if (ln == 0) mbar_arrive(&sm.full[at_h.slot]);
      at_h.step();
    };
    auto wait_empty = [&](const Ring<NS> &r) { return first || wait_warp(&sm.empty[r.slot], r.phase ^ 1, limit); };
    auto issued = [&]() {
      at_n.step();
      if (at_n.slot == 0) first = false;
    };
    bool is_k;
    int j;
    if constexpr (!Q8) {
      constexpr int CPR = D / 8;                        // 16-byte chunks of a row
      constexpr int RPI = 32 / CPR > 0 ? 32 / CPR : 1;  // rows per instruction
      constexpr int LAG = NS - 3;                       // cp.async tiles in flight before the first is handed on
      // TMA: a box of `box` rows and all columns when a block holds the tile, else of one column of 64 elements; the
      // boxes go over the lanes of all producer warps.  box 0: cp.async alone.
      const int box = p.box_rows, cols = box == TK ? D / 64 : 1, per = D / 64 / cols;
      const int boxes = box > 0 ? TK / box * per : 0, bi = ln * C::PW + pw, bc = bi % per;
      const int br = bi < boxes ? bi / per * box : 0, br_q = br / L.block_tokens, br_r = br - br_q * L.block_tokens;
      const uint32_t bytes = (uint32_t)((boxes - pw + C::PW - 1) / C::PW) * box * cols * 128;  // this warp's share
      while (ok && next_tile(is_k, j)) {
        const int slot = at_n.slot;
        uint8_t *dst = sm.ring[slot];
        if (box > 0 && (int64_t)(pc.t0 + j + 1) * TK <= pc.s.kv) {
          int32_t q, rr;
          offset(br_q, br_r, q, rr);
          const int32_t blk = block_of(q);
          if (!(ok = wait_empty(at_n))) break;
          if (ln == 0) {
            if (bytes) mbar_arrive_expect_tx(&sm.full[slot], bytes);
            else mbar_arrive(&sm.full[slot]);
          }
          __syncwarp();
          if (bi < boxes)
            tma_load_5d(dst + bc * (TK * 128) + br * 128, &map, 0, rr, bc, pc.head, blk + (is_k ? 0 : L.num_blocks),
                        &sm.full[slot]);
          if (pending > 0) {  // cp.async tiles before this one
            cp_async_wait<0>();
            for (; pending > 0; --pending) hand_on();
          }
          at_h.step();
          issued();
          continue;
        }
        const int64_t at = place(j, nullptr, is_k);
        if (!(ok = wait_empty(at_n))) break;
        const uint8_t *base = is_k ? L.k : L.v;
        const int ch = ln % CPR;
#pragma unroll
        for (int i = 0; i < RPW; i += RPI) {
          const int rl = i + ln / CPR, r = pw * RPW + rl;
          const int64_t a = __shfl_sync(0xffffffffu, at, rl);
          cp_async16_or_zero(smem_u32(dst + (ch >> 3) * (TK * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4)),
                             base + (a < 0 ? 0 : a) + ch * 16, a >= 0);
        }
        cp_async_commit();
        issued();
        if (++pending > LAG) {
          cp_async_wait<LAG>();
          hand_on();
          --pending;
        }
      }
      cp_async_wait<0>();
      for (; ok && pending > 0; --pending) hand_on();
    } else {
      // 16 codes (two chunks of the 16-bit row) a lane and instruction, through a ring of SD stages that belongs to the
      // thread: what it copies with cp.async it converts itself, so the copies need no barrier
      constexpr int SD = C::SD, LPR = D / 16, RPI = 32 / LPR, IT = RPW / RPI;
      const int lc = ln % LPR, th = pw * 32 + ln;
      uint32_t sb[SD];
#pragma unroll
      for (int i = 0; i < SD; ++i) sb[i] = 127;
      Ring<SD> st_in, st_out;
      int left = 0;  // tiles fetched and not converted
      auto fetch = [&]() {  // the run's next tile into its stage; an empty group when there is none
        uint32_t byte = 127;
        if (ok && next_tile(is_k, j)) {
          const int64_t at = place(j, &byte, is_k);
          const uint8_t *base = is_k ? L.k : L.v;
#pragma unroll
          for (int i = 0; i < IT; ++i) {
            const int64_t a = __shfl_sync(0xffffffffu, at, i * RPI + ln / LPR);
            cp_async16_or_zero(smem_u32(&sm.stage[st_in.slot][i][th]), base + (a < 0 ? 0 : a) + lc * 16, a >= 0);
          }
          st_in.step();
          ++left;
        }
        cp_async_commit();
#pragma unroll
        for (int i = 0; i + 1 < SD; ++i) sb[i] = sb[i + 1];
        sb[SD - 1] = byte;
      };
      for (int g = 0; g < SD; ++g) fetch();
      for (; left > 0; --left) {
        cp_async_wait<SD - 1>();
        if (!(ok = wait_empty(at_n))) break;
        uint8_t *dst = sm.ring[at_n.slot];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int rl = i * RPI + ln / LPR, r = pw * RPW + rl;
          const float k = scale_of(__shfl_sync(0xffffffffu, sb[0], rl));
          const uint4 code = sm.stage[st_out.slot][i][th];
          const uint32_t cw[4] = {code.x, code.y, code.z, code.w};
          uint32_t o[8];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 lo = e4m3x2_to_float2(cw[x] & 0xffffu), hi = e4m3x2_to_float2(cw[x] >> 16);
            o[2 * x] = pack2(lo.x * k, lo.y * k, BF16);
            o[2 * x + 1] = pack2(hi.x * k, hi.y * k, BF16);
          }
          const int ch = 2 * lc;
          uint8_t *row = dst + (ch >> 3) * (TK * 128) + r * 128;
          *(uint4 *)(row + (((ch & 7) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          *(uint4 *)(row + ((((ch & 7) + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        hand_on();
        issued();
        st_out.step();
        fetch();
      }
      cp_async_wait<0>();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::mma));
  }
  if (w == C::SW + C::PW) {
    // ---------------------------------------------------------------- products
    const bool lead = tc::elect_one();
    constexpr uint32_t iqk = idesc_f16(128, TK, BF16, false), ipv = idesc_f16(128, D, BF16, true);
    Ring<NS> at;  // the next tile of the ring to wait for
    uint32_t itb[2] = {0, 0}, pieces[2] = {0, 0};
    const uint32_t ring0 = smem_u32(sm.ring[0]), q0 = smem_u32(sm.q);
    auto wait = [&](uint64_t *bar, uint32_t phase) {
      if (ok) ok = wait_bar(bar, phase, limit);
      return ok;
    };
    auto next_slot = [&](int &slot) {  // waits for the ring's next tile
      slot = at.slot;
      const bool r = wait(&sm.full[at.slot], at.phase);
      at.step();
      tc::fence_after_sync();
      return r;
    };
    auto scores = [&](int b, int sb, int slot) {  // S[sb] = Q[b] K^T
      if (lead) {
        const uint32_t kb = ring0 + slot * C::slot, qb = q0 + b * 128 * D * 2;
        const uint32_t d = tm + C::S0 + sb * C::SN;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t bd = desc128(kb + (k >> 2) * (TK * 128) + (k & 3) * 32, 16, 1024);
          if constexpr (C::QT) mma_ts16(d, tm + C::Q0 + k * 8, bd, iqk, k > 0);
          else mma_ss16(d, desc128(qb + (k >> 2) * 16384 + (k & 3) * 32, 16, 1024), bd, iqk, k > 0);
        }
        tc::mma_commit(&sm.sfull[sb]);
      }
    };
    auto values = [&](int b, int sb, int slot, bool fresh, bool last) {  // O[b] (+)= P[sb] V
      if (lead) {
        const uint32_t vb = ring0 + slot * C::slot;
#pragma unroll
        for (int k = 0; k < TK / 16; ++k)
          mma_ts16(tm + C::O0 + b * D, tm + C::S0 + sb * C::SN + k * 8, desc128(vb + k * 2048, TK * 128, 1024), ipv,
                   !(fresh && k == 0));
        tc::mma_commit(&sm.odone[b]);
        if (last) tc::mma_commit(&sm.fin[b]);
      }
    };
    auto release = [&](int slot) {
      if (lead) tc::mma_commit(&sm.empty[slot]);
    };
    int ks, vs;
    while (ok && next_piece<M, TK>(p, run, pc)) {
      const int nt = pc.t1 - pc.t0;
      const int64_t rows = (int64_t)pc.s.n * p.group - (int64_t)pc.block * M;
      const int nb = NQ == 2 && rows > 128 ? 2 : 1;
      for (int b = 0; b < nb; ++b)
        if (!wait(&sm.qfull[b], pieces[b]++)) break;
      if (!ok || !next_slot(ks)) break;
      if constexpr (NQ == 2) {
        for (int b = 0; b < nb; ++b) scores(b, b, ks);
        release(ks);
        for (int j = 0; j < nt; ++j) {
          if (!next_slot(vs)) break;
          for (int b = 0; b < nb; ++b) {
            if (!wait(&sm.pfull[b], itb[b]++)) break;
            tc::fence_after_sync();
            values(b, b, vs, j == 0, j == nt - 1);
            if (b == nb - 1) release(vs);
            if (j + 1 < nt) {
              if (b == 0 && !next_slot(ks)) break;
              scores(b, b, ks);
              if (b == nb - 1) release(ks);
            }
          }
          if (!ok) break;
        }
      } else {
        uint32_t &it = itb[0];
        scores(0, (int)(it & 1), ks);
        release(ks);
        for (int j = 0; j < nt; ++j, ++it) {
          if (j + 1 < nt) {
            if (!next_slot(ks)) break;
            scores(0, (int)((it + 1) & 1), ks);
            release(ks);
          }
          if (!next_slot(vs) || !wait(&sm.pfull[it & 1], it >> 1)) break;
          tc::fence_after_sync();
          values(0, (int)(it & 1), vs, j == 0, j == nt - 1);
          release(vs);
        }
      }
    }
    // everything issued has completed before TMEM is freed
    if (lead) tc::mma_commit(&sm.drain);
    __syncwarp();
    if (!mbar_wait_bounded(&sm.drain, 0, p.drain_limit_ns)) ok = false;
  }
  if (!ok && ln == 0) report(L.status, LSC_ERR_DEV_TIMEOUT);
  if (tid == 0 && p.ws) workspace_at(p.ws, ctas, M).cut[cta] = cut;
  tc::fence_before_sync();
  __syncthreads();
  if (w == C::SW + C::PW) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tm, 512);
  }
}

template <bool BF16, bool Q8, int D>
cudaError_t launch_one(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  static SmemLimit limit;
  auto *k = chunk_attend_kernel<BF16, Q8, D>;
  const int smem = (int)sizeof(Smem<D, Q8>);
  const cudaError_t e = limit.ensure((const void *)k, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, plan.ctas, kThreads, smem, stream, p, p.map ? *p.map : CUtensorMap{});
}

template <bool BF16, bool Q8>
cudaError_t launch_type(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  switch (p.L.head_dim) {
    case 64: return launch_one<BF16, Q8, 64>(p, plan, stream);
    case 128: return launch_one<BF16, Q8, 128>(p, plan, stream);
    default: return launch_one<BF16, Q8, 256>(p, plan, stream);
  }
}

}  // namespace chunk
}  // namespace kv

cudaError_t launch_kv_attend_chunk_bf16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
cudaError_t launch_kv_attend_chunk_f16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
cudaError_t launch_kv_attend_chunk_e4m3(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);

}  // namespace lsc
