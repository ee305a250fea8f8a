// lsc_kv_attend_chunk.cuh -- attention over a layer of the K/V block pool for
// sequences with many packed rows (lsc_kv_attend.cuh): prefill chunks.
//
// 4 * head_dim operations a (row, position) pair, and K/V tiles that serve 128 or
// 256 rows: the 5th-generation tensor cores bound it.  One CTA per SM walks its
// run of tiles of TK positions with the warps in roles:
//   * two softmax warpgroups, one thread a row: wait for the scores S = Q K^T of a
//     tile in TMEM, weights 2^(s - m) to 16 bits back into the same TMEM columns,
//     sum in a register.  m is a reference, not the exact maximum: O is rescaled
//     (in TMEM, by these threads) only when a row's maximum rose by more than 2^8,
//     so a weight is at most 2^8 and the rescale is rare after the first tiles.
//   * one MMA warp: S = Q K^T, O += P V with P as the TMEM operand, issued so that
//     the products of one tile run while the softmax of another does.
//   * producers: K and V rows through the block table into a shared-memory ring
//     (K(0), V(0), K(1), V(1) ...) in the 128-byte-swizzled layout.  16-bit pools:
//     a warp for K and one for V.  Blocks that are a multiple of 8 tokens come
//     as tiled TMA boxes of rows x 64 elements (x head_dim / 64 when a block holds
//     the tile: then one box a tile; coordinates (element, row, column of 64, head,
//     block) of the layer, element always 0); other block sizes with 16-byte
//     cp.async.  E4M3 pools: four warps each, codes the same two ways into a staging
//     buffer, then bf16 with their scale (exact above bf16's smallest normal).  V
//     rows behind the last position become zeros: here, where they are copied or
//     converted, else by the softmax threads.
// head_dim 64 and 128: two row blocks of 128, one per softmax warpgroup, each with
// its own S and O (S 2 x 128, O 2 x head_dim columns of TMEM), Q in shared memory,
// tiles of 128: one block's softmax runs under the other's products, and a K/V
// tile is fetched once for 256 rows.
// head_dim 256: O takes 256 columns, so one row block, tiles of 64 and two S
// buffers; the warpgroups take the tiles in turn, so that a tile's softmax has two
// tiles' time, and hand the reference m on through shared memory.  Q is a TMEM
// operand (128 columns), which leaves shared memory to K and V and halves what the
// score products read from it.
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

template <int D, bool Q8>
struct Conf {
  static constexpr int NQ = D == 256 ? 1 : 2;   // row blocks of 128
  static constexpr int M = 128 * NQ;
  static constexpr int TK = D == 256 ? 64 : 128;
  static constexpr bool QT = D == 256;          // Q in TMEM
  static constexpr int slot = TK * D * 2;       // bytes of a K or V tile
  static constexpr int NS = Q8 ? (D == 64 ? 6 : D == 128 ? 3 : 4) : (D == 64 ? 8 : D == 128 ? 4 : 6);
  static constexpr int SD = D == 128 ? 1 : 2;   // E4M3: stages of codes
  // warps: 0-7 softmax, 8 MMA, 16-bit pools 9 K and 10 V, E4M3 12-15 K and 16-19 V
  static constexpr int threads = Q8 ? 640 : 384;
  static constexpr int GW = Q8 ? 4 : 1;         // producer warps of a tile
  static constexpr bool hold = !Q8 || TK == 64; // a thread keeps all scores of a tile in registers
  // registers a thread of a softmax warpgroup, the MMA's and E4M3's producers' keeps of those at launch
  static constexpr int soft = Q8 ? 144 : 208, mma = Q8 ? 56 : 80, prod = 64;
  static_assert(2 * soft + mma + (Q8 ? 2 * prod : 0) <= (Q8 ? 5 * 96 : 3 * 168), "more registers than the block has");
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
  alignas(128) uint8_t stage[2][Q8 ? C::SD : 1][Q8 ? C::TK * D : 16];  // E4M3: tiles of codes, K's and V's
  alignas(16) uint8_t rows[8][32][80];  // by softmax warp: 64 bytes of each of its rows, between TMEM and memory
  int32_t bad[3][D];      // first position whose v is NaN, +inf, -inf
  uint64_t full[C::NS], empty[C::NS], sfull[2], pfull[2], qfull[2], odone[2], fin[2], met[2], drain;
  uint64_t ready[2][2], freed[2][2];  // E4M3: by K or V and stage
  uint64_t turn[2][4], swap[2][4];   // one row block: by warpgroup and warp
  float ref[C::NQ == 1 ? 128 : 1];   // a row's reference m
  float2 ml[2][2][C::NQ == 1 ? 128 : 1];  // (m, sum) by piece parity and warpgroup
  uint32_t tmem;
  int32_t any_bad;
  RunScratch run;
};

// Low word of a shared-memory matrix descriptor: start address and leading byte offset.  The high word is the stride
// byte offset (1024: groups of 8 rows of 128 bytes), version 1 (bit 46) and the 128-byte swizzle (bits 61-63 = 2).  A
// descriptor further along is the low word plus bytes / 16, so a product's 16 descriptors need no registers of their own.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | (lbo >> 4) << 16;
}
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;
// Instruction descriptor of kind::f16 with an fp32 accumulator: both operands f16 (0) or bf16 (1).
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool bf16, bool b_mn_major) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_ss16(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(kDescHi),
      "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts16(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(kDescHi),
      "r"(acc)
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

// Codes in the high bytes of two halves -> bf16 bits with the same sign, exponent field and mantissa, worth the codes
// times 2^-120: the exponent bias of e4m3 is 7, of bf16 127, and a subnormal code becomes a subnormal bf16.
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2_bits(uint32_t x) {
  return ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
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

// A walk over the ring's slots of K (from 0) or V (from 1).  Counting modulo a number that is no power of two, or
// dividing by a block size, costs a lone warp a hundred cycles and more each time, so the roles step instead.
template <int NS>
struct Ring {
  int slot;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Ring(int first) : slot(first) {}
  __device__ __forceinline__ void step() {
    slot += 2;
    if (slot >= NS) slot -= NS, phase ^= 1;
  }
};

template <bool BF16, bool Q8, int D>
__global__ void __launch_bounds__(Conf<D, Q8>::threads, 1)
chunk_attend_kernel(const __grid_constant__ KvAttendParams p, const __grid_constant__ CUtensorMap map) {
  using C = Conf<D, Q8>;
  constexpr int NQ = C::NQ, M = C::M, TK = C::TK, NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D, Q8> &sm = *reinterpret_cast<Smem<D, Q8> *>(smem_raw);
  const int tid = threadIdx.x, w = tid >> 5, ln = tid & 31;
  const KvLayer &L = p.L;
  if (w == 8) {
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&sm.full[i], C::GW), mbar_init(&sm.empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.sfull[i], 1), mbar_init(&sm.pfull[i], 4), mbar_init(&sm.qfull[i], NQ == 2 ? 4 : 8);
      mbar_init(&sm.odone[i], 1), mbar_init(&sm.fin[i], 1), mbar_init(&sm.met[i], 4);
      for (int x = 0; x < 2; ++x) mbar_init(&sm.ready[i][x], 1), mbar_init(&sm.freed[i][x], C::GW);
      for (int x = 0; x < 4; ++x) mbar_init(&sm.turn[i][x], 1), mbar_init(&sm.swap[i][x], 1);
    }
    mbar_init(&sm.drain, 1);
    fence_mbar_init();
    sm.any_bad = 0;
  }
  for (int i = tid; i < 3 * D; i += C::threads) (&sm.bad[0][0])[i] = INT32_MAX;
  griddep_wait();
  if (tid == 0) griddep_launch_dependents();
  const int ctas = gridDim.x, cta = blockIdx.x;
  if (cta == 0) check_cu(L, p.b);
  tc::fence_before_sync();
  Run run = find_run<C::threads, M, TK>(p, cta, ctas, sm.run);
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = sm.tmem;
  const uint64_t limit = p.wait_limit_ns;
  bool ok = true;
  Cut cut = {0, 0, 0, 0};
  Piece pc;

  if (w < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::soft));
    // ---------------------------------------------------------------- softmax
    const int b = w >> 2, pair = w & 3, row = pair * 32 + ln;  // warpgroup; row of its row block
    const int block = NQ == 2 ? b : 0;                         // row block
    const uint32_t lane = (uint32_t)(pair * 32) << 16;
    const Workspace ws = workspace_at(p.ws, ctas, M);
    const float c = p.scale_log2;
    auto rows_of = [&](const Piece &q) {  // packed rows of the unit
      const int32_t r = q.s.n * p.group - q.block * M;
      return r < M ? r : M;
    };
    // Rows of Q and of the result move 64 bytes a row and 8 rows an instruction: a lane a row would touch 32 sectors
    // with 16 bytes each (8000 cycles for a unit's rows, measured on short chunks).
    uint8_t(&mine_rows)[32][80] = sm.rows[w];
    const int oct = ln >> 2, part16 = (ln & 3) * 16;
    // two row blocks: this warpgroup's rows to shared memory; one: its half of every row to TMEM
    auto load_q = [&](const Piece &q) {
      const int r = block * 128 + row;
      const int32_t R = q.block * M + r, tok = p.by_group.div(R);
      const uint8_t *src = r < rows_of(q) ? (const uint8_t *)p.q + 2 * ((int64_t)(q.s.row0 + tok) * p.q_stride +
                                                                        (int64_t)(q.head * p.group + (R - tok * p.group)) * D)
                                          : nullptr;
      if (C::QT && src) src += b * D;
      const uint8_t *from[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) from[i] = (const uint8_t *)__shfl_sync(0xffffffffu, (unsigned long long)src, i * 8 + oct);
#pragma unroll 4
      for (int x = 0; x < (C::QT ? D : 2 * D); x += 64) {  // bytes of a row
        uint4 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          y[i] = from[i] ? *(const uint4 *)(from[i] + x + part16) : make_uint4(0, 0, 0, 0);
        if constexpr (C::QT) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) *(uint4 *)&mine_rows[i * 8 + oct][part16] = y[i];
          __syncwarp();
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 z = *(const uint4 *)&mine_rows[ln][i * 16];
            v[4 * i] = z.x, v[4 * i + 1] = z.y, v[4 * i + 2] = z.z, v[4 * i + 3] = z.w;
          }
          tc::tmem_st16(tm + lane + C::Q0 + b * (D / 4) + x / 4, v);
        } else {
          uint8_t *dst = sm.q + b * 128 * D * 2 + (x >> 7) * 16384;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = pair * 32 + i * 8 + oct, ch = ((x >> 4) & 4) + (ln & 3);
            *(uint4 *)(dst + rr * 128 + ((ch ^ (rr & 7)) << 4)) = y[i];
          }
        }
      }
      if constexpr (C::QT) {
        tc::tmem_wait_st();
        tc::fence_before_sync();
      } else {
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (ln == 0) mbar_arrive(&sm.qfull[block]);
    };
    bool have = next_piece<M, TK>(p, run, pc);
    if (have && block * 128 < rows_of(pc)) load_q(pc);
    uint32_t it = 0;     // tiles this row block has been through
    uint32_t slots = 0;  // ring slots of the pieces before this one, modulo 2 NS
    uint32_t meets = 0, done = 0, turns = 0;
    while (have && ok) {
      const int nt = pc.t1 - pc.t0, rows = rows_of(pc);
      const bool mine = block * 128 < rows;
      const int r = block * 128 + row;
      const int32_t R = pc.block * M + r, tok = p.by_group.div(R);
      const int32_t vis = r < rows ? visible(pc.s, tok, p.causal) : 0;
      const int32_t sure = visible(pc.s, p.by_group.div(pc.block * M), p.causal);
      const int32_t full_to = NQ == 2 && b == 1 && mine
                                  ? visible(pc.s, p.by_group.div(pc.block * M + 128), p.causal)
                                  : sure;  // every row of this block sees positions below it
      const bool rows_all = (block + 1) * 128 <= rows;
      float m = -INFINITY, l = 0.f;
      // does the piece reach positions that some row of the unit does not see
      const bool mixed = (pc.s.kv < pc.t1 * TK ? pc.s.kv : pc.t1 * TK) > sure;
      for (int j = 0; j < nt && mine; ++j, ++it) {
        if (NQ == 1 && (int)(it & 1) != b) continue;  // the other warpgroup's
        const uint32_t sa = tm + lane + C::S0 + b * C::SN;
        const int32_t first = (pc.t0 + j) * TK;
        if (!(ok = wait_warp(&sm.sfull[b], NQ == 2 ? it : it >> 1, limit))) break;
        tc::fence_after_sync();
        // a column is seen when first + column < vis
        const bool mask = first + TK > full_to || !rows_all;
        const int32_t seen = vis - first;
        constexpr int NC = TK / 32;                 // chunks of 32 columns
        uint32_t s[C::hold ? NC : 2][32];
        float top;
        tc::tmem_ld32(sa, s[0]);
        wait_ld(s[0]);
        if constexpr (C::hold) {
#pragma unroll
          for (int x = 1; x < NC; ++x) tc::tmem_ld32(sa + 32 * x, s[x]);
          if (mask) hide(s[0], seen);
          top = top_of(s[0]);
#pragma unroll
          for (int x = 1; x < NC; ++x) {
            wait_ld(s[x]);
            if (mask) hide(s[x], seen - 32 * x);
            top = fmaxf(top, top_of(s[x]));
          }
        } else {  // twice through TMEM, the next chunk on its way while one is looked at
          top = -INFINITY;
#pragma unroll
          for (int x = 0; x < NC; ++x) {
            if (x + 1 < NC) tc::tmem_ld32(sa + 32 * x + 32, s[(x + 1) & 1]);
            if (mask) hide(s[x & 1], seen - 32 * x);
            top = fmaxf(top, top_of(s[x & 1]));
            if (x + 1 < NC) wait_ld(s[(x + 1) & 1]);
          }
          tc::tmem_ld32(sa, s[0]);
        }
        const float mt = top * c;  // c > 0
        float old = m;             // the reference that l goes by
        if (NQ == 1 && j > 0) {
          if (!(ok = wait_warp(&sm.turn[b][pair], turns++, limit))) break;
          m = sm.ref[row];
        }
        if (__any_sync(0xffffffffu, mt > m + 8.f)) {  // also the first tile's (m is -inf)
          const float to = fmaxf(m, mt), f = ex2(m - (to == -INFINITY ? 0.f : to));
          m = to;
          if (j > 0) {
            if (!(ok = wait_warp(&sm.odone[block], it - 1, limit))) break;
            tc::fence_after_sync();
            const uint32_t oa = tm + lane + C::O0 + block * D;
#pragma unroll 1
            for (int x = 0; x < D; x += 32) {
              uint32_t o[32];
              tc::tmem_ld32(oa + x, o);
              wait_ld(o);
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tc::tmem_st32(oa + x, o);
            }
          }
          if (NQ == 1) sm.ref[row] = m;
        }
        if (NQ == 1 && j + 1 < nt) {  // the other warpgroup's next tile goes by this reference
          __syncwarp();
          if (ln == 0) mbar_arrive(&sm.turn[b ^ 1][pair]);
        }
        const float ref = m == -INFINITY ? 0.f : m;
        if (__any_sync(0xffffffffu, old != m)) l *= ex2(old - ref);
        const uint64_t c2 = two(c, c), r2 = two(-ref, -ref);
        uint64_t l2 = two(0.f, 0.f);
        if constexpr (!C::hold) wait_ld(s[0]);
#pragma unroll
        for (int x = 0; x < NC; ++x) {
          uint32_t q[16];
          auto &sx = s[C::hold ? x : x & 1];
          if constexpr (!C::hold) {
            if (x + 1 < NC) tc::tmem_ld32(sa + 32 * x + 32, s[(x + 1) & 1]);
            if (mask) hide(sx, seen - 32 * x);
          }
          weights<BF16>(sx, c2, r2, l2, q);
          if constexpr (!C::hold) {
            if (x + 1 < NC) wait_ld(s[(x + 1) & 1]);
          }
          tc::tmem_st16(sa + 16 * x, q);  // over columns that have been read
        }
        const float2 lf = *reinterpret_cast<const float2 *>(&l2);
        l += lf.x + lf.y;
        const int32_t last = first + TK < pc.s.kv ? first + TK : pc.s.kv;
        // positions [max(first, sure), last): some row of the unit does not see them; behind last: a 16-bit block's rows
        // came as they were
        if (last > sure || (!Q8 && last < first + TK)) {
          const uint32_t vi = slots + 2 * j + 1;
          const int slot = (int)(vi % NS);
          if (!(ok = wait_warp(&sm.full[slot], vi / NS, limit))) break;
          if (!Q8)
            for (int i = row; i < (first + TK - last) * (D / 8); i += 128) {
              const int key = last - first + i / (D / 8), ch = i % (D / 8);
              *(uint4 *)(sm.ring[slot] + (ch >> 3) * (TK * 128) + key * 128 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
            }
          const int lo = (sure > first ? sure : first) - first, cnt = last - first - lo;  // cnt <= 0: nothing to search
          // an exponent field of ones carries into the sign's place
          constexpr uint32_t E = BF16 ? 0x7f80 : 0x7c00, up = (0x8000 - E) * 0x10001u;
          auto vec = [&](int i) {
            const int key = lo + i / (D / 8), ch = i % (D / 8);
            return (uint4 *)(sm.ring[slot] + (ch >> 3) * (TK * 128) + key * 128 + (((ch & 7) ^ (key & 7)) << 4));
          };
          uint32_t carry = 0;
#pragma unroll 2
          for (int i = row; i < cnt * (D / 8); i += 128) {
            const uint4 v = *vec(i);
            carry |= ((v.x & 0x7fff7fffu) + up) | ((v.y & 0x7fff7fffu) + up) | ((v.z & 0x7fff7fffu) + up) |
                     ((v.w & 0x7fff7fffu) + up);
          }
          if (carry & 0x80008000u) {
#pragma unroll 1
            for (int i = row; i < cnt * (D / 8); i += 128) {
              uint16_t *e = (uint16_t *)vec(i);
#pragma unroll 1
              for (int x = 0; x < 8; ++x) {
                const uint32_t u = e[x];
                if ((u & E) != E) continue;
                atomicMin(&sm.bad[(u & (E ^ 0x7fff)) ? 0 : (u & 0x8000) ? 2 : 1][i % (D / 8) * 8 + x], first + lo + i / (D / 8));
                e[x] = 0;
              }
            }
            sm.any_bad = 1;
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (ln == 0) mbar_arrive(&sm.pfull[b]);
      }
      if (!ok) break;
      if (NQ == 1) {  // the warpgroups' sums of each row, by the later reference; then both know that Q has been used
        sm.ml[done & 1][b][row] = make_float2(m, l);
        __syncwarp();
        if (ln == 0) mbar_arrive(&sm.swap[b ^ 1][pair]);
        if (!(ok = wait_warp(&sm.swap[b][pair], done, limit))) break;
        const float2 x = sm.ml[done & 1][b ^ 1][row];
        const float to = fmaxf(m, x.x), ref = to == -INFINITY ? 0.f : to;
        // in the same order in both
        const float la = (b == 0 ? l : x.y) * ex2((b == 0 ? m : x.x) - ref), lb = (b == 0 ? x.y : l) * ex2((b == 0 ? x.x : m) - ref);
        l = la + lb;
        m = to;
      }
      const Piece q = pc;
      cut = cut_of(run, q, cta);
      slots = (slots + 2 * (uint32_t)nt) % (2 * NS);
      have = next_piece<M, TK>(p, run, pc);
      if (have && block * 128 < rows_of(pc)) load_q(pc);  // this piece's score products are done
      if (mine) {
        // a barrier of its own: odone may be up to two phases behind here, and a parity tells two apart, not three
        if (!(ok = wait_warp(&sm.fin[block], done++, limit))) break;
        tc::fence_after_sync();
        const bool whole = q.t0 == 0 && q.t1 == q.tiles;
        const bool empty = l == 0.f;
        const float inv = whole ? (empty ? 0.f : 1.f / l) : 1.f;
        const int64_t h = q.head * p.group + (R - tok * p.group), t = q.s.row0 + tok;
        const int64_t slot = (int64_t)(2 * cta + (q.t0 == 0 ? 1 : 0)) * M + r;
        const bool on = r < rows;
        const bool look = mixed && *(volatile int32_t *)&sm.any_bad != 0;
        uint8_t *dst = !on ? nullptr : whole ? (uint8_t *)((uint16_t *)p.out + t * p.out_stride + h * D) : (uint8_t *)(ws.o + slot * D);
        uint8_t *to[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = (uint8_t *)__shfl_sync(0xffffffffu, (unsigned long long)dst, i * 8 + oct);
        const uint32_t oa = tm + lane + C::O0 + block * D;
        constexpr int half = NQ == 1 ? D / 2 : D;  // one row block: each warpgroup writes half of a row
#pragma unroll 1
        for (int x = NQ == 1 ? b * half : 0, end = x + half; x < end; x += 32) {
          uint32_t o[32];
          tc::tmem_ld32(oa + x, o);
          wait_ld(o);
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
          auto rows_out = [&](const uint32_t (&v)[16], int at) {  // 64 bytes of every row
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *(uint4 *)&mine_rows[ln][i * 16] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (to[i]) *(uint4 *)(to[i] + at + part16) = *(const uint4 *)&mine_rows[i * 8 + oct][part16];
          };
          uint32_t v[16];
          if (whole) {
#pragma unroll
            for (int y = 0; y < 16; ++y) v[y] = pack2(__uint_as_float(o[2 * y]), __uint_as_float(o[2 * y + 1]), BF16);
            rows_out(v, x * 2);
          } else {
#pragma unroll
            for (int y = 0; y < 16; ++y) v[y] = o[y];
            rows_out(v, x * 4);
#pragma unroll
            for (int y = 0; y < 16; ++y) v[y] = o[16 + y];
            rows_out(v, x * 4 + 64);
          }
          __syncwarp();
        }
        if (on && (NQ == 2 || b == 0)) {
          if (!whole) ws.ml[slot] = make_float2(m, l);
          else if (p.lse) p.lse[t * p.heads + h] = empty ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
        }
        tc::fence_before_sync();  // these reads before the next piece's products, through pfull
      }
      if (mixed && have) {  // the next unit starts with a clean list: all softmax warps meet before and after it is cleared
        for (int round = 0; round < 2 && ok; ++round, ++meets) {
          if (round == 1 && *(volatile int32_t *)&sm.any_bad)
            for (int i = tid; i < 3 * D; i += 256) (&sm.bad[0][0])[i] = INT32_MAX;
          __syncwarp();
          if (ln == 0) mbar_arrive(&sm.met[b]);
          for (int x = 0; x < 2 && ok; ++x) ok = wait_warp(&sm.met[x], meets, limit);
        }
      }
    }
  } else if (w < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::mma));
  }
  if ((!Q8 && (w == 9 || w == 10)) || (Q8 && w >= 12)) {
    if constexpr (Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::prod));
    // ---------------------------------------------------------------- producers
    const bool is_k = Q8 ? w < 16 : w == 9;
    const uint8_t *base = is_k ? L.k : L.v;
    Ring<NS> at(is_k ? 0 : 1);
    const int64_t row_bytes = (int64_t)L.heads * D * (Q8 ? 1 : 2);
    int32_t blocks_held = 0;  // of the piece's sequence
    // Block i of the piece's sequence, 0 behind its last position; a bad one is recorded and read as block 0.
    auto load_block = [&](int32_t i) {
      if (i >= blocks_held) return 0;
      int32_t blk = __ldg(p.b.table + (int64_t)pc.seq * p.b.max_blocks + i);
      if (blk < 0 || blk >= L.num_blocks) {
        report(L.status, LSC_ERR_OUT_OF_RANGE);
        blk = 0;
      }
      return blk;
    };
    // Table entries [base_i, base_i + 64) of the piece in the lanes' registers, the second half fetched a window ahead:
    // a lookup per tile would cost an L2 round trip.  A tile reaches at most 16 entries; smaller blocks look up directly.
    const bool window = L.block_tokens >= 8;
    int32_t base_i = 0, near = 0, far = 0;
    auto block_of = [&](int32_t i) {  // converged; i may differ between lanes
      if (!window) return load_block(i);
      const int32_t o = i - base_i;
      const int32_t x = __shfl_sync(0xffffffffu, near, o & 31), y = __shfl_sync(0xffffffffu, far, o & 31);
      return o < 32 ? x : y;
    };
    // Block and row of a tile's first position, stepped by a tile; a lane adds its own offset.
    const int32_t tk_q = L.by_block.div(TK), tk_r = TK - tk_q * L.block_tokens;
    int32_t q0 = 0, r0 = 0;
    auto start = [&]() {
      blocks_held = L.by_block.div(pc.s.kv + L.block_tokens - 1);
      q0 = L.by_block.div(pc.t0 * TK);
      r0 = pc.t0 * TK - q0 * L.block_tokens;
      if (window) {
        base_i = q0;
        near = load_block(base_i + ln);
        far = load_block(base_i + 32 + ln);
      }
    };
    auto step = [&]() {
      q0 += tk_q;
      r0 += tk_r;
      if (r0 >= L.block_tokens) r0 -= L.block_tokens, ++q0;
      if (window && q0 - base_i >= 32) {
        base_i += 32;
        near = far;
        far = load_block(base_i + 32 + ln);
      }
    };
    // byte offset in a lane of the row of position `off` of tile j, (oq, orr) = off by blocks; -1 behind the last position
    auto place = [&](int j, int32_t off, int32_t oq, int32_t orr, uint32_t *sb) {
      int32_t q = q0 + oq, rr = r0 + orr;
      if (rr >= L.block_tokens) rr -= L.block_tokens, ++q;
      const int64_t page = (int64_t)block_of(q) * L.page;
      if ((pc.t0 + j) * TK + off >= pc.s.kv) return (int64_t)-1;
      if (Q8) *sb = __ldg(base + page + L.scale_off + (int64_t)rr * L.heads + pc.head);
      return page + (int64_t)rr * row_bytes + (int64_t)pc.head * D * (Q8 ? 1 : 2);
    };
    auto hand_on = [&](int slot) {
      fence_proxy_async_smem();
      __syncwarp();
      if (ln == 0) mbar_arrive(&sm.full[slot]);
    };
    // the ring's first turn passes at once: the phase before a fresh barrier's first one counts as complete
    auto wait_empty = [&]() { return wait_warp(&sm.empty[at.slot], at.phase ^ 1, limit); };
    if constexpr (!Q8) {
      constexpr int CPR = D / 8, RPI = 32 / CPR > 0 ? 32 / CPR : 1;  // 16-byte chunks of a row, rows an instruction
      constexpr int LAG = (NS - 1) / 2;  // cp.async tiles in flight before the first is handed on
      // TMA: a box of `box` rows and all columns when a block holds the tile, else of one column of 64 elements, a box a
      // lane.  box 0: cp.async alone.
      const int box = p.box_rows, cols = box == TK ? D / 64 : 1, per = D / 64 / cols;
      const int boxes = box > 0 ? TK / box * per : 0, bc = ln % per, br = ln < boxes ? ln / per * box : 0;
      const int br_q = L.by_block.div(br), br_r = br - br_q * L.block_tokens;
      int pending = 0;
      uint32_t flying = 0;  // slots that TMA has filled (low byte), in which phase last (the next byte)
      Ring<NS> at_h = at;  // the next tile to hand on
      while (ok && next_piece<M, TK>(p, run, pc)) {
        const int nt = pc.t1 - pc.t0;
        start();
        for (int j = 0; j < nt; ++j, at.step(), step()) {
          uint8_t *dst = sm.ring[at.slot];
          if (box > 0) {
            int32_t q = q0 + br_q, rr = r0 + br_r;
            if (rr >= L.block_tokens) rr -= L.block_tokens, ++q;
            const int32_t blk = block_of(q);
            if (!(ok = wait_empty())) break;
            if (ln == 0) mbar_arrive_expect_tx(&sm.full[at.slot], C::slot);
            __syncwarp();
            if (ln < boxes)
              tma_load_5d(dst + bc * (TK * 128) + br * 128, &map, 0, rr, bc, pc.head, blk + (is_k ? 0 : L.num_blocks),
                          &sm.full[at.slot]);
            flying = flying & ~(0x101u << at.slot) | (1u | at.phase << 8) << at.slot;
            if (pending > 0) {  // cp.async tiles before this one
              cp_async_wait<0>();
              for (; pending > 0; --pending, at_h.step()) hand_on(at_h.slot);
            }
            at_h.step();
            continue;
          }
          int64_t row_at[TK / 32];
#pragma unroll
          for (int g = 0; g < TK / 32; ++g) {
            const int32_t off = g * 32 + ln, oq = L.by_block.div(off);
            row_at[g] = place(j, off, oq, off - oq * L.block_tokens, nullptr);
          }
          if (!(ok = wait_empty())) break;
          const int ch = ln % CPR;
#pragma unroll
          for (int g = 0; g < TK / 32; ++g)
#pragma unroll 4
            for (int i = 0; i < 32; i += RPI) {
              const int r = i + ln / CPR;
              const int64_t a = __shfl_sync(0xffffffffu, row_at[g], r);
              cp_async16_or_zero(smem_u32(dst + (ch >> 3) * (TK * 128) + (g * 32 + r) * 128 + (((ch & 7) ^ (r & 7)) << 4)),
                                 base + (a < 0 ? 0 : a) + ch * 16, a >= 0);
            }
          cp_async_commit();
          if (++pending > LAG) {
            cp_async_wait<LAG>();
            hand_on(at_h.slot);
            at_h.step();
            --pending;
          }
        }
      }
      cp_async_wait<0>();
      for (; ok && pending > 0; --pending, at_h.step()) hand_on(at_h.slot);
      if (!ok)  // a wait gave up: nothing may be in flight when the CTA leaves
        for (int i = 0; i < NS; ++i)
          if (flying >> i & 1) wait_warp(&sm.full[i], flying >> (8 + i), p.drain_limit_ns);
    } else {
      // 16 codes (two chunks of the 16-bit row) a lane and pass, through SD stages of codes per kind.  Tiles come by TMA
      // (the first warp of the four) or with cp.async: each thread copies what it converts itself, so those copies need
      // no barrier.
      constexpr uint32_t kNoRow = 256;
      constexpr int SD = C::SD, LPR = D / 16, RPI = 32 / LPR, RPW = TK / 4, IT = RPW / RPI;
      const int kind = is_k ? 0 : 1, gw = w & 3, lc = ln % LPR, r_first = gw * RPW;
      const int32_t off = r_first + (ln < RPW ? ln : 0), oq = L.by_block.div(off), orr = off - oq * L.block_tokens;
      const int box = p.box_rows, boxes = box > 0 ? TK / box : 0, br = ln < boxes ? ln * box : 0;
      const int br_q = L.by_block.div(br), br_r = br - br_q * L.block_tokens;
      uint32_t sb[SD], uses[SD];  // scale bytes by stage (a load's result stays where it lands, so nothing waits for it early)
      bool tma[SD];
      int nt = 0, j = 0, left = 0;  // tiles fetched and not converted
#pragma unroll
      for (int st = 0; st < SD; ++st) uses[st] = 0, tma[st] = false;
      auto fetch = [&](int st) {  // the run's next tile into a stage; an empty cp.async group when there is none
        sb[st] = 127;
        if (ok && (j < nt || next_piece<M, TK>(p, run, pc))) {
          if (j >= nt) {
            nt = pc.t1 - pc.t0;
            j = 0;
            start();
          }
          const int64_t row_at = place(j, off, oq, orr, &sb[st]);
          if (row_at < 0) sb[st] = kNoRow;
          tma[st] = box > 0;
          if (tma[st]) {
            int32_t q = q0 + br_q, rr = r0 + br_r;
            if (rr >= L.block_tokens) rr -= L.block_tokens, ++q;
            const int32_t blk = block_of(q);
            if (gw == 0) {  // all four warps have read the stage's last tile
              ok = wait_warp(&sm.freed[kind][st], uses[st] ^ 1, limit);
              if (ok && ln == 0) mbar_arrive_expect_tx(&sm.ready[kind][st], TK * D);
              __syncwarp();
              if (ok && ln < boxes)
                tma_load_5d(&sm.stage[kind][st][br * D], &map, 0, rr, 0, pc.head, blk + (is_k ? 0 : L.num_blocks),
                            &sm.ready[kind][st]);
            }
          } else {
            if (gw == 0) {  // keeps in step with the stage's phases
              ok = wait_warp(&sm.freed[kind][st], uses[st] ^ 1, limit);
              if (ok && ln == 0) mbar_arrive(&sm.ready[kind][st]);
            }
#pragma unroll
            for (int i = 0; i < IT; ++i) {
              const int rl = i * RPI + ln / LPR;
              const int64_t a = __shfl_sync(0xffffffffu, row_at, rl);
              cp_async16_or_zero(smem_u32(&sm.stage[kind][st][(r_first + rl) * D + lc * 16]), base + (a < 0 ? 0 : a) + lc * 16,
                                 a >= 0);
            }
          }
          ++left;
          ++j;
          step();
        }
        cp_async_commit();
      };
      auto convert = [&](int st, uint8_t *dst, const bool wide) {
#pragma unroll 4
        for (int i = 0; i < IT; ++i) {
          const int rl = i * RPI + ln / LPR, r = r_first + rl;
          const uint32_t e = __shfl_sync(0xffffffffu, sb[st], rl);
          // 2^(120 + e - 127) as two bf16; beyond bf16's range 2^120, and the rest in a second product (255: NaN)
          // a row behind the last position: 0 times whatever finite bits the block holds
          const uint32_t k1 = e == kNoRow ? 0 : wide && e > 134 ? 0x7b807b80u : (e + 120) * 0x00800080u;
          const uint32_t k2 = e > 134 && e != kNoRow ? (e == 255 ? 0x7fc07fc0u : e * 0x00800080u) : 0x3f803f80u;
          const uint4 code = *(const uint4 *)&sm.stage[kind][st][r * D + lc * 16];
          const uint32_t cw[4] = {code.x, code.y, code.z, code.w};
          uint32_t o[8];
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            o[x] = mul_bf16x2(e4m3x2_to_bf16x2_bits(__byte_perm(cw[x >> 1], 0, x & 1 ? 0x3424 : 0x1404)), k1);
            if (wide) o[x] = mul_bf16x2(o[x], k2);
          }
          const int ch = 2 * lc;
          uint8_t *row = dst + (ch >> 3) * (TK * 128) + r * 128;
          *(uint4 *)(row + (((ch & 7) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          *(uint4 *)(row + ((((ch & 7) + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      };
#pragma unroll
      for (int st = 0; st < SD; ++st) fetch(st);
      while (ok && left > 0) {
#pragma unroll
        for (int st = 0; st < SD; ++st) {
          if (!ok || left == 0) break;
          cp_async_wait<SD - 1>();
          if (!(ok = wait_warp(&sm.ready[kind][st], uses[st], limit)) || !(ok = wait_empty())) break;
          if (__any_sync(0xffffffffu, sb[st] > 134 && sb[st] != kNoRow)) convert(st, sm.ring[at.slot], true);
          else convert(st, sm.ring[at.slot], false);
          hand_on(at.slot);
          if (ln == 0) mbar_arrive(&sm.freed[kind][st]);
          uses[st] ^= 1;
          --left;
          at.step();
          fetch(st);
        }
      }
      if (!ok && gw == 0)  // a wait gave up: nothing may be in flight when the CTA leaves
        for (int st = 0; st < SD; ++st)
          if (tma[st]) wait_warp(&sm.ready[kind][st], uses[st], p.drain_limit_ns);
      cp_async_wait<0>();
    }
  }
  if (w == 8) {
    // ---------------------------------------------------------------- products
    const bool lead = tc::elect_one();
    constexpr uint32_t iqk = idesc_f16(128, TK, BF16, false), ipv = idesc_f16(128, D, BF16, true);
    Ring<NS> rk(0), rv(1);  // the next K and V tile to wait for
    uint32_t itb[2] = {0, 0}, pieces[2] = {0, 0};
    const uint32_t ring0 = smem_u32(sm.ring[0]), q0 = smem_u32(sm.q);
    auto wait = [&](uint64_t *bar, uint32_t phase) {
      if (ok) ok = wait_bar(bar, phase, limit);
      return ok;
    };
    auto next_slot = [&](Ring<NS> &at, int &slot) {  // waits for the ring's next K or V tile
      slot = at.slot;
      const bool r = wait(&sm.full[at.slot], at.phase);
      at.step();
      tc::fence_after_sync();
      return r;
    };
    auto scores = [&](int b, int sb, int slot) {  // S[sb] = Q[b] K^T
      if (lead) {
        const uint32_t kd = desc_lo(ring0 + slot * C::slot, 16), qd = desc_lo(q0 + b * 128 * D * 2, 16);
        const uint32_t d = tm + C::S0 + sb * C::SN;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t kk = kd + ((k >> 2) * (TK * 128) + (k & 3) * 32) / 16;
          if constexpr (C::QT) mma_ts16(d, tm + C::Q0 + k * 8, kk, iqk, k > 0);
          else mma_ss16(d, qd + ((k >> 2) * 16384 + (k & 3) * 32) / 16, kk, iqk, k > 0);
        }
        tc::mma_commit(&sm.sfull[sb]);
      }
    };
    auto values = [&](int b, int sb, int slot, bool fresh, bool last) {  // O[b] (+)= P[sb] V
      if (lead) {
        const uint32_t vd = desc_lo(ring0 + slot * C::slot, TK * 128);
#pragma unroll
        for (int k = 0; k < TK / 16; ++k)
          mma_ts16(tm + C::O0 + b * D, tm + C::S0 + sb * C::SN + k * 8, vd + k * (2048 / 16), ipv, !(fresh && k == 0));
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
      const int32_t rows = pc.s.n * p.group - pc.block * M;
      const int nb = NQ == 2 && rows > 128 ? 2 : 1;
      for (int b = 0; b < nb; ++b)
        if (!wait(&sm.qfull[b], pieces[b]++)) break;
      if (!ok || !next_slot(rk, ks)) break;
      if constexpr (NQ == 2) {
        for (int b = 0; b < nb; ++b) scores(b, b, ks);
        release(ks);
        for (int j = 0; j < nt; ++j) {
          if (!next_slot(rv, vs)) break;
          for (int b = 0; b < nb; ++b) {
            if (!wait(&sm.pfull[b], itb[b]++)) break;
            tc::fence_after_sync();
            values(b, b, vs, j == 0, j == nt - 1);
            if (b == nb - 1) release(vs);
            if (j + 1 < nt) {
              if (b == 0 && !next_slot(rk, ks)) break;
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
            if (!next_slot(rk, ks)) break;
            scores(0, (int)((it + 1) & 1), ks);
            release(ks);
          }
          if (!next_slot(rv, vs) || !wait(&sm.pfull[it & 1], it >> 1)) break;
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
  if (w == 8) {
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
  return launch_pdl(k, plan.ctas, Conf<D, Q8>::threads, smem, stream, p, p.map ? *p.map : CUtensorMap{});
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
