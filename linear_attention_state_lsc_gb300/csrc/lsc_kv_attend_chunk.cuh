// lsc_kv_attend_chunk.cuh -- attention over a layer of the K/V block pool for
// sequences with many packed rows (lsc_kv_attend.cuh): prefill chunks.
//
// 4 * head_dim operations a (row, position) pair, and K/V tiles that serve 128 or
// 256 rows: the 5th-generation tensor cores bound it.  One CTA per SM walks its
// run of tiles of TK positions with the warps in roles:
//   * two softmax warpgroups: a thread waits for the scores S = Q K^T of its row in
//     TMEM, puts weights 2^(s - m) at 16 bits back into the same TMEM columns and
//     keeps the sum in a register.  m is a reference, not the exact maximum: O is
//     rescaled (in TMEM, by these threads) only when a row's maximum rose by more
//     than 2^lag, and m then lies 2^lift below it, so a weight is at most
//     2^(lag + lift) and the rescale is rare after the first tiles.
//   * one MMA warp: S = Q K^T, O += P V with P as the TMEM operand, issued so that
//     the products of one tile run while the softmax of another does.
//   * producers: K and V rows through the block table into a shared-memory ring
//     (K(0), V(0), K(1), V(1) ...) in the 128-byte-swizzled layout.  16-bit pools:
//     a warp for K and one for V.  Blocks that are a multiple of 8 tokens come
//     as tiled TMA boxes of rows x 64 elements (x head_dim / 64 when a block holds
//     the tile: then one box a tile; coordinates (element, row, column of 64, head,
//     block) of the layer, element always 0); other block sizes with 16-byte
//     cp.async.  V rows behind the last position become zeros: here, where they
//     are copied, else by the softmax threads.
// E4M3 pools run on the 8-bit products as they are (converting the codes to bf16 in
// front of the tensor cores took 2.4 ms where this took 1.77, bound by the integer
// pipes).  A row of q, times a power of two that brings it to [128, 256), is the sum
// of two e4m3 rows: four significant bits each, so bf16 is exact down to 2^-9 of the
// row's largest magnitude and off by 2^-18 of it below.  Scores take K's scale per
// position.  A weight is p 2^e with V's scale 2^e, as f16 relative to the row's
// largest contribution (the reference is that of s + e; the sum takes p), and an f16
// is the sum of three e5m2 numbers: its upper byte, the upper byte of the rest, and
// what is left rounded to nearest (in whole numbers: the conversion took 5 % more
// time), together nine bits or more.  The smallest e5m2 number is 2^-16, so weights
// take the room above 1 (2^15 at most): a weight is off by half of its ninth bit or
// by 2^-26 of the row's largest, and a long flat tail behind one large score keeps
// its share (lag 8 and lift 7, 2^-24: 975 us; 6 and 9: 988; 4 and 11, 2^-28, more
// rescaling: 1036; 8 chunks behind up to 16384 as below, with pauses).  So Q K^T takes two 8-bit products, P V three, at
// twice bf16's rate.
// head_dim 64 and 128: two row blocks of 128, one warpgroup and a thread a row
// each, with its own S and O (S 2 x 128, O 2 x head_dim columns of TMEM), Q in
// shared memory, tiles of 128: one block's softmax runs under the other's
// products, and a K/V tile is fetched once for 256 rows.
// head_dim 256: O takes 256 columns, so one row block, tiles of 64 and two S
// buffers in turn; Q is a TMEM operand (128 columns), which leaves shared memory
// to K and V and halves what the score products read from it.  The way from S to
// P is what the products wait for here, so it is made short: both warpgroups take
// each tile, a thread half the columns of a row, and tell each other the largest
// of their halves (bf16, 24 sequences of 1 to 2048 tokens behind up to 8192, runs
// by tiles alone: 817 us; 890 with a thread a row and the tiles in turn; 849 when
// each thread looks at the whole row for the maximum and computes half the
// weights; the pair of head_dim 128 with sixteen softmax warps of 104 registers:
// 1928 us against 1350, so not there).
// Two row blocks: half a tile's weights go to the products while the other half
// is computed (head_dim 128, 4096 tokens behind 28000: 1361 -> 1320 us).
//
// Measured, calls back to back (bf16 products 1923 TFLOP/s): head_dim 128, 4096
// tokens behind 28000, 32 q heads: 1482 us, 1361 TFLOP/s (1300 us with pauses, when
// the power limit is not met; head_dim 64: 1168 us with pauses, 863 TFLOP/s, where
// the softmax has twice the work a product); head_dim 256, mixed as above: 832 us,
// 1120 TFLOP/s (687 with pauses; 2160 over blocks of 12, whose rows are copied one by
// one); E4M3, 8 chunks behind up to 16384: 1039 us, 954 TFLOP/s (996 with pauses).
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

template <int D, bool Q8, bool BF16 = true>
struct Conf {
  static constexpr int NQ = D == 256 ? 1 : 2;   // row blocks of 128
  static constexpr int M = 128 * NQ;
  static constexpr int TK = D == 256 ? 64 : 128;
  static constexpr bool QT = D == 256;          // Q in TMEM
  static constexpr int ES = Q8 ? 1 : 2;         // bytes of an element
  static constexpr int row = D * ES, line = row < 128 ? row : 128;  // bytes of a row, of a swizzled line of it
  static constexpr int slot = TK * row;         // bytes of a K or V tile
  static constexpr int NS = Q8 ? (D == 128 ? 6 : 8) : (D == 64 ? 8 : D == 128 ? 4 : 6);
  static constexpr int SR = Q8 ? 8 : 1;         // E4M3: tiles whose scales are held
  static constexpr int threads = 384;           // warps: 0-7 softmax, 8 MMA, 9 K, 10 V, 11 idle
  static constexpr int NH = 2 / NQ;             // threads of a row
  static constexpr int HC = TK / NH;            // columns of a thread
  // registers a thread of a softmax warpgroup and of the others' keeps of the 168 at launch
  static constexpr int soft = 208, mma = 80;
  static_assert(2 * soft + mma <= 3 * 168, "more registers than the block has");
  // powers of two: how far a row's maximum may rise above the one that set the reference, and how far the reference
  // lies below that (f16 weights, whose smallest is 2^-24, take the room up to 2^15; bf16 has the exponents as it is)
  static constexpr float lag = Q8 ? 6.f : 8.f, lift = Q8 ? 9.f : BF16 ? 0.f : 7.f;
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
  // E4M3, by tile and position: K's scale, V's exponent (bounded) and V's scale
  alignas(16) float ks[C::SR][Q8 ? C::TK : 4], ve[C::SR][Q8 ? C::TK : 4], vs[C::SR][Q8 ? C::TK : 4];
  float up[8][32];        // E4M3, by softmax warp: the power of two of a row of q
  alignas(16) uint8_t rows[8][32][80];  // by softmax warp: 64 bytes of each of its rows, between TMEM and memory
  int32_t bad[Q8 ? 1 : 3][Q8 ? 1 : D];  // first position whose v is NaN, +inf, -inf
  uint64_t full[C::NS], empty[C::NS], sfull[2], phalf[2], pfull[2], qfull[2], odone[2], fin[2], met, drain;
  uint64_t scaled[C::SR];             // E4M3: a tile's scales are there
  uint64_t told[2][8][32];      // NH == 2: a half's part of a row's maximum or sum, behind the turn's number
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
// (64-byte lines: groups of 512 bytes, 64-byte swizzle.)
template <int LINE>
constexpr uint32_t kDescHi = LINE == 64 ? (512 >> 4) | 1u << 14 | 4u << 29 : (1024 >> 4) | 1u << 14 | 2u << 29;
// Instruction descriptor with an fp32 accumulator.  kind::f16: a, b = 0 f16, 1 bf16; kind::f8f6f4: 0 e4m3, 1 e5m2.
__host__ __device__ constexpr uint32_t idesc(int M, int N, uint32_t a, uint32_t b, bool b_mn_major) {
  return (1u << 4) | a << 7 | b << 10 | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
#define LSC_MMA(NAME, KIND)                                                                                          \
  __device__ __forceinline__ void NAME##_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t id, uint32_t acc) { \
    asm volatile(                                                                                                    \
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %4};\n\t"                     \
        "mov.b64 b, {%2, %4};\n\ttcgen05.mma.cta_group::1.kind::" KIND " [%0], a, b, %3, p;\n\t}" ::"r"(d),        \
        "r"(a), "r"(b), "r"(id), "r"(hi), "r"(acc)                                                                   \
        : "memory");                                                                                                 \
  }                                                                                                                  \
  __device__ __forceinline__ void NAME##_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t id, uint32_t acc) { \
    asm volatile(                                                                                                    \
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %4};\n\t"                       \
        "tcgen05.mma.cta_group::1.kind::" KIND " [%0], [%1], b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(id),      \
        "r"(hi), "r"(acc)                                                                                            \
        : "memory");                                                                                                 \
  }
LSC_MMA(mma16, "f16")
LSC_MMA(mma8, "f8f6f4")
#undef LSC_MMA

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

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// v[0..7] -> 8 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ float lo_f(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float hi_f(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }

// E4M3: 32 scores times K's scales (kept in s); returns the largest of s c + e over the seen ones.
__device__ __forceinline__ float scale8(uint32_t (&s)[32], const float *ks, const float *ve, uint64_t c, bool mask,
                                        int32_t seen) {
#pragma unroll
  for (int y = 0; y < 32; y += 4) {
    const ulonglong2 k = *(const ulonglong2 *)(ks + y);
    const uint64_t a = mul2((uint64_t)s[y] | (uint64_t)s[y + 1] << 32, k.x);
    const uint64_t b = mul2((uint64_t)s[y + 2] | (uint64_t)s[y + 3] << 32, k.y);
    s[y] = (uint32_t)a, s[y + 1] = (uint32_t)(a >> 32), s[y + 2] = (uint32_t)b, s[y + 3] = (uint32_t)(b >> 32);
  }
  if (mask) hide(s, seen);
  float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
  for (int y = 0; y < 32; y += 4) {
    const ulonglong2 e = *(const ulonglong2 *)(ve + y);
    const uint64_t a = fma2((uint64_t)s[y] | (uint64_t)s[y + 1] << 32, c, e.x);
    const uint64_t b = fma2((uint64_t)s[y + 2] | (uint64_t)s[y + 3] << 32, c, e.y);
    t0 = fmaxf(t0, fmaxf(lo_f(a), hi_f(a)));
    t1 = fmaxf(t1, fmaxf(lo_f(b), hi_f(b)));
  }
  return fmaxf(t0, t1);
}

// E4M3: p = 2^(s c + r) of 32 scores, added to l; p times V's scale as three e5m2 numbers, four a word in q[0..2].
__device__ __forceinline__ void weights8(const uint32_t (&s)[32], const float *vs, uint64_t c, uint64_t r, bool mask,
                                         int32_t seen, uint64_t &l, uint32_t (&q)[3][8]) {
  uint64_t sum[2] = {0, 0};
#pragma unroll
  for (int y = 0; y < 8; ++y) {
    const ulonglong2 v = *(const ulonglong2 *)(vs + 4 * y);
    uint32_t h[2], t2[2];
    uint32_t t0[2], t1[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int i = 4 * y + 2 * z;
      const uint64_t x = fma2((uint64_t)s[i] | (uint64_t)s[i + 1] << 32, c, r);
      const uint64_t p = two(ex2(lo_f(x)), ex2(hi_f(x)));
      sum[z] = add2(sum[z], p);
      uint64_t w = mul2(p, z ? v.y : v.x);
      if (mask) {  // 0 whatever the scale
        if (i >= seen) w &= 0xffffffff00000000ull;
        if (i + 1 >= seen) w &= 0xffffffffull;
      }
      h[z] = pack2(lo_f(w), hi_f(w), 0);
      t0[z] = h[z] & 0xff00ff00u;
      __half2 rest = __hsub2(*reinterpret_cast<const __half2 *>(&h[z]), *reinterpret_cast<const __half2 *>(&t0[z]));
      t1[z] = *reinterpret_cast<const uint32_t *>(&rest) & 0xff00ff00u;
      rest = __hsub2(rest, *reinterpret_cast<const __half2 *>(&t1[z]));
      t2[z] = *reinterpret_cast<const uint32_t *>(&rest) + 0x00800080u;  // rest >= 0: to nearest in whole numbers
    }
    q[0][y] = __byte_perm(t0[0], t0[1], 0x7531);
    q[1][y] = __byte_perm(t1[0], t1[1], 0x7531);
    q[2][y] = __byte_perm(t2[0], t2[1], 0x7531);
  }
  l = add2(l, add2(sum[0], sum[1]));
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
  using C = Conf<D, Q8, BF16>;
  constexpr int NQ = C::NQ, M = C::M, TK = C::TK, NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem<D, Q8> &sm = *reinterpret_cast<Smem<D, Q8> *>(smem_raw);
  const int tid = threadIdx.x, w = tid >> 5, ln = tid & 31;
  const KvLayer &L = p.L;
  if (w == 8) {
    tc::tmem_alloc(&sm.tmem, 512);
    tc::tmem_relinquish();
  }
  if (C::NH == 2)
    for (int i = tid; i < 2 * 8 * 32; i += C::threads) (&sm.told[0][0][0])[i] = ~0ull;  // no turn's number
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&sm.full[i], 1), mbar_init(&sm.empty[i], 1);
    for (int i = 0; i < C::SR; ++i) mbar_init(&sm.scaled[i], 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.sfull[i], 1), mbar_init(&sm.phalf[i], 4), mbar_init(&sm.pfull[i], 4 * C::NH), mbar_init(&sm.qfull[i], 4 * C::NH);
      mbar_init(&sm.odone[i], 1), mbar_init(&sm.fin[i], 1);
    }
    mbar_init(&sm.met, 8);
    mbar_init(&sm.drain, 1);
    fence_mbar_init();
    sm.any_bad = 0;
  }
  if (!Q8)
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
    const int block = NQ == 2 ? w >> 2 : 0, half = NQ == 2 ? 0 : w >> 2;  // row block; which half of the columns
    const int quad = w & 3, row = quad * 32 + ln;  // row of the block
    const int partner = w ^ 4;                     // NH == 2: the warp with the other half of the same rows
    const uint32_t lane = (uint32_t)(quad * 32) << 16;
    const Workspace ws = workspace_at(p.ws, ctas, M);
    float c = p.scale_log2, c_next = c;  // of this thread's row (E4M3: with q's power of two)
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
      const uint8_t *from[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) from[i] = (const uint8_t *)__shfl_sync(0xffffffffu, (unsigned long long)src, i * 8 + oct);
      auto load = [&](int i, int x) { return from[i] ? *(const uint4 *)(from[i] + x + part16) : make_uint4(0, 0, 0, 0); };
      constexpr int bytes = 2 * D / C::NH;         // of a row, this warpgroup's share
      const int begin = half * bytes;
      // all loads before the first use: a unit's queries are its first latency (head_dim 256: 3300 cycles, 4100 a piece at
      // a time; E4M3, whose scale takes the whole row, 6600 and 9900)
      uint4 own[bytes / 64][4];
#pragma unroll
      for (int x = 0; x < bytes / 64; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) own[x][i] = load(i, begin + 64 * x);
      if constexpr (Q8) {
        uint32_t top[4] = {0, 0, 0, 0};  // magnitudes of bf16 order as whole numbers, two a word
        auto look = [&](int i, const uint4 &y) {
          const uint32_t k = 0x7fff7fffu;
          top[i] = __vmaxu2(top[i], __vmaxu2(__vmaxu2(y.x & k, y.y & k), __vmaxu2(y.z & k, y.w & k)));
        };
        if constexpr (C::NH == 2) {
          uint4 rest[bytes / 64][4];
#pragma unroll
          for (int x = 0; x < bytes / 64; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) rest[x][i] = load(i, (half ^ 1) * bytes + 64 * x);
#pragma unroll
          for (int x = 0; x < bytes / 64; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) look(i, rest[x][i]);
        }
#pragma unroll
        for (int x = 0; x < bytes / 64; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) look(i, own[x][i]);
        float down[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t t = max(top[i] & 0xffffu, top[i] >> 16);
          t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
          t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
          const uint32_t ex = t >> 7;  // 2^(ex - 127) <= the largest magnitude: brought to 2^7, where both powers are normal
          const bool plain = ex < 8 || ex == 255;
          down[i] = plain ? 1.f : __uint_as_float((261 - ex) << 23);
          // an infinity would become a code of 448: a row that is not finite has NaN for its power
          if ((ln & 3) == 0) sm.up[w][i * 8 + oct] = ex < 8 ? 1.f : __uint_as_float(ex == 255 ? 0x7fc00000u : (ex - 7) << 23);
        }
        __syncwarp();
        c_next = p.scale_log2 * sm.up[w][ln];
#pragma unroll
        for (int x = 0; x < bytes; x += 64) {  // 32 elements: 32 bytes of each part
          uint2 part[4][2];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 y = own[x / 64][i];
            const uint32_t in[4] = {y.x, y.y, y.z, y.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float f0 = __uint_as_float(in[e] << 16) * down[i], f1 = __uint_as_float(in[e] & 0xffff0000u) * down[i];
              hi[e] = to_e4m3x2(f0, f1);
              const float2 back = e4m3x2_to_float2(hi[e]);
              lo[e] = to_e4m3x2(f0 - back.x, f1 - back.y);
            }
            part[i][0] = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            part[i][1] = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
          }
          if constexpr (C::QT) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int t = 0; t < 2; ++t) *(uint2 *)&mine_rows[i * 8 + oct][t * 32 + (ln & 3) * 8] = part[i][t];
            __syncwarp();
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint4 y = *(const uint4 *)&mine_rows[ln][t * 32], z = *(const uint4 *)&mine_rows[ln][t * 32 + 16];
              const uint32_t v[8] = {y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
              tmem_st8(tm + lane + C::Q0 + t * (D / 4) + (begin + x) / 8, v);
            }
          } else {
            const int at = (begin + x) / 2 + (ln & 3) * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int t = 0; t < 2; ++t)
                *(uint2 *)(sm.q + block * 128 * D * 2 + t * 128 * D +
                           chunk_at<C::line>(128, quad * 32 + i * 8 + oct, at >> 4) + (at & 8)) = part[i][t];
          }
        }
      } else {
#pragma unroll
        for (int x = 0; x < bytes; x += 64) {
          const uint4(&y)[4] = own[x / 64];
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
            tc::tmem_st16(tm + lane + C::Q0 + (begin + x) / 4, v);
          } else {
            uint8_t *dst = sm.q + block * 128 * D * 2 + ((begin + x) >> 7) * 16384;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rr = quad * 32 + i * 8 + oct, ch = (((begin + x) >> 4) & 4) + (ln & 3);
              *(uint4 *)(dst + rr * 128 + ((ch ^ (rr & 7)) << 4)) = y[i];
            }
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
    uint32_t meets = 0, done = 0, turns = 0, tiles = 0;  // tiles: of the pieces before this one
    // x for the thread that has the other half of the row, against its own.  Value and turn number are one 64-bit word,
    // so a thread itself sees when it is there (a warp's barrier instead: the same with bf16, 1.4 % slower with E4M3).
    // The word was read two turns ago: the partner has told the last turn's since.
    auto exchange = [&](float x, float &other) {
      const uint32_t mine = smem_u32(&sm.told[turns & 1][w][ln]), its = smem_u32(&sm.told[turns & 1][partner][ln]);
      asm volatile("st.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(mine), "l"((uint64_t)turns << 32 | __float_as_uint(x))
                   : "memory");
      uint64_t v, t0 = 0;
      bool there;
      for (uint32_t i = 0;; ++i) {
        asm volatile("ld.relaxed.cta.shared::cta.b64 %0, [%1];" : "=l"(v) : "r"(its) : "memory");
        there = __all_sync(0xffffffffu, (uint32_t)(v >> 32) == turns);
        if (there) break;
        if ((i & 255) == 255) {  // reading the clock takes a microsecond
          const uint64_t t = global_timer_ns();
          if (t0 == 0) t0 = t;
          if (__any_sync(0xffffffffu, t - t0 >= limit)) break;
        }
      }
      other = __uint_as_float((uint32_t)v);
      ++turns;
      return there;
    };
    while (have && ok) {
      c = c_next;
      const int nt = pc.t1 - pc.t0, rows = rows_of(pc);
      const bool mine = block * 128 < rows;
      const int r = block * 128 + row;
      const int32_t R = pc.block * M + r, tok = p.by_group.div(R);
      const int32_t vis = r < rows ? visible(pc.s, tok, p.causal) : 0;
      if (Q8 && vis == 0) c = 1.f;  // sees nothing: zeros, whatever q is (a hidden score is -infinity times c)
      const int32_t sure = visible(pc.s, p.by_group.div(pc.block * M), p.causal);
      const int32_t full_to = NQ == 2 && block == 1 && mine
                                  ? visible(pc.s, p.by_group.div(pc.block * M + 128), p.causal)
                                  : sure;  // every row of this block sees positions below it
      const bool rows_all = (block + 1) * 128 <= rows;
      float m = -INFINITY, l = 0.f;
      // does the piece reach positions that some row of the unit does not see
      const bool mixed = (pc.s.kv < pc.t1 * TK ? pc.s.kv : pc.t1 * TK) > sure;
      for (int j = 0; j < nt && mine; ++j, ++it) {
        const int sb = NQ == 2 ? block : (int)(it & 1);
        const uint32_t s0 = tm + lane + C::S0 + sb * C::SN, sa = s0 + half * C::HC;
        const int32_t first = (pc.t0 + j) * TK;
        if (!(ok = wait_warp(&sm.sfull[sb], NQ == 2 ? it : it >> 1, limit))) break;
        tc::fence_after_sync();
        // a column is seen when first + column < vis
        const bool mask = first + TK > full_to || !rows_all;
        const int32_t seen = vis - first - half * C::HC;  // of this thread's columns
        constexpr int NC = C::HC / 32;              // chunks of 32 columns
        const uint32_t tile = tiles + j, sr = tile % C::SR;  // E4M3: where its scales are
        const int32_t last = first + TK < pc.s.kv ? first + TK : pc.s.kv;
        if (Q8 && !(ok = wait_warp(&sm.scaled[sr], tile / C::SR, limit))) break;
        const bool edge = last > sure || last < first + TK;  // rows of v may have to be cleared
        if (Q8 && edge) {
          // Codes of NaN where some row does not see the position become zeros; the scale says NaN to the rows that see it.
          // Every warp looks at all of them, so none waits for another.  So does whatever lies behind the last position,
          // a share of it by each warp of the row block.
          const uint32_t vi = slots + 2 * j + 1;
          const int slot = (int)(vi % NS);
          if (!(ok = wait_warp(&sm.full[slot], vi / NS, limit))) break;
          constexpr int CH = C::row / 16;
          auto chunk = [&](int i) { return (uint4 *)(sm.ring[slot] + chunk_at<C::line>(TK, i / CH, i % CH)); };
          for (int i = (last - first) * CH + half * 128 + row; i < TK * CH; i += 128 * C::NH) *chunk(i) = make_uint4(0, 0, 0, 0);
#pragma unroll 1
          for (int i = (sure > first ? sure - first : 0) * CH + ln; i < (last - first) * CH; i += 32) {
            const uint4 v = *chunk(i);
            const uint32_t k = 0x7f7f7f7fu, one = 0x01010101u;
            if (((((v.x & k) + one) | ((v.y & k) + one) | ((v.z & k) + one) | ((v.w & k) + one)) & 0x80808080u) == 0) continue;
            *(volatile float *)&sm.vs[sr][i / CH] = __uint_as_float(0x7fc00000u);
            __threadfence_block();
            *chunk(i) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint64_t c2 = two(c, c);
        uint32_t s[NC][32];
        float top;
        tc::tmem_ld32(sa, s[0]);
        wait_ld(s[0]);
#pragma unroll
        for (int x = 1; x < NC; ++x) tc::tmem_ld32(sa + 32 * x, s[x]);
        auto look_at = [&](int x) {
          if constexpr (Q8) return scale8(s[x], &sm.ks[sr][half * C::HC + 32 * x], &sm.ve[sr][half * C::HC + 32 * x], c2, mask, seen - 32 * x);
          if (mask) hide(s[x], seen - 32 * x);
          return top_of(s[x]);
        };
        top = look_at(0);
#pragma unroll
        for (int x = 1; x < NC; ++x) {
          wait_ld(s[x]);
          top = fmaxf(top, look_at(x));
        }
        if (C::NH == 2) {  // the partner's half of the row (it has read its scores too, so the weights may go over them)
          float other;
          if (!(ok = exchange(top, other))) break;
          top = fmaxf(top, other);
        }
        const float mt = Q8 ? top : top * c;  // c > 0
        // also the first tile's (m is -inf); the same in both halves
        if (__any_sync(0xffffffffu, mt > m + (C::lag + C::lift))) {
          const float to = fmaxf(m, mt - C::lift), f = ex2(m - (to == -INFINITY ? 0.f : to));
          m = to;
          l *= f;
          if (j > 0) {
            if (!(ok = wait_warp(&sm.odone[block], it - 1, limit))) break;
            tc::fence_after_sync();
            const uint32_t oa = tm + lane + C::O0 + block * D + half * (D / C::NH);
#pragma unroll 1
            for (int x = 0; x < D / C::NH; x += 32) {
              uint32_t o[32];
              tc::tmem_ld32(oa + x, o);
              wait_ld(o);
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tc::tmem_st32(oa + x, o);
            }
          }
        }
        auto hand = [&](uint64_t *bar) {  // the weights up to here (and the rescaled O) to the products
          tc::tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (ln == 0) mbar_arrive(bar);
        };
        const float ref = m == -INFINITY ? 0.f : m;
        const uint64_t r2 = two(-ref, -ref);
        uint64_t l2 = two(0.f, 0.f);
#pragma unroll
        for (int x = 0; x < NC; ++x) {
          if constexpr (Q8) {
            uint32_t q[3][8];
            weights8(s[x], &sm.vs[sr][half * C::HC + 32 * x], c2, r2, mask, seen - 32 * x, l2, q);
#pragma unroll
            for (int t = 0; t < 3; ++t) tmem_st8(s0 + t * (TK / 4) + half * (C::HC / 4) + 8 * x, q[t]);
          } else {
            uint32_t q[16];
            weights<BF16>(s[x], c2, r2, l2, q);
            tc::tmem_st16(s0 + half * (C::HC / 2) + 16 * x, q);
          }
          if (NQ == 2 && x == NC / 2 - 1 && !edge) hand(&sm.phalf[sb]);
        }
        const float2 lf = *reinterpret_cast<const float2 *>(&l2);
        l += lf.x + lf.y;
        // positions [max(first, sure), last): some row of the unit does not see them; behind last: a block's rows came as
        // they were
        if (!Q8 && edge) {
          const uint32_t vi = slots + 2 * j + 1;
          const int slot = (int)(vi % NS);
          if (!(ok = wait_warp(&sm.full[slot], vi / NS, limit))) break;
          {
            for (int i = half * 128 + row; i < (first + TK - last) * (D / 8); i += 128 * C::NH) {
              const int key = last - first + i / (D / 8), ch = i % (D / 8);
              *(uint4 *)(sm.ring[slot] + (ch >> 3) * (TK * 128) + key * 128 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
            }
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
          for (int i = half * 128 + row; i < cnt * (D / 8); i += 128 * C::NH) {
            const uint4 v = *vec(i);
            carry |= ((v.x & 0x7fff7fffu) + up) | ((v.y & 0x7fff7fffu) + up) | ((v.z & 0x7fff7fffu) + up) |
                     ((v.w & 0x7fff7fffu) + up);
          }
          if (carry & 0x80008000u) {
#pragma unroll 1
            for (int i = half * 128 + row; i < cnt * (D / 8); i += 128 * C::NH) {
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
        if (NQ == 2 && edge) hand(&sm.phalf[sb]);
        hand(&sm.pfull[sb]);
      }
      if (!ok) break;
      if (C::NH == 2) {  // the halves' sums; then both know that Q has been used
        float other;
        if (!(ok = exchange(l, other))) break;
        l += other;  // the same in both
      }
      const Piece q = pc;
      cut = cut_of(run, q, cta);
      slots = (slots + 2 * (uint32_t)nt) % (2 * NS);
      tiles += nt;
      have = next_piece<M, TK>(p, run, pc);
      if (have && block * 128 < rows_of(pc)) load_q(pc);  // this piece's score products are done
      if (mine) {
        // a barrier of its own: odone may be up to two phases behind here, and a parity tells two apart, not three
        if (!(ok = wait_warp(&sm.fin[block], done++, limit))) break;
        tc::fence_after_sync();
        const bool whole = q.t0 == 0 && q.t1 == q.tiles;
        const bool empty = vis == 0;
        const float inv = whole ? (empty ? 0.f : 1.f / l) : 1.f;
        const int64_t h = q.head * p.group + (R - tok * p.group), t = q.s.row0 + tok;
        const int64_t slot = (int64_t)(2 * cta + (q.t0 == 0 ? 1 : 0)) * M + r;
        const bool on = r < rows;
        const bool look = !Q8 && mixed && *(volatile int32_t *)&sm.any_bad != 0;
        uint8_t *dst = !on ? nullptr : whole ? (uint8_t *)((uint16_t *)p.out + t * p.out_stride + h * D) : (uint8_t *)(ws.o + slot * D);
        uint8_t *to[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = (uint8_t *)__shfl_sync(0xffffffffu, (unsigned long long)dst, i * 8 + oct);
        const uint32_t oa = tm + lane + C::O0 + block * D;
#pragma unroll 1
        for (int x = half * (D / C::NH), end = x + D / C::NH; x < end; x += 32) {
          uint32_t o[32];
          tc::tmem_ld32(oa + x, o);
          wait_ld(o);
#pragma unroll
          for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * inv);
          if constexpr (!Q8) {
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
        if (on && half == 0) {
          if (!whole) ws.ml[slot] = make_float2(m, l);
          else if (p.lse) p.lse[t * p.heads + h] = empty ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
        }
        tc::fence_before_sync();  // these reads before the next piece's products, through pfull
      }
      if (!Q8 && mixed && have) {  // the next unit starts with a clean list: all softmax warps meet before and after it is cleared
        for (int round = 0; round < 2 && ok; ++round, ++meets) {
          if (round == 1 && *(volatile int32_t *)&sm.any_bad)
            for (int i = tid; i < 3 * D; i += 256) (&sm.bad[0][0])[i] = INT32_MAX;
          __syncwarp();
          if (ln == 0) mbar_arrive(&sm.met);
          ok = wait_warp(&sm.met, meets, limit);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::mma));
  }
  if (w == 9 || w == 10) {
    // ---------------------------------------------------------------- producers
    const bool is_k = w == 9;
    const uint8_t *base = is_k ? L.k : L.v;
    Ring<NS> at(is_k ? 0 : 1);
    const int64_t row_bytes = (int64_t)L.heads * C::row;
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
      blocks_held = pc.s.kv > 0 ? L.by_block.div(pc.s.kv - 1) + 1 : 0;  // block_tokens more could pass 31 bits
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
    // E4M3: the scale bytes of a tile's positions lane, lane + 32 ... 127 behind the last one; looked up a tile ahead
    uint32_t sb[TK / 32];
    auto load_scales = [&](int j) {
#pragma unroll
      for (int g = 0; g < TK / 32; ++g) {
        const int32_t off = g * 32 + ln, oq = L.by_block.div(off);
        int32_t q = q0 + oq, rr = r0 + off - oq * L.block_tokens;
        if (rr >= L.block_tokens) rr -= L.block_tokens, ++q;
        const int64_t page = (int64_t)block_of(q) * L.page;
        sb[g] = (pc.t0 + j) * TK + off < pc.s.kv ? __ldg(base + page + L.scale_off + (int64_t)rr * L.heads + pc.head) : 127;
      }
    };
    // into tile slot sr of the scales
    auto put_scales = [&](int sr) {
#pragma unroll
      for (int g = 0; g < TK / 32; ++g) {
        if (is_k) {
          sm.ks[sr][g * 32 + ln] = scale_of(sb[g]);
        } else {
          sm.vs[sr][g * 32 + ln] = scale_of(sb[g]);
          sm.ve[sr][g * 32 + ln] = v_exponent(sb[g]);
        }
      }
      __syncwarp();
      if (ln == 0) mbar_arrive(&sm.scaled[sr]);
    };
    // byte offset in a lane of the row of position `off` of tile j, (oq, orr) = off by blocks; -1 behind the last position
    auto place = [&](int j, int32_t off, int32_t oq, int32_t orr) {
      int32_t q = q0 + oq, rr = r0 + orr;
      if (rr >= L.block_tokens) rr -= L.block_tokens, ++q;
      const int64_t page = (int64_t)block_of(q) * L.page;
      if ((pc.t0 + j) * TK + off >= pc.s.kv) return (int64_t)-1;
      return page + (int64_t)rr * row_bytes + (int64_t)pc.head * C::row;
    };
    auto hand_on = [&](int slot) {
      fence_proxy_async_smem();
      __syncwarp();
      if (ln == 0) mbar_arrive(&sm.full[slot]);
    };
    // the ring's first turn passes at once: the phase before a fresh barrier's first one counts as complete
    auto wait_empty = [&]() { return wait_warp(&sm.empty[at.slot], at.phase ^ 1, limit); };
    constexpr int CPR = C::row / 16, RPI = 32 / CPR > 0 ? 32 / CPR : 1;  // 16-byte chunks of a row, rows an instruction
    constexpr int LAG = (NS - 1) / 2;  // cp.async tiles in flight before the first is handed on
    // TMA: a box of `box` rows and all lines when a block holds the tile, else of one line, a box a lane.  box 0: cp.async.
    constexpr int LINES = C::row / C::line;
    const int box = p.box_rows, per = box == TK ? 1 : LINES;
    const int boxes = box > 0 ? TK / box * per : 0, bc = ln % per, br = ln < boxes ? ln / per * box : 0;
    const int br_q = L.by_block.div(br), br_r = br - br_q * L.block_tokens;
    int pending = 0;
    uint32_t flying = 0;  // slots that TMA has filled (low byte), in which phase last (the next byte)
    Ring<NS> at_h = at;   // the next tile to hand on
    int sr = 0;
    while (ok && next_piece<M, TK>(p, run, pc)) {
      const int nt = pc.t1 - pc.t0;
      start();
      if (Q8) load_scales(0);
      for (int j = 0; j < nt; ++j, at.step()) {
        uint8_t *dst = sm.ring[at.slot];
        if (box > 0) {
          int32_t q = q0 + br_q, rr = r0 + br_r;
          if (rr >= L.block_tokens) rr -= L.block_tokens, ++q;
          const int32_t blk = block_of(q);
          if (!(ok = wait_empty())) break;
          if (ln == 0) mbar_arrive_expect_tx(&sm.full[at.slot], C::slot);
          __syncwarp();
          if (ln < boxes)
            tma_box(dst + bc * (TK * 128) + br * C::line, &map, rr, bc, pc.head, blk + (is_k ? 0 : L.num_blocks),
                    &sm.full[at.slot]);
          flying = flying & ~(0x101u << at.slot) | (1u | at.phase << 8) << at.slot;
        } else {
          int64_t row_at[TK / 32];
#pragma unroll
          for (int g = 0; g < TK / 32; ++g) {
            const int32_t off = g * 32 + ln, oq = L.by_block.div(off);
            row_at[g] = place(j, off, oq, off - oq * L.block_tokens);
          }
          if (!(ok = wait_empty())) break;
          const int ch = ln % CPR;
#pragma unroll
          for (int g = 0; g < TK / 32; ++g)
#pragma unroll 4
            for (int i = 0; i < 32; i += RPI) {
              const int r = i + ln / CPR;
              const int64_t a = __shfl_sync(0xffffffffu, row_at[g], r);
              cp_async16_or_zero(smem_u32(dst + chunk_at<C::line>(TK, g * 32 + r, ch)), base + (a < 0 ? 0 : a) + ch * 16, a >= 0);
            }
          cp_async_commit();
          if (++pending > LAG) {
            cp_async_wait<LAG>();
            hand_on(at_h.slot);
            at_h.step();
            --pending;
          }
        }
        if (Q8) {
          put_scales(sr);
          if (++sr == C::SR) sr = 0;
        }
        step();
        if (Q8 && j + 1 < nt) load_scales(j + 1);
      }
    }
    cp_async_wait<0>();
    for (; ok && pending > 0; --pending, at_h.step()) hand_on(at_h.slot);
    if (!ok)  // a wait gave up: nothing may be in flight when the CTA leaves
      for (int i = 0; i < NS; ++i)
        if (flying >> i & 1) wait_warp(&sm.full[i], flying >> (8 + i), p.drain_limit_ns);
  }
  if (w == 8) {
    // ---------------------------------------------------------------- products
    const bool lead = tc::elect_one();
    constexpr uint32_t hi = kDescHi<C::line>;
    constexpr uint32_t ty = BF16 && !Q8 ? 1 : 0;  // Q8: q and K e4m3, weights e5m2
    constexpr uint32_t iqk = idesc(128, TK, ty, ty, false), ipv = idesc(128, D, Q8 ? 1 : ty, ty, true);
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
        if constexpr (Q8) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
              const uint32_t kk = kd + ((k >> 2) * (TK * 128) + (k & 3) * 32) / 16;
              if constexpr (C::QT) mma8_ts(d, tm + C::Q0 + t * (D / 4) + k * 8, kk, hi, iqk, t + k > 0);
              else mma8_ss(d, qd + (t * 128 * D + k * 32) / 16, kk, hi, iqk, t + k > 0);
            }
        } else {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t kk = kd + ((k >> 2) * (TK * 128) + (k & 3) * 32) / 16;
            if constexpr (C::QT) mma16_ts(d, tm + C::Q0 + k * 8, kk, hi, iqk, k > 0);
            else mma16_ss(d, qd + ((k >> 2) * 16384 + (k & 3) * 32) / 16, kk, hi, iqk, k > 0);
          }
        }
        tc::mma_commit(&sm.sfull[sb]);
      }
    };
    // O[b] (+)= P[sb] V over half `part` of the tile's positions (NQ == 2: else all)
    auto values = [&](int b, int sb, int slot, int part, bool fresh, bool last) {
      if (lead) {
        const uint32_t vd = desc_lo(ring0 + slot * C::slot, TK * 128);
        const uint32_t od = tm + C::O0 + b * D, pa = tm + C::S0 + sb * C::SN;
        constexpr int step = Q8 ? 32 : 16, KN = TK / step / NQ;
        const int k0 = part * KN;
#pragma unroll
        for (int t = 0; t < (Q8 ? 3 : 1); ++t)
#pragma unroll
          for (int k = 0; k < KN; ++k) {
            const uint32_t acc = !(fresh && part + t + k == 0);
            if constexpr (Q8) mma8_ts(od, pa + t * (TK / 4) + (k0 + k) * 8, vd + (k0 + k) * (32 * C::line / 16), hi, ipv, acc);
            else mma16_ts(od, pa + (k0 + k) * 8, vd + (k0 + k) * (2048 / 16), hi, ipv, acc);
          }
        if (part == NQ - 1) {
          tc::mma_commit(&sm.odone[b]);
          if (last) tc::mma_commit(&sm.fin[b]);
        }
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
            if (!wait(&sm.phalf[b], itb[b])) break;
            tc::fence_after_sync();
            values(b, b, vs, 0, j == 0, j == nt - 1);
            if (!wait(&sm.pfull[b], itb[b]++)) break;
            tc::fence_after_sync();
            values(b, b, vs, 1, j == 0, j == nt - 1);
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
          values(0, (int)(it & 1), vs, 0, j == 0, j == nt - 1);
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
