// lsc_kv_attend_rows.cuh -- attention over a layer of the K/V block pool for
// sequences with few packed rows (lsc_kv_attend.cuh): decode steps where blocks do
// not fit TMA boxes, and over E4M3 pools a few speculated tokens and short chunks.
// Up to 16 * MT rows a unit, MT 1 (and 4 for E4M3).
//
// K and V are read once, so HBM bounds it: 4 * head_dim bytes a position and kv
// head at 16 bits against 4 * head_dim * rows operations, at 16 rows 16
// operations a byte where the tensor cores of an SM do 290.  mma.sync
// (m16n8k16) is enough for that and keeps scores, weights and sums in
// registers; tcgen05 would want 128 rows and a trip through TMEM each way.
//
// A CTA walks its run of tiles of kTK positions.  All its threads keep a ring of
// kST - 1 tiles of K and V rows in flight with 16-byte cp.async (rows found
// through the block table a tile ahead; padded rows, so ldmatrix meets no bank
// twice; rows behind the last position are zeros and are not read).  Per tile
// each of the 8 warps
//   * multiplies the rows of q with its 8 positions (scores in registers), takes
//     the largest of each row and shares it through shared memory,
//   * forms the weights 2^(s - m) against the running maximum of all warps (m lies
//     2^15 below it for f16 weights, whose smallest is 2^-24), adds them to its part
//     of the sum, and writes them, 16-bit, to shared memory,
//   * multiplies all weights of the tile with its share of v's columns.
// Every warp rescales its own columns when m grew; the sums meet at the end.
// Measured, E4M3, 128 sequences of 8 tokens behind 500 to 8000, 32 q heads, 8 heads of
// 128 (32 rows a unit): 1.08 GB in 1115 us, 1.0 TB/s, 14 % of a copy's rate.  One token
// a sequence, blocks of 12: bf16, 64 sequences behind 64 to 16384, 2 heads of 256: 230
// us, 4.4 TB/s; E4M3, 128 behind 500 to 8000: 459 us, 2.3 TB/s.  The barriers of a tile
// and the copies' issue bound it.
//
// E4M3 pools: codes go to f16 exactly (one conversion per two codes), so the
// products run in f16; K's scale multiplies the scores.  V's scale 2^e joins the
// weight: the running maximum is that of s + e, the weight 2^(s + e - m) is
// rounded to f16 relative to the largest contribution, and the sum takes
// 2^(s - m).  q's rows are brought to [1, 2) by a power of two that the
// scores take back, so bf16 q loses nothing that counts in f16.
//
// Positions that only some rows of a unit see (the new tokens of a causal chunk)
// may hold infinities and NaN, and 0 * NaN would reach the rows that do not
// see them.  Such a tile's v is searched: what is not finite is put to zero
// and added again, at the end, to the rows that see it.
#pragma once

#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_attend.cuh"
#include "lsc_ptx.h"

namespace lsc {
namespace kv {
namespace rows {

constexpr int kTK = 64;
constexpr int kThreads = 256;

// Ring depth and CTAs per SM: what keeps about 100 KB or more in flight per SM,
// with two CTAs where they fit (one's products run under the other's barriers).
template <int ES, int D, int MT>
struct Conf {
  static constexpr int RB = D * ES + 16;           // bytes of a K or V row in the ring
  static constexpr int stage = 2 * kTK * RB;
  static constexpr int occ = MT == 1 && D * ES <= 256 ? 2 : 1;
  static constexpr int ST = D * ES >= 256 ? (MT == 1 ? 3 : 5) : D * ES == 128 ? 5 : 6;
};

template <int ES, int D, int MT>
struct Smem {
  using C = Conf<ES, D, MT>;
  alignas(128) uint8_t ring[C::ST][C::stage];
  alignas(16) uint16_t w[16 * MT][kTK + 8];                    // weights of the tile
  int64_t at[C::ST][kTK];                          // byte offset of a position's row in a lane, -1: none
  float top[8][16 * MT];                           // a warp's largest score of a row
  float part[8][16 * MT];                          // a warp's part of a row's sum
  float qs[16 * MT];                               // E4M3: the power of two of a row of q
  int32_t vis[16 * MT];                            // positions a row sees
  float ks[ES == 1 ? C::ST : 1][kTK], vs[ES == 1 ? C::ST : 1][kTK];  // E4M3: scales of the tile's rows
  int32_t bad[ES == 1 ? 1 : 3][ES == 1 ? 1 : D];   // first position whose v is NaN, +inf, -inf
  alignas(16) uint16_t q[MT == 1 ? 1 : 16 * MT][MT == 1 ? 8 : D + 8];
  RunScratch run;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// BF16: the products' type (q's type; f16 for E4M3 pools).  ES: pool bytes per
// element (1: E4M3).
template <bool BF16, int ES, int D, int MT>
__global__ void __launch_bounds__(kThreads, (Conf<ES, D, MT>::occ))
rows_attend_kernel(const __grid_constant__ KvAttendParams p) {
  using C = Conf<ES, D, MT>;
  constexpr bool Q8 = ES == 1;
  constexpr int M = 16 * MT, ST = C::ST, RB = C::RB;
  constexpr int CPR = D * ES / 16;               // 16-byte chunks of a row
  constexpr int KS = D / 16;                     // k steps of a score
  constexpr int PV_WARPS = Q8 && D == 64 ? 4 : 8;  // warps that share v's columns (16 at least for E4M3)
  constexpr int COLS = D / PV_WARPS, NT = COLS / 8;
  constexpr float lift = BF16 ? 0.f : 15.f;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<ES, D, MT> &sm = *reinterpret_cast<Smem<ES, D, MT> *>(smem_raw);
  const int tid = threadIdx.x, w = tid >> 5, ln = tid & 31, g = ln >> 2, tq = ln & 3;
  griddep_wait();
  if (tid == 0) griddep_launch_dependents();
  const KvLayer &L = p.L;
  const int ctas = gridDim.x, cta = blockIdx.x;
  if (cta == 0) check_cu(L, p.b);
  const Workspace ws = workspace_at(p.ws, ctas, M);
  Run run = find_run<kThreads, M, kTK>(p, cta, ctas, sm.run);
  Piece pc;
  Cut cut = {0, 0, 0, 0};
  while (next_piece<M, kTK>(p, run, pc)) {
    const int R = pc.s.n * p.group < M ? pc.s.n * p.group : M;  // this launch's units have one block
    const int nt = pc.t1 - pc.t0;
    const int32_t kv = pc.s.kv;
    const int32_t *table = p.b.table + (int64_t)pc.seq * p.b.max_blocks;
    const int64_t row_bytes = (int64_t)L.heads * D * ES;
    const int64_t head_off = (int64_t)pc.head * D * ES;
    // where position `key` of the tile lies
    auto place = [&](int tile, int i) -> int64_t {
      const int32_t key = (pc.t0 + tile) * kTK + i;
      if (tile >= nt || key >= kv) return -1;
      const int32_t b = L.by_block.div(key);
      int32_t blk = table[b];
      if (blk < 0 || blk >= L.num_blocks) {
        report(L.status, LSC_ERR_OUT_OF_RANGE);
        blk = 0;
      }
      return (int64_t)blk * L.page + (int64_t)(key - b * L.block_tokens) * row_bytes;
    };
    auto issue = [&](int tile) {
      const int st = tile % ST;
      if (tile < nt) {
        const uint32_t base = smem_u32(sm.ring[st]);
#pragma unroll
        for (int c = tid; c < kTK * CPR; c += kThreads) {
          const int key = c / CPR, ch = c - key * CPR;
          const int64_t at = sm.at[st][key];
          const uint8_t *src = (at < 0 ? L.k : L.k + at + head_off) + ch * 16;
          const uint8_t *srv = (at < 0 ? L.v : L.v + at + head_off) + ch * 16;
          cp_async16_or_zero(base + key * RB + ch * 16, src, at >= 0);
          cp_async16_or_zero(base + (kTK + key) * RB + ch * 16, srv, at >= 0);
        }
      }
      cp_async_commit();
    };
    // E4M3: thread i < 128 reads the scale byte of position i & 63 (K, then V)
    auto scale_byte_of = [&](int tile) -> uint32_t {
      if (!Q8 || tid >= 2 * kTK || tile >= nt) return 127;
      const int key = tid & (kTK - 1);
      const int32_t pos = (pc.t0 + tile) * kTK + key;
      if (pos >= kv) return 127;
      const int32_t b = L.by_block.div(pos);
      const int32_t blk = table[b];
      if (blk < 0 || blk >= L.num_blocks) return 127;
      const uint8_t *lane = (tid < kTK ? L.k : L.v) + (int64_t)blk * L.page + L.scale_off;
      return lane[(int64_t)(pos - b * L.block_tokens) * L.heads + pc.head];
    };
    auto put_scale = [&](int tile, uint32_t byte) {
      if (Q8 && tid < 2 * kTK) (tid < kTK ? sm.ks : sm.vs)[tile % ST][tid & (kTK - 1)] = scale_of(byte);
    };

    __syncthreads();  // the last piece's shared memory is free
    if (tid < kTK)
#pragma unroll
      for (int s = 0; s < ST - 1; ++s) sm.at[s][tid] = place(s, tid);
    if (tid < M) sm.vis[tid] = tid < R ? visible(pc.s, p.by_group.div(tid), p.causal) : 0;
    if (!Q8)
      for (int i = tid; i < 3 * D; i += kThreads) (&sm.bad[0][0])[i] = INT32_MAX;
    // q: rows of 16-bit elements, for E4M3 as f16 times a power of two and with the elements of each group of 16 in
    // the order in which a lane meets the codes (4 consecutive ones per lane); at MT == 1 through the ring to registers
    uint16_t *sq = MT == 1 ? (uint16_t *)sm.ring[ST - 1] : &sm.q[0][0];
    constexpr int QS = D + 8;
    for (int r = w; r < M; r += kThreads / 32) {
      const int32_t tok = p.by_group.div(r);
      const uint16_t *src = (const uint16_t *)p.q + (int64_t)(pc.s.row0 + tok) * p.q_stride +
                            (int64_t)(pc.head * p.group + (r - tok * p.group)) * D;
      if constexpr (!Q8) {
        for (int c = ln; c < D / 8; c += 32)
          *(uint4 *)(sq + r * QS + c * 8) = r < R ? *(const uint4 *)(src + c * 8) : make_uint4(0, 0, 0, 0);
      } else {
        float x[D / 32];
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          const uint16_t b = r < R ? src[ln + 32 * e] : 0;
          x[e] = p.dtype == LSC_BF16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
          top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        // 2^k <= the largest magnitude < 2^(k + 1), where that is a normal number
        const uint32_t ex = top >> 23;
        const bool plain = ex == 0 || ex == 255;
        const float up = plain ? 1.f : __uint_as_float(ex << 23), down = plain ? 1.f : inv_scale_of(ex);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          const int d = ln + 32 * e, i = d & 15;
          // lane t of four holds dims 4t .. 4t+3 as k = 2t, 2t+1, 2t+8, 2t+9
          const int k = (i >> 2) * 2 + (i & 1) + ((i & 2) ? 8 : 0);
          sq[r * QS + (d & ~15) + k] = __half_as_ushort(__float2half_rn(x[e] * down));
        }
        if (ln == 0) sm.qs[r] = up;
      }
    }
    __syncthreads();
    uint32_t qf[MT == 1 ? KS : 1][4];
    if constexpr (MT == 1) {
#pragma unroll
      for (int k = 0; k < KS; ++k) ldsm4(qf[k], smem_u32(sq + (ln & 15) * QS + k * 16 + (ln >> 4) * 8));
    }
    uint32_t next_byte = 0;
#pragma unroll
    for (int s = 0; s < ST - 1; ++s) {
      issue(s);
      put_scale(s, scale_byte_of(s));
    }
    int64_t next_at = tid < kTK ? place(ST - 1, tid) : -1;
    next_byte = scale_byte_of(ST - 1);

    float m[MT][2], l[MT][2], o[MT][NT][4], qsc[MT][2];
    int32_t vis[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m[i][h] = -INFINITY;
        l[i][h] = 0.f;
        vis[i][h] = sm.vis[16 * i + 8 * h + g];
        qsc[i][h] = p.scale_log2 * (Q8 ? sm.qs[16 * i + 8 * h + g] : 1.f);
#pragma unroll
        for (int n = 0; n < NT; ++n) o[i][n][2 * h] = o[i][n][2 * h + 1] = 0.f;
      }
    const int32_t sure = visible(pc.s, 0, p.causal);  // every row sees positions below this

    for (int j = 0; j < nt; ++j) {
      const int st = j % ST;
      if (tid < kTK) sm.at[(j + ST - 1) % ST][tid] = next_at;  // tile j - 1's entry: its loads were issued long ago
      put_scale(j + ST - 1, next_byte);                         // as are tile j - 1's scales used (barrier below its products)
      cp_async_wait<ST - 2>();
      __syncthreads();  // tile j is here; nobody reads tile j - 1 any more
      issue(j + ST - 1);
      next_at = tid < kTK ? place(j + ST, tid) : -1;
      next_byte = scale_byte_of(j + ST);
      const uint32_t kb = smem_u32(sm.ring[st]), vb = kb + kTK * RB;
      const int32_t first = (pc.t0 + j) * kTK;
      const int32_t last = first + kTK < kv ? first + kTK : kv;
      if (last > sure) {  // positions [max(first, sure), last): some row does not see them
        const int lo = (sure > first ? sure : first) - first, cnt = last - first - lo;
        uint8_t *v = sm.ring[st] + kTK * RB;
        if constexpr (Q8) {
          for (int i = tid; i < cnt * D; i += kThreads) {
            const int key = lo + i / D;
            uint8_t &c = v[key * RB + i % D];
            if ((c & 0x7f) == 0x7f) {
              c = 0;
              sm.vs[st][key] = __uint_as_float(0x7fc00000u);
            }
          }
        } else {
          for (int i = tid; i < cnt * D; i += kThreads) {
            const int key = lo + i / D, d = i % D;
            uint16_t &c = *(uint16_t *)(v + key * RB + d * 2);
            constexpr uint16_t E = BF16 ? 0x7f80 : 0x7c00;
            if ((c & E) == E) {
              atomicMin(&sm.bad[(c & (E ^ 0x7fff)) ? 0 : (c & 0x8000) ? 2 : 1][d], first + key);
              c = 0;
            }
          }
        }
        __syncthreads();
      }
      // ---- scores of this warp's positions 8 w .. 8 w + 7
      float s[MT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
      const uint32_t ka = kb + (8 * w + (ln & 7)) * RB + (ln >> 3) * 16;
      constexpr int PER = Q8 ? 4 : 2;  // k steps per ldmatrix.x4
#pragma unroll
      for (int k0 = 0; k0 < KS; k0 += PER) {
        uint32_t b[4];
        ldsm4(b, ka + k0 * 16 * ES);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
          uint32_t b0, b1;
          if constexpr (Q8) b0 = e4m3x2_to_f16x2(b[k] & 0xffffu), b1 = e4m3x2_to_f16x2(b[k] >> 16);
          else b0 = b[2 * k], b1 = b[2 * k + 1];
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            if constexpr (MT == 1) {
              mma<BF16>(s[i], qf[k0 + k], b0, b1);
            } else {
              uint32_t a[4];
              ldsm4(a, smem_u32(&sm.q[16 * i + (ln & 15)][(k0 + k) * 16 + (ln >> 4) * 8]));
              mma<BF16>(s[i], a, b0, b1);
            }
          }
        }
      }
      // lane (g, tq) has rows g, g + 8 and positions 2 tq, 2 tq + 1 of the warp's eight
      const int kp = 8 * w + 2 * tq;
      float vx[2] = {1.f, 1.f}, kx[2] = {1.f, 1.f}, ve[2] = {0.f, 0.f};
      if constexpr (Q8) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          kx[e] = sm.ks[st][kp + e];
          vx[e] = sm.vs[st][kp + e];
          ve[e] = v_exponent((__float_as_uint(vx[e]) >> 23) & 255);
        }
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float t = -INFINITY;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = s[i][2 * h + e] * qsc[i][h];
            if constexpr (Q8) x *= kx[e];
            x = first + kp + e < vis[i][h] ? x : -INFINITY;
            s[i][2 * h + e] = x;
            t = fmaxf(t, x + ve[e]);
          }
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
          if (tq == 0) sm.top[w][16 * i + 8 * h + g] = t - lift;
        }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * i + 8 * h + g;
          float t = m[i][h];
#pragma unroll
          for (int x = 0; x < 8; ++x) t = fmaxf(t, sm.top[x][r]);
          const float ref = t == -INFINITY ? 0.f : t, keep = exp2f(m[i][h] - ref);
          m[i][h] = t;
          l[i][h] *= keep;
#pragma unroll
          for (int n = 0; n < NT; ++n) o[i][n][2 * h] *= keep, o[i][n][2 * h + 1] *= keep;
          const float p0 = exp2f(s[i][2 * h] - ref), p1 = exp2f(s[i][2 * h + 1] - ref);
          l[i][h] += p0 + p1;
          // a position that the row does not see has weight 0 whatever its scale
          const float w0 = Q8 ? (first + kp < vis[i][h] ? p0 * vx[0] : 0.f) : p0;
          const float w1 = Q8 ? (first + kp + 1 < vis[i][h] ? p1 * vx[1] : 0.f) : p1;
          *(uint32_t *)&sm.w[r][kp] = pack2(w0, w1, BF16);
        }
      __syncthreads();
      // ---- weights times this warp's columns of v
      if (w < PV_WARPS) {
#pragma unroll
        for (int k = 0; k < kTK / 16; k += 2) {  // 32 positions
          uint32_t a[MT][2][4];
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              ldsm4(a[i][y], smem_u32(&sm.w[16 * i + (ln & 15)][(k + y) * 16 + (ln >> 4) * 8]));
          // four 8 x 8 matrices: positions 0-7, 8-15, 16-23, 24-31 of one group of 16 bytes
          const uint32_t va = vb + (k * 16 + ln) * RB + w * COLS * ES;
#pragma unroll
          for (int c = 0; c < COLS * ES / 16; ++c) {
            uint32_t b[4];
            ldsm4t(b, va + c * 16);
            if constexpr (Q8) {
#pragma unroll
              for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int odd = 0; odd < 2; ++odd) {  // columns 2 i, then 2 i + 1, of the 16
                  const uint32_t sel = odd ? 0x31 : 0x20;
                  const uint32_t b0 = e4m3x2_to_f16x2(__byte_perm(b[2 * y], 0, sel) & 0xffffu);
                  const uint32_t b1 = e4m3x2_to_f16x2(__byte_perm(b[2 * y + 1], 0, sel) & 0xffffu);
#pragma unroll
                  for (int i = 0; i < MT; ++i) mma<BF16>(o[i][2 * c + odd], a[i][y], b0, b1);
                }
            } else {
#pragma unroll
              for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int i = 0; i < MT; ++i) mma<BF16>(o[i][c], a[i][y], b[2 * y], b[2 * y + 1]);
            }
          }
        }
      }
    }
    // ---- the piece's end: sums of all warps, then rows out or to the workspace
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = l[i][h];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (tq == 0) sm.part[w][16 * i + 8 * h + g] = x;
      }
    __syncthreads();
    cp_async_wait<0>();
    const bool whole = pc.t0 == 0 && pc.t1 == pc.tiles;
    const int64_t slot = (int64_t)(2 * cta + (pc.t0 == 0 ? 1 : 0)) * M;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * i + 8 * h + g;
        if (r >= R) continue;
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < 8; ++x) sum += sm.part[x][r];
        const bool empty = vis[i][h] == 0;
        const float inv = whole ? (empty ? 0.f : 1.f / sum) : 1.f;
        const int32_t tok = p.by_group.div(r);
        const int64_t t = pc.s.row0 + tok, hd = (int64_t)pc.head * p.group + (r - tok * p.group);
        if (w == 0 && tq == 0) {
          if (!whole) ws.ml[slot + r] = make_float2(m[i][h], sum);
          else if (p.lse) p.lse[t * p.heads + hd] = empty ? -INFINITY : (m[i][h] + log2f(sum)) * 0.693147180559945309f;
        }
        if (w >= PV_WARPS) continue;
        uint16_t *out = (uint16_t *)p.out + t * p.out_stride + hd * D;
        float *part = ws.o + (slot + r) * D;
#pragma unroll
        for (int n = 0; n < NT; n += Q8 ? 2 : 1) {
          if constexpr (Q8) {  // four columns in a row: even and odd ones are in two tiles
            const int d = w * COLS + n * 8 + 4 * tq;
            const float x0 = o[i][n][2 * h] * inv, x1 = o[i][n + 1][2 * h] * inv, x2 = o[i][n][2 * h + 1] * inv,
                        x3 = o[i][n + 1][2 * h + 1] * inv;
            if (whole) {
              const int bf = p.dtype == LSC_BF16;
              *(uint2 *)(out + d) = make_uint2(pack2(x0, x1, bf), pack2(x2, x3, bf));
            } else {
              *(float4 *)(part + d) = make_float4(x0, x1, x2, x3);
            }
          } else {
            const int d = w * COLS + n * 8 + 2 * tq;
            float x[2] = {o[i][n][2 * h] * inv, o[i][n][2 * h + 1] * inv};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (sm.bad[1][d + e] < vis[i][h]) x[e] += INFINITY;
              if (sm.bad[2][d + e] < vis[i][h]) x[e] -= INFINITY;
              if (sm.bad[0][d + e] < vis[i][h]) x[e] = __uint_as_float(0x7fc00000u);
            }
            if (whole) *(uint32_t *)(out + d) = pack2(x[0], x[1], BF16);
            else *(float2 *)(part + d) = make_float2(x[0], x[1]);
          }
        }
      }
    cut = cut_of(run, pc, cta);
  }
  if (tid == 0 && p.ws) ws.cut[cta] = cut;
}

template <bool BF16, int ES, int D, int MT>
cudaError_t launch_one(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  static SmemLimit limit;
  const int smem = (int)sizeof(Smem<ES, D, MT>);
  auto *k = rows_attend_kernel<BF16, ES, D, MT>;
  const cudaError_t e = limit.ensure((const void *)k, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, plan.ctas, kThreads, smem, stream, p);
}

// One type's kernels, by head size and rows.
template <bool BF16, int ES, int D>
cudaError_t launch_size(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  if constexpr (ES == 1)  // 16-bit pools: more than 16 rows are the chunk kernel's
    if (plan.M > 16) return launch_one<BF16, ES, D, 4>(p, plan, stream);
  return launch_one<BF16, ES, D, 1>(p, plan, stream);
}

template <bool BF16, int ES>
cudaError_t launch_type(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream) {
  switch (p.L.head_dim) {
    case 64: return launch_size<BF16, ES, 64>(p, plan, stream);
    case 128: return launch_size<BF16, ES, 128>(p, plan, stream);
    default: return launch_size<BF16, ES, 256>(p, plan, stream);
  }
}

template <int ES, int D>
constexpr int occ_of(int M) { return M == 16 ? Conf<ES, D, 1>::occ : Conf<ES, D, ES == 1 ? 4 : 1>::occ; }

}  // namespace rows
}  // namespace kv

cudaError_t launch_kv_attend_rows_bf16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
cudaError_t launch_kv_attend_rows_f16(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
cudaError_t launch_kv_attend_rows_e4m3(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);

}  // namespace lsc
