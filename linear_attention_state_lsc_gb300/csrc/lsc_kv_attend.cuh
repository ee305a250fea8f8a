// lsc_kv_attend.cuh -- what the tensor-core forms of lsc_kv_attend share: how the
// work is cut, where parts of a cut unit go, and how they are joined.
//
// A unit is one kv head of a sequence with up to M packed rows: packed row R of
// a (sequence, kv head) is q head R % group of new token R / group, so the heads
// that share K and V are rows of one tile and K/V is read once for all of
// them.  A unit's work is its tiles of TK positions, up to the last one that
// any of its rows sees (at least one, so that a unit that sees nothing still
// writes its zeros).  All tiles of all units, in the order (sequence, kv head,
// row block, tile), are cut into equal runs, one per CTA: lengths that differ
// between sequences do not leave SMs idle, and a single long sequence spreads
// over all of them.  The cut is computed on the device from the lengths, so a
// captured graph follows them.
//
// A run that holds all tiles of a unit writes its rows; parts of a cut unit go
// to the workspace as (maximum, sum, unnormalised fp32 row), and a second launch
// joins them in tile order.  A CTA has at most two parts: slot 0, the rest of a
// unit that began in an earlier CTA, and slot 1, the beginning of one that goes
// on in the next.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "lsc_internal.h"
#include "lsc_kv_batch.cuh"
#include "lsc_ptx.h"

namespace lsc {
namespace kv {

// A CTA's record of the unit that begins in it and is cut: `more` CTAs after it
// hold the rest (0: none).
struct Cut {
  int32_t seq, head, block, more;
};

struct Workspace {
  Cut *cut;    // [ctas]
  float2 *ml;  // [ctas][2][M]
  float *o;    // [ctas][2][M][D]
};

__host__ __device__ __forceinline__ size_t workspace_size(int ctas, int M, int D) {
  return (size_t)ctas * (sizeof(Cut) + 2 * (size_t)M * (sizeof(float2) + (size_t)D * sizeof(float)));
}
__host__ __device__ __forceinline__ Workspace workspace_at(uint8_t *ws, int ctas, int M) {
  Workspace w;
  w.o = nullptr;
  w.cut = (Cut *)ws;
  w.ml = (float2 *)(ws + (size_t)ctas * sizeof(Cut));
  w.o = (float *)(ws + (size_t)ctas * (sizeof(Cut) + 2 * (size_t)M * sizeof(float2)));
  return w;
}

// Row blocks of M packed rows of a sequence.
template <int M>
__device__ __forceinline__ int32_t row_blocks(const Seq &s, int32_t group) {
  return (int32_t)(((int64_t)s.n * group + M - 1) / M);
}

// Tiles of one row block.
template <int M, int TK>
__device__ __forceinline__ int32_t block_tiles(const Seq &s, int32_t group, int32_t causal, int32_t block) {
  int64_t last = (int64_t)(block + 1) * M - 1;
  const int64_t rows = (int64_t)s.n * group;
  if (last >= rows) last = rows - 1;
  int32_t v = visible(s, (int32_t)(last / group), causal);
  const int32_t t = (int32_t)(((int64_t)v + TK - 1) / TK);
  return t < 1 ? 1 : t;
}

template <int M, int TK>
__device__ __forceinline__ int64_t seq_tiles(const Seq &s, int32_t group, int32_t causal) {
  const int32_t nb = row_blocks<M>(s, group);
  if (!causal) return nb ? (int64_t)nb * block_tiles<M, TK>(s, group, causal, 0) : 0;
  int64_t t = 0;
  for (int32_t b = 0; b < nb; ++b) t += block_tiles<M, TK>(s, group, causal, b);
  return t;
}

// Where a CTA's run is: the walk over its pieces.
struct Run {
  int64_t pos, end, chunk;  // tile indexes in the order of all tiles; pos == end: done
  int32_t seq, head, block, tile;
};

struct Piece {
  Seq s;
  int32_t seq, head, block;
  int32_t t0, t1, tiles;  // tiles [t0, t1) of the unit's `tiles`
};

struct RunScratch {
  int64_t warp_sum[32];
  int64_t total, before;
  int32_t seq;
};

// Sum over the block of x; every thread gets the total.  NT threads, all present.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t x, RunScratch &sc, int64_t *inclusive) {
  const int ln = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (ln >= o) x += y;
  }
  if (ln == 31) sc.warp_sum[w] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    const int64_t y = sc.warp_sum[i];
    if (i < w) before += y;
    all += y;
  }
  __syncthreads();
  *inclusive = before + x;
  return all;
}

// The run of CTA `cta` of `ctas`; called by all NT threads.
template <int NT, int M, int TK>
__device__ __forceinline__ Run find_run(const KvAttendParams &p, int cta, int ctas, RunScratch &sc) {
  const int H = p.L.heads;
  int64_t total = 0, mine = 0, incl = 0;
  for (int32_t i0 = 0; i0 < p.b.n_seq; i0 += NT) {
    const int32_t i = i0 + threadIdx.x;
    mine = i < p.b.n_seq
               ? seq_tiles<M, TK>(attend_seq(p.L, p.b, i, p.max_seq, p.max_kv), p.group, p.causal)
               : 0;
    total += block_scan<NT>(mine, sc, &incl);
  }
  total *= H;
  Run r;
  r.chunk = (total + ctas - 1) / ctas;
  if (r.chunk < 1) r.chunk = 1;
  r.pos = (int64_t)cta * r.chunk;
  r.end = r.pos + r.chunk < total ? r.pos + r.chunk : total;
  r.seq = r.head = r.block = r.tile = 0;
  if (r.pos >= r.end) {
    r.pos = r.end;
    return r;
  }
  int64_t base = 0;
  for (int32_t i0 = 0; i0 < p.b.n_seq; i0 += NT) {
    const int32_t i = i0 + threadIdx.x;
    if (p.b.n_seq > NT) {  // else the first pass left this thread's values
      mine = i < p.b.n_seq
                 ? seq_tiles<M, TK>(attend_seq(p.L, p.b, i, p.max_seq, p.max_kv), p.group, p.causal)
                 : 0;
      const int64_t all = block_scan<NT>(mine, sc, &incl);
      if (mine > 0 && (base + incl - mine) * H <= r.pos && r.pos < (base + incl) * H) {
        sc.seq = i;
        sc.before = (base + incl - mine) * H;
        sc.total = mine;
      }
      base += all;
    } else if (mine > 0 && (incl - mine) * H <= r.pos && r.pos < incl * H) {
      sc.seq = i;
      sc.before = (incl - mine) * H;
      sc.total = mine;
    }
  }
  __syncthreads();
  r.seq = sc.seq;
  const int64_t off = r.pos - sc.before;
  r.head = (int32_t)(off / sc.total);
  int64_t rem = off - (int64_t)r.head * sc.total;
  const Seq s = attend_seq(p.L, p.b, r.seq, p.max_seq, p.max_kv);
  for (;;) {
    const int32_t t = block_tiles<M, TK>(s, p.group, p.causal, r.block);
    if (rem < t) break;
    rem -= t;
    ++r.block;
  }
  r.tile = (int32_t)rem;
  return r;
}

// The next piece of the run; false when it is done.
template <int M, int TK>
__device__ __forceinline__ bool next_piece(const KvAttendParams &p, Run &r, Piece &q) {
  if (r.pos >= r.end) return false;
  Seq s = attend_seq(p.L, p.b, r.seq, p.max_seq, p.max_kv);
  while (r.block >= row_blocks<M>(s, p.group)) {  // past this head's blocks (or a sequence without new tokens)
    r.block = 0;
    if (row_blocks<M>(s, p.group) == 0 || ++r.head == p.L.heads) {
      r.head = 0;
      ++r.seq;
      s = attend_seq(p.L, p.b, r.seq, p.max_seq, p.max_kv);
    }
  }
  q.s = s;
  q.seq = r.seq;
  q.head = r.head;
  q.block = r.block;
  q.tiles = block_tiles<M, TK>(s, p.group, p.causal, r.block);
  q.t0 = r.tile;
  const int64_t left = r.end - r.pos;
  q.t1 = q.tiles - q.t0 <= left ? q.tiles : q.t0 + (int32_t)left;
  r.pos += q.t1 - q.t0;
  r.tile = 0;
  ++r.block;
  return true;
}

// The CTA's record, given its last piece (after next_piece moved past it).
__device__ __forceinline__ Cut cut_of(const Run &r, const Piece &q, int cta) {
  Cut c = {q.seq, q.head, q.block, 0};
  if (q.t0 == 0 && q.t1 < q.tiles) c.more = (int32_t)((r.pos + (q.tiles - q.t1) - 1) / r.chunk) - cta;
  return c;
}

// Dense addresses of a packed row.
__device__ __forceinline__ int64_t row_token(const Seq &s, int32_t group, int64_t R) { return s.row0 + R / group; }

__device__ __forceinline__ uint32_t pack2(float x, float y, int bf16) {
  if (bf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// 16 bytes global -> shared, or zeros when `on` is false (nothing is read then).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

}  // namespace kv

// ---- launches (lsc_kv_attend_rows_*.cu, lsc_kv_attend_chunk.cu, lsc_kv_attend_join.cu) ----
struct AttendPlan {
  int32_t ctas;    // runs
  int32_t M;       // rows of a unit
  size_t ws_bytes; // of this launch's part of the workspace
  bool may_cut;    // false: every unit is one tile, so no run can cut one
};
cudaError_t launch_kv_attend_rows(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
cudaError_t launch_kv_attend_join(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
AttendPlan plan_kv_attend_rows(const KvAttendParams &p);
cudaError_t launch_kv_attend_chunk(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
AttendPlan plan_kv_attend_chunk(const KvAttendParams &p);

}  // namespace lsc
