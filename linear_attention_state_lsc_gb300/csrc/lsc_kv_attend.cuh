// lsc_kv_attend.cuh -- what the tensor-core forms of lsc_kv_attend share: how the
// work is cut, where parts of a cut unit go, and how they are joined.
//
// A unit is one kv head of a sequence (decode: a group of up to four) with up to M packed rows: packed row R of
// a (sequence, kv head) is q head R % group of new token R / group, so the heads
// that share K and V are rows of one tile and K/V is read once for all of
// them.  A unit's work is its tiles of TK positions, up to the last one that
// any of its rows sees (at least one, so that a unit that sees nothing still
// writes its zeros).  Before its tiles a unit has `lead` counts for the time that
// it takes besides them.  All counts of all units, in the order (sequence, kv head,
// row block, count), are cut into equal runs, one per CTA: lengths that differ
// between sequences do not leave SMs idle, and a single long sequence spreads
// over all of them.  The cut is computed on the device from the lengths, so a
// captured graph follows them.
//
// Units that are short for everybody (p.whole: by the host's bound of the
// lengths) are not cut: each counts as one in the order above, and a run is of
// whole units.  Joining the parts of a 256-row unit costs as much time as eight of
// its tiles.
//
// A run that holds all tiles of a unit writes its rows; parts of a cut unit go
// to the workspace as (maximum, sum, unnormalised fp32 row), and a second launch
// joins them in tile order.  A CTA has at most two parts: slot 0, the rest of a
// unit that began in an earlier CTA, and slot 1, the beginning of one that goes
// on in the next.
#pragma once

#include <cuda.h>
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

// Counts here are below 2^31 (the host sends larger calls to the CUDA cores).

// Row blocks of M packed rows of a sequence.
template <int M>
__device__ __forceinline__ int32_t row_blocks(const Seq &s, int32_t group) {
  return (s.n * group + M - 1) / M;
}

// Tiles of one row block.
template <int M, int TK>
__device__ __forceinline__ int32_t block_tiles(const KvAttendParams &p, const Seq &s, int32_t block) {
  const int32_t rows = s.n * p.group, last = (block + 1) * M < rows ? (block + 1) * M - 1 : rows - 1;
  const int32_t t = (visible(s, p.by_group.div(last), p.causal) + TK - 1) / TK;
  return t < 1 ? 1 : t;
}

// Counts of one kv head of a sequence.
template <int M, int TK>
__device__ __forceinline__ int32_t seq_tiles(const KvAttendParams &p, int32_t i) {
  if (i >= p.b.n_seq) return 0;
  const Seq s = attend_seq(p.L, p.b, i, p.max_seq, p.max_kv);
  const int32_t nb = row_blocks<M>(s, p.group);
  int32_t t = 0;
  if (p.whole) return nb;
#pragma unroll 1
  for (int32_t b = 0; b < nb; ++b) t += p.lead + block_tiles<M, TK>(p, s, b);
  return t;
}

// Where a CTA's run is: the walk over its pieces.
struct Run {
  int32_t pos, end, chunk;  // in the order of all counts; pos == end: done
  int32_t seq, head, block, count;
};

struct Piece {
  Seq s;
  int32_t seq, head, block;
  int32_t t0, t1, tiles;  // tiles [t0, t1) of the unit's `tiles`
};

struct RunScratch {
  int32_t warp_sum[32];
  int32_t total, before, seq;
};

// Inclusive sum over the block of x, and the block's total.  NT threads, all present.
template <int NT>
__device__ __forceinline__ int32_t block_scan(int32_t x, RunScratch &sc, int32_t *inclusive) {
  const int ln = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (ln >= o) x += y;
  }
  if (ln == 31) sc.warp_sum[w] = x;
  __syncthreads();
  const int32_t ws = ln < NT / 32 ? sc.warp_sum[ln] : 0;
  const int32_t before = __reduce_add_sync(0xffffffffu, ln < w ? ws : 0), all = __reduce_add_sync(0xffffffffu, ws);
  __syncthreads();
  *inclusive = before + x;
  return all;
}

// The run of CTA `cta` of `ctas`; called by all NT threads.
template <int NT, int M, int TK>
__device__ __forceinline__ Run find_run(const KvAttendParams &p, int cta, int ctas, RunScratch &sc) {
  const int H = p.groups;
  int32_t total = 0, mine = 0, incl = 0;
  bool down = false;
#pragma unroll 1
  for (int32_t i0 = 0; i0 < p.b.n_seq; i0 += NT) {
    const int32_t i = i0 + threadIdx.x;
    down |= i < p.b.n_seq && p.b.cu[i + 1] < p.b.cu[i];
    mine = seq_tiles<M, TK>(p, i);
    total += block_scan<NT>(mine, sc, &incl);
  }
  total *= H;
  // Sequences that overlap (recorded by check_cu) could count past 31 bits: no work then.
  if (__syncthreads_or(down)) total = 0;
  Run r;
  r.chunk = (total + ctas - 1) / ctas;
  if (r.chunk < p.min_run) r.chunk = p.min_run;
  r.pos = cta * r.chunk;
  r.end = r.pos + r.chunk < total ? r.pos + r.chunk : total;
  r.seq = r.head = r.block = r.count = 0;
  if (r.pos >= r.end) {
    r.pos = r.end;
    return r;
  }
  int32_t base = 0;
#pragma unroll 1
  for (int32_t i0 = 0; i0 < p.b.n_seq; i0 += NT) {
    int32_t all = 0;
    if (p.b.n_seq > NT) {  // else the first pass left this thread's values
      mine = seq_tiles<M, TK>(p, i0 + threadIdx.x);
      all = block_scan<NT>(mine, sc, &incl);
    }
    if (mine > 0 && (base + incl - mine) * H <= r.pos && r.pos < (base + incl) * H) {
      sc.seq = i0 + threadIdx.x;
      sc.before = (base + incl - mine) * H;
      sc.total = mine;
    }
    base += all;
  }
  __syncthreads();
  r.seq = sc.seq;
  int32_t rem = r.pos - sc.before;
  r.head = rem / sc.total;
  rem -= r.head * sc.total;
  if (p.whole) {
    r.block = rem;
    return r;
  }
  const Seq s = attend_seq(p.L, p.b, r.seq, p.max_seq, p.max_kv);
#pragma unroll 1
  for (;;) {
    const int32_t t = p.lead + block_tiles<M, TK>(p, s, r.block);
    if (rem < t) break;
    rem -= t;
    ++r.block;
  }
  r.count = rem;
  return r;
}

// The next piece of the run; false when it is done.
template <int M, int TK>
__device__ __forceinline__ bool next_piece(const KvAttendParams &p, Run &r, Piece &q) {
  if (r.pos >= r.end) return false;
  Seq s = attend_seq(p.L, p.b, r.seq, p.max_seq, p.max_kv);
#pragma unroll 1
  while (r.block >= row_blocks<M>(s, p.group)) {  // past this head's blocks (or a sequence without new tokens)
    r.block = 0;
    if (s.n == 0 || ++r.head == p.groups) {
      r.head = 0;
      ++r.seq;
      s = attend_seq(p.L, p.b, r.seq, p.max_seq, p.max_kv);
    }
  }
  q.s = s;
  q.seq = r.seq;
  q.head = r.head;
  q.block = r.block;
  q.tiles = block_tiles<M, TK>(p, s, r.block);
  if (p.whole) {
    q.t0 = 0;
    q.t1 = q.tiles;
    r.pos += 1;
  } else {
    const int32_t c0 = r.count - p.lead, rest = q.tiles - c0, left = r.end - r.pos;
    const int32_t c = rest < left ? rest : left;
    q.t0 = c0 > 0 ? c0 : 0;
    q.t1 = c0 + c;
    r.pos += c;
    if (q.t1 <= 0) return false;  // the run ends before the unit's first tile
  }
  r.count = 0;
  ++r.block;
  return true;
}

// The CTA's record, given its last piece (after next_piece moved past it).
__device__ __forceinline__ Cut cut_of(const Run &r, const Piece &q, int cta) {
  Cut c = {q.seq, q.head, q.block, 0};
  if (q.t0 == 0 && q.t1 < q.tiles) c.more = (r.pos + (q.tiles - q.t1) - 1) / r.chunk - cta;
  return c;
}

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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Byte of 16-byte chunk ch of row r in a swizzled tile of `rows` rows: columns of LINE bytes, chunks xor the row's low bits
// (lines of 64 bytes: pairs of rows share 128).
template <int LINE>
__device__ __forceinline__ uint32_t chunk_at(int rows, int r, int ch) {
  if constexpr (LINE == 64) return r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
  else return (ch >> 3) * (rows * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

// Tiled TMA load of one box of a layer's rows (this CTA's shared memory), completing on `bar`.
__device__ __forceinline__ void tma_box(void *dst, const CUtensorMap *map, int row, int col, int head, int block,
                                        uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(0), "r"(row), "r"(col), "r"(head), "r"(block), "r"(smem_u32(bar))
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

}  // namespace kv

// ---- plans and launches (lsc_kv_attend_join.cu; a type's kernels in lsc_kv_attend_{decode,rows,chunk}_*.cu) ----
struct AttendPlan {
  int32_t ctas;    // runs
  int32_t M;       // rows of a unit, `together` heads' worth
  int32_t TK;      // positions of a tile
  int32_t together;  // kv heads of a unit
  size_t ws_bytes;
  bool may_cut;    // false: units are not cut
  int32_t min_run; // tiles of a run at least
  int32_t lead;    // tiles' worth of time that a unit takes besides its tiles
};
cudaError_t launch_kv_attend_rows(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
cudaError_t launch_kv_attend_decode(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
AttendPlan plan_kv_attend_decode(const KvAttendParams &p, bool side_by_side = true);
cudaError_t launch_kv_attend_join(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
AttendPlan plan_kv_attend_rows(const KvAttendParams &p);
cudaError_t launch_kv_attend_chunk(const KvAttendParams &p, const AttendPlan &plan, cudaStream_t stream);
AttendPlan plan_kv_attend_chunk(const KvAttendParams &p);

}  // namespace lsc
