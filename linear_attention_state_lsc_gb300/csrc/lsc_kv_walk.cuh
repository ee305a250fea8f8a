// lsc_kv_walk.cuh -- how the warps of a row kernel share a step's tokens: all items (a
// token's rows are a number of them) in token order are cut into equal runs, one a
// warp, so a warp finds a sequence and a block once for the tokens that share them,
// no barrier paces it, and a handful of tokens still spreads over many warps.
#pragma once

#include <cuda_runtime.h>

#include "lsc_internal.h"
#include "lsc_kv_batch.cuh"

namespace lsc {
namespace kv {

constexpr int kWalkThreads = 256, kWalkWarps = kWalkThreads / 32;

// Items [begin, end) of this warp; item = token * per_token + rest.
struct WarpRun {
  int64_t begin, end;
};
__device__ __forceinline__ WarpRun warp_run(int64_t items) {
  const int64_t warps = (int64_t)gridDim.x * kWalkWarps, w = (int64_t)blockIdx.x * kWalkWarps + (threadIdx.x >> 5);
  return {items * w / warps, items * (w + 1) / warps};
}
// CTAs for that: an item a warp at least, `occ` CTAs an SM at most.
inline int walk_grid(int64_t items, int num_sms, int occ) {
  const int64_t need = (items + kWalkWarps - 1) / kWalkWarps, most = (int64_t)num_sms * occ;
  return (int)(need < most ? need : most);
}

// Where the warp's tokens sit, in token order.  All lanes of the warp call at() together and hold the same.
struct PlaceWalk {
  int32_t c0 = 0, c1 = -1, seq = -1, kv = 0;  // the last token's sequence; c1 < 0: none yet
  int32_t block = -1;                         // and its block of that sequence
  int64_t page = 0;                           // byte of it in a lane, -1: a bad one

  // The last entry of cu_seqlens that is <= t, 32 at a time; -1: none.
  static __device__ __forceinline__ int32_t search(const KvBatch &b, int32_t t) {
    int32_t lo = -1, hi = b.n_seq + 1;
    while (hi - lo > 1) {
      const int32_t step = (hi - lo - 1 + 31) / 32, i = lo + 1 + (int32_t)(threadIdx.x & 31) * step;
      const bool le = i < hi && i > lo && b.cu[i] <= t;
      const int32_t n = __popc(__ballot_sync(0xffffffffu, le));
      if (n == 0) break;
      lo += 1 + (n - 1) * step;
      hi = hi < lo + step ? hi : lo + step;
    }
    return lo;
  }

  // Row of token t in its block, its page in `page`; -1: no row in the cache, -2: the token belongs to no sequence.
  __device__ __forceinline__ int32_t at(const KvLayer &L, const KvBatch &b, int32_t t) {
    if (!(c0 <= t && t < c1)) {
      seq = search(b, t);
      if (seq < 0 || seq >= b.n_seq) {
        c1 = -1;
        return -2;
      }
      c0 = b.cu[seq];
      c1 = b.cu[seq + 1];
      kv = checked_kv(L, b, b.kv[seq]);
      block = -1;
      if (!(c0 <= t && t < c1)) return -1;
    }
    const int64_t pos = (int64_t)kv - ((int64_t)c1 - c0) + (t - c0);
    if (pos < 0) return -1;
    const int32_t q = L.by_block.div((int32_t)pos);
    if (q != block) {
      const int32_t blk = b.table[(int64_t)seq * b.max_blocks + q];
      block = q;
      page = (int64_t)blk * L.page;
      if ((uint32_t)blk >= (uint32_t)L.num_blocks) {
        report(L.status, LSC_ERR_OUT_OF_RANGE);
        page = -1;
      }
    }
    return page < 0 ? -1 : (int32_t)pos - q * L.block_tokens;
  }
};

}  // namespace kv
}  // namespace lsc
