// lsc_kv.cu -- host side of the attention K/V block pool (include/lsc_kv.h):
// layout, views, copy_prefix's validation and launch plans, and the argument
// checks of append, rotary positions, gather and attend.  The copy kernel is
// kv_copy_kernel in lsc_copy.cu; append and gather are in lsc_kv_rows.cu (E2M1 pools:
// lsc_kv_rows4.cu), rotary positions in lsc_kv_rotary.cu, attend in lsc_kv_attend_*.
//
// Sources, cited by page title and section:
//   [VA] "非连续 KV Cache" §3, §3.2, §3.4 (page-strided block views, separate K
//        and V views, the merged two-lane view)
//   [KP] "Kapitsa 源码拆解 05：前缀缓存与模型状态恢复", figure 2 (copy_prefix)
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <new>
#include <vector>

#include "lsc_internal.h"
#include "lsc_kv_attend.cuh"
#include "lsc_kv.h"

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct lsc_kv_pool {
  lsc_kv_pool_desc d;
  int device = -1;  // -1: host-only pool (no GPU when created)
  int num_sms = 0;
  uint8_t *base = nullptr;
  bool owns_base = false;
  int64_t bits = 0, row_bytes = 0, payload = 0, lane_bytes = 0, region_bytes = 0;
  int32_t scale_off = 0;        // E4M3, E2M1: page offset of the scale bytes
  int32_t scale_row = 0;        // and scale bytes of a token row
  int32_t *status = nullptr;    // device error word
  int32_t box_rows = 0;         // rows of a TMA box of `maps`
  int32_t box_decode = 0;       // and of `maps_decode`
  std::vector<CUtensorMap> maps, maps_decode;  // per layer; empty: none
  EncodeTiled encode = nullptr;                // null: no maps to be had
};

namespace {

int esize(int32_t dtype) {
  switch (dtype) {
    case LSC_F32: return 4;
    case LSC_BF16: return 2;
    case LSC_F16: return 2;
    case LSC_E4M3: return 1;
    default: return 0;
  }
}

int bits_of(int32_t dtype) { return dtype == LSC_E2M1 ? 4 : 8 * esize(dtype); }

// Bound of every device-side wait (mbarrier), in nanoseconds.
constexpr uint64_t kWaitLimitNs = 1000000000ull;

// Host-side fault injection for the tests: LSC_FAULT=<name>.
bool fault(const char *name) {
  const char *f = getenv("LSC_FAULT");
  return f && strcmp(f, name) == 0;
}

// [VA] §3: block stride = physical page size / element size, so the page must
// hold the logical block and divide by the element size; 16-byte vector copies
// add page % 16 == 0.
int describe(const lsc_kv_pool_desc *d, lsc_kv_pool *g) {
  if (!d || d->num_layers <= 0 || d->num_blocks <= 0 || d->block_tokens <= 0 || d->num_kv_heads <= 0 ||
      d->head_dim <= 0)
    return LSC_ERR_INVALID_ARG;
  const int bits = bits_of(d->dtype);
  if (!bits) return LSC_ERR_INVALID_ARG;
  if (d->dtype == LSC_E2M1 && d->head_dim % 16 != 0) return LSC_ERR_LAYOUT;
  g->d = *d;
  g->bits = bits;
  const int64_t elements = (int64_t)d->num_kv_heads * d->head_dim;
  if (bits == 4 && elements > INT32_MAX - 1023) return LSC_ERR_LAYOUT;  // rows are walked in stretches of up to 1024, in 32 bits
  g->row_bytes = bits == 4 ? elements / 2 : elements * (bits / 8);
  g->payload = g->row_bytes * d->block_tokens;
  if (bits <= 8) {  // codes, then one scale byte per (row, head), or per 16 elements of it, at the next 16 B boundary
    const int64_t off = (g->payload + 15) / 16 * 16;
    if (off > INT32_MAX) return LSC_ERR_LAYOUT;
    g->scale_off = (int32_t)off;
    const int64_t scales = bits == 8 ? d->num_kv_heads : elements / 16;
    if (bits == 4 && scales > (INT32_MAX - off) / d->block_tokens) return LSC_ERR_LAYOUT;
    g->scale_row = (int32_t)scales;
    g->payload = off + scales * d->block_tokens;
  }
  if (d->page_bytes < g->payload || (bits > 8 && d->page_bytes % (bits / 8))) return LSC_ERR_LAYOUT;
  if (d->page_bytes % 16) return LSC_ERR_MISALIGNED;
  g->lane_bytes = (int64_t)d->num_blocks * d->page_bytes;
  g->region_bytes = 2 * g->lane_bytes;
  return LSC_OK;
}

// TMA maps of the layers' rows, for attend: coordinates (element of a column, row
// of a block, column of 128 bytes, kv head, block; V's blocks follow K's), a box
// of one column, or of all when it has a whole tile's rows.  A box never leaves its
// block: its rows are the largest power of two that divides block_tokens, up to
// the tile's.  128-byte swizzle (rows of 64 or 32 bytes: 64- or 32-byte).  Without maps (blocks that are
// no multiple of 8 tokens, other types and sizes) the kernels copy rows themselves.
// One region's map: `blocks` pages of each lane, heads of head_dim elements of `bits` bits.
bool encode_map(EncodeTiled encode, CUtensorMap *map, void *region, int32_t dtype, int bits, int32_t block_tokens,
                int32_t heads, int32_t head_dim, int64_t page, int64_t blocks, int tile, int box) {
  const int row = head_dim * bits / 8, col = row < 128 ? row : 128;  // bytes
  const int es = bits == 16 ? 2 : 1;  // of the map's elements
  const CUtensorMapDataType type = es == 1             ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : dtype == LSC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapSwizzle swizzle = col == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
                                     : col == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                 : CU_TENSOR_MAP_SWIZZLE_128B;
  const cuuint64_t dims[5] = {(cuuint64_t)(col / es), (cuuint64_t)block_tokens, (cuuint64_t)(row / col),
                              (cuuint64_t)heads, 2 * (cuuint64_t)blocks};
  const cuuint64_t strides[4] = {(cuuint64_t)heads * row, (cuuint64_t)col, (cuuint64_t)row, (cuuint64_t)page};
  const cuuint32_t boxes[5] = {(cuuint32_t)(col / es), (cuuint32_t)box, box == tile ? (cuuint32_t)(row / col) : 1, 1, 1};
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return encode(map, type, 5, region, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_maps(const lsc_kv_pool *p, EncodeTiled encode, int tile, int box, std::vector<CUtensorMap> *out) {
  const lsc_kv_pool_desc &d = p->d;
  try {
    out->resize(d.num_layers);
  } catch (...) {
    return false;
  }
  for (int32_t l = 0; l < d.num_layers; ++l)
    if (!encode_map(encode, &(*out)[l], p->base + (int64_t)l * p->region_bytes, d.dtype, (int)p->bits, d.block_tokens,
                    d.num_kv_heads, d.head_dim, d.page_bytes, d.num_blocks, tile, box))
      return false;
  return true;
}

// Positions of a chunk kernel's tile.
int chunk_tile(int head_dim) { return head_dim == 256 ? 64 : 128; }

void make_maps(lsc_kv_pool *p) {
  const lsc_kv_pool_desc &d = p->d;
  const int D = d.head_dim, most = d.block_tokens & -d.block_tokens;
  if (d.dtype == LSC_F32 || (D != 64 && D != 128 && D != 256)) return;
  void *fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess || !fn) {
    cudaGetLastError();
    return;
  }
  p->encode = (EncodeTiled)fn;
  if (most < 8) return;  // a swizzle pattern is 8 rows
  const int tile = chunk_tile(D), keys = lsc::kv_decode_keys(D, (int)p->bits);
  const int box = std::min(most, tile), box_decode = std::min(most, keys);
  std::vector<CUtensorMap> maps, decode;
  if ((d.dtype != LSC_E2M1 && !encode_maps(p, p->encode, tile, box, &maps)) ||  // E2M1: decode alone takes boxes
      !encode_maps(p, p->encode, keys, box_decode, &decode))
    return;
  p->maps.swap(maps);
  p->maps_decode.swap(decode);
  p->box_rows = p->maps.empty() ? 0 : box;
  p->box_decode = box_decode;
}

// Allocations by a thread that is capturing a stream: allowed while this lives (they touch no stream).
struct WhileCapturing {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  WhileCapturing() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~WhileCapturing() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

// The status word, cleared on a stream of its own: the default stream may be waiting for one that is being captured.
int32_t *make_status() {
  int32_t *word = nullptr;
  if (cudaMalloc(&word, 256) != cudaSuccess) return nullptr;
  cudaStream_t s;
  bool ok = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking) == cudaSuccess;
  if (ok) {
    ok = cudaMemsetAsync(word, 0, 256, s) == cudaSuccess && cudaStreamSynchronize(s) == cudaSuccess;
    cudaStreamDestroy(s);
  }
  if (ok) return word;
  cudaFree(word);
  return nullptr;
}

int check_device(const lsc_kv_pool *p) {
  if (p->device < 0) return LSC_ERR_CUDA;  // host-only pool
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return LSC_ERR_CUDA;
  }
  return dev == p->device ? LSC_OK : LSC_ERR_WRONG_DEVICE;
}

lsc::KvLayer layer_of(const lsc_kv_pool *p, int32_t layer) {
  lsc::KvLayer L{};
  L.k = p->base + (int64_t)layer * p->region_bytes;
  L.v = L.k + p->lane_bytes;
  L.page = p->d.page_bytes;
  L.num_blocks = p->d.num_blocks;
  L.block_tokens = p->d.block_tokens;
  L.heads = p->d.num_kv_heads;
  L.head_dim = p->d.head_dim;
  L.dtype = p->d.dtype;
  L.scale_off = p->scale_off;
  L.status = p->status;
  L.by_block.set((uint32_t)p->d.block_tokens);
  return L;
}

bool misaligned(const void *q, uintptr_t a) { return ((uintptr_t)q % a) != 0; }

// The checks every step call shares; out receives the batch.
int check_batch(const lsc_kv_pool *p, const lsc_kv_batch &b, lsc::KvBatch *out) {
  if (b.n_seq < 0 || b.total_tokens < 0 || b.max_blocks < 0 || b.reserved != 0) return LSC_ERR_INVALID_ARG;
  if (b.n_seq > 0 && (!b.cu_seqlens || !b.kv_lens || (b.max_blocks > 0 && !b.block_table))) return LSC_ERR_INVALID_ARG;
  if (misaligned(b.cu_seqlens, 4) || misaligned(b.kv_lens, 4) || misaligned(b.block_table, 4))
    return LSC_ERR_MISALIGNED;
  // the kernels step past the last position by up to a few tiles, in 32 bits
  const int64_t held = std::min<int64_t>((int64_t)b.max_blocks * p->d.block_tokens, LSC_KV_MAX_TOKENS);
  *out = {b.n_seq, b.total_tokens, b.max_blocks, (int32_t)held, b.block_table, b.cu_seqlens, b.kv_lens};
  return LSC_OK;
}

// The dense side of append and gather.
int check_rows(const lsc_kv_pool *p, int32_t layer, const lsc_kv_batch &b, const void *k, const void *v, int32_t dtype,
               int32_t reserved, int64_t k_stride, int64_t v_stride, lsc::KvRowsParams *r) {
  if (layer < 0 || layer >= p->d.num_layers) return LSC_ERR_OUT_OF_RANGE;
  const int rc = check_batch(p, b, &r->b);
  if (rc != LSC_OK) return rc;
  if (reserved != 0 || (dtype != LSC_F32 && dtype != LSC_BF16 && dtype != LSC_F16)) return LSC_ERR_INVALID_ARG;
  const int64_t row = (int64_t)p->d.num_kv_heads * p->d.head_dim;
  if ((k_stride != 0 && k_stride < row) || (v_stride != 0 && v_stride < row)) return LSC_ERR_INVALID_ARG;
  if (b.n_seq > 0 && b.total_tokens > 0 && (!k || !v)) return LSC_ERR_INVALID_ARG;
  if (misaligned(k, esize(dtype)) || misaligned(v, esize(dtype))) return LSC_ERR_MISALIGNED;
  r->L = layer_of(p, layer);
  r->k = const_cast<void *>(k);
  r->v = const_cast<void *>(v);
  r->k_stride = k_stride ? k_stride : row;
  r->v_stride = v_stride ? v_stride : row;
  r->dtype = dtype;
  r->by_heads.set((uint32_t)p->d.num_kv_heads);
  return check_device(p);
}

// 2^64 times the fraction of a turn in an angle of f radians, cut to whole numbers (off by 2 at most): f / (2 pi) as a sum of two doubles (the product
// with 1 / (2 pi), itself two doubles, and what its rounding left).
uint64_t turns_of(double f) {
  constexpr double kInv2Pi = 0x1.45f306dc9c883p-3, kInv2PiLow = -0x1.6b01ec5417056p-57;
  if (f < 0) return 0 - turns_of(-f);
  const double hi = f * kInv2Pi, lo = std::fma(f, kInv2Pi, -hi) + f * kInv2PiLow;  // |lo| < 2^-38: see kMostFreq
  return (uint64_t)((hi - std::floor(hi)) * 0x1p64) + (uint64_t)(int64_t)(lo * 0x1p64);
}
constexpr double kMostFreq = 65536.0;

// head_dim, and whether any rows are to be turned; out receives the launch parameters.
int check_rotary(const lsc_rotary &a, int32_t head_dim, int32_t total_tokens, bool any, lsc::KvRotaryParams *r) {
  const int32_t half = a.rotary_dim / 2;
  if (a.rotary_dim <= 0 || a.rotary_dim % 2 != 0 || a.rotary_dim > head_dim || half > lsc::kRotaryPairs)
    return LSC_ERR_INVALID_ARG;
  if (a.axes <= 0 || a.axes > LSC_ROTARY_MAX_AXES || (a.interleaved != 0 && a.interleaved != 1) ||
      !std::isfinite(a.scale) || !a.inv_freq || (a.axis_stride != 0 && a.axis_stride < total_tokens) ||
      (any && !a.positions))
    return LSC_ERR_INVALID_ARG;
  if ((uintptr_t)a.positions % 4 != 0) return LSC_ERR_MISALIGNED;
  for (int32_t i = 0; i < half; ++i) {
    if (!(std::fabs(a.inv_freq[i]) <= kMostFreq) || (a.pair_axis && a.pair_axis[i] >= a.axes)) return LSC_ERR_INVALID_ARG;
    r->r.turns[i] = turns_of(a.inv_freq[i]);
    r->r.axis[i] = a.pair_axis ? a.pair_axis[i] : 0;
  }
  r->r.positions = a.positions;
  r->r.axis_stride = a.axis_stride ? a.axis_stride : total_tokens;
  r->r.scale = a.scale;
  r->r.half = half;
  r->r.interleaved = a.interleaved;
  r->by_half.set((uint32_t)half);
  return LSC_OK;
}

// Rows of a token that one call of the rotary kernel takes at most.
constexpr int64_t kRotaryHeads = 1 << 24;

// The dense rows that are turned dense to dense.
int check_turned(const void *x, const void *out, int32_t heads, int32_t head_dim, int32_t dtype, int64_t x_stride,
                 int64_t out_stride, bool any, lsc::KvRotaryParams *r) {
  const int64_t row = (int64_t)heads * head_dim;
  if ((x_stride != 0 && x_stride < row) || (out_stride != 0 && out_stride < row)) return LSC_ERR_INVALID_ARG;
  r->x_stride = x_stride ? x_stride : row;
  r->out_stride = out_stride ? out_stride : row;
  if (any && (!x || !out)) return LSC_ERR_INVALID_ARG;
  if (x == out && r->x_stride != r->out_stride) return LSC_ERR_INVALID_ARG;
  if (misaligned(x, esize(dtype)) || misaligned(out, esize(dtype))) return LSC_ERR_MISALIGNED;
  r->x = x;
  r->out = const_cast<void *>(out);
  r->heads = heads;
  r->head_dim = head_dim;
  r->dtype = dtype;
  return LSC_OK;
}

// attend's arguments; out receives the launch parameters without the workspace.
int check_attend(const lsc_kv_pool *p, int32_t layer, const lsc_kv_attend_args *a, lsc::KvAttendParams *r) {
  if (!p || !a) return LSC_ERR_INVALID_ARG;
  if (layer < 0 || layer >= p->d.num_layers) return LSC_ERR_OUT_OF_RANGE;
  const int rc = check_batch(p, a->batch, &r->b);
  if (rc != LSC_OK) return rc;
  const int32_t H = p->d.num_kv_heads, D = p->d.head_dim;
  if (a->num_q_heads <= 0 || a->num_q_heads % H != 0) return LSC_ERR_INVALID_ARG;
  if (a->dtype != LSC_F32 && a->dtype != LSC_BF16 && a->dtype != LSC_F16) return LSC_ERR_INVALID_ARG;
  if (!(a->scale > 0.f) || std::isinf(a->scale * 1.44269504088896341f) || (a->causal != 0 && a->causal != 1)) return LSC_ERR_INVALID_ARG;
  if (a->max_seq_tokens < 0 || a->max_kv_tokens < 0) return LSC_ERR_INVALID_ARG;
  const int64_t row = (int64_t)a->num_q_heads * D;
  if ((a->q_stride != 0 && a->q_stride < row) || (a->out_stride != 0 && a->out_stride < row)) return LSC_ERR_INVALID_ARG;
  if (a->batch.n_seq > 0 && a->batch.total_tokens > 0 && (!a->q || !a->out)) return LSC_ERR_INVALID_ARG;
  if (D > 512) return LSC_ERR_UNSUPPORTED;
  if (misaligned(a->q, esize(a->dtype)) || misaligned(a->out, esize(a->dtype)) || misaligned(a->lse, 4) ||
      misaligned(a->workspace, 16))
    return LSC_ERR_MISALIGNED;
  r->L = layer_of(p, layer);
  r->q = a->q;
  r->out = a->out;
  r->lse = a->lse;
  r->q_stride = a->q_stride ? a->q_stride : row;
  r->out_stride = a->out_stride ? a->out_stride : row;
  r->dtype = a->dtype;
  r->heads = a->num_q_heads;
  r->group = a->num_q_heads / H;
  r->causal = a->causal;
  r->scale_log2 = a->scale * 1.44269504088896341f;
  r->max_seq = a->max_seq_tokens ? std::min(a->max_seq_tokens, a->batch.total_tokens) : a->batch.total_tokens;
  r->max_kv = a->max_kv_tokens ? std::min(a->max_kv_tokens, r->b.held) : r->b.held;
  r->by_group.set((uint32_t)r->group);
  r->num_sms = p->num_sms;
  r->map = p->maps.empty() ? nullptr : &p->maps[layer];
  r->box_rows = p->box_rows;
  r->map_decode = p->maps_decode.empty() ? nullptr : &p->maps_decode[layer];
  r->box_decode = p->box_decode;
  r->wait_limit_ns = fault("timeout0") ? 0 : kWaitLimitNs;
  r->drain_limit_ns = kWaitLimitNs;
  return LSC_OK;
}

// Which kernel a call takes, by sizes, types and alignment: the decode kernel when
// every sequence has kDecodeMost packed rows at most and the blocks have TMA maps,
// else the few-row kernel up to kDecodeMost (E4M3 pools: kRowsMost), the chunk
// kernel when a sequence may have more, the CUDA cores for what none of them
// takes.  64 sequences of 8 tokens behind 64 to 16384, 64 packed rows: bf16, few-row
// kernel 398 us, chunk kernel 193; of 3 tokens, 24 rows: 382 and 189; one sequence
// of 4 behind 1000: 23 and 25.  bf16, 128 sequences of 8 tokens behind 500 to 8000, 8
// heads, 32 rows: head_dim 64, 829 and 386, head_dim 128, 1068 and 436; 4 such
// sequences of 5: 46 and 34, 56 and 38; one of 8 behind 1000: 22 and 24, 23 and 27.
// E4M3, 128 sequences of 8 tokens, head_dim 128: 1115 and 1131.  E2M1 pools have no
// few-row kernel: the chunk kernel takes what the decode kernel does not.
constexpr int32_t kDecodeMost = 16, kRowsMost = 64;
constexpr int64_t kMostCounts = 1 << 30;
enum Form { kAny, kDecode, kRows, kChunk };

bool tensor_core_types(const lsc::KvAttendParams &r) {
  const int D = r.L.head_dim;
  return r.dtype != LSC_F32 && (r.L.dtype == r.dtype || r.L.dtype == LSC_E4M3 || r.L.dtype == LSC_E2M1) && (D == 64 || D == 128 || D == 256);
}

Form attend_form(const lsc::KvAttendParams &r, lsc::AttendPlan *plan) {
  *plan = lsc::AttendPlan{};
  const uintptr_t mis = (uintptr_t)r.q | (uintptr_t)r.out | (uintptr_t)(r.q_stride * 2) | (uintptr_t)(r.out_stride * 2);
  const bool q8 = r.L.dtype == LSC_E4M3;
  if (!tensor_core_types(r) || (mis & 15) != 0) return kAny;
  // the tensor-core kernels count packed rows and the units' tiles in 31 bits
  const int64_t rows = (int64_t)r.max_seq * r.group;
  if (rows > INT32_MAX - 1024) return kAny;
  Form form = kChunk;
  int64_t blocks = r.b.n_seq;  // row blocks of all sequences at most; the two forms for few rows have one a sequence
  if (rows <= kDecodeMost && r.box_decode > 0) {
    form = kDecode;
    *plan = lsc::plan_kv_attend_decode(r);
  } else if (rows <= (q8 ? kRowsMost : kDecodeMost) && r.L.dtype != LSC_E2M1) {  // E2M1: the chunk kernel copies any blocks
    form = kRows;
    *plan = lsc::plan_kv_attend_rows(r);
  } else {
    if (q8 && r.dtype != LSC_BF16) return kAny;  // q is two e4m3 rows there, too few bits for f16
    *plan = lsc::plan_kv_attend_chunk(r);
    blocks += (int64_t)r.b.total_tokens * r.group / plan->M;
  }
  // a run ends one run's length behind the last count at most
  if (blocks * r.L.heads <= kMostCounts / (r.max_kv / plan->TK + 1 + plan->lead)) return form;
  *plan = lsc::AttendPlan{};
  return kAny;
}

// E2M1 chunks of many row blocks: the batch's rows are first made f16 in the workspace (lsc_kv_rows4.cu) and the f16
// chunk kernels take them, to the bits of the E2M1 chunk kernel.  The host knows the sequences' row blocks on average and
// the workspace by the bounds of the lengths; beyond kExpandMost bytes of it, and below expand_blocks blocks, the E2M1
// chunk kernel converts each tile it meets.  16 sequences behind 4000 to 8000, 2, 4 and 6 blocks each, expanded and
// converted by tile: 8 heads of 128: 301 and 277, 468 and 515, 589 and 758 us; 2 heads of 256: 125 and 82, 175 and 143, 184
// and 202 us.  (Batches whose sequences differ are judged by their average all the same: 4096 tokens behind 28000 take
// 1324 us, and with 16 single tokens beside them, not expanded, 2164.)
int64_t expand_blocks(int head_dim) { return head_dim == 256 ? 6 : 4; }
constexpr int64_t kExpandMost = (int64_t)4 << 30;

int64_t up16(int64_t x) { return (x + 15) / 16 * 16; }

// Bytes for n_seq sequences.
int64_t expand_bytes(const lsc::KvAttendParams &r, int64_t n_seq) {
  const int64_t blocks = n_seq * (((int64_t)r.max_kv + lsc::kExpandTokens - 1) / lsc::kExpandTokens);
  const int64_t row = (int64_t)r.L.heads * r.L.head_dim * 2, most = kExpandMost + 1;
  if (blocks > most / (lsc::kExpandTokens * 2) / row) return most;
  return up16(blocks * 4) + 2 * blocks * lsc::kExpandTokens * row;
}

// Sequences that the step's rows fill with that many row blocks each.
int64_t expand_seqs(const lsc::KvAttendParams &r, int M) {
  return (int64_t)r.b.total_tokens * r.group / (M * expand_blocks(r.L.head_dim));
}

bool expands(const lsc_kv_pool *p, const lsc::KvAttendParams &r, const lsc::AttendPlan &plan) {
  return r.L.dtype == LSC_E2M1 && p->encode && r.max_kv > 0 && r.b.n_seq <= expand_seqs(r, plan.M) &&
         expand_bytes(r, r.b.n_seq) <= kExpandMost;
}

// The step's layer and batch as the f16 chunk kernels see them, over `space`; map receives its TMA map.
bool expand_layer(const lsc_kv_pool *p, uint8_t *space, lsc::KvAttendParams *r, lsc::KvExpand *x, CUtensorMap *map) {
  lsc::KvLayer &L = r->L;
  const int32_t blocks = (r->max_kv + lsc::kExpandTokens - 1) / lsc::kExpandTokens;
  const int64_t all = (int64_t)r->b.n_seq * blocks, page = (int64_t)lsc::kExpandTokens * L.heads * L.head_dim * 2;
  *x = lsc::KvExpand{};
  x->table = (int32_t *)space;
  x->k = (uint16_t *)(space + up16(all * 4));
  x->v = (uint16_t *)((uint8_t *)x->k + all * page);
  x->blocks = blocks;
  const int tile = chunk_tile(L.head_dim);
  if (!encode_map(p->encode, map, x->k, LSC_F16, 16, lsc::kExpandTokens, L.heads, L.head_dim, page, all, tile, tile))
    return false;
  L.k = (uint8_t *)x->k;
  L.v = (uint8_t *)x->v;
  L.page = page;
  L.num_blocks = (int32_t)all;
  L.block_tokens = lsc::kExpandTokens;
  L.dtype = LSC_F16;  // code times scale is exact in it
  L.scale_off = 0;
  L.by_block.set(lsc::kExpandTokens);
  r->b.table = x->table;
  r->b.max_blocks = blocks;
  r->map = map;
  r->box_rows = tile;
  return true;
}

// What every call of these sizes or smaller ones needs: the most over the forms that one of them may take, each at its
// largest sizes.  A form's need grows with every size; for decode with and without heads side by side, which smaller
// sizes may do without.
size_t attend_workspace(const lsc_kv_pool *p, lsc::KvAttendParams r) {
  if (!tensor_core_types(r)) return 0;
  const bool q8 = r.L.dtype == LSC_E4M3, q4 = r.L.dtype == LSC_E2M1;
  const int32_t max_seq = r.max_seq, few = q8 ? kRowsMost : kDecodeMost;
  size_t most = 0;
  auto rows_up_to = [&](int32_t rows) {
    r.max_seq = std::min(max_seq, rows / r.group);
    return r.max_seq > 0;
  };
  if (r.box_decode > 0 && rows_up_to(kDecodeMost))
    most = std::max(lsc::plan_kv_attend_decode(r).ws_bytes, lsc::plan_kv_attend_decode(r, false).ws_bytes);
  if ((q8 || r.box_decode == 0) && !q4 && rows_up_to(few)) most = std::max(most, lsc::plan_kv_attend_rows(r).ws_bytes);
  r.max_seq = max_seq;
  if (((int64_t)max_seq * r.group > few && !(q8 && r.dtype != LSC_BF16)) || (q4 && r.box_decode == 0)) {
    const lsc::AttendPlan plan = lsc::plan_kv_attend_chunk(r);
    most = std::max(most, plan.ws_bytes);
    if (q4 && p->encode && r.max_kv > 0) {  // the rows of fewer sequences, or of shorter ones, may be just within what is allowed
      const int64_t seqs = std::min<int64_t>(r.b.n_seq, expand_seqs(r, plan.M));
      if (seqs > 0) most = up16(most) + std::min(expand_bytes(r, seqs), kExpandMost);
    }
  }
  return most;
}

}  // namespace

extern "C" {

int lsc_kv_pool_required_bytes(const lsc_kv_pool_desc *desc, size_t *total_bytes) {
  if (!total_bytes) return LSC_ERR_INVALID_ARG;
  lsc_kv_pool g;
  const int rc = describe(desc, &g);
  if (rc != LSC_OK) return rc;
  *total_bytes = (size_t)g.d.num_layers * (size_t)g.region_bytes;
  return LSC_OK;
}

int lsc_kv_pool_create(const lsc_kv_pool_desc *desc, void *device_base, size_t base_bytes, lsc_kv_pool **out) {
  if (!out) return LSC_ERR_INVALID_ARG;
  *out = nullptr;
  lsc_kv_pool *p = new (std::nothrow) lsc_kv_pool();
  if (!p) return LSC_ERR_NO_MEMORY;
  int rc = describe(desc, p);
  if (rc != LSC_OK) {
    delete p;
    return rc;
  }
  const size_t need = (size_t)p->d.num_layers * (size_t)p->region_bytes;
  if (device_base) {
    if ((uintptr_t)device_base % 256) {
      delete p;
      return LSC_ERR_MISALIGNED;
    }
    if (base_bytes < need) {
      delete p;
      return LSC_ERR_NO_MEMORY;
    }
  }
  int ndev = 0;
  if (cudaGetDeviceCount(&ndev) != cudaSuccess || ndev == 0) {
    cudaGetLastError();
    if (!device_base) {
      delete p;
      return LSC_ERR_CUDA;
    }
    p->base = (uint8_t *)device_base;  // host-only: views, no copies
    *out = p;
    return LSC_OK;
  }
  if (cudaGetDevice(&p->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&p->num_sms, cudaDevAttrMultiProcessorCount, p->device) != cudaSuccess) {
    cudaGetLastError();
    delete p;
    return LSC_ERR_CUDA;
  }
  const WhileCapturing allowed;
  p->status = make_status();
  if (!p->status) {
    cudaGetLastError();
    delete p;
    return LSC_ERR_NO_MEMORY;
  }
  if (device_base) {
    p->base = (uint8_t *)device_base;
  } else {
    if (cudaMalloc(&p->base, need) != cudaSuccess) {
      cudaGetLastError();
      cudaFree(p->status);
      delete p;
      return LSC_ERR_NO_MEMORY;
    }
    p->owns_base = true;
  }
  make_maps(p);
  *out = p;
  return LSC_OK;
}

int lsc_kv_pool_destroy(lsc_kv_pool *p) {
  if (!p) return LSC_ERR_INVALID_ARG;
  int rc = LSC_OK;
  if (p->device >= 0) {
    if (p->owns_base && cudaDeviceSynchronize() != cudaSuccess) rc = LSC_ERR_CUDA;
    const WhileCapturing allowed;
    if (p->owns_base) cudaFree(p->base);
    if (cudaFree(p->status) != cudaSuccess) {  // waits for the work that may still write it
      cudaGetLastError();
      rc = LSC_ERR_CUDA;
    }
  }
  delete p;
  return rc;
}

int lsc_kv_pool_layer_view(const lsc_kv_pool *p, int32_t layer, lsc_kv_layer_view *v) {
  if (!p || !v) return LSC_ERR_INVALID_ARG;
  if (layer < 0 || layer >= p->d.num_layers) return LSC_ERR_OUT_OF_RANGE;
  std::memset(v, 0, sizeof(*v));
  uint8_t *region = p->base + (int64_t)layer * p->region_bytes;
  v->region = region;
  v->region_bytes = p->region_bytes;
  v->k = region;
  v->v = region + p->lane_bytes;
  v->shape[0] = p->d.num_blocks;
  v->shape[1] = p->d.block_tokens;
  v->shape[2] = p->d.num_kv_heads;
  v->shape[3] = p->d.head_dim;
  v->strides[0] = p->d.page_bytes * 8 / p->bits;
  v->strides[1] = (int64_t)p->d.num_kv_heads * p->d.head_dim;
  v->strides[2] = p->d.head_dim;
  v->strides[3] = 1;
  v->lane_stride = p->lane_bytes * 8 / p->bits;
  v->page_bytes = p->d.page_bytes;
  v->payload_bytes = p->payload;
  v->row_bytes = p->row_bytes;
  v->dtype = p->d.dtype;
  v->scale_offset = p->scale_off;
  return LSC_OK;
}

int lsc_kv_pool_status(lsc_kv_pool *p, void *stream, int32_t *host_status) {
  lsc::TraceRange trace_("lsc_kv_pool_status");
  if (!p || !host_status) return LSC_ERR_INVALID_ARG;
  const int rc = check_device(p);
  if (rc != LSC_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  int32_t word = 0;
  if (cudaMemcpyAsync(&word, p->status, sizeof(int32_t), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemsetAsync(p->status, 0, sizeof(int32_t), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return LSC_ERR_CUDA;
  *host_status = word;
  return LSC_OK;
}

int lsc_copy_prefix(lsc_kv_pool *p, const lsc_kv_copy_op *ops, int32_t n_ops, void *stream, void *done_event,
                    int64_t *bytes_copied) {
  lsc::TraceRange trace_("lsc_copy_prefix");
  if (!p || n_ops < 0 || (n_ops > 0 && !ops)) return LSC_ERR_INVALID_ARG;
  const int32_t B = p->d.num_blocks;
  // validate every copying op before enqueueing anything
  std::vector<int32_t> dst_owner;
  try {
    dst_owner.assign(B, -1);
  } catch (...) {
    return LSC_ERR_NO_MEMORY;
  }
  int64_t bytes = 0;
  int32_t n_copy = 0, last_copy = -1;
  for (int32_t r = 0; r < n_ops; ++r) {
    const lsc_kv_copy_op &o = ops[r];
    if (o.reserved != 0 || o.n_tokens < 0 || o.n_tokens > p->d.block_tokens) return LSC_ERR_INVALID_ARG;
    if (o.n_tokens == 0) continue;
    if (o.src_block < 0 || o.src_block >= B || o.dst_block < 0 || o.dst_block >= B) return LSC_ERR_OUT_OF_RANGE;
    if (dst_owner[o.dst_block] >= 0) return LSC_ERR_DUP_DST;
    dst_owner[o.dst_block] = r;
    bytes += (int64_t)o.n_tokens * (p->row_bytes + p->scale_row) * 2 * p->d.num_layers;
    ++n_copy;
    last_copy = r;
  }
  for (int32_t r = 0; r < n_ops; ++r)
    if (ops[r].n_tokens > 0 && dst_owner[ops[r].src_block] >= 0) return LSC_ERR_SRC_IS_DST;
  const int rc = check_device(p);
  if (rc != LSC_OK) return rc;
  cudaStream_t s = (cudaStream_t)stream;
  if (n_copy > 0) {
    static thread_local lsc::KvPlan plan;  // 30 KB: kept off the stack
    plan.base = p->base;
    plan.region_bytes = p->region_bytes;
    plan.lane_bytes = p->lane_bytes;
    plan.page = p->d.page_bytes;
    plan.row_bytes = p->row_bytes;
    plan.chunk_bytes = 32 << 10;
    plan.num_layers = p->d.num_layers;
    plan.chunks_per_op = (int32_t)((p->row_bytes * p->d.block_tokens + plan.chunk_bytes - 1) / plan.chunk_bytes);
    plan.scale_off = p->scale_off;
    plan.scale_row = p->scale_row;
    plan.n_ops = 0;
    for (int32_t r = 0; r < n_ops; ++r) {
      if (ops[r].n_tokens == 0) continue;
      plan.op[plan.n_ops++] = make_int3(ops[r].src_block, ops[r].dst_block, ops[r].n_tokens);
      if (plan.n_ops == lsc::kKvPlanMaxOps || r == last_copy) {
        if (lsc::launch_kv_copy(plan, p->num_sms, s) != cudaSuccess) {
          cudaGetLastError();
          return LSC_ERR_CUDA;
        }
        plan.n_ops = 0;
      }
    }
  }
  if (done_event && cudaEventRecord((cudaEvent_t)done_event, s) != cudaSuccess) {
    cudaGetLastError();
    return LSC_ERR_CUDA;
  }
  if (bytes_copied) *bytes_copied = bytes;
  return LSC_OK;
}

int lsc_kv_append(lsc_kv_pool *p, int32_t layer, const lsc_kv_append_args *a, void *stream) {
  lsc::TraceRange trace_("lsc_kv_append");
  if (!p || !a) return LSC_ERR_INVALID_ARG;
  lsc::KvRowsParams r{};
  const int rc = check_rows(p, layer, a->batch, a->k, a->v, a->dtype, a->reserved, a->k_stride, a->v_stride, &r);
  if (rc != LSC_OK) return rc;
  if (r.b.n_seq == 0 || r.b.total_tokens == 0) return LSC_OK;
  if (lsc::launch_kv_append(r, p->num_sms, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return LSC_ERR_CUDA;
  }
  return LSC_OK;
}

int lsc_kv_append_rotated(lsc_kv_pool *p, int32_t layer, const lsc_kv_append_rotated_args *a, void *stream) {
  lsc::TraceRange trace_("lsc_kv_append_rotated");
  if (!p || !a) return LSC_ERR_INVALID_ARG;
  const lsc_kv_append_args &k = a->append;
  lsc::KvRowsParams rows{};
  lsc::KvRotaryParams r{};
  int rc = check_rows(p, layer, k.batch, k.k, k.v, k.dtype, k.reserved, k.k_stride, k.v_stride, &rows);
  if (rc != LSC_OK && rc != LSC_ERR_CUDA && rc != LSC_ERR_WRONG_DEVICE) return rc;
  const int device_rc = rc;  // after the arguments
  const bool any = k.batch.n_seq > 0 && k.batch.total_tokens > 0;
  if (a->num_q_heads < 0 || a->reserved != 0) return LSC_ERR_INVALID_ARG;
  rc = check_turned(a->q, a->q_out, a->num_q_heads, p->d.head_dim, k.dtype, a->q_stride, a->q_out_stride,
                    any && a->num_q_heads > 0, &r);
  if (rc == LSC_OK) rc = check_rotary(a->rotary, p->d.head_dim, k.batch.total_tokens, any, &r);
  if (rc != LSC_OK) return rc;
  if ((int64_t)a->num_q_heads + 2 * (int64_t)p->d.num_kv_heads > kRotaryHeads) return LSC_ERR_UNSUPPORTED;
  if (device_rc != LSC_OK) return device_rc;
  if (!any) return LSC_OK;
  r.L = rows.L;
  r.b = rows.b;
  r.k = rows.k;
  r.v = rows.v;
  r.k_stride = rows.k_stride;
  r.v_stride = rows.v_stride;
  if (lsc::launch_kv_rotary(r, p->num_sms, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return LSC_ERR_CUDA;
  }
  return LSC_OK;
}

int lsc_rotate(const lsc_rotate_args *a, void *stream) {
  lsc::TraceRange trace_("lsc_rotate");
  if (!a || a->total_tokens < 0 || a->num_heads <= 0 || a->head_dim <= 0) return LSC_ERR_INVALID_ARG;
  if (a->dtype != LSC_F32 && a->dtype != LSC_BF16 && a->dtype != LSC_F16) return LSC_ERR_INVALID_ARG;
  lsc::KvRotaryParams r{};
  const bool any = a->total_tokens > 0;
  int rc = check_turned(a->x, a->out, a->num_heads, a->head_dim, a->dtype, a->x_stride, a->out_stride, any, &r);
  if (rc == LSC_OK) rc = check_rotary(a->rotary, a->head_dim, a->total_tokens, any, &r);
  if (rc != LSC_OK) return rc;
  if (a->num_heads > kRotaryHeads) return LSC_ERR_UNSUPPORTED;
  int device = -1, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
    cudaGetLastError();
    return LSC_ERR_CUDA;
  }
  if (!any) return LSC_OK;
  r.b.total_tokens = a->total_tokens;
  if (lsc::launch_kv_rotary(r, sms, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return LSC_ERR_CUDA;
  }
  return LSC_OK;
}

int lsc_kv_gather(lsc_kv_pool *p, int32_t layer, const lsc_kv_gather_args *a, void *stream) {
  lsc::TraceRange trace_("lsc_kv_gather");
  if (!p || !a) return LSC_ERR_INVALID_ARG;
  lsc::KvRowsParams r{};
  const int rc = check_rows(p, layer, a->batch, a->k, a->v, a->dtype, a->reserved, a->k_stride, a->v_stride, &r);
  if (rc != LSC_OK) return rc;
  if (r.b.n_seq == 0 || r.b.total_tokens == 0) return LSC_OK;
  if (lsc::launch_kv_gather(r, p->num_sms, (cudaStream_t)stream) != cudaSuccess) {
    cudaGetLastError();
    return LSC_ERR_CUDA;
  }
  return LSC_OK;
}

int lsc_kv_attend_workspace_bytes(const lsc_kv_pool *p, const lsc_kv_attend_args *a, size_t *bytes) {
  if (!bytes) return LSC_ERR_INVALID_ARG;
  lsc::KvAttendParams r{};
  const int rc = check_attend(p, 0, a, &r);
  if (rc != LSC_OK) return rc;
  if (p->device < 0) return LSC_ERR_CUDA;  // host-only pool: the need depends on the device
  *bytes = r.b.n_seq == 0 || r.b.total_tokens == 0 ? 0 : attend_workspace(p, r);
  return LSC_OK;
}

int lsc_kv_attend(lsc_kv_pool *p, int32_t layer, const lsc_kv_attend_args *a, void *stream) {
  lsc::TraceRange trace_("lsc_kv_attend");
  lsc::KvAttendParams r{};
  int rc = check_attend(p, layer, a, &r);
  if (rc != LSC_OK) return rc;
  rc = check_device(p);
  if (rc != LSC_OK) return rc;
  if (r.b.n_seq == 0 || r.b.total_tokens == 0) return LSC_OK;
  lsc::AttendPlan plan;
  const Form form = attend_form(r, &plan);
  cudaStream_t s = (cudaStream_t)stream;
  void *ws = a->workspace;
  bool expand = form == kChunk && expands(p, r, plan);
  const size_t parts = expand ? up16(plan.ws_bytes) : plan.ws_bytes;
  size_t need = parts + (expand ? expand_bytes(r, r.b.n_seq) : 0);
  if (ws && need > 0 && a->workspace_bytes < attend_workspace(p, r)) return LSC_ERR_INVALID_ARG;
  if (!ws && expand && (fault("no_rows") || cudaMallocAsync(&ws, need, s) != cudaSuccess)) {  // by tile, then: the same bits
    cudaGetLastError();
    ws = nullptr;
    expand = false;
    need = plan.ws_bytes;
  }
  if (!ws && need > 0 && cudaMallocAsync(&ws, need, s) != cudaSuccess) {
    cudaGetLastError();
    return LSC_ERR_NO_MEMORY;
  }
  if (plan.ws_bytes > 0) r.ws = (uint8_t *)ws;
  r.whole = !plan.may_cut;
  r.min_run = plan.min_run;
  r.lead = plan.lead;
  r.groups = r.L.heads / std::max(plan.together, 1);
  cudaError_t e = cudaSuccess;
  CUtensorMap map;
  if (expand) {
    const lsc::KvAttendParams held = r;
    lsc::KvExpand x;
    e = expand_layer(p, (uint8_t *)ws + parts, &r, &x, &map) ? lsc::launch_kv_expand(held, x, s) : cudaErrorUnknown;
  }
  if (e == cudaSuccess)
    e = form == kAny      ? lsc::launch_kv_attend_any(r, s)
        : form == kDecode ? lsc::launch_kv_attend_decode(r, plan, s)
        : form == kRows   ? lsc::launch_kv_attend_rows(r, plan, s)
                          : lsc::launch_kv_attend_chunk(r, plan, s);
  if (e == cudaSuccess && plan.may_cut) e = lsc::launch_kv_attend_join(r, plan, s);
  if (need > 0 && !a->workspace && cudaFreeAsync(ws, s) != cudaSuccess && e == cudaSuccess) e = cudaErrorUnknown;
  if (e != cudaSuccess) {
    cudaGetLastError();
    return LSC_ERR_CUDA;
  }
  return LSC_OK;
}

}  // extern "C"
