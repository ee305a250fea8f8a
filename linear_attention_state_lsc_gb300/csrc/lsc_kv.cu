// lsc_kv.cu -- host side of the attention K/V block pool (include/lsc_kv.h):
// layout, views, copy_prefix's validation and launch plans, and the argument
// checks of append, gather and attend.  The copy kernel is kv_copy_kernel in
// lsc_copy.cu; append and gather are in lsc_kv_rows.cu.
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

struct lsc_kv_pool {
  lsc_kv_pool_desc d;
  int device = -1;  // -1: host-only pool (no GPU when created)
  int num_sms = 0;
  uint8_t *base = nullptr;
  bool owns_base = false;
  int64_t es = 0, row_bytes = 0, payload = 0, lane_bytes = 0, region_bytes = 0;
  int32_t scale_off = 0;        // E4M3: page offset of the scale bytes
  int32_t *status = nullptr;    // device error word
  int32_t box_rows = 0;         // rows of a TMA box of `maps`
  int32_t box_decode = 0;       // and of `maps_decode`
  std::vector<CUtensorMap> maps, maps_decode;  // per layer; empty: none
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
  const int es = esize(d->dtype);
  if (!es) return LSC_ERR_INVALID_ARG;
  g->d = *d;
  g->es = es;
  g->row_bytes = (int64_t)d->num_kv_heads * d->head_dim * es;
  g->payload = g->row_bytes * d->block_tokens;
  if (d->dtype == LSC_E4M3) {  // codes, then one scale byte per (row, head) at the next 16 B boundary
    const int64_t off = (g->payload + 15) / 16 * 16;
    if (off > INT32_MAX) return LSC_ERR_LAYOUT;
    g->scale_off = (int32_t)off;
    g->payload = off + (int64_t)d->block_tokens * d->num_kv_heads;
  }
  if (d->page_bytes < g->payload || d->page_bytes % es) return LSC_ERR_LAYOUT;
  if (d->page_bytes % 16) return LSC_ERR_MISALIGNED;
  g->lane_bytes = (int64_t)d->num_blocks * d->page_bytes;
  g->region_bytes = 2 * g->lane_bytes;
  return LSC_OK;
}

// TMA maps of the layers' rows, for attend: coordinates (element of a column, row
// of a block, column of 128 bytes, kv head, block; V's blocks follow K's), a box
// of one column, or of all when it has a whole tile's rows.  A box never leaves its
// block: its rows are the largest power of two that divides block_tokens, up to
// the tile's.  128-byte swizzle (64 bytes a row: 64-byte).  Without maps (blocks that are
// no multiple of 8 tokens, other types and sizes) the kernels copy rows themselves.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool encode_maps(const lsc_kv_pool *p, EncodeTiled encode, int tile, int box, std::vector<CUtensorMap> *out) {
  const lsc_kv_pool_desc &d = p->d;
  const int row = d.head_dim * (int)p->es, col = row < 128 ? row : 128;  // bytes
  const CUtensorMapDataType type = d.dtype == LSC_E4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : d.dtype == LSC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapSwizzle swizzle = col == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  const cuuint64_t dims[5] = {(cuuint64_t)(col / p->es), (cuuint64_t)d.block_tokens, (cuuint64_t)(row / col),
                              (cuuint64_t)d.num_kv_heads, 2 * (cuuint64_t)d.num_blocks};
  const cuuint64_t strides[4] = {(cuuint64_t)p->row_bytes, (cuuint64_t)col, (cuuint64_t)row, (cuuint64_t)d.page_bytes};
  const cuuint32_t boxes[5] = {(cuuint32_t)(col / p->es), (cuuint32_t)box, box == tile ? (cuuint32_t)(row / col) : 1, 1, 1};
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  try {
    out->resize(d.num_layers);
  } catch (...) {
    return false;
  }
  for (int32_t l = 0; l < d.num_layers; ++l)
    if (encode(&(*out)[l], type, 5, p->base + (int64_t)l * p->region_bytes, dims, strides, boxes, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}

void make_maps(lsc_kv_pool *p) {
  const lsc_kv_pool_desc &d = p->d;
  const int D = d.head_dim, most = d.block_tokens & -d.block_tokens;
  if (d.dtype == LSC_F32 || (D != 64 && D != 128 && D != 256) || most < 8) return;  // a swizzle pattern is 8 rows
  void *fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess || !fn) {
    cudaGetLastError();
    return;
  }
  const int tile = D == 256 ? 64 : 128, keys = lsc::kv_decode_keys(D, (int)p->es);
  const int box = std::min(most, tile), box_decode = std::min(most, keys);
  std::vector<CUtensorMap> maps, decode;
  if (!encode_maps(p, (EncodeTiled)fn, tile, box, &maps) ||
      !encode_maps(p, (EncodeTiled)fn, keys, box_decode, &decode))
    return;
  p->maps.swap(maps);
  p->maps_decode.swap(decode);
  p->box_rows = box;
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
// E4M3, 128 sequences of 8 tokens, head_dim 128: 1115 and 1131.
constexpr int32_t kDecodeMost = 16, kRowsMost = 64;
constexpr int64_t kMostCounts = 1 << 30;
enum Form { kAny, kDecode, kRows, kChunk };

bool tensor_core_types(const lsc::KvAttendParams &r) {
  const int D = r.L.head_dim;
  return r.dtype != LSC_F32 && (r.L.dtype == r.dtype || r.L.dtype == LSC_E4M3) && (D == 64 || D == 128 || D == 256);
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
  } else if (rows <= (q8 ? kRowsMost : kDecodeMost)) {
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

// What every call of these sizes or smaller ones needs: the most over the forms that one of them may take, each at its
// largest sizes.  A form's need grows with every size; for decode with and without heads side by side, which smaller
// sizes may do without.
size_t attend_workspace(lsc::KvAttendParams r) {
  if (!tensor_core_types(r)) return 0;
  const bool q8 = r.L.dtype == LSC_E4M3;
  const int32_t max_seq = r.max_seq, few = q8 ? kRowsMost : kDecodeMost;
  size_t most = 0;
  auto rows_up_to = [&](int32_t rows) {
    r.max_seq = std::min(max_seq, rows / r.group);
    return r.max_seq > 0;
  };
  if (r.box_decode > 0 && rows_up_to(kDecodeMost))
    most = std::max(lsc::plan_kv_attend_decode(r).ws_bytes, lsc::plan_kv_attend_decode(r, false).ws_bytes);
  if ((q8 || r.box_decode == 0) && rows_up_to(few)) most = std::max(most, lsc::plan_kv_attend_rows(r).ws_bytes);
  r.max_seq = max_seq;
  if ((int64_t)max_seq * r.group > few && !(q8 && r.dtype != LSC_BF16))
    most = std::max(most, lsc::plan_kv_attend_chunk(r).ws_bytes);
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
  v->strides[0] = p->d.page_bytes / p->es;
  v->strides[1] = (int64_t)p->d.num_kv_heads * p->d.head_dim;
  v->strides[2] = p->d.head_dim;
  v->strides[3] = 1;
  v->lane_stride = p->lane_bytes / p->es;
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
  const int32_t scale_row = p->d.dtype == LSC_E4M3 ? p->d.num_kv_heads : 0;
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
    bytes += (int64_t)o.n_tokens * (p->row_bytes + scale_row) * 2 * p->d.num_layers;
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
    plan.scale_row = scale_row;
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
  *bytes = r.b.n_seq == 0 || r.b.total_tokens == 0 ? 0 : attend_workspace(r);
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
  if (plan.ws_bytes > 0) {
    if (ws && a->workspace_bytes < attend_workspace(r)) return LSC_ERR_INVALID_ARG;
    if (!ws && cudaMallocAsync(&ws, plan.ws_bytes, s) != cudaSuccess) {
      cudaGetLastError();
      return LSC_ERR_NO_MEMORY;
    }
    r.ws = (uint8_t *)ws;
  }
  r.whole = !plan.may_cut;
  r.min_run = plan.min_run;
  r.lead = plan.lead;
  r.groups = r.L.heads / std::max(plan.together, 1);
  cudaError_t e = form == kAny    ? lsc::launch_kv_attend_any(r, s)
                  : form == kDecode ? lsc::launch_kv_attend_decode(r, plan, s)
                  : form == kRows ? lsc::launch_kv_attend_rows(r, plan, s)
                                  : lsc::launch_kv_attend_chunk(r, plan, s);
  if (e == cudaSuccess && plan.may_cut) e = lsc::launch_kv_attend_join(r, plan, s);
  if (plan.ws_bytes > 0 && !a->workspace && cudaFreeAsync(ws, s) != cudaSuccess && e == cudaSuccess) e = cudaErrorUnknown;
  if (e != cudaSuccess) {
    cudaGetLastError();
    return LSC_ERR_CUDA;
  }
  return LSC_OK;
}

}  // extern "C"
