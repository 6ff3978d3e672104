// csa2_api.cu -- the C ABI declared in include/csa2.h: argument checks, the
// cache layout in caller memory, TMA tensor maps, and launch scheduling of
// the kernels in k_append.cu, k_index.cu, k_topk.cu and k_attn.cu.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <initializer_list>
#include <memory>
#include <mutex>
#include <new>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "csa2.h"
#include "csa2_kernels.h"

namespace {
// One NVTX range per C call, named after the call (shows in Nsight
// timelines; without an attached tool the push and pop return at once).
struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};
}  // namespace
#define CSA2_RANGE() NvtxRange csa2_nvtx_range_(__func__)

// Scratch of csa2_index_topk_decode_static, for callers that cannot allocate:
// a fixed array in the library's device image (one per GPU that loads it).
static __device__ __align__(256) uint8_t g_static_scratch[CSA2_STATIC_SCRATCH_BYTES];

using namespace csa2;

struct csa2_cache {
  csa2_config_t cfg;
  int32_t batch;
  int32_t group;       // channels per scale
  int32_t scale_bytes; // per entry
  std::vector<int64_t> cap, off, len;
  int64_t total;
  int64_t max_cap;
  uint8_t* base;
  size_t bytes;
  int32_t* d_len;
  uint32_t* d_err;
  uint8_t* codes;
  uint8_t* scales;
  uint16_t* idxk;       // CSA2_IDX_BF16 keys
  uint8_t* idx_codes;   // CSA2_IDX_MXFP4 keys: codes [idx_rows, 64], scales [idx_rows, 4]
  uint8_t* idx_scales;
  int64_t idx_rows;     // total rounded up to whole 512-key chunks (MXFP4 keys)
  CUtensorMap tm_k;    // indexer keys, 128-row boxes (contiguous tiles)
  CUtensorMap tm_k8;   // indexer keys, one 8-key block per box (pool mode)
  CUtensorMap tm_kq;   // MXFP4 key codes, 128-key tiles in the permuted row order
  CUtensorMap tm_kc8;  // MXFP4 key codes, one 8-key block per box (pool mode)
  int dev;             // device of the cache
  int num_sms;
  int index_sms;       // SMs the indexer's persistent grid may occupy
  int64_t wait_cycles; // bounded-wait limit of the kernels (0: their default)
  int32_t inject;      // fault injection for tests (kInjectNoKeyLoads)
};

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

csa2_status_t check_cfg(const csa2_config_t* c) {
  if (!c) return CSA2_ERR_INVALID_ARG;
  if (c->head_dim != kHeadDim || c->idx_dim != kIdxDim || c->idx_heads != kIdxHeads)
    return CSA2_ERR_UNSUPPORTED;
  if (c->n_heads <= 0 || c->n_heads % kAttnHeadGroup != 0 || c->n_heads > 128)
    return CSA2_ERR_UNSUPPORTED;
  if (c->topk <= 0 || c->topk % 128 != 0 || c->topk > 2048) return CSA2_ERR_UNSUPPORTED;
  if (c->swa < 0 || c->swa > 128) return CSA2_ERR_UNSUPPORTED;
  if (c->ratio < 1 || c->ratio > 16) return CSA2_ERR_UNSUPPORTED;
  if (c->layout != CSA2_KV_L32_UE8M0 && c->layout != CSA2_KV_L16_E4M3) return CSA2_ERR_UNSUPPORTED;
  if (c->idx_layout != CSA2_IDX_BF16 && c->idx_layout != CSA2_IDX_MXFP4) return CSA2_ERR_UNSUPPORTED;
  return CSA2_OK;
}

struct Layout {
  size_t len_off, err_off, codes_off, scales_off, idxk_off, idxs_off, total;
};

static_assert(CSA2_MAX_ATTN_LAYERS == kAttnMaxLayers, "layers of one readout launch");

// Rows of the MXFP4 key arrays: the entries rounded up to 512-key chunks.
int64_t mxfp4_rows(int64_t total) { return (total + 511) / 512 * 512; }

Layout layout_for(const csa2_config_t* c, int64_t total) {
  Layout L;
  const int g = c->layout == CSA2_KV_L16_E4M3 ? 16 : 32;
  L.len_off = 0;
  L.err_off = 0;  // filled below
  L.codes_off = 0;
  size_t o = 0;
  L.len_off = o;
  o = align_up(o + 4096 * sizeof(int32_t), kAlign);  // up to 4096 sequences of lengths
  L.err_off = o;
  o = align_up(o + sizeof(uint32_t), kAlign);
  L.codes_off = o;
  o = align_up(o + (size_t)total * (kHeadDim / 2), kAlign);
  L.scales_off = o;
  o = align_up(o + (size_t)total * (kHeadDim / g), kAlign);
  L.idxk_off = o;
  if (c->idx_layout == CSA2_IDX_MXFP4) {
    // E2M1 codes and UE8M0 scales, each holding whole 512-key chunks (the
    // indexer reads keys in aligned tiles of up to 512 keys; rows past
    // `total` are never valid entries)
    const size_t rows = (size_t)mxfp4_rows(total);
    o = align_up(o + rows * (kIdxDim / 2), kAlign);
    L.idxs_off = o;
    o = align_up(o + rows * (kIdxDim / 32), kAlign);
  } else {
    o = align_up(o + (size_t)total * kIdxDim * 2, kAlign);
    L.idxs_off = 0;
  }
  L.total = o;
  return L;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 2-D bf16 tensor [rows, cols] (row stride cols * 2 bytes), 128B-swizzled
// boxes of [box_rows, box_cols]; out-of-range rows read as zero.
bool make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_cols,
              uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn || rows == 0) return false;
  cuuint64_t gdim[2] = {cols, rows};
  cuuint64_t gstride[1] = {cols * 2};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), gdim, gstride, box,
            es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// MXFP4 key codes as bytes [rows, row_bytes] (64: one key per row, 64-byte
// swizzle; 128: two keys per row, 128-byte swizzle), boxes of box_rows rows:
// the K-major layouts of the block-scaled MMA's operands.
bool make_code_map(CUtensorMap* m, const void* base, uint64_t rows, uint32_t row_bytes,
                   uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn || rows == 0) return false;
  cuuint64_t gdim[2] = {row_bytes, rows};
  cuuint64_t gstride[1] = {row_bytes};
  cuuint32_t box[2] = {row_bytes, box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), gdim, gstride, box,
            es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// MXFP4 key codes in aligned 128-key tiles with their rows permuted: key
// 4 r + q of a tile (r < 32, q < 4) lands in shared-memory row 32 q + r (64-
// byte rows, the 64-byte swizzle).  With the keys in that order, the tile's
// UE8M0 scale words in their natural order are exactly the scale atom of
// the block-scaled MMA (row 32 q + r at byte 16 r + 4 q), so a tile's scales
// are one contiguous copy.  The view is (64 bytes, r, q, tile) with strides
// (1, 256, 64, 8192); rows must be a multiple of 128.  (The box's rows are
// exactly one swizzle span wide: with a wider swizzle than the row, the TMA
// would lay each row out at the swizzle span.)
bool make_perm_map(CUtensorMap* m, const void* base, int64_t rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn || rows <= 0 || rows % 128 != 0) return false;
  cuuint64_t gdim[4] = {64, 32, 4, (cuuint64_t)(rows / 128)};
  cuuint64_t gstride[3] = {256, 64, 8192};
  cuuint32_t box[4] = {64, 32, 4, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), gdim, gstride, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Indexer keys [rows, 128] bf16 seen as (64 columns, rows, 2 halves): one
// box of (64, 8, 2) is a whole block of 8 keys, landing in shared memory as
// two 1 KB 128B-swizzled atoms (columns 0-63, then 64-127).
bool make_block_map(CUtensorMap* m, const void* base, uint64_t rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn || rows == 0) return false;
  cuuint64_t gdim[3] = {64, rows, 2};
  cuuint64_t gstride[2] = {kIdxDim * 2, 128};
  cuuint32_t box[3] = {64, (cuuint32_t)kHsiBlock, 2};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), gdim, gstride, box,
            es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaStream_t S(csa2_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

csa2_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA; }

int64_t score_ld(int64_t n) { return std::max<int64_t>(4, (n + 3) / 4 * 4); }

// The indexer kernel for the cache's key storage: bf16 keys (TMA, kind::f16
// MMAs), or MXFP4 keys (E2M1 codes by TMA, block-scaled kind::mxf4 MMAs,
// queries rounded to MXFP4 on chip from q_idx).  `pool` selects the
// pool-mode tensor map of bf16 keys.
cudaError_t launch_index_any(const csa2_cache* c, IndexParams& ip, const CUtensorMap& tm_q,
                             const void* q_idx, int grid, cudaStream_t s, bool pool = false) {
  if (c->cfg.idx_layout == CSA2_IDX_MXFP4) {
    ip.idx_codes = c->idx_codes;
    ip.idx_scales = c->idx_scales;
    ip.idx_total = c->total;
    ip.q_idx = static_cast<const uint16_t*>(q_idx);
    return launch_index_fp4(ip, c->tm_kq, c->tm_kc8, grid, s);
  }
  return launch_index(ip, pool ? c->tm_k8 : c->tm_k, tm_q, grid, s);
}

// Append / compress segments: rows of one launch grouped by sequence.
csa2_status_t run_append(csa2_cache* c, int mode, int32_t n_seqs, const int32_t* seq_ids,
                         const int32_t* n_rows_in, const float* entries, const void* c_tok,
                         const float* z_tok, const void* idx_k, float* entries_out,
                         csa2_stream_t stream) {
  if (!c || n_seqs < 0 || (n_seqs > 0 && (!seq_ids || !n_rows_in))) return CSA2_ERR_INVALID_ARG;
  const int m = c->cfg.ratio;
  std::vector<int64_t> new_len(c->len);
  int64_t total_rows = 0;
  for (int i = 0; i < n_seqs; ++i) {
    const int32_t s = seq_ids[i];
    const int32_t n = n_rows_in[i];
    if (s < 0 || s >= c->batch || n < 0) return CSA2_ERR_INVALID_ARG;
    if (mode == 2 && n % m != 0) return CSA2_ERR_INVALID_ARG;
    const int64_t ne = mode == 2 ? n / m : n;
    new_len[s] += ne;
    if (new_len[s] > c->cap[s]) return CSA2_ERR_CAPACITY;
    total_rows += ne;
  }
  if (total_rows == 0) return CSA2_OK;
  if (!idx_k || !aligned16(idx_k)) return CSA2_ERR_INVALID_ARG;
  if (mode == 1 && (!entries || !aligned16(entries))) return CSA2_ERR_INVALID_ARG;
  if (mode == 2 && (!c_tok || !z_tok || !aligned16(c_tok) || !aligned16(z_tok)))
    return CSA2_ERR_INVALID_ARG;
  if (entries_out && !aligned16(entries_out)) return CSA2_ERR_INVALID_ARG;

  std::vector<int64_t> cur(c->len);
  int64_t src = 0;
  int i = 0;
  while (i < n_seqs) {
    AppendParams p;
    std::memset(&p, 0, sizeof(p));
    p.mode = mode;
    p.ratio = m;
    p.layout = c->cfg.layout;
    p.dim = kHeadDim;
    p.entries = entries;
    p.c_tok = static_cast<const uint16_t*>(c_tok);
    p.z_tok = z_tok;
    p.idx_k = static_cast<const uint16_t*>(idx_k);
    p.entries_out = entries_out;
    p.codes = c->codes;
    p.scales = c->scales;
    p.cache_idxk = c->idxk;
    p.idx_mxfp4 = c->cfg.idx_layout == CSA2_IDX_MXFP4 ? 1 : 0;
    p.idx_codes = c->idx_codes;
    p.idx_scales = c->idx_scales;
    p.d_len = c->d_len;
    p.total = c->total;
    p.err = c->d_err;
    int64_t rows = 0;
    while (i < n_seqs && p.n_segs < kMaxAppendSegs) {
      const int32_t s = seq_ids[i];
      const int64_t ne = mode == 2 ? n_rows_in[i] / m : n_rows_in[i];
      AppendSeg& g = p.seg[p.n_segs++];
      g.first = rows;
      g.src_row = src;
      g.dst_row = c->off[s] + cur[s];
      g.seq = s;
      cur[s] += ne;
      g.new_len = (int32_t)cur[s];
      rows += ne;
      src += ne;
      ++i;
    }
    p.rows = rows;
    cudaError_t e = launch_append(p, S(stream));
    if (e != cudaSuccess) return CSA2_ERR_CUDA;
  }
  c->len = new_len;
  return CSA2_OK;
}

}  // namespace

extern "C" {

int32_t csa2_version(void) { return 1; }

const char* csa2_status_string(csa2_status_t s) {
  switch (s) {
    case CSA2_OK: return "ok";
    case CSA2_ERR_INVALID_ARG: return "invalid argument";
    case CSA2_ERR_UNSUPPORTED: return "unsupported configuration";
    case CSA2_ERR_CAPACITY: return "capacity exceeded";
    case CSA2_ERR_CUDA: return "CUDA error";
    case CSA2_ERR_OOM: return "out of memory";
    case CSA2_ERR_TIMEOUT: return "device wait timed out";
    case CSA2_ERR_DEVICE: return "device-side check failed";
  }
  return "unknown status";
}

size_t csa2_cache_bytes(const csa2_config_t* cfg, int32_t batch, const int64_t* capacity) {
  if (check_cfg(cfg) != CSA2_OK || batch <= 0 || batch > 4096 || !capacity) return 0;
  int64_t total = 0;
  for (int i = 0; i < batch; ++i) {
    if (capacity[i] < 0 || capacity[i] > (int64_t)INT32_MAX) return 0;
    total += capacity[i];
  }
  if (total <= 0) return 0;
  return layout_for(cfg, total).total;
}

csa2_status_t csa2_cache_create(const csa2_config_t* cfg, int32_t batch, const int64_t* capacity,
                                void* dev_mem, size_t bytes, csa2_stream_t stream,
                                csa2_cache_t** out) {
  CSA2_RANGE();
  if (!out) return CSA2_ERR_INVALID_ARG;
  *out = nullptr;
  csa2_status_t st = check_cfg(cfg);
  if (st != CSA2_OK) return st;
  if (batch <= 0 || batch > 4096 || !capacity || !dev_mem) return CSA2_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(dev_mem) & (kAlign - 1)) != 0) return CSA2_ERR_INVALID_ARG;
  const size_t need = csa2_cache_bytes(cfg, batch, capacity);
  if (need == 0) return CSA2_ERR_INVALID_ARG;
  if (bytes < need) return CSA2_ERR_CAPACITY;

  csa2_cache* c = new (std::nothrow) csa2_cache();
  if (!c) return CSA2_ERR_OOM;
  c->cfg = *cfg;
  c->batch = batch;
  c->group = cfg->layout == CSA2_KV_L16_E4M3 ? 16 : 32;
  c->scale_bytes = kHeadDim / c->group;
  c->cap.assign(capacity, capacity + batch);
  c->off.resize(batch + 1);
  c->len.assign(batch, 0);
  c->off[0] = 0;
  c->max_cap = 0;
  for (int i = 0; i < batch; ++i) {
    c->off[i + 1] = c->off[i] + capacity[i];
    c->max_cap = std::max(c->max_cap, capacity[i]);
  }
  c->total = c->off[batch];
  const Layout L = layout_for(cfg, c->total);
  c->base = static_cast<uint8_t*>(dev_mem);
  c->bytes = bytes;
  c->d_len = reinterpret_cast<int32_t*>(c->base + L.len_off);
  c->d_err = reinterpret_cast<uint32_t*>(c->base + L.err_off);
  c->codes = c->base + L.codes_off;
  c->scales = c->base + L.scales_off;
  const bool mx = cfg->idx_layout == CSA2_IDX_MXFP4;
  c->idxk = mx ? nullptr : reinterpret_cast<uint16_t*>(c->base + L.idxk_off);
  c->idx_codes = mx ? c->base + L.idxk_off : nullptr;
  c->idx_scales = mx ? c->base + L.idxs_off : nullptr;
  c->idx_rows = mx ? mxfp4_rows(c->total) : 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    delete c;
    return CSA2_ERR_CUDA;
  }
  c->dev = dev;
  c->index_sms = c->num_sms;
  c->wait_cycles = 0;
  c->inject = 0;
  if (!mx && (!make_map(&c->tm_k, c->idxk, (uint64_t)c->total, kIdxDim, 64, 128) ||
              !make_block_map(&c->tm_k8, c->idxk, (uint64_t)c->total))) {
    delete c;
    return CSA2_ERR_CUDA;
  }
  if (mx && (!make_perm_map(&c->tm_kq, c->idx_codes, c->idx_rows) ||
             !make_code_map(&c->tm_kc8, c->idx_codes, (uint64_t)c->total, kIdxDim / 2, kHsiBlock))) {
    delete c;
    return CSA2_ERR_CUDA;
  }
  if (cudaMemsetAsync(c->base, 0, L.codes_off, S(stream)) != cudaSuccess) {
    delete c;
    return CSA2_ERR_CUDA;
  }
  *out = c;
  return CSA2_OK;
}

csa2_status_t csa2_cache_destroy(csa2_cache_t* c) {
  CSA2_RANGE();
  if (!c) return CSA2_ERR_INVALID_ARG;
  delete c;
  return CSA2_OK;
}

csa2_status_t csa2_cache_set_index_sms(csa2_cache_t* c, int32_t n_sms) {
  CSA2_RANGE();
  if (!c || n_sms < 0) return CSA2_ERR_INVALID_ARG;
  c->index_sms = (n_sms == 0 || n_sms > c->num_sms) ? c->num_sms : n_sms;
  return CSA2_OK;
}

csa2_status_t csa2_cache_set_wait_limit(csa2_cache_t* c, int64_t cycles) {
  CSA2_RANGE();
  if (!c || cycles < 0) return CSA2_ERR_INVALID_ARG;
  c->wait_cycles = cycles;
  return CSA2_OK;
}

csa2_status_t csa2_cache_inject_fault(csa2_cache_t* c, int32_t fault) {
  CSA2_RANGE();
  if (!c || (fault != CSA2_FAULT_NONE && fault != CSA2_FAULT_INDEX_NO_KEY_LOADS))
    return CSA2_ERR_INVALID_ARG;
  c->inject = fault == CSA2_FAULT_INDEX_NO_KEY_LOADS ? kInjectNoKeyLoads : 0;
  return CSA2_OK;
}

csa2_status_t csa2_cache_reset(csa2_cache_t* c, csa2_stream_t stream) {
  CSA2_RANGE();
  if (!c) return CSA2_ERR_INVALID_ARG;
  std::fill(c->len.begin(), c->len.end(), 0);
  return cuda_status(cudaMemsetAsync(c->d_len, 0, sizeof(int32_t) * c->batch, S(stream)));
}

csa2_status_t csa2_cache_length(const csa2_cache_t* c, int32_t seq, int64_t* n) {
  CSA2_RANGE();
  if (!c || !n || seq < 0 || seq >= c->batch) return CSA2_ERR_INVALID_ARG;
  *n = c->len[seq];
  return CSA2_OK;
}

csa2_status_t csa2_cache_views(const csa2_cache_t* c, csa2_cache_views_t* v) {
  CSA2_RANGE();
  if (!c || !v) return CSA2_ERR_INVALID_ARG;
  v->codes = c->codes;
  v->scales = c->scales;
  v->idx_k = c->idxk;
  v->idx_codes = c->idx_codes;
  v->idx_scales = c->idx_scales;
  v->lengths = c->d_len;
  v->entry_offset = c->off.data();
  v->total = c->total;
  v->batch = c->batch;
  v->group = c->group;
  return CSA2_OK;
}

csa2_status_t csa2_compress(int32_t ratio, int64_t n_out, int32_t dim, const void* c_tok,
                            const float* z_tok, float* out, csa2_stream_t stream) {
  CSA2_RANGE();
  if (ratio < 1 || ratio > 16 || n_out < 0 || dim <= 0 || dim % 16 != 0 || dim > kHeadDim)
    return ratio > 16 || dim > kHeadDim ? CSA2_ERR_UNSUPPORTED : CSA2_ERR_INVALID_ARG;
  if (n_out == 0) return CSA2_OK;
  if (!c_tok || !z_tok || !out || !aligned16(c_tok) || !aligned16(z_tok) || !aligned16(out))
    return CSA2_ERR_INVALID_ARG;
  AppendParams p;
  std::memset(&p, 0, sizeof(p));
  p.mode = 0;
  p.ratio = ratio;
  p.dim = dim;
  p.n_segs = 1;
  p.rows = n_out;
  p.seg[0].first = 0;
  p.c_tok = static_cast<const uint16_t*>(c_tok);
  p.z_tok = z_tok;
  p.entries_out = out;
  return cuda_status(launch_append(p, S(stream)));
}

csa2_status_t csa2_append_entries(csa2_cache_t* c, int32_t n_seqs, const int32_t* seq_ids,
                                  const int32_t* n_new, const float* entries, const void* idx_k,
                                  csa2_stream_t stream) {
  CSA2_RANGE();
  return run_append(c, 1, n_seqs, seq_ids, n_new, entries, nullptr, nullptr, idx_k, nullptr,
                    stream);
}

csa2_status_t csa2_append_tokens(csa2_cache_t* c, int32_t n_seqs, const int32_t* seq_ids,
                                 const int32_t* n_tok, const void* c_tok, const float* z_tok,
                                 const void* idx_k, float* entries_out, csa2_stream_t stream) {
  CSA2_RANGE();
  return run_append(c, 2, n_seqs, seq_ids, n_tok, nullptr, c_tok, z_tok, idx_k, entries_out,
                    stream);
}

size_t csa2_index_workspace_bytes(const csa2_cache_t* c, int32_t n_queries) {
  if (!c || n_queries < 0) return 0;
  return (size_t)n_queries * ((size_t)score_ld(c->max_cap) * sizeof(float) +
                              kKeyHistBinsHost * sizeof(uint32_t)) +
         topk_seg_bytes(n_queries, c->max_cap);
}

size_t csa2_index_prefill_workspace_bytes(const csa2_cache_t* c, int32_t seq, int32_t n_queries) {
  if (!c || seq < 0 || seq >= c->batch || n_queries < 0) return 0;
  size_t b = (size_t)n_queries * (size_t)score_ld(c->cap[seq]) * sizeof(float);
  if (c->cfg.idx_layout == CSA2_IDX_BF16) b += (size_t)n_queries * kKeyHistBinsHost * sizeof(uint32_t);
  return b;
}

size_t csa2_topk_workspace_bytes(int32_t n_rows, int64_t max_valid) {
  if (n_rows < 0 || max_valid < 0) return 0;
  return topk_seg_bytes(n_rows, max_valid);
}

}  // extern "C"

namespace {
csa2_status_t topk_impl(int32_t n_rows, const void* scores, int64_t ld, const int64_t* n_valid,
                        int32_t k, const uint32_t* key_hist, int32_t* idx_out, float* score_out,
                        void* workspace, size_t ws_bytes, csa2_stream_t stream, bool bf16) {
  if (n_rows < 0 || k <= 0 || k > 4096) return CSA2_ERR_INVALID_ARG;
  if (n_rows == 0) return CSA2_OK;
  if (!scores || !n_valid || !idx_out || ld < 0) return CSA2_ERR_INVALID_ARG;
  const size_t esz = bf16 ? 2 : 4;
  int64_t max_valid = 0;
  for (int r = 0; r < n_rows; ++r) {
    if (n_valid[r] < 0 || n_valid[r] > ld || n_valid[r] > (int64_t)INT32_MAX)
      return CSA2_ERR_INVALID_ARG;
    max_valid = std::max(max_valid, n_valid[r]);
  }
  const bool seg = key_hist && workspace && aligned16(workspace) && topk_segments(max_valid) > 2 &&
                   ws_bytes >= topk_seg_bytes(n_rows, max_valid) &&
                   topk_segments(max_valid) <= 1024;
  const int n_seg = topk_segments(max_valid);
  for (int r0 = 0; r0 < n_rows; r0 += kTopkTab) {
    const int nr = std::min(kTopkTab, n_rows - r0);
    TopkParams* p = new (std::nothrow) TopkParams();
    if (!p) return CSA2_ERR_OOM;
    p->scores = reinterpret_cast<const float*>(static_cast<const uint8_t*>(scores) +
                                               (size_t)r0 * ld * esz);
    p->score_bf16 = bf16 ? 1 : 0;
    p->ld = ld;
    p->rows = nr;
    p->k = k;
    p->idx_out = idx_out + (int64_t)r0 * k;
    p->score_out = score_out ? score_out + (int64_t)r0 * k : nullptr;
    p->key_hist = key_hist ? key_hist + (int64_t)r0 * kKeyHistBinsHost : nullptr;
    p->seg_ws = seg ? static_cast<uint32_t*>(workspace) +
                          (size_t)r0 * topk_seg_bytes(1, max_valid) / sizeof(uint32_t)
                    : nullptr;
    p->n_seg = seg ? n_seg : 0;
    p->formula = 0;
    for (int r = 0; r < nr; ++r) p->n_valid[r] = n_valid[r0 + r];
    cudaError_t e = launch_topk(*p, S(stream));
    delete p;
    if (e != cudaSuccess) return CSA2_ERR_CUDA;
  }
  return CSA2_OK;
}
}  // namespace

extern "C" {

csa2_status_t csa2_topk(int32_t n_rows, const float* scores, int64_t ld, const int64_t* n_valid,
                        int32_t k, const uint32_t* key_hist, int32_t* idx_out, float* score_out,
                        void* workspace, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_RANGE();
  return topk_impl(n_rows, scores, ld, n_valid, k, key_hist, idx_out, score_out, workspace,
                   ws_bytes, stream, false);
}

csa2_status_t csa2_topk_bf16(int32_t n_rows, const uint16_t* scores, int64_t ld,
                             const int64_t* n_valid, int32_t k, const uint32_t* key_hist,
                             int32_t* idx_out, float* score_out, void* workspace, size_t ws_bytes,
                             csa2_stream_t stream) {
  CSA2_RANGE();
  return topk_impl(n_rows, scores, ld, n_valid, k, key_hist, idx_out, score_out, workspace,
                   ws_bytes, stream, true);
}

}  // extern "C"

namespace {

// Scores of decode queries [q0, q0 + n) into scores (row stride ld): one
// indexer launch per chunk of up to kMaxIdxGroups queries.
// Entries query i sees: its sequence's appended entries, or with a token
// position those causally visible there, (s + 1) * ratio - 1 <= pos.
int64_t visible_of(const csa2_cache_t* c, int32_t s, const int64_t* q_pos, int i) {
  const int64_t len = c->len[s];
  if (!q_pos) return len;
  return std::min<int64_t>(len, (q_pos[i] + 1) / c->cfg.ratio);
}

csa2_status_t run_index_decode(const csa2_cache_t* c, int32_t nq, const void* q_idx,
                               const float* w, const int32_t* seq_ids, void* scores, int64_t ld,
                               uint32_t* key_hist, csa2_stream_t stream, IndexParams* ip,
                               bool bf16 = false, const int64_t* q_pos = nullptr) {
  const size_t esz = bf16 ? 2 : 4;
  const uint16_t* qb = static_cast<const uint16_t*>(q_idx);
  if (key_hist &&
      cudaMemsetAsync(key_hist, 0, (size_t)nq * kKeyHistBinsHost * sizeof(uint32_t), S(stream)) !=
          cudaSuccess)
    return CSA2_ERR_CUDA;
  // keys per decode tile: 512 for MXFP4 keys, 256 for bf16 keys
  const bool mx = c->cfg.idx_layout == CSA2_IDX_MXFP4;
  const int64_t tile_e = mx ? 512 : 256;
  for (int q0 = 0; q0 < nq; q0 += kMaxIdxGroups) {
    const int n = std::min(kMaxIdxGroups, nq - q0);
    std::memset(ip, 0, sizeof(IndexParams));
    ip->w = w + (int64_t)q0 * kIdxHeads;
    ip->scores = reinterpret_cast<float*>(static_cast<uint8_t*>(scores) + (size_t)q0 * ld * esz);
    ip->score_bf16 = bf16 ? 1 : 0;
    ip->ld = ld;
    ip->key_hist = key_hist ? key_hist + (int64_t)q0 * kKeyHistBinsHost : nullptr;
    ip->err = c->d_err;
    ip->nq = n;
    ip->qpg = 1;
    ip->n_groups = n;
    ip->prefill = 0;
    ip->ratio = c->cfg.ratio;
    ip->wait_cycles = c->wait_cycles;
    ip->inject = c->inject;
    ip->tile_prefix[0] = 0;
    for (int i = 0; i < n; ++i) {
      const int s = seq_ids ? seq_ids[q0 + i] : q0 + i;
      const int64_t nv = visible_of(c, s, q_pos, q0 + i);
      ip->entry_base[i] = c->off[s];
      ip->nvis[i] = (int32_t)nv;
      // MXFP4 decode tiles are aligned 512-key chunks: a sequence starting
      // inside one begins `lead` keys into its first tile
      const int64_t lead = (mx && nv > 0) ? (c->off[s] & 511) : 0;
      ip->tile_prefix[i + 1] = ip->tile_prefix[i] + (int32_t)((nv + lead + tile_e - 1) / tile_e);
    }
    CUtensorMap tm_q;
    const uint16_t* qn = qb + (int64_t)q0 * kIdxHeads * kIdxDim;
    if (!make_map(&tm_q, qn, (uint64_t)n * kIdxHeads, kIdxDim, 64, 32)) return CSA2_ERR_CUDA;
    const int tiles = ip->tile_prefix[n];
    if (tiles > 0) {
      const int grid = std::min(c->index_sms, tiles);
      if (launch_index_any(c, *ip, tm_q, qn, grid, S(stream)) != cudaSuccess) return CSA2_ERR_CUDA;
    }
  }
  return CSA2_OK;
}

csa2_status_t check_decode_queries(const csa2_cache_t* c, int32_t nq, const void* q_idx,
                                   const float* w, const int32_t* seq_ids) {
  if (!q_idx || !w || !aligned16(q_idx) || !aligned16(w)) return CSA2_ERR_INVALID_ARG;
  if (seq_ids) {
    for (int i = 0; i < nq; ++i)
      if (seq_ids[i] < 0 || seq_ids[i] >= c->batch) return CSA2_ERR_INVALID_ARG;
  } else if (nq > c->batch) {
    return CSA2_ERR_INVALID_ARG;
  }
  return CSA2_OK;
}

}  // namespace

extern "C" {

csa2_status_t csa2_index_scores_decode(const csa2_cache_t* c, int32_t nq, const void* q_idx,
                                       const float* w, const int32_t* seq_ids, float* scores,
                                       int64_t ld, uint32_t* key_hist, csa2_stream_t stream) {
  CSA2_RANGE();
  if (!c || nq < 0) return CSA2_ERR_INVALID_ARG;
  if (nq == 0) return CSA2_OK;
  csa2_status_t st = check_decode_queries(c, nq, q_idx, w, seq_ids);
  if (st != CSA2_OK) return st;
  if (!scores || !aligned16(scores) || ld % 4 != 0) return CSA2_ERR_INVALID_ARG;
  for (int i = 0; i < nq; ++i)
    if (c->len[seq_ids ? seq_ids[i] : i] > ld) return CSA2_ERR_CAPACITY;
  IndexParams* ip = new (std::nothrow) IndexParams();
  if (!ip) return CSA2_ERR_OOM;
  if (key_hist && !aligned16(key_hist)) { delete ip; return CSA2_ERR_INVALID_ARG; }
  st = run_index_decode(c, nq, q_idx, w, seq_ids, scores, ld, key_hist, stream, ip);
  delete ip;
  return st;
}

}  // extern "C"

namespace {
csa2_status_t index_topk_decode_impl(const csa2_cache_t* c, int32_t nq, const void* q_idx,
                                     const float* w, const int32_t* seq_ids, int32_t* topk_idx,
                                     float* topk_score, void* workspace, size_t ws_bytes,
                                     csa2_stream_t stream, bool bf16,
                                     const int64_t* q_pos = nullptr) {
  if (!c || nq < 0) return CSA2_ERR_INVALID_ARG;
  if (nq == 0) return CSA2_OK;
  csa2_status_t st = check_decode_queries(c, nq, q_idx, w, seq_ids);
  if (st != CSA2_OK) return st;
  if (q_pos)
    for (int i = 0; i < nq; ++i)
      if (q_pos[i] < 0) return CSA2_ERR_INVALID_ARG;
  if (!topk_idx || !workspace || !aligned16(workspace)) return CSA2_ERR_INVALID_ARG;
  if (ws_bytes < csa2_index_workspace_bytes(c, nq)) return CSA2_ERR_CAPACITY;
  // bf16 rows: a multiple of 8 scores keeps every row 16-byte aligned (and
  // the bf16 layout never needs more bytes than the fp32 one)
  const int64_t ld = bf16 ? (c->max_cap + 7) / 8 * 8 : score_ld(c->max_cap);
  const size_t esz = bf16 ? 2 : 4;
  uint8_t* scores = static_cast<uint8_t*>(workspace);
  uint32_t* key_hist = reinterpret_cast<uint32_t*>(scores + (size_t)nq * ld * esz);
  uint32_t* seg_ws = key_hist + (int64_t)nq * kKeyHistBinsHost;
  IndexParams* ip = new (std::nothrow) IndexParams();
  TopkParams* tp = new (std::nothrow) TopkParams();
  if (!ip || !tp) { delete ip; delete tp; return CSA2_ERR_OOM; }
  st = run_index_decode(c, nq, q_idx, w, seq_ids, scores, ld, key_hist, stream, ip, bf16, q_pos);
  const int k = c->cfg.topk;
  for (int q0 = 0; q0 < nq && st == CSA2_OK; q0 += kTopkTab) {
    const int n = std::min(kTopkTab, nq - q0);
    std::memset(tp, 0, sizeof(TopkParams));
    tp->scores = reinterpret_cast<const float*>(scores + (size_t)q0 * ld * esz);
    tp->score_bf16 = bf16 ? 1 : 0;
    tp->ld = ld;
    tp->rows = n;
    tp->k = k;
    tp->idx_out = topk_idx + (int64_t)q0 * k;
    tp->score_out = topk_score ? topk_score + (int64_t)q0 * k : nullptr;
    tp->key_hist = key_hist + (int64_t)q0 * kKeyHistBinsHost;
    // segments pay from three on: rows of up to two (16384 scores) are
    // compacted by the row kernel in one block-wide pass, one launch
    const bool use_seg = topk_segments(c->max_cap) <= 1024 && topk_segments(c->max_cap) > 2;
    tp->seg_ws = use_seg ? seg_ws + (size_t)q0 * topk_seg_bytes(1, c->max_cap) / sizeof(uint32_t)
                         : nullptr;
    tp->n_seg = use_seg ? topk_segments(c->max_cap) : 0;
    tp->formula = 0;
    tp->err = c->d_err;
    for (int i = 0; i < n; ++i)
      tp->n_valid[i] = visible_of(c, seq_ids ? seq_ids[q0 + i] : q0 + i, q_pos, q0 + i);
    if (launch_topk(*tp, S(stream)) != cudaSuccess) st = CSA2_ERR_CUDA;
  }
  delete ip;
  delete tp;
  return st;
}
}  // namespace

extern "C" {

csa2_status_t csa2_index_topk_decode(const csa2_cache_t* c, int32_t nq, const void* q_idx,
                                     const float* w, const int32_t* seq_ids, int32_t* topk_idx,
                                     float* topk_score, void* workspace, size_t ws_bytes,
                                     csa2_stream_t stream) {
  CSA2_RANGE();
  return index_topk_decode_impl(c, nq, q_idx, w, seq_ids, topk_idx, topk_score, workspace,
                                ws_bytes, stream, false);
}

csa2_status_t csa2_index_topk(const csa2_cache_t* c, int32_t nq, const void* q_idx,
                              const float* w, const int32_t* seq_of_q, const int64_t* q_pos,
                              int32_t* topk_idx, float* topk_score, void* workspace,
                              size_t ws_bytes, csa2_stream_t stream) {
  CSA2_RANGE();
  if (!q_pos) return CSA2_ERR_INVALID_ARG;
  return index_topk_decode_impl(c, nq, q_idx, w, seq_of_q, topk_idx, topk_score, workspace,
                                ws_bytes, stream, false, q_pos);
}

csa2_status_t csa2_index_topk_decode_bf16(const csa2_cache_t* c, int32_t nq, const void* q_idx,
                                          const float* w, const int32_t* seq_ids,
                                          int32_t* topk_idx, float* topk_score, void* workspace,
                                          size_t ws_bytes, csa2_stream_t stream) {
  CSA2_RANGE();
  return index_topk_decode_impl(c, nq, q_idx, w, seq_ids, topk_idx, topk_score, workspace,
                                ws_bytes, stream, true);
}

csa2_status_t csa2_index_scores_decode_bf16(const csa2_cache_t* c, int32_t nq, const void* q_idx,
                                            const float* w, const int32_t* seq_ids,
                                            uint16_t* scores, int64_t ld, uint32_t* key_hist,
                                            csa2_stream_t stream) {
  CSA2_RANGE();
  if (!c || nq < 0) return CSA2_ERR_INVALID_ARG;
  if (nq == 0) return CSA2_OK;
  csa2_status_t st = check_decode_queries(c, nq, q_idx, w, seq_ids);
  if (st != CSA2_OK) return st;
  if (!scores || !aligned16(scores) || ld % 8 != 0) return CSA2_ERR_INVALID_ARG;
  for (int i = 0; i < nq; ++i)
    if (c->len[seq_ids ? seq_ids[i] : i] > ld) return CSA2_ERR_CAPACITY;
  if (key_hist && !aligned16(key_hist)) return CSA2_ERR_INVALID_ARG;
  IndexParams* ip = new (std::nothrow) IndexParams();
  if (!ip) return CSA2_ERR_OOM;
  st = run_index_decode(c, nq, q_idx, w, seq_ids, scores, ld, key_hist, stream, ip, true);
  delete ip;
  return st;
}

csa2_status_t csa2_index_scores_prefill(const csa2_cache_t* c, int32_t seq, int32_t nq,
                                        int64_t pos0, const void* q_idx, const float* w,
                                        float* scores, int64_t ld, uint32_t* key_hist,
                                        csa2_stream_t stream) {
  CSA2_RANGE();
  if (!c || nq < 0 || seq < 0 || seq >= c->batch || pos0 < 0) return CSA2_ERR_INVALID_ARG;
  if (nq == 0) return CSA2_OK;
  if (!q_idx || !w || !scores || !aligned16(q_idx) || !aligned16(w) || !aligned16(scores) ||
      ld % 4 != 0 || (key_hist && !aligned16(key_hist)))
    return CSA2_ERR_INVALID_ARG;
  if (ld < c->len[seq]) return CSA2_ERR_CAPACITY;
  // queries sharing one tile of keys in the MMA: 8 (N = 256) on bf16 keys,
  // 4 (N = 128) on MXFP4 keys, whose tensor memory also holds the scales
  const bool mx = c->cfg.idx_layout == CSA2_IDX_MXFP4;
  // the score-key histograms come from the bf16 indexer's epilogue (the
  // MXFP4 kernel's shared memory has no room for eight of them)
  if (key_hist && mx) return CSA2_ERR_UNSUPPORTED;
  if (key_hist &&
      cudaMemsetAsync(key_hist, 0, (size_t)nq * kKeyHistBinsHost * sizeof(uint32_t), S(stream)) !=
          cudaSuccess)
    return CSA2_ERR_CUDA;
  const int kQpg = mx ? 4 : 8;
  const int m = c->cfg.ratio;
  const int64_t len = c->len[seq];
  const uint16_t* qb = static_cast<const uint16_t*>(q_idx);
  IndexParams* ip = new (std::nothrow) IndexParams();
  if (!ip) return CSA2_ERR_OOM;
  csa2_status_t st = CSA2_OK;
  const int per_launch = kMaxIdxGroups * kQpg;
  for (int q0 = 0; q0 < nq && st == CSA2_OK; q0 += per_launch) {
    const int n = std::min(per_launch, nq - q0);
    const int groups = (n + kQpg - 1) / kQpg;
    std::memset(ip, 0, sizeof(IndexParams));
    ip->w = w + (int64_t)q0 * kIdxHeads;
    ip->scores = scores + (int64_t)q0 * ld;
    ip->ld = ld;
    ip->key_hist = key_hist ? key_hist + (int64_t)q0 * kKeyHistBinsHost : nullptr;
    ip->err = c->d_err;
    ip->nq = n;
    ip->qpg = kQpg;
    ip->n_groups = groups;
    ip->prefill = 1;
    ip->pre_base = c->off[seq];
    ip->pos0 = pos0 + q0;
    ip->pre_len = (int32_t)len;
    ip->ratio = m;
    ip->wait_cycles = c->wait_cycles;
    ip->inject = c->inject;
    ip->tile_prefix[0] = 0;
    for (int g = 0; g < groups; ++g) {
      const int64_t last = std::min<int64_t>((int64_t)g * kQpg + kQpg, n) - 1;
      const int64_t nv = std::min<int64_t>(len, (ip->pos0 + last + 1) / m);
      // MXFP4 tiles are aligned 128-key chunks (the first one `lead` keys
      // before the sequence start)
      const int64_t lead = (mx && nv > 0) ? (c->off[seq] & 127) : 0;
      ip->tile_prefix[g + 1] = ip->tile_prefix[g] + (int32_t)((nv + lead + 127) / 128);
    }
    CUtensorMap tm_q;
    const uint16_t* qn = qb + (int64_t)q0 * kIdxHeads * kIdxDim;
    if (!make_map(&tm_q, qn, (uint64_t)n * kIdxHeads, kIdxDim, 64, 32 * kQpg)) {
      st = CSA2_ERR_CUDA;
      break;
    }
    const int tiles = ip->tile_prefix[groups];
    if (tiles > 0) {
      const int grid = std::min(c->index_sms, tiles);
      if (launch_index_any(c, *ip, tm_q, qn, grid, S(stream)) != cudaSuccess) st = CSA2_ERR_CUDA;
    }
  }
  delete ip;
  return st;
}

csa2_status_t csa2_index_topk_prefill(const csa2_cache_t* c, int32_t seq, int32_t nq, int64_t pos0,
                                      const void* q_idx, const float* w, int32_t* topk_idx,
                                      float* topk_score, void* workspace, size_t ws_bytes,
                                      csa2_stream_t stream) {
  CSA2_RANGE();
  if (!c || nq < 0 || seq < 0 || seq >= c->batch || pos0 < 0) return CSA2_ERR_INVALID_ARG;
  if (nq == 0) return CSA2_OK;
  if (!topk_idx || !workspace || !aligned16(workspace)) return CSA2_ERR_INVALID_ARG;
  if (ws_bytes < csa2_index_prefill_workspace_bytes(c, seq, nq)) return CSA2_ERR_CAPACITY;
  const int64_t ld = score_ld(c->cap[seq]);
  // workspace: scores [nq, ld], then (bf16 keys) the score-key histograms
  // [nq, 2048] that the indexer builds for the top-k's first digit
  float* scores = static_cast<float*>(workspace);
  uint32_t* key_hist = c->cfg.idx_layout == CSA2_IDX_BF16
                           ? reinterpret_cast<uint32_t*>(scores + (size_t)nq * ld)
                           : nullptr;
  csa2_status_t st =
      csa2_index_scores_prefill(c, seq, nq, pos0, q_idx, w, scores, ld, key_hist, stream);
  if (st != CSA2_OK) return st;
  TopkParams* tp = new (std::nothrow) TopkParams();
  if (!tp) return CSA2_ERR_OOM;
  tp->scores = scores;
  tp->key_hist = key_hist;
  tp->ld = ld;
  tp->rows = nq;
  tp->k = c->cfg.topk;
  tp->idx_out = topk_idx;
  tp->score_out = topk_score;
  tp->formula = 1;
  tp->err = c->d_err;
  tp->pre_len = (int32_t)c->len[seq];
  tp->ratio = c->cfg.ratio;
  tp->pos0 = pos0;
  if (launch_topk(*tp, S(stream)) != cudaSuccess) st = CSA2_ERR_CUDA;
  delete tp;
  return st;
}

size_t csa2_sparse_attn_workspace_bytes(const csa2_cache_t* c, int32_t n_queries) {
  if (!c || n_queries < 0) return 0;
  return kAttnSplitToken;
}

}  // extern "C"

namespace {
// Epilogue options into the launch parameters; false when they are invalid.
// Epilogue options of layer `ly` of a launch (sink, FP8 window rows), and
// the launch's output RoPE (shared by its layers); false when they are
// invalid.
bool apply_opts(AttnParams* p, AttnLayer* ly, const csa2_attn_opts_t* opts, bool decode,
                int32_t q0, int64_t row0) {
  if (!opts) return true;
  ly->sink = opts->sink;
  const bool f8 = opts->swa_codes || opts->swa_rope || opts->swa_scales;
  if (f8) {
    if (!opts->swa_codes || !opts->swa_rope || !opts->swa_scales || !aligned16(opts->swa_codes) ||
        !aligned16(opts->swa_rope) || (reinterpret_cast<uintptr_t>(opts->swa_scales) & 7u))
      return false;
    ly->swa_codes = opts->swa_codes + row0 * 448;
    ly->swa_rope = static_cast<const uint16_t*>(opts->swa_rope) + row0 * 64;
    ly->swa_scales = opts->swa_scales + row0 * 8;
  }
  if (opts->rope_out) {
    if (decode && !opts->rope_pos) return false;
    if (opts->rope_base < 0.0 || opts->rope_base != opts->rope_base) return false;
    p->rope_out = 1;
    p->rope_pos = decode ? opts->rope_pos + q0 : nullptr;
    const double base = opts->rope_base > 0.0 ? opts->rope_base : 10000.0;
    for (int t = 0; t < 32; ++t) p->rope_theta[t] = std::pow(base, -(double)t / 32.0);
  }
  return true;
}
}  // namespace

extern "C" {

csa2_status_t csa2_sparse_attn_decode(const csa2_cache_t* c, int32_t nq, const int32_t* seq_ids,
                                      const void* q, const void* swa_kv, const int32_t* swa_len,
                                      const int32_t* topk_idx, float scale, void* out, float* lse,
                                      void* workspace, size_t ws_bytes, csa2_stream_t stream) {
  CSA2_RANGE();
  return csa2_sparse_attn_decode_ex(c, nq, seq_ids, q, swa_kv, swa_len, topk_idx, scale, out, lse,
                                    workspace, ws_bytes, nullptr, stream);
}

csa2_status_t csa2_sparse_attn_decode_ex(const csa2_cache_t* c, int32_t nq,
                                         const int32_t* seq_ids, const void* q,
                                         const void* swa_kv, const int32_t* swa_len,
                                         const int32_t* topk_idx, float scale, void* out,
                                         float* lse, void* workspace, size_t ws_bytes,
                                         const csa2_attn_opts_t* opts, csa2_stream_t stream) {
  CSA2_RANGE();
  return csa2_sparse_attn_decode_layers(c, 1, nq, seq_ids, &q, &swa_kv, swa_len, topk_idx, scale,
                                        &out, &lse, workspace, ws_bytes, &opts, stream);
}

csa2_status_t csa2_sparse_attn_decode_layers(const csa2_cache_t* c, int32_t n_layers, int32_t nq,
                                             const int32_t* seq_ids, const void* const* q,
                                             const void* const* swa_kv, const int32_t* swa_len,
                                             const int32_t* topk_idx, float scale,
                                             void* const* out, float* const* lse,
                                             void* workspace, size_t ws_bytes,
                                             const csa2_attn_opts_t* const* opts,
                                             csa2_stream_t stream) {
  CSA2_RANGE();
  if (!c || nq < 0 || n_layers < 1 || n_layers > CSA2_MAX_ATTN_LAYERS || !q || !out)
    return CSA2_ERR_INVALID_ARG;
  if (nq == 0) return CSA2_OK;
  const int W = c->cfg.swa;
  if (!topk_idx || !aligned16(topk_idx)) return CSA2_ERR_INVALID_ARG;
  const csa2_attn_opts_t* o0 = opts ? opts[0] : nullptr;
  for (int l = 0; l < n_layers; ++l) {
    const csa2_attn_opts_t* ol = opts ? opts[l] : nullptr;
    if (!q[l] || !out[l] || !aligned16(q[l]) || !aligned16(out[l])) return CSA2_ERR_INVALID_ARG;
    const bool f8 = ol && ol->swa_codes;
    const void* sw = swa_kv ? swa_kv[l] : nullptr;
    if (W > 0 && !f8 && (!sw || !aligned16(sw))) return CSA2_ERR_INVALID_ARG;
    if (lse && lse[l] && !aligned16(lse[l])) return CSA2_ERR_INVALID_ARG;
    // the output RoPE is one setting for the launch: every layer the same
    const bool r0 = o0 && o0->rope_out, rl = ol && ol->rope_out;
    if (r0 != rl || (rl && (ol->rope_pos != o0->rope_pos || ol->rope_base != o0->rope_base)))
      return CSA2_ERR_INVALID_ARG;
  }
  if (workspace && !aligned16(workspace)) return CSA2_ERR_INVALID_ARG;
  if (seq_ids)
    for (int i = 0; i < nq; ++i)
      if (seq_ids[i] < 0 || seq_ids[i] >= c->batch) return CSA2_ERR_INVALID_ARG;
  if (!seq_ids && nq > c->batch) return CSA2_ERR_INVALID_ARG;
  const int H = c->cfg.n_heads, k = c->cfg.topk, G = H / kAttnHeadGroup;
  AttnParams* p = new (std::nothrow) AttnParams();
  AttnMaps* maps = new (std::nothrow) AttnMaps();
  if (!p || !maps) { delete p; delete maps; return CSA2_ERR_OOM; }
  csa2_status_t st = CSA2_OK;
  for (int q0 = 0; q0 < nq && st == CSA2_OK; q0 += kAttnTab) {
    const int n = std::min(kAttnTab, nq - q0);
    // two CTAs per (query, head group) when the pairs still fit the SMs in
    // one wave: a second wave of split CTAs costs more than unsplit CTAs
    // leaving some SMs idle
    const bool split = workspace && ws_bytes >= kAttnSplitToken &&
                       2 * (int64_t)n_layers * n * G <= c->num_sms;
    std::memset(p, 0, sizeof(AttnParams));
    p->topk_idx = topk_idx + (int64_t)q0 * k;
    p->swa_len = swa_len ? swa_len + q0 : nullptr;
    p->codes = c->codes;
    p->scales = c->scales;
    p->n_layers = n_layers;
    p->err = c->d_err;
    p->nq = n;
    p->n_heads = H;
    p->topk = k;
    p->swa = W;
    p->layout = c->cfg.layout;
    p->scale = scale;
    p->scale_log2 = scale * 1.4426950408889634f;
    p->prefill = 0;
    p->splits = split ? 2 : 1;
    p->wait_cycles = c->wait_cycles;
    for (int i = 0; i < n; ++i) {
      const int s = seq_ids ? seq_ids[q0 + i] : q0 + i;
      p->q_base[i] = c->off[s];
      p->q_len[i] = (int32_t)c->len[s];
    }
    for (int l = 0; l < n_layers && st == CSA2_OK; ++l) {
      AttnLayer& ly = p->layer[l];
      const csa2_attn_opts_t* ol = opts ? opts[l] : nullptr;
      ly.out = static_cast<uint16_t*>(out[l]) + (int64_t)q0 * H * kHeadDim;
      ly.lse = (lse && lse[l]) ? lse[l] + (int64_t)q0 * H : nullptr;
      if (!apply_opts(p, &ly, ol, true, q0, (int64_t)q0 * W)) { st = CSA2_ERR_INVALID_ARG; break; }
      const uint16_t* qb = static_cast<const uint16_t*>(q[l]) + (int64_t)q0 * H * kHeadDim;
      if (!make_map(&maps->q[l], qb, (uint64_t)n * H, kHeadDim, 64, kAttnHeadGroup)) {
        st = CSA2_ERR_CUDA;
        break;
      }
      if (W > 0 && !(ol && ol->swa_codes)) {
        const uint16_t* sb = static_cast<const uint16_t*>(swa_kv[l]) + (int64_t)q0 * W * kHeadDim;
        if (!make_map(&maps->swa[l], sb, (uint64_t)n * W, kHeadDim, 64, 128)) { st = CSA2_ERR_CUDA; break; }
      } else {
        maps->swa[l] = maps->q[l];
      }
    }
    if (st == CSA2_OK && launch_attn(*p, *maps, S(stream)) != cudaSuccess) st = CSA2_ERR_CUDA;
  }
  delete p;
  delete maps;
  return st;
}

csa2_status_t csa2_sparse_attn_prefill(const csa2_cache_t* c, int32_t seq, int32_t nq,
                                       int64_t pos0, const void* q, const void* swa_kv,
                                       int64_t swa_pos0, int64_t n_swa_rows,
                                       const int32_t* topk_idx, float scale, void* out, float* lse,
                                       csa2_stream_t stream) {
  CSA2_RANGE();
  return csa2_sparse_attn_prefill_ex(c, seq, nq, pos0, q, swa_kv, swa_pos0, n_swa_rows, topk_idx,
                                     scale, out, lse, nullptr, stream);
}

csa2_status_t csa2_sparse_attn_prefill_ex(const csa2_cache_t* c, int32_t seq, int32_t nq,
                                          int64_t pos0, const void* q, const void* swa_kv,
                                          int64_t swa_pos0, int64_t n_swa_rows,
                                          const int32_t* topk_idx, float scale, void* out,
                                          float* lse, const csa2_attn_opts_t* opts,
                                          csa2_stream_t stream) {
  CSA2_RANGE();
  return csa2_sparse_attn_prefill_layers(c, seq, 1, nq, pos0, &q, &swa_kv, swa_pos0, n_swa_rows,
                                         topk_idx, scale, &out, &lse, &opts, stream);
}

csa2_status_t csa2_sparse_attn_prefill_layers(const csa2_cache_t* c, int32_t seq, int32_t n_layers,
                                              int32_t nq, int64_t pos0, const void* const* q,
                                              const void* const* swa_kv, int64_t swa_pos0,
                                              int64_t n_swa_rows, const int32_t* topk_idx,
                                              float scale, void* const* out, float* const* lse,
                                              const csa2_attn_opts_t* const* opts,
                                              csa2_stream_t stream) {
  CSA2_RANGE();
  if (!c || nq < 0 || seq < 0 || seq >= c->batch || pos0 < 0 || n_layers < 1 ||
      n_layers > CSA2_MAX_ATTN_LAYERS || !q || !out)
    return CSA2_ERR_INVALID_ARG;
  if (nq == 0) return CSA2_OK;
  const int W = c->cfg.swa;
  if (!topk_idx || !aligned16(topk_idx)) return CSA2_ERR_INVALID_ARG;
  if (W > 0 && (swa_pos0 < 0 || swa_pos0 > pos0 || n_swa_rows <= 0 ||
                pos0 + nq - 1 - swa_pos0 >= n_swa_rows))
    return CSA2_ERR_INVALID_ARG;
  const csa2_attn_opts_t* o0 = opts ? opts[0] : nullptr;
  for (int l = 0; l < n_layers; ++l) {
    const csa2_attn_opts_t* ol = opts ? opts[l] : nullptr;
    if (!q[l] || !out[l] || !aligned16(q[l]) || !aligned16(out[l])) return CSA2_ERR_INVALID_ARG;
    if (lse && lse[l] && !aligned16(lse[l])) return CSA2_ERR_INVALID_ARG;
    const bool f8 = ol && ol->swa_codes;
    const void* sw = swa_kv ? swa_kv[l] : nullptr;
    if (W > 0 && !f8 && (!sw || !aligned16(sw))) return CSA2_ERR_INVALID_ARG;
    const bool r0 = o0 && o0->rope_out, rl = ol && ol->rope_out;
    if (r0 != rl || (rl && ol->rope_base != o0->rope_base)) return CSA2_ERR_INVALID_ARG;
  }
  const int H = c->cfg.n_heads, k = c->cfg.topk;
  AttnParams* p = new (std::nothrow) AttnParams();
  AttnMaps* maps = new (std::nothrow) AttnMaps();
  if (!p || !maps) { delete p; delete maps; return CSA2_ERR_OOM; }
  std::memset(p, 0, sizeof(AttnParams));
  p->topk_idx = topk_idx;
  p->codes = c->codes;
  p->scales = c->scales;
  p->n_layers = n_layers;
  p->err = c->d_err;
  p->nq = nq;
  p->n_heads = H;
  p->topk = k;
  p->swa = W;
  p->layout = c->cfg.layout;
  p->scale = scale;
  p->scale_log2 = scale * 1.4426950408889634f;
  p->prefill = 1;
  p->pre_base = c->off[seq];
  p->pre_len = (int32_t)c->len[seq];
  p->pos0 = pos0;
  p->swa_pos0 = swa_pos0;
  p->splits = 1;
  p->wait_cycles = c->wait_cycles;
  csa2_status_t st = CSA2_OK;
  for (int l = 0; l < n_layers && st == CSA2_OK; ++l) {
    AttnLayer& ly = p->layer[l];
    const csa2_attn_opts_t* ol = opts ? opts[l] : nullptr;
    ly.out = static_cast<uint16_t*>(out[l]);
    ly.lse = lse ? lse[l] : nullptr;
    if (!apply_opts(p, &ly, ol, false, 0, 0)) { st = CSA2_ERR_INVALID_ARG; break; }
    if (!make_map(&maps->q[l], q[l], (uint64_t)nq * H, kHeadDim, 64, kAttnHeadGroup)) {
      st = CSA2_ERR_CUDA;
      break;
    }
    if (W > 0 && !(ol && ol->swa_codes)) {
      if (!make_map(&maps->swa[l], swa_kv[l], (uint64_t)n_swa_rows, kHeadDim, 64, 128)) {
        st = CSA2_ERR_CUDA;
        break;
      }
    } else {
      maps->swa[l] = maps->q[l];
    }
  }
  if (st == CSA2_OK && launch_attn(*p, *maps, S(stream)) != cudaSuccess) st = CSA2_ERR_CUDA;
  delete p;
  delete maps;
  return st;
}

// Device address of g_static_scratch for the current device (host code
// cannot use the symbol itself as a device pointer).  It is looked up again
// on every call made while `stream` is not being captured, so a new context
// (after a device reset) gets its own address; a call during a capture uses
// the address the last uncaptured call found and is refused with
// CSA2_ERR_UNSUPPORTED when there is none (the lookup may load the module,
// which a capture must not contain).
static csa2_status_t static_scratch_ptr(cudaStream_t stream, void** out) {
  static std::mutex mu;
  static void* ptrs[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return CSA2_ERR_CUDA;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cs) != cudaSuccess) return CSA2_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (cs == cudaStreamCaptureStatusNone) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_static_scratch) != cudaSuccess) return CSA2_ERR_CUDA;
    ptrs[dev] = p;
  } else if (!ptrs[dev]) {
    return CSA2_ERR_UNSUPPORTED;
  }
  *out = ptrs[dev];
  return CSA2_OK;
}

csa2_status_t csa2_index_topk_decode_static(const csa2_cache_t* c, int32_t nq, const void* q_idx,
                                            const float* w, const int32_t* seq_ids,
                                            int32_t* topk_idx, float* topk_score,
                                            csa2_stream_t stream) {
  CSA2_RANGE();
  if (!c || nq < 0) return CSA2_ERR_INVALID_ARG;
  if (nq == 0) return CSA2_OK;
  csa2_status_t st = check_decode_queries(c, nq, q_idx, w, seq_ids);
  if (st != CSA2_OK) return st;
  if (!topk_idx) return CSA2_ERR_INVALID_ARG;
  const int64_t ld = score_ld(c->max_cap);
  const size_t need = (size_t)nq * ((size_t)ld * sizeof(float) + kKeyHistBinsHost * sizeof(uint32_t));
  if (need > CSA2_STATIC_SCRATCH_BYTES) return CSA2_ERR_CAPACITY;
  void* scratch = nullptr;
  st = static_scratch_ptr(S(stream), &scratch);
  if (st != CSA2_OK) return st;
  float* scores = static_cast<float*>(scratch);
  uint32_t* key_hist = reinterpret_cast<uint32_t*>(scores + (int64_t)nq * ld);
  // parameter blocks on the stack: this path touches no heap
  IndexParams ip;
  st = run_index_decode(c, nq, q_idx, w, seq_ids, scores, ld, key_hist, stream, &ip);
  const int k = c->cfg.topk;
  TopkParams tp;
  for (int q0 = 0; q0 < nq && st == CSA2_OK; q0 += kTopkTab) {
    const int n = std::min(kTopkTab, nq - q0);
    std::memset(&tp, 0, sizeof(TopkParams));
    tp.scores = scores + (int64_t)q0 * ld;
    tp.ld = ld;
    tp.rows = n;
    tp.k = k;
    tp.idx_out = topk_idx + (int64_t)q0 * k;
    tp.score_out = topk_score ? topk_score + (int64_t)q0 * k : nullptr;
    tp.key_hist = key_hist + (int64_t)q0 * kKeyHistBinsHost;
    tp.seg_ws = nullptr;   // one CTA per row: no segment scratch
    tp.n_seg = 0;
    tp.formula = 0;
    tp.err = c->d_err;
    for (int i = 0; i < n; ++i) tp.n_valid[i] = c->len[seq_ids ? seq_ids[q0 + i] : q0 + i];
    if (launch_topk(tp, S(stream)) != cudaSuccess) st = CSA2_ERR_CUDA;
  }
  return st;
}

// ---------------------------------------------------------------- HSI
static int64_t hsi_ld_b(int64_t max_valid) {
  return score_ld((max_valid + kHsiBlock - 1) / kHsiBlock);
}

size_t csa2_hsi_pool_workspace_bytes(int32_t n_rows, int64_t max_valid) {
  if (n_rows < 0 || max_valid < 0) return 0;
  return (size_t)n_rows * (size_t)hsi_ld_b(max_valid) * sizeof(float);
}

csa2_status_t csa2_hsi_pool(int32_t n_rows, const float* scores, int64_t ld,
                            const int64_t* n_valid, int32_t block, int32_t max_blocks,
                            int32_t* pool_blocks, void* workspace, size_t ws_bytes,
                            csa2_stream_t stream) {
  CSA2_RANGE();
  if (n_rows < 0 || ld < 0) return CSA2_ERR_INVALID_ARG;
  if (block != kHsiBlock || max_blocks <= 0 || max_blocks % 16 != 0 || max_blocks > 4096)
    return CSA2_ERR_UNSUPPORTED;
  if (n_rows == 0) return CSA2_OK;
  if (!scores || !n_valid || !pool_blocks || !workspace || !aligned16(workspace))
    return CSA2_ERR_INVALID_ARG;
  int64_t max_valid = 0;
  for (int r = 0; r < n_rows; ++r) {
    if (n_valid[r] < 0 || n_valid[r] > ld) return CSA2_ERR_INVALID_ARG;
    max_valid = std::max(max_valid, n_valid[r]);
  }
  if (ws_bytes < csa2_hsi_pool_workspace_bytes(n_rows, max_valid)) return CSA2_ERR_CAPACITY;
  const int64_t ld_b = hsi_ld_b(max_valid);
  float* bmax = static_cast<float*>(workspace);
  HsiParams* hp = new (std::nothrow) HsiParams();
  TopkParams* tp = new (std::nothrow) TopkParams();
  if (!hp || !tp) { delete hp; delete tp; return CSA2_ERR_OOM; }
  csa2_status_t st = CSA2_OK;
  for (int r0 = 0; r0 < n_rows && st == CSA2_OK; r0 += kHsiTab) {
    const int n = std::min(kHsiTab, n_rows - r0);
    std::memset(hp, 0, sizeof(HsiParams));
    hp->rows = n;
    hp->scores = scores + (int64_t)r0 * ld;
    hp->ld = ld;
    hp->bmax = bmax + (int64_t)r0 * ld_b;
    hp->ld_b = ld_b;
    for (int i = 0; i < n; ++i) hp->n[i] = n_valid[r0 + i];
    if (launch_block_max(*hp, S(stream)) != cudaSuccess) { st = CSA2_ERR_CUDA; break; }
    // the blocks with the highest block scores, ties to the lower block
    std::memset(tp, 0, sizeof(TopkParams));
    tp->scores = hp->bmax;
    tp->ld = ld_b;
    tp->rows = n;
    tp->k = max_blocks;
    tp->idx_out = pool_blocks + (int64_t)r0 * max_blocks;
    tp->formula = 0;
    for (int i = 0; i < n; ++i) tp->n_valid[i] = (n_valid[r0 + i] + kHsiBlock - 1) / kHsiBlock;
    if (launch_topk(*tp, S(stream)) != cudaSuccess) st = CSA2_ERR_CUDA;
  }
  delete hp;
  delete tp;
  return st;
}

size_t csa2_index_reindex_workspace_bytes(const csa2_cache_t* c, int32_t n_queries,
                                          int32_t max_blocks) {
  if (!c || n_queries < 0 || max_blocks <= 0) return 0;
  const int64_t slots = (int64_t)max_blocks * kHsiBlock;
  return (size_t)n_queries * ((size_t)slots * sizeof(float) + kKeyHistBinsHost * 4 +
                              (size_t)c->cfg.topk * 4) +
         topk_seg_bytes(n_queries, slots);
}

csa2_status_t csa2_index_topk_reindex_decode(const csa2_cache_t* c, int32_t nq, const void* q_idx,
                                             const float* w, const int32_t* seq_ids,
                                             const int32_t* pool_blocks, int32_t max_blocks,
                                             int32_t* topk_idx, float* topk_score,
                                             void* workspace, size_t ws_bytes,
                                             csa2_stream_t stream) {
  CSA2_RANGE();
  if (!c || nq < 0) return CSA2_ERR_INVALID_ARG;
  if (max_blocks <= 0 || max_blocks % 16 != 0 || max_blocks > 4096) return CSA2_ERR_UNSUPPORTED;
  if (nq == 0) return CSA2_OK;
  csa2_status_t st = check_decode_queries(c, nq, q_idx, w, seq_ids);
  if (st != CSA2_OK) return st;
  if (!pool_blocks || !topk_idx || !workspace || !aligned16(workspace)) return CSA2_ERR_INVALID_ARG;
  if (ws_bytes < csa2_index_reindex_workspace_bytes(c, nq, max_blocks)) return CSA2_ERR_CAPACITY;
  const int64_t slots = (int64_t)max_blocks * kHsiBlock;
  float* pscores = static_cast<float*>(workspace);
  uint32_t* key_hist = reinterpret_cast<uint32_t*>(pscores + (int64_t)nq * slots);
  int32_t* sel = reinterpret_cast<int32_t*>(key_hist + (int64_t)nq * kKeyHistBinsHost);
  uint32_t* seg_ws = reinterpret_cast<uint32_t*>(sel + (int64_t)nq * c->cfg.topk);
  const int k = c->cfg.topk;
  IndexParams* ip = new (std::nothrow) IndexParams();
  TopkParams* tp = new (std::nothrow) TopkParams();
  HsiParams* hp = new (std::nothrow) HsiParams();
  if (!ip || !tp || !hp) { delete ip; delete tp; delete hp; return CSA2_ERR_OOM; }
  const uint16_t* qb = static_cast<const uint16_t*>(q_idx);
  if (cudaMemsetAsync(key_hist, 0, (size_t)nq * kKeyHistBinsHost * 4, S(stream)) != cudaSuccess)
    st = CSA2_ERR_CUDA;
  // tiles of 32 blocks (256 slots) over bf16 keys, of 64 blocks (512 slots)
  // over MXFP4 keys; a last tile holds what remains of max_blocks (a
  // multiple of 16)
  const int blocks_per_tile = c->cfg.idx_layout == CSA2_IDX_MXFP4 ? 64 : 32;
  const int pool_tiles = (max_blocks + blocks_per_tile - 1) / blocks_per_tile;
  for (int q0 = 0; q0 < nq && st == CSA2_OK; q0 += kMaxIdxGroups) {
    const int n = std::min(kMaxIdxGroups, nq - q0);
    // ---- the pool positions' scores (indexer in pool mode)
    std::memset(ip, 0, sizeof(IndexParams));
    ip->w = w + (int64_t)q0 * kIdxHeads;
    ip->scores = pscores + (int64_t)q0 * slots;
    ip->ld = slots;
    ip->key_hist = key_hist + (int64_t)q0 * kKeyHistBinsHost;
    ip->pool = pool_blocks + (int64_t)q0 * max_blocks;
    ip->pool_blocks = max_blocks;
    ip->err = c->d_err;
    ip->nq = n;
    ip->qpg = 1;
    ip->n_groups = n;
    ip->ratio = c->cfg.ratio;
    ip->wait_cycles = c->wait_cycles;
    ip->inject = c->inject;
    ip->tile_prefix[0] = 0;
    for (int i = 0; i < n; ++i) {
      const int s = seq_ids ? seq_ids[q0 + i] : q0 + i;
      ip->entry_base[i] = c->off[s];
      ip->nvis[i] = (int32_t)c->len[s];
      ip->tile_prefix[i + 1] = ip->tile_prefix[i] + pool_tiles;
    }
    CUtensorMap tm_q;
    const uint16_t* qn = qb + (int64_t)q0 * kIdxHeads * kIdxDim;
    if (!make_map(&tm_q, qn, (uint64_t)n * kIdxHeads, kIdxDim, 64, 32)) {
      st = CSA2_ERR_CUDA;
      break;
    }
    const int grid = std::min(c->index_sms, ip->tile_prefix[n]);
    if (launch_index_any(c, *ip, tm_q, qn, grid, S(stream), true) != cudaSuccess) {
      st = CSA2_ERR_CUDA;
      break;
    }
    // ---- top-k over the pool slots (ties to the lower slot = lower entry)
    std::memset(tp, 0, sizeof(TopkParams));
    tp->scores = ip->scores;
    tp->ld = slots;
    tp->rows = n;
    tp->k = k;
    tp->idx_out = sel + (int64_t)q0 * k;
    tp->score_out = topk_score ? topk_score + (int64_t)q0 * k : nullptr;
    tp->key_hist = ip->key_hist;
    // a pool of at most two segments (16384 slots) is compacted by the row
    // kernel itself in one block-wide pass: one launch instead of two
    const bool use_seg = topk_segments(slots) > 2;
    tp->seg_ws = use_seg ? seg_ws + (size_t)q0 * topk_seg_bytes(1, slots) / sizeof(uint32_t)
                         : nullptr;
    tp->n_seg = use_seg ? topk_segments(slots) : 0;
    tp->formula = 0;
    tp->err = c->d_err;
    for (int i = 0; i < n; ++i) tp->n_valid[i] = slots;
    if (launch_topk(*tp, S(stream)) != cudaSuccess) { st = CSA2_ERR_CUDA; break; }
    // ---- pool slots back to entry indices
    std::memset(hp, 0, sizeof(HsiParams));
    hp->rows = n;
    hp->sel = tp->idx_out;
    hp->k = k;
    hp->pool = ip->pool;
    hp->pool_blocks = max_blocks;
    hp->out = topk_idx + (int64_t)q0 * k;
    hp->score_out = tp->score_out;
    hp->err = c->d_err;
    for (int i = 0; i < n; ++i) hp->n[i] = ip->nvis[i];
    if (launch_pool_map(*hp, S(stream)) != cudaSuccess) st = CSA2_ERR_CUDA;
  }
  delete ip;
  delete tp;
  delete hp;
  return st;
}

}  // extern "C"

// ---------------------------------------------------------------- trees of drafts
namespace {

// A tree call's queries, one record per draft in call order: the fields of
// TreeQuery with `rows` the whole path (self included) and win_n the depth;
// win_row is the sequence's position in the call.
struct TreePlan {
  TreeQuery* q = nullptr;
  int64_t nq = 0;
  int32_t max_draft = 0;
  ~TreePlan() { delete[] q; }
};

// Depth and path (bit a: draft a is on it, self included) of each draft.
bool tree_paths(int32_t n, const int32_t* parent, int32_t* depth, uint64_t* path) {
  for (int t = 0; t < n; ++t) {
    const int32_t a = parent[t];
    if (a < -1 || a >= t) return false;
    depth[t] = a < 0 ? 0 : depth[a] + 1;
    path[t] = (a < 0 ? 0ull : path[a]) | (1ull << t);
  }
  return true;
}

// Checks a tree against the cache and fills the plan.  Every sequence at
// most once; its cache must hold exactly floor(pos0 / ratio) committed
// entries and the entries of its drafts.
csa2_status_t plan_tree(const csa2_cache* c, const csa2_tree_t* t, TreePlan* plan) {
  if (!c || !t || t->n_seqs < 0) return CSA2_ERR_INVALID_ARG;
  if (t->n_seqs == 0) return CSA2_OK;
  if (!t->n_draft || !t->pos0 || t->n_seqs > c->batch) return CSA2_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return CSA2_ERR_CUDA;
  if (dev != c->dev) return CSA2_ERR_INVALID_ARG;
  uint64_t seen[4096 / 64] = {};
  int64_t nq = 0;
  for (int i = 0; i < t->n_seqs; ++i) {
    const int32_t s = t->seq_ids ? t->seq_ids[i] : i, n = t->n_draft[i];
    if (s < 0 || s >= c->batch || n < 0 || t->pos0[i] < 0 ||
        t->pos0[i] > INT64_MAX - CSA2_MAX_DRAFT)
      return CSA2_ERR_INVALID_ARG;
    if (n > CSA2_MAX_DRAFT) return CSA2_ERR_UNSUPPORTED;
    if ((seen[s >> 6] >> (s & 63)) & 1u) return CSA2_ERR_INVALID_ARG;
    seen[s >> 6] |= 1ull << (s & 63);
    nq += n;
    plan->max_draft = std::max(plan->max_draft, n);
  }
  if (nq > 0 && !t->parent) return CSA2_ERR_INVALID_ARG;
  plan->q = new (std::nothrow) TreeQuery[(size_t)std::max<int64_t>(nq, 1)];
  if (!plan->q) return CSA2_ERR_OOM;
  plan->nq = nq;
  int64_t first = 0;
  for (int i = 0; i < t->n_seqs; ++i) {
    const int32_t s = t->seq_ids ? t->seq_ids[i] : i, n = t->n_draft[i];
    int32_t depth[CSA2_MAX_DRAFT];
    uint64_t path[CSA2_MAX_DRAFT];
    if (!tree_paths(n, t->parent ? t->parent + first : nullptr, depth, path))
      return CSA2_ERR_INVALID_ARG;
    const int64_t m = c->cfg.ratio, pos0 = t->pos0[i];
    uint64_t own = 0;   // drafts that complete a block, and so own an entry
    for (int j = 0; j < n; ++j)
      if ((pos0 + depth[j] + 1) % m == 0) own |= 1ull << j;
    const int64_t n_com = pos0 / m;
    if (c->len[s] != n_com + __builtin_popcountll(own)) return CSA2_ERR_INVALID_ARG;
    for (int j = 0; j < n; ++j) {
      TreeQuery& q = plan->q[first + j];
      q.base = c->off[s];
      q.pos = pos0 + depth[j];
      q.rows = path[j];
      q.ents = 0;
      for (uint64_t b = path[j] & own; b; b &= b - 1) {
        const uint64_t bit = b & (~b + 1);
        q.ents |= 1ull << __builtin_popcountll(own & (bit - 1));
      }
      q.len = (int32_t)c->len[s];
      q.n_com = (int32_t)n_com;
      q.win_row = i;
      q.win_n = depth[j];
      q.draft0 = (int32_t)first;
    }
    first += n;
  }
  return CSA2_OK;
}

int64_t tree_columns(const TreeQuery& q) { return q.n_com + __builtin_popcountll(q.ents); }

// Scores of a planned tree into rows of stride ld.
csa2_status_t run_index_tree(const csa2_cache* c, const csa2_tree_t* t, const TreePlan& plan,
                             const void* q_idx, const float* w, float* scores, int64_t ld,
                             uint32_t* key_hist, csa2_stream_t stream) {
  const int64_t nq = plan.nq;
  const bool mx = c->cfg.idx_layout == CSA2_IDX_MXFP4;
  TreeIndexParams* ip = new (std::nothrow) TreeIndexParams();
  if (!ip) return CSA2_ERR_OOM;
  csa2_status_t st = CSA2_OK;
  if (plan.max_draft == 1) {
    // a single draft a sequence sees every entry: the decode indexer
    int32_t* ids = new (std::nothrow) int32_t[(size_t)nq];
    if (!ids) { delete ip; return CSA2_ERR_OOM; }
    int64_t k = 0;
    for (int i = 0; i < t->n_seqs; ++i)
      if (t->n_draft[i]) ids[k++] = t->seq_ids ? t->seq_ids[i] : i;
    st = run_index_decode(c, (int32_t)nq, q_idx, w, ids, scores, ld, key_hist, stream, ip);
    delete[] ids;
    delete ip;
    return st;
  }
  if (key_hist &&
      cudaMemsetAsync(key_hist, 0, (size_t)nq * kKeyHistBinsHost * sizeof(uint32_t), S(stream)) !=
          cudaSuccess) {
    delete ip;
    return CSA2_ERR_CUDA;
  }
  // queries that share a tile of keys
  const int qpg = mx ? 4 : plan.max_draft <= 2 ? 2 : plan.max_draft <= 4 ? 4 : 8;
  // keys of a tile.  MXFP4: 512 (a stage's waits once in four M-groups: 101
  // drafts of 4 trees over 128K 80 us, with 256 96), 256 when there would be fewer such
  // tiles than SMs (29 drafts over 4096: 5.2 us, with 512 5.8)
  int64_t tiles512 = 0;
  for (int i = 0; mx && i < t->n_seqs; ++i) {
    const int s = t->seq_ids ? t->seq_ids[i] : i;
    tiles512 += (int64_t)((t->n_draft[i] + 3) / 4) * ((c->len[s] + 511) / 512);
  }
  const int tile = !mx ? 128 : tiles512 >= c->num_sms ? 512 : 256;
  const uint16_t* qb = static_cast<const uint16_t*>(q_idx);
  int64_t q0 = 0, done = 0;   // queries before this launch, queries of the sequence already taken
  int seq = 0;
  while (seq < t->n_seqs && st == CSA2_OK) {
    std::memset(ip, 0, sizeof(TreeIndexParams));
    int n = 0, groups = 0;
    while (seq < t->n_seqs) {
      const int T = t->n_draft[seq];
      if (done >= T) { ++seq; done = 0; continue; }
      // a sequence's drafts in groups of nearly equal size
      const int ng = (T + qpg - 1) / qpg;
      const int g = (int)(done * ng / T) + (done * ng % T != 0);
      const int size = (int)((int64_t)(g + 1) * T / ng - done);
      if (n + size > kMaxTreeQueries || groups >= kMaxTreeQueries) break;
      const TreeQuery& q = plan.q[q0 + n];
      ip->q_first[groups] = n;
      ip->n_com[groups] = q.n_com;
      ip->entry_base[groups] = q.base;
      ip->nvis[groups] = q.len;
      for (int j = 0; j < size; ++j) ip->ents[n + j] = plan.q[q0 + n + j].ents;
      const int64_t lead = (mx && q.len > 0) ? (q.base & (tile - 1)) : 0;
      ip->tile_prefix[groups + 1] =
          ip->tile_prefix[groups] + (int32_t)((q.len + lead + tile - 1) / tile);
      n += size;
      ++groups;
      done += size;
    }
    ip->q_first[groups] = n;
    if (n == 0) break;
    ip->w = w + q0 * kIdxHeads;
    ip->scores = scores + q0 * ld;
    ip->ld = ld;
    ip->key_hist = key_hist ? key_hist + q0 * kKeyHistBinsHost : nullptr;
    ip->err = c->d_err;
    ip->nq = n;
    ip->qpg = qpg;
    ip->n_groups = groups;
    ip->tile_keys = tile;
    ip->ratio = c->cfg.ratio;
    ip->wait_cycles = c->wait_cycles;
    ip->inject = c->inject;
    const uint16_t* qn = qb + q0 * kIdxHeads * kIdxDim;
    const int tiles = ip->tile_prefix[groups];
    q0 += n;
    if (tiles == 0) continue;
    const int grid = std::min(c->index_sms, tiles);
    cudaError_t e;
    if (mx) {
      ip->idx_codes = c->idx_codes;
      ip->idx_scales = c->idx_scales;
      ip->idx_total = c->total;
      ip->q_idx = qn;
      e = launch_index_fp4_tree(*ip, c->tm_kq, grid, S(stream));
    } else {
      CUtensorMap tm_q;
      if (!make_map(&tm_q, qn, (uint64_t)n * kIdxHeads, kIdxDim, 64, 32 * qpg)) {
        st = CSA2_ERR_CUDA;
        break;
      }
      e = launch_index_tree(*ip, c->tm_k, tm_q, grid, S(stream));
    }
    if (e != cudaSuccess) st = CSA2_ERR_CUDA;
  }
  delete ip;
  return st;
}

}  // namespace

extern "C" {

csa2_status_t csa2_tree_paths(int32_t n_draft, const int32_t* parent, int32_t* depth,
                              uint64_t* path) {
  CSA2_RANGE();
  if (n_draft < 0) return CSA2_ERR_INVALID_ARG;
  if (n_draft > CSA2_MAX_DRAFT) return CSA2_ERR_UNSUPPORTED;
  if (n_draft == 0) return CSA2_OK;
  if (!parent) return CSA2_ERR_INVALID_ARG;
  int32_t d[CSA2_MAX_DRAFT];
  uint64_t pt[CSA2_MAX_DRAFT];
  if (!tree_paths(n_draft, parent, d, pt)) return CSA2_ERR_INVALID_ARG;
  if (depth) std::memcpy(depth, d, sizeof(int32_t) * n_draft);
  if (path) std::memcpy(path, pt, sizeof(uint64_t) * n_draft);
  return CSA2_OK;
}

csa2_status_t csa2_index_scores_tree(const csa2_cache_t* c, const csa2_tree_t* tree,
                                     const void* q_idx, const float* w, float* scores, int64_t ld,
                                     uint32_t* key_hist, csa2_stream_t stream) {
  CSA2_RANGE();
  TreePlan plan;
  csa2_status_t st = plan_tree(c, tree, &plan);
  if (st != CSA2_OK || plan.nq == 0) return st;
  if (!q_idx || !w || !scores || !aligned16(q_idx) || !aligned16(w) || !aligned16(scores) ||
      ld % 4 != 0 || (key_hist && !aligned16(key_hist)))
    return CSA2_ERR_INVALID_ARG;
  if (key_hist && c->cfg.idx_layout == CSA2_IDX_MXFP4) return CSA2_ERR_UNSUPPORTED;
  for (int64_t i = 0; i < plan.nq; ++i)
    if (tree_columns(plan.q[i]) > ld) return CSA2_ERR_CAPACITY;
  return run_index_tree(c, tree, plan, q_idx, w, scores, ld, key_hist, stream);
}

csa2_status_t csa2_index_topk_tree(const csa2_cache_t* c, const csa2_tree_t* tree,
                                   const void* q_idx, const float* w, int32_t* topk_idx,
                                   float* topk_score, void* workspace, size_t ws_bytes,
                                   csa2_stream_t stream) {
  CSA2_RANGE();
  TreePlan plan;
  csa2_status_t st = plan_tree(c, tree, &plan);
  if (st != CSA2_OK || plan.nq == 0) return st;
  if (!q_idx || !w || !aligned16(q_idx) || !aligned16(w) || !topk_idx || !aligned16(topk_idx) ||
      !workspace || !aligned16(workspace))
    return CSA2_ERR_INVALID_ARG;
  const int64_t nq = plan.nq;
  if (ws_bytes < csa2_index_workspace_bytes(c, (int32_t)nq)) return CSA2_ERR_CAPACITY;
  const int64_t ld = score_ld(c->max_cap);
  const bool mx = c->cfg.idx_layout == CSA2_IDX_MXFP4;
  float* scores = static_cast<float*>(workspace);
  uint32_t* hist = reinterpret_cast<uint32_t*>(scores + nq * ld);
  uint32_t* seg_ws = hist + nq * kKeyHistBinsHost;
  // the histograms come from the bf16 indexer's epilogue, or, for trees of one
  // draft, from the decode indexer of either key format (the MXFP4 indexer's
  // shared memory has room for one query's, not for a group's four)
  uint32_t* key_hist = mx && plan.max_draft > 1 ? nullptr : hist;
  st = run_index_tree(c, tree, plan, q_idx, w, scores, ld, key_hist, stream);
  if (st != CSA2_OK) return st;
  TopkParams* tp = new (std::nothrow) TopkParams();
  TreeMapParams* mp = new (std::nothrow) TreeMapParams();
  if (!tp || !mp) { delete tp; delete mp; return CSA2_ERR_OOM; }
  const int k = c->cfg.topk;
  for (int64_t q0 = 0; q0 < nq && st == CSA2_OK; q0 += kTopkTab) {
    const int n = (int)std::min<int64_t>(kTopkTab, nq - q0);
    std::memset(tp, 0, sizeof(TopkParams));
    tp->scores = scores + q0 * ld;
    tp->ld = ld;
    tp->rows = n;
    tp->k = k;
    tp->idx_out = topk_idx + q0 * k;
    tp->score_out = topk_score ? topk_score + q0 * k : nullptr;
    tp->key_hist = key_hist ? key_hist + q0 * kKeyHistBinsHost : nullptr;
    const int n_seg = topk_segments(c->max_cap);
    const bool seg = key_hist && n_seg > 2 && n_seg <= 1024;
    tp->seg_ws = seg ? seg_ws + (size_t)q0 * topk_seg_bytes(1, c->max_cap) / sizeof(uint32_t)
                     : nullptr;
    tp->n_seg = seg ? n_seg : 0;
    tp->err = c->d_err;
    // columns of a path whose entries are the first drafts' are entries already
    bool map = false;
    mp->rows = n;
    mp->k = k;
    mp->idx = tp->idx_out;
    for (int i = 0; i < n; ++i) {
      const TreeQuery& q = plan.q[q0 + i];
      tp->n_valid[i] = tree_columns(q);
      mp->n_com[i] = q.n_com;
      mp->ents[i] = q.ents;
      map = map || (q.ents & (q.ents + 1)) != 0;
    }
    if (launch_topk(*tp, S(stream)) != cudaSuccess ||
        (map && launch_tree_map(*mp, S(stream)) != cudaSuccess))
      st = CSA2_ERR_CUDA;
  }
  delete tp;
  delete mp;
  return st;
}

csa2_status_t csa2_sparse_attn_tree(const csa2_cache_t* c, const csa2_tree_t* tree,
                                    int32_t n_layers, const csa2_tree_layer_t* layers,
                                    const int32_t* swa_len, const int32_t* topk_idx, float scale,
                                    int32_t rope_out, double rope_base, void* workspace,
                                    size_t ws_bytes, csa2_stream_t stream) {
  CSA2_RANGE();
  TreePlan plan;
  csa2_status_t st = plan_tree(c, tree, &plan);
  if (st != CSA2_OK) return st;
  if (n_layers < 1 || n_layers > CSA2_MAX_ATTN_LAYERS || !layers) return CSA2_ERR_INVALID_ARG;
  if (rope_out && !(rope_base >= 0.0 && std::isfinite(rope_base))) return CSA2_ERR_INVALID_ARG;
  const int W = c->cfg.swa;
  for (int i = 0; swa_len && i < tree->n_seqs; ++i)
    if (swa_len[i] < 0 || swa_len[i] > W || swa_len[i] > tree->pos0[i]) return CSA2_ERR_INVALID_ARG;
  const int64_t nq = plan.nq;
  if (nq == 0) return CSA2_OK;
  if (!topk_idx || !aligned16(topk_idx) || (workspace && !aligned16(workspace)))
    return CSA2_ERR_INVALID_ARG;
  auto off16 = [](const void* x) { return !x || !aligned16(x); };
  for (int l = 0; l < n_layers; ++l) {
    const csa2_tree_layer_t& y = layers[l];
    if (off16(y.q) || off16(y.out) || (y.lse && !aligned16(y.lse))) return CSA2_ERR_INVALID_ARG;
    if (W == 0) continue;
    if (y.swa_codes || y.swa_rope || y.swa_scales || y.draft_codes || y.draft_rope ||
        y.draft_scales) {
      if (off16(y.swa_codes) || off16(y.swa_rope) || off16(y.draft_codes) ||
          off16(y.draft_rope) || !y.swa_scales || !y.draft_scales ||
          (reinterpret_cast<uintptr_t>(y.swa_scales) & 7u) ||
          (reinterpret_cast<uintptr_t>(y.draft_scales) & 7u))
        return CSA2_ERR_INVALID_ARG;
    } else if (off16(y.swa_kv) || off16(y.draft_kv)) {
      return CSA2_ERR_INVALID_ARG;
    }
  }
  const int H = c->cfg.n_heads, k = c->cfg.topk, G = H / kAttnHeadGroup;
  TreeAttnParams* p = new (std::nothrow) TreeAttnParams();
  AttnMaps* maps = new (std::nothrow) AttnMaps();
  if (!p || !maps) { delete p; delete maps; return CSA2_ERR_OOM; }
  for (int64_t q0 = 0; q0 < nq && st == CSA2_OK; q0 += kMaxTreeQueries) {
    const int n = (int)std::min<int64_t>(kMaxTreeQueries, nq - q0);
    std::memset(p, 0, sizeof(TreeAttnParams));
    p->topk_idx = topk_idx + q0 * k;
    p->codes = c->codes;
    p->scales = c->scales;
    p->n_layers = n_layers;
    p->err = c->d_err;
    p->nq = n;
    p->n_heads = H;
    p->topk = k;
    p->swa = W;
    p->layout = c->cfg.layout;
    p->scale = scale;
    p->scale_log2 = scale * 1.4426950408889634f;
    // as in decode: two CTAs per (query, head group) while the pairs fit the
    // SMs in one wave
    p->splits = workspace && ws_bytes >= kAttnSplitToken &&
                        2 * (int64_t)n_layers * n * G <= c->num_sms
                    ? 2
                    : 1;
    p->wait_cycles = c->wait_cycles;
    if (rope_out) {
      p->rope_out = 1;
      const double base = rope_base > 0.0 ? rope_base : 10000.0;
      for (int t = 0; t < 32; ++t) p->rope_theta[t] = std::pow(base, -(double)t / 32.0);
    }
    for (int i = 0; i < n; ++i) {
      TreeQuery& q = p->tq[i];
      q = plan.q[q0 + i];
      // the window: the deepest W drafts of the path, then committed rows
      // back to W rows in all
      const int s = q.win_row;
      while (__builtin_popcountll(q.rows) > W) q.rows &= q.rows - 1;
      const int have = swa_len ? swa_len[s] : (int)std::min<int64_t>(W, tree->pos0[s]);
      q.win_n = std::max(0, std::min(have, W - (int)__builtin_popcountll(q.rows)));
      q.win_row = s * W + have - q.win_n;
    }
    for (int l = 0; l < n_layers && st == CSA2_OK; ++l) {
      const csa2_tree_layer_t& y = layers[l];
      AttnLayer& ly = p->layer[l];
      ly.out = static_cast<uint16_t*>(y.out) + q0 * H * kHeadDim;
      ly.lse = y.lse ? y.lse + q0 * H : nullptr;
      ly.sink = y.sink;
      TreeLayer& tl = p->tree[l];
      const uint16_t* qb = static_cast<const uint16_t*>(y.q) + q0 * H * kHeadDim;
      if (!make_map(&maps->q[l], qb, (uint64_t)n * H, kHeadDim, 64, kAttnHeadGroup)) {
        st = CSA2_ERR_CUDA;
        break;
      }
      maps->swa[l] = maps->q[l];
      if (W == 0) continue;
      if (y.swa_codes) {
        ly.swa_codes = y.swa_codes;
        ly.swa_rope = static_cast<const uint16_t*>(y.swa_rope);
        ly.swa_scales = y.swa_scales;
        tl.draft_codes = y.draft_codes;
        tl.draft_rope = static_cast<const uint16_t*>(y.draft_rope);
        tl.draft_scales = y.draft_scales;
      } else {
        tl.draft = static_cast<const uint16_t*>(y.draft_kv);
        if (!make_map(&maps->swa[l], y.swa_kv, (uint64_t)tree->n_seqs * W, kHeadDim, 64, 128)) {
          st = CSA2_ERR_CUDA;
          break;
        }
      }
    }
    if (st == CSA2_OK && launch_attn_tree(*p, *maps, S(stream)) != cudaSuccess) st = CSA2_ERR_CUDA;
  }
  delete p;
  delete maps;
  return st;
}

csa2_status_t csa2_cache_accept_tree(csa2_cache_t* c, const csa2_tree_t* tree,
                                     const int32_t* accepted, csa2_stream_t stream) {
  CSA2_RANGE();
  TreePlan plan;
  csa2_status_t st = plan_tree(c, tree, &plan);
  if (st != CSA2_OK) return st;
  if (tree->n_seqs == 0) return CSA2_OK;
  if (!accepted) return CSA2_ERR_INVALID_ARG;
  for (int i = 0; i < tree->n_seqs; ++i)
    if (accepted[i] < -1 || accepted[i] >= tree->n_draft[i]) return CSA2_ERR_INVALID_ARG;
  AcceptParams* p = new (std::nothrow) AcceptParams();
  if (!p) return CSA2_ERR_OOM;
  int64_t first = 0;
  for (int i0 = 0; i0 < tree->n_seqs && st == CSA2_OK; i0 += kAcceptTab) {
    const int n = std::min(kAcceptTab, tree->n_seqs - i0);
    p->n_segs = n;
    p->scale_bytes = c->scale_bytes;
    p->codes = c->codes;
    p->scales = c->scales;
    p->idxk = c->idxk;
    p->idx_codes = c->idx_codes;
    p->idx_scales = c->idx_scales;
    p->d_len = c->d_len;
    for (int i = 0; i < n; ++i) {
      const int t = i0 + i, s = tree->seq_ids ? tree->seq_ids[t] : t;
      const int64_t n_com = tree->pos0[t] / c->cfg.ratio;
      const uint64_t keep = accepted[t] >= 0 ? plan.q[first + accepted[t]].ents : 0;
      first += tree->n_draft[t];
      p->seg[i] = {c->off[s] + n_com, keep, s, (int32_t)(n_com + __builtin_popcountll(keep))};
    }
    if (launch_accept(*p, S(stream)) != cudaSuccess) { st = CSA2_ERR_CUDA; break; }
    for (int i = 0; i < n; ++i) c->len[p->seg[i].seq] = p->seg[i].new_len;
  }
  delete p;
  return st;
}

// ---------------------------------------------------------------- norm + rotation
csa2_status_t csa2_norm_rope(int32_t n_parts, const csa2_norm_part_t* parts, float eps,
                             double rope_base, csa2_stream_t stream) {
  CSA2_RANGE();
  if (n_parts < 0 || n_parts > CSA2_MAX_NORM_PARTS || (n_parts > 0 && !parts))
    return CSA2_ERR_INVALID_ARG;
  if (!(eps >= 1e-30f && eps <= 1.0f) || !(rope_base == 0.0 || rope_base >= 1.0) ||
      !std::isfinite(rope_base))
    return CSA2_ERR_INVALID_ARG;
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.eps = eps;
  const double base = rope_base > 0.0 ? rope_base : 10000.0;
  for (int i = 0; i < n_parts; ++i) {
    const csa2_norm_part_t& a = parts[i];
    if (a.n_tokens < 0 || a.n_heads < 1) return CSA2_ERR_INVALID_ARG;
    if (a.dim != 64 && a.dim != 128 && a.dim != 256 && a.dim != 512) return CSA2_ERR_UNSUPPORTED;
    if (a.rope_dim < 0 || a.rope_dim > a.dim || a.rope_dim % 8 != 0) return CSA2_ERR_INVALID_ARG;
    if (a.rope_dim > 2 * kNormMaxPairs) return CSA2_ERR_UNSUPPORTED;
    if ((a.x_fp32 != 0 && a.x_fp32 != 1) || (a.out_fp32 != 0 && a.out_fp32 != 1))
      return CSA2_ERR_INVALID_ARG;
    if (a.n_tokens == 0) continue;
    if (a.n_tokens > kNormMaxRows / a.n_heads) return CSA2_ERR_UNSUPPORTED;
    if (!a.x || !a.out || !aligned16(a.x) || !aligned16(a.out) ||
        (a.weight && !aligned16(a.weight)) || (a.rope_dim > 0 && !a.pos) ||
        (reinterpret_cast<uintptr_t>(a.pos) & 7u))
      return CSA2_ERR_INVALID_ARG;
    const int64_t xa = a.x_fp32 ? 4 : 8, oa = a.out_fp32 ? 4 : 8;   // elements of 16 bytes
    // the stride of an axis of one is not used
    if ((a.n_tokens > 1 && (a.x_token_stride % xa || a.out_token_stride % oa)) ||
        (a.n_heads > 1 && (a.x_head_stride % xa || a.out_head_stride % oa)))
      return CSA2_ERR_INVALID_ARG;
    // strides that lay two heads of the output over each other
    const int64_t ot = std::llabs(a.out_token_stride), oh = std::llabs(a.out_head_stride);
    if ((a.n_tokens > 1 && ot < a.dim) || (a.n_heads > 1 && oh < a.dim) ||
        (a.n_tokens > 1 && a.n_heads > 1 && ot == oh))
      return CSA2_ERR_INVALID_ARG;
    NormPart& d = p.part[p.n_parts];
    d.x = a.x;
    d.out = a.out;
    d.weight = a.weight;
    d.pos = a.pos;
    d.n_tokens = a.n_tokens;
    d.n_heads = a.n_heads;
    d.dim = a.dim;
    d.rope_dim = a.rope_dim;
    d.norm = a.norm;
    d.x_fp32 = a.x_fp32;
    d.out_fp32 = a.out_fp32;
    d.x_token = a.x_token_stride;
    d.x_head = a.x_head_stride;
    d.out_token = a.out_token_stride;
    d.out_head = a.out_head_stride;
    // parts of one rotated width share a row of frequencies
    int row = 0;
    while (row < p.n_parts && p.part[row].rope_dim != a.rope_dim) ++row;
    d.rope_table = row;
    if (row == p.n_parts)
      for (int t = 0; t < a.rope_dim / 2; ++t) {
        // 2^64 * base^(-2t / rope_dim) / (2 pi), below one turn as base >= 1
        const double f = std::pow(base, -2.0 * t / a.rope_dim) * 0.15915494309189535;
        p.turns[row][t] = (uint64_t)(f * 18446744073709551616.0);
      }
    ++p.n_parts;
  }
  if (p.n_parts == 0) return CSA2_OK;
  return cuda_status(launch_norm_rope(p, S(stream)));
}

}  // extern "C"

namespace {
// Reads and clears a sticky error word (synchronises the stream).
csa2_status_t read_error_word(uint32_t* d_err, csa2_stream_t stream, int32_t* device_status) {
  uint32_t word = 0;
  if (cudaMemcpyAsync(&word, d_err, sizeof(word), cudaMemcpyDeviceToHost, S(stream)) !=
          cudaSuccess ||
      cudaStreamSynchronize(S(stream)) != cudaSuccess)
    return CSA2_ERR_CUDA;
  if (word && cudaMemsetAsync(d_err, 0, sizeof(uint32_t), S(stream)) != cudaSuccess)
    return CSA2_ERR_CUDA;
  *device_status = (word & kErrTimeoutBit) ? CSA2_ERR_TIMEOUT
                   : (word & kErrIndexBit) ? CSA2_ERR_DEVICE
                                           : CSA2_OK;
  return CSA2_OK;
}
}  // namespace

extern "C" {

csa2_status_t csa2_swa_fp8_quantise(int64_t n_rows, const void* rows, uint8_t* codes, void* rope,
                                    uint8_t* scales, csa2_stream_t stream) {
  CSA2_RANGE();
  if (n_rows < 0) return CSA2_ERR_INVALID_ARG;
  if (n_rows == 0) return CSA2_OK;
  if (!rows || !codes || !rope || !scales || !aligned16(rows) || !aligned16(codes) ||
      !aligned16(rope) || (reinterpret_cast<uintptr_t>(scales) & 7u))
    return CSA2_ERR_INVALID_ARG;
  return cuda_status(launch_swa_fp8(static_cast<const uint16_t*>(rows), n_rows, codes,
                                    static_cast<uint16_t*>(rope), scales, S(stream)));
}

csa2_status_t csa2_get_device_error(const csa2_cache_t* c, csa2_stream_t stream,
                                    int32_t* device_status) {
  CSA2_RANGE();
  if (!c || !device_status) return CSA2_ERR_INVALID_ARG;
  return read_error_word(c->d_err, stream, device_status);
}

}  // extern "C"

// ---------------------------------------------------------------- window rows in a cache
namespace {

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

// The arrays of a cache, checked.
csa2_status_t window_rows(const csa2_window_t* w, WinRows* r) {
  if (!w || w->n_seqs < 0 || w->swa < 1 || w->n_first < 0 || (w->fp8 != 0 && w->fp8 != 1))
    return CSA2_ERR_INVALID_ARG;
  if (w->swa > 128 || w->n_first > CSA2_MAX_FIRST ||
      (int64_t)w->n_seqs * (w->swa + w->n_first) > (int64_t)1 << 31)
    return CSA2_ERR_UNSUPPORTED;
  std::memset(r, 0, sizeof(*r));
  r->n_seqs = w->n_seqs;
  r->swa = w->swa;
  r->n_first = w->n_first;
  r->fp8 = w->fp8;
  r->pos = w->pos;
  r->err = w->error;
  if (w->fp8) {
    r->codes = w->codes;
    r->rope = static_cast<uint16_t*>(w->rope);
    r->scales = w->scales;
  } else {
    r->rows = static_cast<uint16_t*>(w->rows);
  }
  if (w->n_seqs == 0) return CSA2_OK;
  if (!w->pos || !aligned16(w->pos) || (reinterpret_cast<uintptr_t>(w->error) & 3u))
    return CSA2_ERR_INVALID_ARG;
  const bool ok = w->fp8 ? r->codes && r->rope && r->scales && aligned16(r->codes) &&
                               aligned16(r->rope) && aligned8(r->scales)
                         : r->rows && aligned16(r->rows);
  return ok ? CSA2_OK : CSA2_ERR_INVALID_ARG;
}

// Sequences of a call's segments: in range, and (once) no two alike.
csa2_status_t check_sequences(const csa2_window_t* w, int32_t n, const int32_t* ids, bool once) {
  if (!ids) return n <= w->n_seqs ? CSA2_OK : CSA2_ERR_INVALID_ARG;
  if (once && n > w->n_seqs) return CSA2_ERR_INVALID_ARG;
  std::unique_ptr<uint8_t[]> seen;
  if (once) {
    seen.reset(new (std::nothrow) uint8_t[(size_t)w->n_seqs / 8 + 1]());
    if (!seen) return CSA2_ERR_OOM;
  }
  for (int32_t i = 0; i < n; ++i) {
    const int32_t s = ids[i];
    if (s < 0 || s >= w->n_seqs) return CSA2_ERR_INVALID_ARG;
    if (!once) continue;
    if ((seen[s >> 3] >> (s & 7)) & 1u) return CSA2_ERR_INVALID_ARG;
    seen[s >> 3] |= (uint8_t)(1u << (s & 7));
  }
  return CSA2_OK;
}

// Rows of drafts in the cache's form.
csa2_status_t draft_rows(const csa2_window_t* w, const void* kv, const uint8_t* codes,
                         const void* rope, const uint8_t* scales, WinDrafts* d) {
  *d = {};
  if (w->fp8) {
    if (!codes || !rope || !scales || !aligned16(codes) || !aligned16(rope) || !aligned8(scales))
      return CSA2_ERR_INVALID_ARG;
    d->codes = codes;
    d->rope = static_cast<const uint16_t*>(rope);
    d->scales = scales;
  } else {
    if (!kv || !aligned16(kv)) return CSA2_ERR_INVALID_ARG;
    d->rows = static_cast<const uint16_t*>(kv);
  }
  return CSA2_OK;
}
WinDrafts drafts_from(WinDrafts d, int64_t row) {
  if (d.rows) d.rows += row * kHeadDim;
  if (d.codes) d.codes += row * 448;
  if (d.rope) d.rope += row * 64;
  if (d.scales) d.scales += row * 8;
  return d;
}

// Checks a tree's own numbers; `w`: against the sequences of a cache, too.
// *n_queries: its drafts; their paths into *paths.
csa2_status_t check_tree(const csa2_tree_t* t, const csa2_window_t* w, int64_t* n_queries,
                         std::unique_ptr<uint64_t[]>* paths) {
  if (!t || t->n_seqs < 0) return CSA2_ERR_INVALID_ARG;
  *n_queries = 0;
  if (t->n_seqs == 0) return CSA2_OK;
  if (!t->n_draft || (w && !t->pos0)) return CSA2_ERR_INVALID_ARG;
  if (w) {
    const csa2_status_t st = check_sequences(w, t->n_seqs, t->seq_ids, true);
    if (st != CSA2_OK) return st;
  }
  for (int i = 0; i < t->n_seqs; ++i) {
    if (t->n_draft[i] < 0) return CSA2_ERR_INVALID_ARG;
    if (w && (t->pos0[i] < 0 || t->pos0[i] > INT64_MAX - CSA2_MAX_DRAFT))
      return CSA2_ERR_INVALID_ARG;
    if (t->n_draft[i] > CSA2_MAX_DRAFT) return CSA2_ERR_UNSUPPORTED;
    *n_queries += t->n_draft[i];
  }
  if (*n_queries > INT32_MAX) return CSA2_ERR_UNSUPPORTED;
  if (*n_queries > 0 && !t->parent) return CSA2_ERR_INVALID_ARG;
  if (paths) {
    paths->reset(new (std::nothrow) uint64_t[(size_t)std::max<int64_t>(*n_queries, 1)]);
    if (!*paths) return CSA2_ERR_OOM;
  }
  int64_t first = 0;
  for (int i = 0; i < t->n_seqs; ++i) {
    int32_t depth[CSA2_MAX_DRAFT];
    uint64_t path[CSA2_MAX_DRAFT];
    if (!tree_paths(t->n_draft[i], t->parent ? t->parent + first : nullptr, depth, path))
      return CSA2_ERR_INVALID_ARG;
    if (paths) std::copy(path, path + t->n_draft[i], paths->get() + first);
    first += t->n_draft[i];
  }
  return CSA2_OK;
}

// How many drafts the deeper of two paths has that the other has not.
int path_more(uint64_t a, uint64_t b) {
  if (__builtin_popcountll(a) > __builtin_popcountll(b)) std::swap(a, b);
  return __builtin_popcountll(b & ~a);
}

// A tree's drafts branch by branch: each before its children, a child's whole
// branch before the next child's.
void branch_order(int n, const int32_t* parent, int* order) {
  int child[CSA2_MAX_DRAFT + 1], next[CSA2_MAX_DRAFT];   // [0]: of the root
  std::fill(child, child + n + 1, -1);
  for (int t = n - 1; t >= 0; --t) {
    next[t] = child[parent[t] + 1];
    child[parent[t] + 1] = t;
  }
  int at = n > 0 ? child[0] : -1;
  for (int k = 0; k < n; ++k) {
    order[k] = at;
    if (child[at + 1] >= 0) {
      at = child[at + 1];
      continue;
    }
    while (at >= 0 && next[at] < 0) at = parent[at];
    if (at >= 0) at = next[at];
  }
}

// Bytes that a call reads or writes (none where p is NULL).
struct Bytes {
  const void* p;
  int64_t n;
};
// Whether nothing that is written lies over what is read, or over what else is written:
// CTAs store outputs while others have yet to load.
bool apart(std::initializer_list<Bytes> written, std::initializer_list<Bytes> read) {
  auto over = [](const Bytes& a, const Bytes& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.n > 0 && b.n > 0 && (x < y ? y - x < (uintptr_t)a.n : x - y < (uintptr_t)b.n);
  };
  for (const Bytes* a = written.begin(); a != written.end(); ++a) {
    for (const Bytes& b : read)
      if (over(*a, b)) return false;
    for (const Bytes* b = a + 1; b != written.end(); ++b)
      if (over(*a, *b)) return false;
  }
  return true;
}
// The same for the outputs of an attention over a cache and drafts.
bool apart_attn(const WinRows& w, const WinDrafts& d, int64_t nq, int32_t n_heads, const void* q,
                const void* out, const WinAttnCommon& p) {
  const int64_t n = (int64_t)w.n_seqs * (w.swa + w.n_first), size = nq * n_heads * kHeadDim * 2;
  return apart({{out, size}, {p.lse, nq * n_heads * 4}},
               {{q, size}, {p.sink, n_heads * 4},
                {w.rows, n * kHeadDim * 2}, {w.codes, n * 448}, {w.rope, n * 128}, {w.scales, n * 8},
                {w.pos, n * 8},
                {d.rows, nq * kHeadDim * 2}, {d.codes, nq * 448}, {d.rope, nq * 128}, {d.scales, nq * 8}});
}

// What the three attention calls share.
csa2_status_t window_attn_common(int32_t n_heads, float scale, const csa2_window_opts_t* o,
                                 WinAttnCommon* p) {
  if (!std::isfinite(scale)) return CSA2_ERR_INVALID_ARG;
  if (n_heads != 64 && n_heads != 128) return CSA2_ERR_UNSUPPORTED;
  p->n_heads = n_heads;
  p->scale_log2 = scale * 1.4426950408889634f;
  p->wait_cycles = kWaitCycles;
  if (!o) return CSA2_OK;
  if ((o->rope_out != 0 && o->rope_out != 1) || (o->sink && !aligned16(o->sink)) ||
      (o->lse && !aligned16(o->lse)) || o->wait_cycles < 0 || o->withhold < 0 ||
      (reinterpret_cast<uintptr_t>(o->error) & 3u))
    return CSA2_ERR_INVALID_ARG;
  if (o->wait_cycles) p->wait_cycles = o->wait_cycles;
  p->withhold = o->withhold;
  p->sink = o->sink;
  p->lse = o->lse;
  if (o->rope_out) {
    if (!(o->rope_base == 0.0 || o->rope_base >= 1.0) || !std::isfinite(o->rope_base))
      return CSA2_ERR_INVALID_ARG;
    p->rope_out = 1;
    const double base = o->rope_base > 0.0 ? o->rope_base : 10000.0;
    for (int t = 0; t < 32; ++t)
      p->turns[t] = (uint64_t)(std::pow(base, -t / 32.0) * 0.15915494309189535 * 18446744073709551616.0);
  }
  return CSA2_OK;
}

bool sm_count(int* n) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess &&
         cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
}

// Queries [n * n_heads, 512] as 64-row boxes of 64 channels.
bool window_map(const void* q, int64_t n, int32_t n_heads, CUtensorMap* m) {
  return make_map(m, q, (uint64_t)n * n_heads, kHeadDim, 64, 64);
}

constexpr int32_t kWinRowLimit = INT32_MAX / 128;   // queries: rows of a map count in int32

}  // namespace

extern "C" {

csa2_status_t csa2_window_reset(const csa2_window_t* w, int32_t seq, csa2_stream_t stream) {
  CSA2_RANGE();
  WinRows r;
  const csa2_status_t st = window_rows(w, &r);
  if (st != CSA2_OK) return st;
  if (seq < -1 || seq >= w->n_seqs) return CSA2_ERR_INVALID_ARG;
  const size_t W = (size_t)w->swa, F = (size_t)w->n_first, n = (size_t)w->n_seqs;
  cudaError_t e = cudaSuccess;
  if (seq < 0) {
    if (n) e = cudaMemsetAsync(r.pos, 0xFF, n * (W + F) * 8, S(stream));
    if (e == cudaSuccess && r.err) e = cudaMemsetAsync(r.err, 0, sizeof(uint32_t), S(stream));
  } else {
    e = cudaMemsetAsync(r.pos + seq * W, 0xFF, W * 8, S(stream));
    if (e == cudaSuccess && F)
      e = cudaMemsetAsync(r.pos + n * W + seq * F, 0xFF, F * 8, S(stream));
  }
  return cuda_status(e);
}

csa2_status_t csa2_window_append(const csa2_window_t* w, int32_t n_segs, const int32_t* seq_ids,
                                 const int32_t* n_rows, const int64_t* pos0, const void* rows,
                                 void* rounded, csa2_stream_t stream) {
  CSA2_RANGE();
  WinRows r;
  csa2_status_t st = window_rows(w, &r);
  if (st != CSA2_OK) return st;
  if (n_segs < 0) return CSA2_ERR_INVALID_ARG;
  st = check_sequences(w, n_segs, seq_ids, true);
  if (st != CSA2_OK) return st;
  int64_t total = n_rows ? 0 : n_segs;
  for (int32_t i = 0; n_rows && i < n_segs; ++i) {
    if (n_rows[i] < 0) return CSA2_ERR_INVALID_ARG;
    total += n_rows[i];
  }
  if (total > INT32_MAX) return CSA2_ERR_UNSUPPORTED;
  if (total == 0) return CSA2_OK;
  if (!pos0 || !rows || !aligned8(pos0) || !aligned16(rows) || (rounded && !aligned16(rounded)))
    return CSA2_ERR_INVALID_ARG;
  // in place, or apart: rows are read by the warps that round them
  const uintptr_t from = reinterpret_cast<uintptr_t>(rows), to = reinterpret_cast<uintptr_t>(rounded);
  if (rounded && to != from && (to < from ? from - to : to - from) < (uintptr_t)total * kHeadDim * 2)
    return CSA2_ERR_INVALID_ARG;
  WinAppendParams* p = new (std::nothrow) WinAppendParams();
  if (!p) return CSA2_ERR_OOM;
  p->w = r;
  p->identity = !seq_ids && !n_rows;
  int64_t row = 0;
  for (int32_t i = 0; i < n_segs && st == CSA2_OK;) {
    const int32_t n = p->identity ? n_segs : std::min(kWinSegs, n_segs - i);
    p->pos0 = pos0 + i;
    p->rows = static_cast<const uint16_t*>(rows) + row * kHeadDim;
    p->rounded = rounded ? static_cast<uint16_t*>(rounded) + row * kHeadDim : nullptr;
    p->n_segs = n;
    p->seq0 = i;
    if (p->identity) {
      p->n_rows = n;
    } else {
      p->first[0] = 0;
      for (int32_t k = 0; k < n; ++k) {
        p->first[k + 1] = p->first[k] + (n_rows ? n_rows[i + k] : 1);
        p->seq[k] = seq_ids ? seq_ids[i + k] : i + k;
      }
      p->n_rows = p->first[n];
    }
    if (p->n_rows > 0) st = cuda_status(launch_window_append(*p, S(stream)));
    row += p->n_rows;
    i += n;
  }
  delete p;
  return st;
}

csa2_status_t csa2_window_read(const csa2_window_t* w, int32_t n_segs, const int32_t* seq_ids,
                               const int64_t* end, int32_t n_rows, void* out, uint8_t* codes,
                               void* rope, uint8_t* scales, void* first, csa2_stream_t stream) {
  CSA2_RANGE();
  WinRows r;
  csa2_status_t st = window_rows(w, &r);
  if (st != CSA2_OK) return st;
  if (n_segs < 0 || n_rows < 1 || n_rows > w->swa) return CSA2_ERR_INVALID_ARG;
  st = check_sequences(w, n_segs, seq_ids, false);
  if (st != CSA2_OK) return st;
  const bool fp8 = codes || rope || scales;
  if (fp8 && (out || !w->fp8 || !codes || !rope || !scales || !aligned16(codes) ||
              !aligned16(rope) || !aligned8(scales)))
    return CSA2_ERR_INVALID_ARG;
  if (n_segs == 0) return CSA2_OK;
  if ((!fp8 && (!out || !aligned16(out))) || !end || !aligned8(end) || (first && !aligned16(first)))
    return CSA2_ERR_INVALID_ARG;
  WinReadParams* p = new (std::nothrow) WinReadParams();
  if (!p) return CSA2_ERR_OOM;
  p->w = r;
  p->n_rows = n_rows;
  p->identity = !seq_ids;
  for (int32_t i = 0; i < n_segs && st == CSA2_OK;) {
    const int32_t n = p->identity ? n_segs : std::min(2 * kWinSegs, n_segs - i);
    const int64_t at = (int64_t)i * n_rows;
    p->end = end + i;
    p->out = out ? static_cast<uint16_t*>(out) + at * kHeadDim : nullptr;
    p->codes = fp8 ? codes + at * 448 : nullptr;
    p->rope = fp8 ? static_cast<uint16_t*>(rope) + at * 64 : nullptr;
    p->scales = fp8 ? scales + at * 8 : nullptr;
    p->first = first && w->n_first
                   ? static_cast<uint16_t*>(first) + (int64_t)i * w->n_first * kHeadDim
                   : nullptr;
    p->n_segs = n;
    p->seq0 = i;
    if (seq_ids) std::copy(seq_ids + i, seq_ids + i + n, p->seq);
    st = cuda_status(launch_window_read(*p, S(stream)));
    i += n;
  }
  delete p;
  return st;
}

csa2_status_t csa2_window_accept_tree(const csa2_window_t* w, const csa2_tree_t* t,
                                      const int32_t* accepted, const void* draft_kv,
                                      const uint8_t* draft_codes, const void* draft_rope,
                                      const uint8_t* draft_scales, csa2_stream_t stream) {
  CSA2_RANGE();
  WinRows r;
  csa2_status_t st = window_rows(w, &r);
  int64_t nq = 0;
  if (st == CSA2_OK) st = check_tree(t, w, &nq, nullptr);
  if (st != CSA2_OK || nq == 0) return st;
  WinDrafts d;
  st = draft_rows(w, draft_kv, draft_codes, draft_rope, draft_scales, &d);
  if (st != CSA2_OK) return st;
  if (!accepted || (reinterpret_cast<uintptr_t>(accepted) & 3u)) return CSA2_ERR_INVALID_ARG;
  WinAcceptParams* p = new (std::nothrow) WinAcceptParams();
  if (!p) return CSA2_ERR_OOM;
  int64_t row = 0;
  for (int32_t i = 0; i < t->n_seqs && st == CSA2_OK;) {
    p->w = r;
    p->d = drafts_from(d, row);
    p->accepted = accepted + i;
    p->n_trees = 0;
    p->first[0] = 0;
    const int64_t row0 = row;
    while (i < t->n_seqs && p->n_trees < kWinTrees &&
           p->first[p->n_trees] + t->n_draft[i] <= kWinDrafts) {
      const int k = p->n_trees++;
      p->pos0[k] = t->pos0[i];
      p->seq[k] = t->seq_ids ? t->seq_ids[i] : i;
      p->first[k + 1] = p->first[k] + t->n_draft[i];
      for (int j = 0; j < t->n_draft[i]; ++j)
        p->parent[p->first[k] + j] = (int8_t)t->parent[row + j];
      row += t->n_draft[i++];
    }
    if (row > row0) st = cuda_status(launch_window_accept(*p, S(stream)));
  }
  delete p;
  return st;
}

csa2_status_t csa2_window_attn_decode(const csa2_window_t* w, int32_t n_heads, int32_t nq,
                                      const int32_t* seq_ids, const void* q, const int64_t* pos,
                                      float scale, void* out, const csa2_window_opts_t* opts,
                                      csa2_stream_t stream) {
  CSA2_RANGE();
  WinRows r;
  csa2_status_t st = window_rows(w, &r);
  if (st != CSA2_OK) return st;
  if (nq < 0) return CSA2_ERR_INVALID_ARG;
  st = check_sequences(w, nq, seq_ids, false);
  if (st != CSA2_OK) return st;
  WinDecodeParams* p = new (std::nothrow) WinDecodeParams();
  if (!p) return CSA2_ERR_OOM;
  st = window_attn_common(n_heads, scale, opts, p);
  if (st == CSA2_OK && nq > kWinRowLimit) st = CSA2_ERR_UNSUPPORTED;
  if (st == CSA2_OK && nq > 0 &&
      (!q || !out || !pos || !aligned16(q) || !aligned16(out) || !aligned8(pos) ||
       !apart_attn(r, {}, nq, n_heads, q, out, *p) ||
       !apart({{out, (int64_t)nq * n_heads * kHeadDim * 2}, {p->lse, (int64_t)nq * n_heads * 4}},
              {{pos, (int64_t)nq * 8}})))
    st = CSA2_ERR_INVALID_ARG;
  int sms = 0;
  if (st == CSA2_OK && nq > 0 && !sm_count(&sms)) st = CSA2_ERR_CUDA;
  p->w = r;
  p->err = r.err;
  p->identity = !seq_ids;
  float* const lse = p->lse;
  for (int32_t i = 0; i < nq && st == CSA2_OK;) {
    const int32_t n = p->identity ? nq : std::min(kWinQueries, nq - i);
    const int64_t row = (int64_t)i * n_heads;
    p->nq = n;
    p->pos = pos + i;
    p->seq0 = i;
    if (seq_ids) std::copy(seq_ids + i, seq_ids + i + n, p->seq);
    p->lse = lse ? lse + row : nullptr;
    p->out = static_cast<uint16_t*>(out) + row * kHeadDim;
    CUtensorMap mq;
    if (!window_map(static_cast<const uint16_t*>(q) + row * kHeadDim, n, n_heads, &mq) ||
        launch_window_decode(*p, mq, sms, S(stream)) != cudaSuccess)
      st = CSA2_ERR_CUDA;
    i += n;
  }
  delete p;
  return st;
}

csa2_status_t csa2_window_attn_tree(const csa2_window_t* w, const csa2_tree_t* t, int32_t n_heads,
                                    const void* q, const void* draft_kv,
                                    const uint8_t* draft_codes, const void* draft_rope,
                                    const uint8_t* draft_scales, float scale, void* out,
                                    const csa2_window_opts_t* opts, csa2_stream_t stream) {
  CSA2_RANGE();
  WinRows r;
  csa2_status_t st = window_rows(w, &r);
  if (st != CSA2_OK) return st;
  int64_t nq = 0;
  std::unique_ptr<uint64_t[]> paths;
  st = check_tree(t, w, &nq, &paths);
  if (st != CSA2_OK) return st;
  WinTreeParams* p = new (std::nothrow) WinTreeParams();
  if (!p) return CSA2_ERR_OOM;
  st = window_attn_common(n_heads, scale, opts, p);
  if (st == CSA2_OK && nq > kWinRowLimit) st = CSA2_ERR_UNSUPPORTED;
  WinDrafts d = {};
  if (st == CSA2_OK && nq > 0) {
    st = draft_rows(w, draft_kv, draft_codes, draft_rope, draft_scales, &d);
    if (st == CSA2_OK && (!q || !out || !aligned16(q) || !aligned16(out) ||
                          !apart_attn(r, d, nq, n_heads, q, out, *p)))
      st = CSA2_ERR_INVALID_ARG;
  }
  int sms = 0;
  if (st == CSA2_OK && nq > 0 && !sm_count(&sms)) st = CSA2_ERR_CUDA;
  p->w = r;
  p->err = r.err;
  float* const lse = p->lse;
  int64_t row = 0;
  for (int32_t i = 0; i < t->n_seqs && st == CSA2_OK;) {
    // whole trees (of at most 64 drafts each) up to the tables' sizes
    p->d = drafts_from(d, row);
    p->nq = 0;
    p->n_items = 0;
    int k = 0;
    const int64_t row0 = row;
    for (; i < t->n_seqs && k < kWinTreeTrees && p->nq + t->n_draft[i] <= kWinTreeQueries; ++i, ++k) {
      p->pos0[k] = t->pos0[i];
      p->seq[k] = t->seq_ids ? t->seq_ids[i] : i;
      p->first[k] = p->nq;
      const uint64_t* path = &paths[(size_t)row];
      const int n = t->n_draft[i], first = p->nq;
      int order[CSA2_MAX_DRAFT];
      branch_order(n, t->parent + row, order);
      for (int j = 0; j < n; ++j) {
        // neighbours share an item of 128 heads if the deeper one's path has
        // few drafts that the other's has not
        const bool two = n_heads == 64 && j + 1 < n &&
                         path_more(path[order[j]], path[order[j + 1]]) <= kWinPairDrafts;
        p->item[p->n_items++] = (uint16_t)(p->nq | (two ? 0x8000 : 0));
        for (const int end = j + two; ; ++j) {
          p->query[p->nq] = (uint16_t)(first + order[j]);
          p->path[p->nq] = path[order[j]];
          p->tree[p->nq++] = (int16_t)k;
          if (j == end) break;
        }
      }
      row += t->n_draft[i];
    }
    if (p->nq == 0) continue;
    // The first item of a tree, and of a CTA, costs about half as much again (its rows
    // come out of the cache): CTAs at a tree's border get fewer.  In halves of an item.
    p->n_ctas = std::min({p->n_items, sms, kWinTreeCtas});
    int b = 0;
    for (int k = 0; k < p->n_items; ++k) {
      int64_t cost = 2 * k + p->tree[p->item[k] & 0x7FFF], all = 2 * p->n_items + p->tree[p->nq - 1] + 1;
      if (p->n_ctas == p->n_items) cost = k, all = p->n_items;   // one each
      while (b < p->n_ctas && cost * p->n_ctas >= b * all) p->start[b++] = (uint16_t)k;
    }
    while (b <= kWinTreeCtas) p->start[b++] = (uint16_t)p->n_items;
    const int64_t at = row0 * n_heads;
    p->lse = lse ? lse + at : nullptr;
    p->out = static_cast<uint16_t*>(out) + at * kHeadDim;
    CUtensorMap mq;
    if (!window_map(static_cast<const uint16_t*>(q) + at * kHeadDim, p->nq, n_heads, &mq) ||
        launch_window_tree(*p, mq, sms, S(stream)) != cudaSuccess)
      st = CSA2_ERR_CUDA;
  }
  delete p;
  return st;
}

csa2_status_t csa2_window_attn_prefill(int32_t n_heads, int32_t nq, int64_t pos0, const void* q,
                                       const void* rows, int64_t rows_pos0, int64_t n_rows,
                                       int32_t swa, const void* first, int32_t n_first, float scale,
                                       void* out, const csa2_window_opts_t* opts,
                                       csa2_stream_t stream) {
  CSA2_RANGE();
  if (nq < 0 || swa < 1 || n_first < 0 || pos0 < 0 || rows_pos0 < 0 || n_rows < 0)
    return CSA2_ERR_INVALID_ARG;
  if (swa > 128 || n_first > CSA2_MAX_FIRST) return CSA2_ERR_UNSUPPORTED;
  WinPrefillParams p;
  std::memset(&p, 0, sizeof(p));
  const csa2_status_t st = window_attn_common(n_heads, scale, opts, &p);
  if (st != CSA2_OK) return st;
  if (nq == 0) return CSA2_OK;
  if (nq > kWinRowLimit) return CSA2_ERR_UNSUPPORTED;
  if (pos0 > INT64_MAX - nq || rows_pos0 > pos0 || n_rows > INT64_MAX - rows_pos0 ||
      pos0 + nq > rows_pos0 + n_rows || !q || !rows || !out || !aligned16(q) || !aligned16(rows) ||
      !aligned16(out) || (first && !aligned16(first)) || (n_first > 0 && rows_pos0 > 0 && !first))
    return CSA2_ERR_INVALID_ARG;
  // rows that are loaded: the chunk's and its window's, in blocks of 8, and first tokens
  const int64_t size = (int64_t)nq * n_heads * kHeadDim * 2, row = kHeadDim * 2;
  const int64_t lo = std::max<int64_t>(pos0 - rows_pos0 - swa - 16, 0);
  const Bytes band = {reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(rows) + (uintptr_t)lo * row),
                      (pos0 - rows_pos0 - lo + nq + std::min<int64_t>(rows_pos0 + n_rows - pos0 - nq, 8)) * row};
  if (!apart({{out, size}, {p.lse, (int64_t)nq * n_heads * 4}},
             {{q, size}, {p.sink, n_heads * 4}, band, {rows, std::min<int64_t>(n_rows, n_first) * row},
              {first, n_first * row}}))
    return CSA2_ERR_INVALID_ARG;
  p.w.swa = swa;
  p.w.n_first = n_first;
  p.out = static_cast<uint16_t*>(out);
  p.err = opts ? opts->error : nullptr;
  p.nq = nq;
  p.band = static_cast<const uint16_t*>(rows);
  p.first = static_cast<const uint16_t*>(first);
  p.pos0 = pos0;
  p.band0 = rows_pos0;
  p.n_band = n_rows;
  int sms = 0;
  CUtensorMap mq;
  if (!sm_count(&sms) || !window_map(q, nq, n_heads, &mq)) return CSA2_ERR_CUDA;
  return cuda_status(launch_window_prefill(p, mq, sms, S(stream)));
}

csa2_status_t csa2_window_device_error(const csa2_window_t* w, csa2_stream_t stream,
                                       int32_t* device_status) {
  CSA2_RANGE();
  if (!w || !device_status || !w->error) return CSA2_ERR_INVALID_ARG;
  return read_error_word(w->error, stream, device_status);
}

// ---------------------------------------------------------------- verification of drafts
csa2_status_t csa2_verify_tree(const csa2_tree_t* t, const csa2_verify_t* v, csa2_stream_t stream) {
  CSA2_RANGE();
  int64_t nq = 0;
  csa2_status_t st = check_tree(t, nullptr, &nq, nullptr);
  if (st != CSA2_OK) return st;
  if (!v || v->vocab < 1 || v->ld < v->vocab || (v->fp32 != 0 && v->fp32 != 1))
    return CSA2_ERR_INVALID_ARG;
  if (v->vocab > 1 << 30) return CSA2_ERR_UNSUPPORTED;
  if (t->n_seqs == 0) return CSA2_OK;
  const uintptr_t el = v->fp32 ? 3u : 1u;
  auto off = [](const void* x, uintptr_t mask) { return (reinterpret_cast<uintptr_t>(x) & mask) != 0; };
  if (!v->accepted || !v->next_token || off(v->accepted, 3) || off(v->next_token, 3) ||
      off(v->target, el) || off(v->target_root, el) || off(v->draft, el) || off(v->draft_root, el) ||
      off(v->token, 3) || off(v->temperature, 3) || off(v->uniform, 3) || off(v->noise, 3))
    return CSA2_ERR_INVALID_ARG;
  if (nq > 0 && (!v->token || !v->target)) return CSA2_ERR_INVALID_ARG;
  if (v->temperature && ((nq > 0 && !v->uniform) || !v->noise || v->noise_ld < v->vocab))
    return CSA2_ERR_INVALID_ARG;
  // draft logits for every node with children, or for none
  if (v->draft_root ? !v->target_root || (nq > 0 && !v->draft)
                    : v->draft != nullptr && v->target_root != nullptr)
    return CSA2_ERR_INVALID_ARG;
  if (!v->target_root) {   // one root child at most: the token drawn before
    int64_t first = 0;
    for (int i = 0; i < t->n_seqs; ++i) {
      for (int j = 1; j < t->n_draft[i]; ++j)
        if (t->parent[first + j] < 0) return CSA2_ERR_INVALID_ARG;
      first += t->n_draft[i];
    }
  }
  int sms = 0;
  if (!sm_count(&sms)) return CSA2_ERR_CUDA;
  VerifyParams* p = new (std::nothrow) VerifyParams();
  if (!p) return CSA2_ERR_OOM;
  const int64_t bytes = v->fp32 ? 4 : 2;
  const int cluster = verify_cluster(t->n_seqs, v->vocab, sms);
  p->ld = v->ld;
  p->noise_ld = v->noise_ld;
  p->vocab = v->vocab;
  int64_t row = 0;
  auto rows_from = [&](const void* x, int64_t r) -> const void* {
    return x ? static_cast<const uint8_t*>(x) + r * v->ld * bytes : nullptr;
  };
  for (int32_t i = 0; i < t->n_seqs && st == CSA2_OK;) {
    p->token = v->token ? v->token + row : nullptr;
    p->uniform = v->uniform ? v->uniform + row : nullptr;
    p->target = rows_from(v->target, row);
    p->draft = rows_from(v->draft, row);
    p->root = rows_from(v->target_root, i);
    p->draft_root = rows_from(v->draft_root, i);
    p->temperature = v->temperature ? v->temperature + i : nullptr;
    p->noise = v->noise ? v->noise + i * v->noise_ld : nullptr;
    p->accepted = v->accepted + i;
    p->next_token = v->next_token + i;
    p->n_trees = 0;
    p->first[0] = 0;
    while (i < t->n_seqs && p->n_trees < kVerifyTrees &&
           p->first[p->n_trees] + t->n_draft[i] <= kVerifyDrafts) {
      const int k = p->n_trees++;
      p->first[k + 1] = p->first[k] + t->n_draft[i];
      for (int j = 0; j < t->n_draft[i]; ++j)
        p->parent[p->first[k] + j] = (int8_t)t->parent[row + j];
      row += t->n_draft[i++];
    }
    st = cuda_status(launch_verify(*p, v->fp32 != 0, cluster, S(stream)));
  }
  delete p;
  return st;
}

}  // extern "C"
