// csa2_kernels.h -- host-side launch interface between the C ABI layer
// (csa2_api.cu) and the kernel translation units.  Internal to the library.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace csa2 {

// Sticky device error word bits (see csa2_get_device_error).
constexpr uint32_t kErrTimeoutBit = 1u;
constexpr uint32_t kErrIndexBit = 2u;

// Launch attribute: programmatic stream serialisation (the kernel's launch
// overlaps the end of the previous kernel in the stream; the kernel waits for
// it with griddepcontrol.wait before its first global memory access).
inline cudaLaunchAttribute pdl_attribute() {
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

constexpr int kHeadDim = 512;     // main-KV latent / attention head dim
constexpr int kIdxDim = 128;      // indexer head dim
constexpr int kIdxHeads = 32;     // indexer heads
constexpr int kCodeBytes = kHeadDim / 2;
constexpr int kKeyHistBinsHost = 2048;   // score-key histogram bins (top 11 key bits)

// ---------------------------------------------------------------- append
constexpr int kMaxAppendSegs = 64;
struct AppendSeg {
  int64_t first;     // first output row of this segment within the launch
  int64_t src_row;   // first input entry row (entries mode) or entry-block row
  int64_t dst_row;   // first cache row
  int32_t seq;
  int32_t new_len;   // sequence length after the append
};
struct AppendParams {
  int32_t mode;      // 0 compress only, 1 append entries, 2 append tokens
  int32_t ratio;
  int32_t layout;    // 0 = L32_UE8M0, 1 = L16_E4M3
  int32_t dim;       // channels (compress-only may differ from kHeadDim)
  int32_t n_segs;
  int64_t rows;      // output rows in this launch
  AppendSeg seg[kMaxAppendSegs];
  const float* entries;
  const uint16_t* c_tok;
  const float* z_tok;
  const uint16_t* idx_k;
  float* entries_out;
  uint8_t* codes;
  uint8_t* scales;
  uint16_t* cache_idxk;
  int32_t idx_mxfp4;         // 1: indexer keys quantised to MXFP4 (codes + scales below)
  uint8_t* idx_codes;
  uint8_t* idx_scales;
  int32_t* d_len;
  int64_t total;             // cache rows (bounds checks of the debug build)
  uint32_t* err;             // nullable device error word
};
cudaError_t launch_append(const AppendParams& p, cudaStream_t s);

// ---------------------------------------------------------------- indexer
constexpr int kMaxIdxGroups = 1024;
// Fault injection for tests of the timeout path: the indexer's producer
// issues no key loads, so the MMA and epilogue waits run out with nothing in
// flight (no copy, no MMA).
constexpr int32_t kInjectNoKeyLoads = 1;
// ~2^31 cycles (about one second at GB300 clocks) before a wait gives up,
// unless the launch sets a limit of its own (csa2_cache_set_wait_limit).
constexpr long long kWaitCycles = 1ll << 31;
struct IndexParams {
  const float* w;          // [nq, 32]
  float* scores;           // [nq, ld]
  int64_t ld;
  uint32_t* key_hist;      // nullable [nq, 2048] score-key histogram (qpg == 1 only)
  int32_t score_bf16;      // 1: scores are stored as bf16 (uint16 [nq, ld], nearest even)
  const uint16_t* q_idx;     // MXFP4 keys (k_index_fp4): bf16 queries [nq, 32, 128]
  const uint8_t* idx_codes;  // MXFP4 keys (k_index_fp4): E2M1 codes [idx_total, 64]
  const uint8_t* idx_scales; // MXFP4 keys: UE8M0 scales [idx_total, 4]
  int64_t idx_total;         // MXFP4 keys: rows in the cache
  const int32_t* pool;     // nullable: pool mode, [nq, pool_blocks] block ids (-1 unused)
  int32_t pool_blocks;     // blocks per pool row (multiple of 16)
  uint32_t* err;
  int32_t nq;
  int32_t qpg;             // queries per group (1 decode, 8 prefill; MXFP4 keys: 4)
  int32_t n_groups;
  int32_t prefill;         // 1: visibility from positions
  int64_t pre_base;        // prefill: entry offset of the sequence
  int64_t pos0;            // prefill: position of query 0
  int32_t pre_len;         // prefill: entries in the sequence
  int32_t ratio;
  int64_t wait_cycles;     // bounded-wait limit in cycles (0: the default, ~2^31)
  int32_t inject;          // kInjectNoKeyLoads: the producer issues no key loads (tests)
  int32_t tile_prefix[kMaxIdxGroups + 1];  // cumulative tiles per group (128 entries; the
                                           // MXFP4 kernel: 256 for one query per group)
  int64_t entry_base[kMaxIdxGroups];       // decode: entry offset of the group's sequence
  int32_t nvis[kMaxIdxGroups];             // decode: visible entries of the group's query
};
// Trees of drafted tokens: a group is up to qpg consecutive queries of one
// sequence; tiles cover the sequence's committed entries and the drafts'
// entries after them.  Query q sees the committed entries (columns 0 ..
// n_com - 1 of its row) and the drafts' entries of its own path (bit e of
// ents[q]: entry n_com + e), which follow in order without gaps.  Tables of
// at most kMaxTreeQueries queries a launch, so that all of the parameters
// stay below 32764 bytes.
constexpr int kMaxTreeQueries = 512;
struct TreeIndexParams : IndexParams {
  int32_t q_first[kMaxTreeQueries + 1];  // first query of each group
  int32_t n_com[kMaxTreeQueries];        // committed entries of the group's sequence
  uint64_t ents[kMaxTreeQueries];        // per query: its path's entries
  int32_t tile_keys;                     // keys of a tile: 128 (bf16 keys), 256 or 512 (MXFP4 keys)
};
int index_smem_bytes(int qpg);
cudaError_t launch_index_tree(const TreeIndexParams& p, const CUtensorMap& tm_k,
                              const CUtensorMap& tm_q, int grid, cudaStream_t s);
cudaError_t launch_index(const IndexParams& p, const CUtensorMap& tm_k, const CUtensorMap& tm_q,
                         int grid, cudaStream_t s);
// MXFP4 keys (codes [idx_rows, 64], scales [idx_rows, 4], idx_rows a
// multiple of 512): tm_kq views the codes as aligned 128-key tiles in the
// permuted row order of the kernel (key 4 r + q of a tile in shared-memory
// row 32 q + r, 64-byte rows, 64-byte swizzle), tm_kc8 as [idx_total, 64]
// in boxes of 8 rows (pool blocks, 64-byte swizzle).  qpg is 1 (decode,
// pool mode) or 4 (prefill).  Decode tiles (no pool) are the aligned 512-key
// chunks: a sequence at key row off has ceil((n + off % 512) / 512) tiles;
// prefill tiles the aligned 128-key chunks, ceil((n + off % 128) / 128) per
// group.
int index_fp4_smem_bytes();
cudaError_t launch_index_fp4(const IndexParams& p, const CUtensorMap& tm_kq,
                             const CUtensorMap& tm_kc8, int grid, cudaStream_t s);
cudaError_t launch_index_fp4_tree(const TreeIndexParams& p, const CUtensorMap& tm_kq, int grid,
                                  cudaStream_t s);

// ---------------------------------------------------------------- trees of drafts
// Selected columns of the rows above back to entries: column c >= n_com of
// row r becomes entry n_com + (the (c - n_com)-th set bit of ents[r]).
constexpr int kTreeMapTab = 1024;
struct TreeMapParams {
  int32_t rows;   // <= kTreeMapTab
  int32_t k;
  int32_t* idx;   // [rows, k], rewritten
  int32_t n_com[kTreeMapTab];
  uint64_t ents[kTreeMapTab];
};
cudaError_t launch_tree_map(const TreeMapParams& p, cudaStream_t s);

// Accepted paths: of the drafts' entries at rows row0 .. of a sequence, those
// of `keep` (bit e: row row0 + e) move up to row0, row0 + 1, ...
constexpr int kAcceptTab = 512;
struct AcceptSeg {
  int64_t row0;
  uint64_t keep;
  int32_t seq;
  int32_t new_len;
};
struct AcceptParams {
  int32_t n_segs;       // <= kAcceptTab
  int32_t scale_bytes;  // 16 or 32 per entry
  uint8_t* codes;
  uint8_t* scales;
  uint16_t* idxk;       // bf16 indexer keys, or null: idx_codes and idx_scales
  uint8_t* idx_codes;
  uint8_t* idx_scales;
  int32_t* d_len;
  AcceptSeg seg[kAcceptTab];
};
cudaError_t launch_accept(const AcceptParams& p, cudaStream_t s);

// ---------------------------------------------------------------- norm + rotation
constexpr int kNormMaxParts = 8;
constexpr int kNormMaxPairs = 64;     // rotated channels / 2
constexpr int64_t kNormMaxRows = (int64_t)1 << 31;   // heads of a tensor: 256 GB of the narrowest
struct NormPart {
  const void* x;
  void* out;
  const float* weight;      // nullable [dim]
  const int64_t* pos;       // [n_tokens], null without rotation
  int64_t n_tokens;
  int64_t x_token, x_head, out_token, out_head;   // strides in elements
  int32_t n_heads;
  int32_t dim;              // 64, 128, 256 or 512
  int32_t rope_dim;         // rotated channels (the last of the head)
  int32_t norm;             // 0: no norm (weight still applies)
  int32_t x_fp32, out_fp32;
  int32_t rope_table;       // row of NormParams::turns
};
struct NormParams {
  NormPart part[kNormMaxParts];
  int64_t block0[kNormMaxParts + 1];   // first block of each part
  int32_t n_parts;
  float eps;
  // frequency of channel pair t in turns per position, as a 64-bit fraction:
  // base^(-2t / rope_dim) / (2 pi) * 2^64
  uint64_t turns[kNormMaxParts][kNormMaxPairs];
};
cudaError_t launch_norm_rope(const NormParams& p, cudaStream_t s);

// ---------------------------------------------------------------- HSI
constexpr int kHsiBlock = 8;   // positions per block of the candidate pool
struct HsiParams {
  int32_t rows;              // <= kHsiTab
  // block max: bmax[r, b] = max of scores[r, 8 b .. 8 b + 7] over the row's
  // n[r] positions, for b < ceil(n[r] / 8)
  const float* scores;
  int64_t ld;
  float* bmax;
  int64_t ld_b;
  // pool map: out[r, j] = pool[r, s / 8] * 8 + s % 8 for s = sel[r, j];
  // -1 for unused slots and for entries >= n[r]
  const int32_t* sel;
  int32_t k;
  const int32_t* pool;
  int32_t pool_blocks;
  int32_t* out;
  float* score_out;          // nullable: zeroed where out is -1
  uint32_t* err;             // nullable device error word (debug-build checks)
  int64_t n[1024];
};
constexpr int kHsiTab = 1024;
cudaError_t launch_block_max(const HsiParams& p, cudaStream_t s);
cudaError_t launch_pool_map(const HsiParams& p, cudaStream_t s);

// ---------------------------------------------------------------- top-k
constexpr int kTopkMaxRowsPerLaunch = 65535;
constexpr int kTopkTab = 1024;
struct TopkParams {
  const float* scores;       // row r at scores + r * ld
  int64_t ld;
  int32_t rows;
  int32_t k;
  const uint32_t* key_hist;  // nullable [rows, 2048] score-key histogram
  int32_t* idx_out;          // [rows, k]
  float* score_out;          // nullable [rows, k]
  int32_t formula;           // 1: n_valid(r) = min(len, (pos0 + r + 1) / ratio)
  int32_t pre_len;
  int32_t ratio;
  int64_t pos0;
  int32_t score_bf16;        // 1: scores are bf16 (uint16 [rows, ld])
  uint32_t* seg_ws;          // nullable: per-segment candidate buffers (see topk_seg_bytes)
  int32_t n_seg;             // segments per row when seg_ws is set
  uint32_t* err;             // nullable device error word (debug-build checks)
  int64_t n_valid[kTopkTab]; // formula == 0: per-row valid counts
};
// Segmented candidate compaction (rows with a score-key histogram): scratch
// bytes for `rows` rows of up to `max_valid` scores, and its segment count.
constexpr int kTopkSegLen = 8192;
int topk_segments(int64_t max_valid);
size_t topk_seg_bytes(int32_t rows, int64_t max_valid);
cudaError_t launch_topk(const TopkParams& p, cudaStream_t s);

// ---------------------------------------------------------------- attention
constexpr int kAttnTab = 1024;
constexpr int kAttnMaxLayers = 8;
// What differs between the layers of one readout launch (the layers of a
// group share the cache, the selection and the windows' geometry).
struct AttnLayer {
  uint16_t* out;             // bf16 [nq, n_heads, 512]
  float* lse;                // nullable [nq, n_heads]
  const float* sink;         // nullable [n_heads]: per-head sink logit z' (units of scale * q.kv)
  const uint8_t* swa_codes;  // FP8 window rows (nullable): E4M3 codes [rows, 448]
  const uint16_t* swa_rope;  //   bf16 RoPE channels [rows, 64]
  const uint8_t* swa_scales; //   UE8M0 scales [rows, 8]
};
// The layers' query rows and bf16 window rows as TMA tensor maps.
struct AttnMaps {
  CUtensorMap q[kAttnMaxLayers];
  CUtensorMap swa[kAttnMaxLayers];
};
struct AttnCommon {
  const int32_t* topk_idx;   // [nq, topk]
  const int32_t* swa_len;    // decode: nullable [nq]
  const uint8_t* codes;
  const uint8_t* scales;
  int32_t n_layers;          // layers of the launch; blocks are (layer, query, head group, split)
  int32_t splits;            // CTAs per (query, 64-head group): 1, or 2 (a cluster)
  uint32_t* err;
  int32_t nq;
  int32_t n_heads;
  int32_t topk;
  int32_t swa;               // window size W
  int32_t layout;
  float scale_log2;          // scale * log2(e)
  float scale;
  int32_t prefill;
  int64_t pre_base;          // prefill: entry offset of the sequence
  int32_t pre_len;           // prefill: entries in the sequence
  int64_t pos0;              // prefill: position of query 0
  int64_t swa_pos0;          // prefill: position of swa row 0
  const int64_t* rope_pos;   // decode: [nq] query positions for the output RoPE(-i)
  int32_t rope_out;          // 1: rotate the last 64 output channels by -position
  double rope_theta[32];     // RoPE frequencies base^(-2t/64) of the 32 channel pairs
  int64_t wait_cycles;       // bounded-wait limit in cycles (0: the default, ~2^31)
  AttnLayer layer[kAttnMaxLayers];
};
struct AttnParams : AttnCommon {
  int64_t q_base[kAttnTab];  // decode: entry offset of each query's sequence
  int32_t q_len[kAttnTab];   // decode: entries of each query's sequence
};
// Trees of drafted tokens: one record per query (at most kMaxTreeQueries a
// launch: the parameters stay below 32764 bytes).
struct TreeQuery {
  int64_t base;              // entry offset of the sequence
  int64_t pos;               // position of the draft
  uint64_t ents;             // drafts' entries on the query's path (bit e: entry n_com + e)
  uint64_t rows;             // drafts whose window rows it sees (bit t: draft t)
  int32_t len;               // entries of the sequence, the drafts' among them
  int32_t n_com;             // committed entries
  int32_t win_row;           // first committed window row it sees
  int32_t win_n;             // committed window rows it sees
  int32_t draft0;            // row of the sequence's first draft
};
struct TreeLayer {
  const uint16_t* draft;         // bf16 rows of the drafts [n_queries, 512], or the FP8 form:
  const uint8_t* draft_codes;
  const uint16_t* draft_rope;
  const uint8_t* draft_scales;
};
struct TreeAttnParams : AttnCommon {
  TreeLayer tree[kAttnMaxLayers];
  TreeQuery tq[kMaxTreeQueries];
};
cudaError_t launch_swa_fp8(const uint16_t* rows, int64_t n, uint8_t* codes, uint16_t* rope,
                           uint8_t* scales, cudaStream_t s);
int attn_smem_bytes();
constexpr int kAttnHeadGroup = 64;
// The two-CTA decode split needs no scratch memory: a caller opts in by
// passing a workspace of at least this many bytes.
constexpr size_t kAttnSplitToken = 16;
cudaError_t launch_attn(const AttnParams& p, const AttnMaps& maps, cudaStream_t s);
cudaError_t launch_attn_tree(const TreeAttnParams& p, const AttnMaps& maps, cudaStream_t s);
static_assert(sizeof(TreeIndexParams) + 2 * sizeof(CUtensorMap) < 32764, "kernel parameters");
static_assert(sizeof(TreeAttnParams) + sizeof(AttnMaps) < 32764, "kernel parameters");

// ---------------------------------------------------------------- window rows in a cache
// Arrays of csa2_window_t.
struct WinRows {
  int32_t n_seqs, swa, n_first, fp8;
  uint16_t* rows;
  uint8_t* codes;
  uint16_t* rope;
  uint8_t* scales;
  int64_t* pos;
  uint32_t* err;
};
// Segments of one launch (tables of at most 32764 bytes of parameters).
constexpr int kWinSegs = 2048;
struct WinAppendParams {
  WinRows w;
  const uint16_t* rows;
  uint16_t* rounded;
  const int64_t* pos0;       // of the launch's first segment
  int64_t n_rows;            // of the launch
  int32_t n_segs;
  int32_t identity;          // segment i is one row of sequence seq0 + i (no table)
  int32_t seq0;
  int32_t first[kWinSegs + 1];   // first row of each segment
  int32_t seq[kWinSegs];
};
cudaError_t launch_window_append(const WinAppendParams& p, cudaStream_t s);
struct WinReadParams {
  WinRows w;
  const int64_t* end;        // of the launch's first segment
  uint16_t* out;
  uint8_t* codes;
  uint16_t* rope;
  uint8_t* scales;
  uint16_t* first;
  int32_t n_rows;
  int32_t n_segs;
  int32_t identity;
  int32_t seq0;
  int32_t seq[2 * kWinSegs];
};
cudaError_t launch_window_read(const WinReadParams& p, cudaStream_t s);

// Rows of drafts in the cache's form.
struct WinDrafts {
  const uint16_t* rows;
  const uint8_t* codes;
  const uint16_t* rope;
  const uint8_t* scales;
};
constexpr int kWinTrees = 512;
constexpr int kWinDrafts = 12288;
struct WinAcceptParams {
  WinRows w;
  WinDrafts d;               // from the launch's first draft on
  const int32_t* accepted;   // of the launch's first tree
  int32_t n_trees;
  int64_t pos0[kWinTrees];
  int32_t seq[kWinTrees];
  int32_t first[kWinTrees + 1];
  int8_t parent[kWinDrafts];
};
cudaError_t launch_window_accept(const WinAcceptParams& p, cudaStream_t s);

// Attention of window layers.
struct WinAttnCommon {
  WinRows w;                 // decode, trees; swa and n_first in a chunk, too
  uint16_t* out;
  float* lse;
  const float* sink;
  uint32_t* err;
  long long wait_cycles;     // bounded-wait limit in cycles (kWaitCycles, if nothing else is asked for)
  int32_t withhold;          // tests: from its n-th item on a CTA loads no queries (0: it does)
  int32_t n_heads;
  int32_t nq;                // queries of the launch
  float scale_log2;          // scale * log2(e)
  int32_t rope_out;
  uint64_t turns[32];        // 2^64 * base^(-2t/64) / (2 pi): the output rotation
};
constexpr int kWinQueries = 4096;
struct WinDecodeParams : WinAttnCommon {
  const int64_t* pos;        // of the launch's first query
  int32_t identity;          // query i is of sequence seq0 + i
  int32_t seq0;
  int32_t seq[kWinQueries];
};
constexpr int kWinTreeQueries = 1536;
constexpr int kWinTreeTrees = 512;
constexpr int kWinTreeCtas = 256;
// Of a tree's two queries that share an item of 128 heads: drafts of the deeper
// one's path that the other's has not.
constexpr int kWinPairDrafts = 8;
struct WinTreeParams : WinAttnCommon {
  WinDrafts d;               // from the first draft of the launch's first tree on
  int64_t pos0[kWinTreeTrees];
  int32_t seq[kWinTreeTrees];
  int32_t first[kWinTreeTrees];       // a tree's first draft row
  // queries, a tree's so that neighbours have much of their paths in common
  uint64_t path[kWinTreeQueries];     // the drafts on the path, itself included
  int16_t tree[kWinTreeQueries];
  uint16_t query[kWinTreeQueries];    // its row of q and of the outputs
  uint16_t item[kWinTreeQueries];     // of an item: its first query; the top bit: it has two
  int32_t n_items;
  // CTA b has items start[b] .. start[b + 1] - 1 (where an item has one CTA)
  int32_t n_ctas;
  uint16_t start[kWinTreeCtas + 1];
};
struct WinPrefillParams : WinAttnCommon {
  const uint16_t* band;
  const uint16_t* first;
  int64_t pos0, band0, n_band;
};
cudaError_t launch_window_decode(const WinDecodeParams& p, const CUtensorMap& q, int sms,
                                 cudaStream_t s);
cudaError_t launch_window_tree(const WinTreeParams& p, const CUtensorMap& q, int sms,
                               cudaStream_t s);
cudaError_t launch_window_prefill(const WinPrefillParams& p, const CUtensorMap& q, int sms,
                                  cudaStream_t s);
static_assert(sizeof(WinAppendParams) < 32764 && sizeof(WinReadParams) < 32764 &&
              sizeof(WinAcceptParams) < 32764, "kernel parameters");
static_assert(sizeof(WinDecodeParams) + 3 * sizeof(CUtensorMap) < 32764 &&
              sizeof(WinTreeParams) + 3 * sizeof(CUtensorMap) < 32764, "kernel parameters");

// ---------------------------------------------------------------- verification of drafts
constexpr int kVerifyTrees = 512;
constexpr int kVerifyDrafts = 16384;
struct VerifyParams {
  const int32_t* token;      // of the launch's first draft
  const void* target;
  const void* root;
  const void* draft;
  const void* draft_root;
  const float* temperature;
  const float* uniform;
  const float* noise;
  int32_t* accepted;
  int32_t* next_token;
  int64_t ld, noise_ld;
  int32_t vocab;
  int32_t n_trees;
  int32_t first[kVerifyTrees + 1];
  int8_t parent[kVerifyDrafts];
};
int verify_cluster(int64_t n_trees, int32_t vocab, int sms);
cudaError_t launch_verify(const VerifyParams& p, bool fp32, int cluster, cudaStream_t s);
static_assert(sizeof(VerifyParams) < 32764, "kernel parameters");

}  // namespace csa2
