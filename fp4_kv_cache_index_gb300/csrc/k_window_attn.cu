// k_window_attn.cu -- attention of window layers: the newest rows and a few
// first tokens, key and value the same row (blog reading of the DeepSeek-V4
// report, section 4.1), for one token a sequence or a tree of drafts (rows in
// a cache, bf16 or FP8) and for a chunk of a prompt (a band of bf16 rows).
//
// A window is at most 128 rows and the first tokens are at most 8, so all keys
// of a query, or of two neighbouring tokens of a chunk, fit one tile of 144
// rows: the softmax has one step, with no running maximum to carry.  An item
// is up to 128 query rows (two tokens of 64 heads of a chunk, or the heads of
// one token):
//     S[128 x 144] = Q[128 x 512] KV[144 x 512]^T      (K-major A and B)
//     O[128 x 512] = P[128 x 144] KV[144 x 512]        (A in tensor memory,
//                                                       B MN-major)
// on tcgen05 with fp32 accumulators; the swizzled rows in shared memory serve
// both products.  Q is needed once and streams through small stages in
// channel blocks of 64; P goes from the softmax's registers to tensor memory, as
// bf16, the type that the MMA multiplies the rows in (their sum is one of the rounded
// values, so the weights still add up to 1; outputs are off by 0.0019 of themselves
// where fp32 probabilities and the same output rounding give 0.0017); O is made in
// two halves of 256 channels, since both halves, S and P do not fit the 512 columns
// together.  A CTA takes neighbouring items: in a
// chunk the rows stay in shared memory as a ring of 17 blocks of 8 positions
// (and one of first tokens), of which one is replaced every 8 tokens; of a tree
// they stay too, but for the slots that the next paths take otherwise.
//
// A tree's drafts of 64 heads go two an item, in the order of its branches, so
// that neighbours have most of their paths in common: the slots are the less deep
// one's, and what only the other's path has is in up to 8 more.  Each query has its
// own mask of the 144 slots.  (One draft an item: 73 us where this took 50, 1024
// drafts.)
//
// What bounds it.  The chunk: HBM, q in and the outputs out (8192 tokens of 64 heads
// are 1.08 GB: 214 us, 74 % of the copy rate); an item's S (32 MMAs of 155 cycles,
// which read Q and the rows from shared memory), softmax, products and stores are a
// chain of which only half of the next S and the second half of the stores run
// beside something else.  Decode: the same chain once (27000 cycles, of which the
// rows 11000, S 5000, the softmax 3000, products and outputs 5000): 14.2 us for 128
// sequences; for one, four CTAs share the outputs: 10.9 us.  509 sequences of 128 heads, 186 MB: 51 us, four rounds of it.
// Trees: 1024 drafts 48 us, three to four items a CTA.
//
// Code is fetched cold by most CTAs, once for each instruction that a single pass
// executes: the softmax and the outputs are loops over 16 and 32 columns although
// they read tensor memory twice for it (unrolled, with all columns in registers, the
// first item's softmax took 10700 cycles, now 4000; the chunk 224 us).
//
// Roles: warp 0 loads Q (TMA), warp 1 issues the MMAs, warps 2 and 3 load
// rows, warps 4-11 (two for each quadrant of tensor memory lanes) do the
// softmax and the outputs and take rows out of a cache.  (Sixteen such warps, with 96
// registers a thread: 224 us instead of 215, the trees 57 instead of 50.)
//
// Every wait has a limit.  A warp whose wait ran out signals nothing more and goes on to
// no rows, since tables that it has not seen complete may hold anything; it leaves with
// the other warps of its role, where these meet at a named barrier (`ok` is then the
// same in all of them), else at once.  What waits for it runs out in turn.
#include <cuda_fp16.h>

#include <type_traits>

#include "csa2_device.cuh"
#include "csa2_kernels.h"

namespace csa2 {
namespace {

// Twelve warps: three on each of an SM's four schedulers, which leaves a
// thread 168 registers (with a fourth it would be 128).
constexpr int kThreads = 384;
constexpr int kSlots = 144;             // rows of the tile
constexpr int kRing = 17;               // blocks of 8 window rows
constexpr int kFirstSlot = 8 * 16;      // first tokens, decode and trees
constexpr int kMoreSlot = 8 * 17;       // drafts of one of an item's two queries only
static_assert(kMoreSlot + kWinPairDrafts <= kSlots, "slots");
constexpr int kChunkFirst = 8 * kRing;  // first tokens, chunks
constexpr int kBlk = kSlots * 128;      // bytes of a 64-channel block of rows
constexpr int kBox = 64 * 128;          // Q: 64 rows x 64 channels
constexpr int kQBytes = 8 * kBox;       // a stage is a box or two, in turn
constexpr int kMaxStages = 8;
constexpr int kOutBox = 32 * 64;        // outputs: 32 rows x 32 channels
constexpr int kLoadWarps = 2, kSoftWarps = 8;
constexpr int kRowWarps = kLoadWarps + kSoftWarps;
constexpr int kMaxParts = 4;            // of an item's rows, by channels

constexpr int kKvOff = 0;
constexpr int kQOff = kKvOff + 8 * kBlk;
constexpr int kOutOff = kQOff + kQBytes;              // a box for each softmax warp
constexpr int kSmallOff = kOutOff + kSoftWarps * kOutBox;
struct Small {
  float red[2][128];            // [half of the columns][row]: maxima, then sums
  float2 rope[2][32];           // [token]: cos, sin of each channel pair
  int64_t at[2][2];             // [item parity][token]: its position
  uint32_t vis[2][2][5];        // [item parity][token]: rows that it sees
  uint32_t bad[5];              // rows that hold an infinity or a NaN (chunks)
  alignas(4) uint8_t bad8[kRing + 1][4];   // the same, 8 rows of each block, by quarter of its loads
  uint32_t bad_cb[kSoftWarps][5];          // the same (caches), by block of channels
  // cache: [item parity] what each slot takes: a row of the cache (-2), none
  // (-1) or a draft of the tree
  int8_t slot[2][kSlots];
  // trees: a path's drafts by depth (each loading warp's own), and [item parity]
  // the slots that the item takes otherwise than the one before it (or, of its
  // tree's first item, those that take drafts), and how many those are
  uint8_t draft[kLoadWarps][64], list[2][kSlots];
  int32_t n_list[2];
  uint32_t tmem;
  uint64_t q_full[kMaxStages], q_empty[kMaxStages];
  // a wait tells neighbouring phases of a barrier apart only: those whose two
  // sides may be two items apart are two, for items in turn
  uint64_t kv_full[2][kMaxParts], kv_empty[2], s_full, p_full, o_full, o_empty, tab_full, end;
};
constexpr int kSmemBytes = kSmallOff + (int)sizeof(Small);
static_assert(kSmemBytes <= 232448, "shared memory");

// Tensor memory columns: O (a half), S, P.
constexpr uint32_t kOCol = 0, kSCol = 256, kPCol = 400;

__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

__device__ __forceinline__ void named_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The same, and whether `ok` holds for all of them: warps whose waits ran out
// leave a loop together, so that none is left at a barrier.
__device__ __forceinline__ bool named_bar_and(int id, int threads, bool ok) {
  int all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %3, 0;\n"
      " barrier.cta.red.and.pred q, %1, %2, p;\n selp.s32 %0, 1, 0, q;\n}"
      : "=r"(all)
      : "r"(id), "r"(threads), "r"(ok ? 1 : 0)
      : "memory");
  return all != 0;
}

// Whether one of the eight bf16 of a piece is an infinity or a NaN: an
// exponent of all ones carries into the bit above it.
__device__ __forceinline__ bool not_finite(const uint4& v) {
  const uint32_t c = 0x00800080u, m = 0x7F807F80u;
  return ((((v.x & m) + c) | ((v.y & m) + c) | ((v.z & m) + c) | ((v.w & m) + c)) & 0x80008000u) != 0u;
}

// Eight E4M3 codes (two words) -> eight bf16 times a power of two, exact (in bf16's
// normal range).  E4M3's seven lower bits four places up in a bf16 are its value times 2^-120,
// subnormal numbers too; the sign goes to the top.
__device__ __forceinline__ uint4 e4m3_eight(uint32_t w0, uint32_t w1, uint32_t factor) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = prmt(i < 2 ? w0 : w1, 0u, (i & 1) ? 0x3424u : 0x1404u);   // a code on top of each half
    o[i] = bf16x2_mul(((t >> 4) & 0x07F007F0u) | (t & 0x80008000u), factor);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// Sixteen codes of rows with scale 2^(byte - 127); whether one of them is a NaN (all
// seven bits set) or the value is above bf16's range: then they come as zeros.  By
// all lanes of a warp.  The factor 2^(byte - 7) is a bf16 up to byte 134; above, which
// rows of ordinary values do not have, there is a second one.
__device__ __forceinline__ bool e4m3_sixteen(uint4 v, uint32_t byte, uint4& lo, uint4& hi) {
  const uint32_t m = 0x7F7F7F7Fu, c = 0x01010101u;
  bool bad = ((((v.x & m) + c) | ((v.y & m) + c) | ((v.z & m) + c) | ((v.w & m) + c)) & 0x80808080u) != 0u;
  if (bad) v = make_uint4(0u, 0u, 0u, 0u);
  const uint32_t f = (min(byte, 134u) + 120u) * 0x00800080u;
  lo = e4m3_eight(v.x, v.y, f);
  hi = e4m3_eight(v.z, v.w, f);
  if (__any_sync(0xffffffffu, byte > 134u)) {
    const uint32_t g = (max(byte, 134u) - 7u) * 0x00800080u;   // 2^(byte - 134)
    uint32_t* const x[2] = {&lo.x, &hi.x};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i >> 2][i & 3] = bf16x2_mul(x[i >> 2][i & 3], g);
    if (not_finite(lo) || not_finite(hi)) {
      bad = true;
      lo = hi = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  return bad;
}

// 16 bytes to shared memory, asynchronously, around the L1.
__device__ __forceinline__ void copy_async(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Until at most n groups of this thread's copies are left.
template <int n>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

template <class P>
constexpr bool kIsChunk = std::is_same<P, WinPrefillParams>::value;
template <class P>
constexpr bool kIsTree = std::is_same<P, WinTreeParams>::value;

template <class P, bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    k_window_attn(const __grid_constant__ P p, const __grid_constant__ CUtensorMap tm_q,
                  const int split) {
  constexpr bool kChunk = kIsChunk<P>, kTree = kIsTree<P>;
  // parts of the rows that the products can begin with
  constexpr int kParts = kChunk || kTree || kFp8 ? 1 : kMaxParts, kLast = kParts - 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* kv = smem + kKvOff;
  Small& sm = *reinterpret_cast<Small*>(smem + kSmallOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = p.n_heads;
  const bool pair = (kChunk || kTree) && H == 64;   // an item is up to two tokens
  int n_items = p.nq;
  if constexpr (kTree) n_items = p.n_items;
  else if (pair) n_items = (p.nq + 1) / 2;
  // With few items each has `split` CTAs, which all make its S and softmax and a
  // part of its output channels, 256 of them (or the 128 of a quarter) at a time.
  const int part = (int)blockIdx.x % split;
  int item0 = (int)blockIdx.x / split, item1 = item0 + 1;
  if (split == 1) {
    if constexpr (kTree) {
      item0 = p.start[blockIdx.x];
      item1 = p.start[blockIdx.x + 1];
    } else {
      item0 = (int)((int64_t)n_items * blockIdx.x / gridDim.x);
      item1 = (int)((int64_t)n_items * (blockIdx.x + 1) / gridDim.x);
    }
  }
  const int width = split == 4 ? 128 : 256, ch0 = kHeadDim / split * part, ch1 = ch0 + kHeadDim / split;
  const int W = p.w.swa, F = p.w.n_first;
  // stages of Q: four of two boxes, or eight of one (the tensor core reads two
  // boxes' rows from each, those behind the first are of no account)
  const int boxes = H / 64 * (pair ? 2 : 1);
  const uint32_t stages = boxes == 2 ? 4u : 8u, stage_bytes = (uint32_t)boxes * kBox;

  if (tid == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sm.q_full[s], 1);
      mbar_init(&sm.q_empty[s], 1);
    }
    for (int i = 0; i < 2 * kMaxParts; ++i)
      mbar_init(&sm.kv_full[i / kMaxParts][i % kMaxParts], kChunk ? kLoadWarps : kSoftWarps);
    mbar_init(&sm.kv_empty[0], 1);
    mbar_init(&sm.kv_empty[1], 1);
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.p_full, kSoftWarps);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_empty, kSoftWarps);
    mbar_init(&sm.tab_full, kLoadWarps);
    mbar_init(&sm.end, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
  }
  if (warp == 1) { tmem_alloc(&sm.tmem, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  griddep_wait();
  uint32_t* err = p.err;
  const long long& wl = p.wait_cycles;
  auto whole_warp = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };

  // warps that load rows: 0 and 1, and of a cache (and a chunk's first window)
  // 2-9, the softmax's
  const int lw = warp - 2;
  const bool loader = warp == 2 || warp == 3, soft = warp >= 4;

  auto tokens_of = [&](int item) -> int {
    if constexpr (kTree) return 1 + (p.item[item] >> 15);
    else return pair ? min(2, p.nq - 2 * item) : 1;
  };
  auto first_token = [&](int item) -> int {
    if constexpr (kTree) return p.item[item] & 0x7FFF;
    else return pair ? 2 * item : item;
  };
  // the query of a token of an item: its row of q and of the outputs
  auto query_row = [&](int item, int tk) -> int {
    if constexpr (kTree) return p.query[first_token(item) + tk];
    else return first_token(item) + tk;
  };
  auto piece = [&](int slot, int cb, int k) {
    return reinterpret_cast<uint4*>(kv + cb * kBlk + slot * 128 + ((k ^ (slot & 7)) << 4));
  };
  // the newest block of 8 positions that an item sees
  auto block_of = [&](int item) -> int64_t {
    if constexpr (kChunk) return (p.pos0 + first_token(item) + tokens_of(item) - 1) >> 3;
    else return 0;
  };
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  bool ok = true;

  // ---------------------------------------------------------- rows, chunks
  // Ring block a holds the positions 8 g .. 8 g + 7 of the newest g = a mod 17
  // that is not above g_hi (g_mod: g_hi mod 17); positions out of the band are
  // zeros.
  auto chunk_block_pos = [&](int64_t g_hi, int g_mod, int a) -> int64_t {
    const int d = g_mod - a;
    return 8 * (g_hi - (d < 0 ? d + kRing : d));
  };
  // A quarter of a block's rows (unit v of 4): four 16-byte pieces a lane, of
  // row lane / 4.  Kept in x[]; written by chunk_store.
  auto chunk_load = [&](int64_t g_hi, int g_mod, int a, int v, uint4 (&x)[4]) {
    if constexpr (kChunk) {
      const int r = lane >> 2;
      const uint16_t* src = nullptr;
      if (a < kRing) {
        const int64_t row = chunk_block_pos(g_hi, g_mod, a) + r - p.band0;
        if (row >= 0 && row < p.n_band) src = p.band + row * kHeadDim;
      } else if (r < F) {
        if (r >= p.band0) {
          if (r - p.band0 < p.n_band) src = p.band + (r - p.band0) * kHeadDim;
        } else if (p.first) {
          src = p.first + r * kHeadDim;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = src ? ldg_now_v4(src + 8 * (4 * (4 * v + i) + (lane & 3))) : zero;
    }
  };
  auto chunk_store = [&](int a, int v, const uint4 (&x)[4]) {
    const int r = lane >> 2, slot = 8 * a + r;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 4 * (4 * v + i) + (lane & 3);
      const bool b = not_finite(x[i]);
      bad |= b;
      // a probability of 0 times such a value would not be 0
      *piece(slot, c >> 3, c & 7) = b ? zero : x[i];
    }
    const uint32_t any = __ballot_sync(0xffffffffu, bad);
    const uint32_t rows = __ballot_sync(0xffffffffu, lane < 8 && ((any >> (4 * lane)) & 15u));
    if (lane == 0) sm.bad8[a][v] = (uint8_t)rows;
  };
  // Which rows hold an infinity or a NaN: slots 32 word .. of the lanes.
  auto chunk_bad = [&](int word) {
    const int j = 32 * word + lane;
    uint32_t q = 0;
    if (j < kSlots) q = *reinterpret_cast<const uint32_t*>(sm.bad8[j >> 3]);
    const bool b = ((q | (q >> 8) | (q >> 16) | (q >> 24)) >> (j & 7)) & 1u;
    const uint32_t m = __ballot_sync(0xffffffffu, b);
    if (lane == 0) sm.bad[word] = m;
  };

  // ---------------------------------------------------------- rows, cache
  struct Query {
    int64_t at, pos0;   // its position; positions from pos0 on are drafts'
    int64_t ring, first;   // the sequence's rows in the cache
    int32_t draft0;
    int at_mod;
  };
  auto query_of = [&](int q) -> Query {
    Query t = {};
    int32_t seq = 0;
    if constexpr (kTree) {
      const int tr = p.tree[q];
      t.pos0 = p.pos0[tr];
      t.at = t.pos0 + __popcll(p.path[q]) - 1;
      t.draft0 = p.first[tr];
      seq = p.seq[tr];
    } else if constexpr (!kChunk) {
      t.at = max((long long)__ldg(p.pos + q), -1ll);   // (what is W below it has to stay negative)
      t.pos0 = INT64_MAX;
      seq = p.identity ? p.seq0 + q : p.seq[q];
    }
    t.at_mod = t.at >= 0 ? (int)(t.at % W) : 0;
    t.ring = (int64_t)seq * W;
    t.first = (int64_t)p.w.n_seqs * W + (int64_t)seq * F;
    return t;
  };
  // An item's query whose rows the slots take: of a tree's two the one that is
  // less deep, whose window begins no later.  Its depth-k draft and the other's
  // are of one position; what only the other one's path has goes to slots of its own.
  auto base_of = [&](int item) -> int {
    const int q = first_token(item);
    if constexpr (kTree) {
      if (tokens_of(item) > 1 && __popcll(p.path[q + 1]) < __popcll(p.path[q])) return q + 1;
    }
    return q;
  };
  // What slot j takes (sm.slot), and x, the position of that row.  Ring row j holds
  // the position that is j mod W among the W newest up to the query's; slot 128 + f
  // first token f.  A row of the cache counts only if it holds that position.
  auto slot_of = [&](const Query& t, int j, int64_t& x) -> int {
    int64_t row = 0;
    x = -1;
    if (j < W) {
      int d = t.at_mod - j;
      if (d < 0) d += W;
      x = t.at - d;
      if (x < F) x = -1;
      row = t.ring + j;
    } else if (j >= kFirstSlot && j - kFirstSlot < F && j - kFirstSlot <= t.at) {
      x = j - kFirstSlot;
      row = t.first + x;
    }
    if (x < 0) return -1;
    if (kTree && x >= t.pos0) return CSA2_IN_BOUNDS(x - t.pos0 < 64, err) ? sm.draft[lw & 1][x - t.pos0] : -1;
    if (!CSA2_IN_BOUNDS(is_window_row(p.w, row), err)) return -1;
    return p.w.pos[row] == x ? -2 : -1;
  };

  // Whether an item is of the tree of the one before it, whose rows are still
  // there.
  auto same_tree = [&](int item) {
    if constexpr (kTree) return item > item0 && p.tree[first_token(item)] == p.tree[first_token(item - 1)];
    else return false;
  };
  // Tables of an item, by the two loading warps (a warp's `ok` is the same in its lanes):
  // the rows that each token sees (of a cache: what each slot takes), and its position.
  auto item_tables = [&](int item) {
    const int par = (item - item0) & 1;
    const int n_tok = tokens_of(item), t0 = first_token(item);
    int64_t at = 0, at_1 = 0;   // the tokens' positions
    if constexpr (kChunk) {
      at = p.pos0 + t0;
      at_1 = at + 1;
      const int64_t hi = at + n_tok - 1;
      const int g_mod = (int)((hi >> 3) % kRing);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int word = 2 * k + lw, j = 32 * word + lane;
        if (word > 4) break;
        int64_t x = -1;
        bool first = false;
        if (j < kChunkFirst) {
          x = chunk_block_pos(hi >> 3, g_mod, j >> 3) + (j & 7);
          if (x < F || x < p.band0) x = -1;
        } else if (j < kSlots) {
          first = true;
          x = j - kChunkFirst < F ? j - kChunkFirst : -1;
        }
        const bool v0 = x >= 0 && x <= at && (first || x > at - W);
        const bool v1 = n_tok > 1 && x >= 0 && x <= hi && (first || x > hi - W);
        const uint32_t m0 = __ballot_sync(0xffffffffu, v0), m1 = __ballot_sync(0xffffffffu, v1);
        if (lane == 0) {
          sm.vis[par][0][word] = m0;
          sm.vis[par][1][word] = m1;
        }
      }
    } else {
      const int base = base_of(item);
      const Query t = query_of(base);
      at = t.at;
      uint64_t path = 0, other = 0;
      int64_t at1 = 0;
      int mine = 0;               // the base's place in the item
      if constexpr (kTree) {
        path = p.path[base];
        mine = base - t0;
        if (n_tok > 1) {
          other = p.path[2 * t0 + 1 - base];
          at1 = t.pos0 + __popcll(other) - 1;
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int b = lane + 32 * h;
          if ((path >> b) & 1ull) sm.draft[lw][__popcll(path & ((1ull << b) - 1ull))] = (uint8_t)b;
        }
        __syncwarp();
        at_1 = mine ? t.at : at1;
        if (mine) at = at1;
      }
      int v[3];
      int64_t x[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) {   // the tags' loads together
        const int j = 32 * (2 * k + lw) + lane;
        x[k] = -1;
        v[k] = j < kMoreSlot ? slot_of(t, j, x[k]) : -1;
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int word = 2 * k + lw, j = 32 * word + lane;
        if (word > 4) break;
        const bool near = j >= kFirstSlot || x[k] > at1 - W;
        const uint32_t m = __ballot_sync(0xffffffffu, v[k] != -1);
        if constexpr (kTree) {
          bool sees = n_tok > 1 && near && (v[k] == -2 || (v[k] >= 0 && ((other >> (v[k] & 63)) & 1ull)));
          if (j >= kMoreSlot && j < kSlots) {
            // the other path's drafts that this one has not
            uint64_t left = other & ~path;
            for (int i = kMoreSlot; i < j; ++i) left &= left - 1ull;
            if (left) {
              v[k] = __ffsll((long long)left) - 1;
              const int64_t y = t.pos0 + __popcll(other & ((1ull << v[k]) - 1ull));
              sees = y < F || y > at1 - W;
            }
          }
          const uint32_t m1 = __ballot_sync(0xffffffffu, sees);
          if (lane == 0) sm.vis[par][mine ^ 1][word] = m1;
        }
        if (j < kSlots) sm.slot[par][j] = (int8_t)v[k];
        if (lane == 0) sm.vis[par][mine][word] = m;
      }
      if constexpr (kTree) {
        named_bar(3, 32 * kLoadWarps);   // both warps' halves
        if (lw == 1) {
          const bool same = same_tree(item);
          int n = 0;
          for (int j = lane; j < 160; j += 32) {
            bool put = false;
            if (j < kSlots) {
              const int now = sm.slot[par][j], old = sm.slot[par ^ 1][j];
              put = same ? now != old : now >= 0 || (item > item0 && j >= kMoreSlot && old >= 0);
            }
            const uint32_t m = __ballot_sync(0xffffffffu, put);
            if (put) sm.list[par][n + __popc(m & ((1u << lane) - 1u))] = (uint8_t)j;
            n += __popc(m);
          }
          if (lane == 0) sm.n_list[par] = n;
        }
        named_bar(3, 32 * kLoadWarps);
      }
    }
    if (lw == 0 && lane == 0) {
      sm.at[par][0] = at;
      sm.at[par][1] = at_1;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.tab_full);
  };
  // Trees: the rows of the listed slots, drafts' and those that take the places of
  // the last path's.  A warp has channel blocks cb0, cb0 + 2, .. (kBlocks of them),
  // 8 rows x 4 pieces of 16 bytes at a time, `ready` comes between the first loads
  // and the first stores.
  auto listed_rows = [&](const Query& t, int par, int cb0, auto blocks, auto ready) {
    if constexpr (kTree) {
      constexpr int kBlocks = decltype(blocks)::value, kFlight = 4;
      const int r8 = lane >> 2, c4 = lane & 3;
      const int n = sm.n_list[par], jobs = (n + 7) / 8 * kBlocks;
      // whether any of these blocks' rows is marked in sm.bad_cb, or is to be
      bool marks = lane < 5 * kBlocks && sm.bad_cb[cb0 + 2 * (lane / 5 % kBlocks)][lane % 5] != 0u;
      int j0 = 0;
#pragma unroll 1
      do {
        uint4 d[kFlight], e[kFlight];
        uint32_t byte[kFlight];
        int slot[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const int at = (j0 + i) / kBlocks * 8 + r8, cb = cb0 + 2 * (i % kBlocks);
          slot[i] = -1;
          d[i] = e[i] = zero;
          byte[i] = 0u;
          if (at >= n) continue;
          slot[i] = sm.list[par][at];
          if (!CSA2_IN_BOUNDS(slot[i] < kSlots, err)) slot[i] = 0;
          const int what = sm.slot[par][slot[i]];
          if (what == -1) continue;
          const WinDrafts& x = p.d;
          const int64_t row = what >= 0 ? (int64_t)t.draft0 + what
                              : slot[i] < W ? t.ring + slot[i] : t.first + slot[i] - kFirstSlot;
          if (!CSA2_IN_BOUNDS(what >= 0 ? row < p.nq : is_window_row(p.w, row), err)) continue;
          if (kFp8 && cb < 7) {
            d[i] = ldg_now_v4((what >= 0 ? x.codes : p.w.codes) + row * 448 + 64 * cb + 16 * c4);
            byte[i] = ldg_now_u8((what >= 0 ? x.scales : p.w.scales) + row * 8 + cb);
          } else {
            const uint16_t* src = kFp8 ? (what >= 0 ? x.rope : p.w.rope) + row * 64
                                       : (what >= 0 ? x.rows : p.w.rows) + row * kHeadDim + 64 * cb;
            d[i] = ldg_now_v4(src + 8 * c4);
            e[i] = ldg_now_v4(src + 32 + 8 * c4);
          }
        }
        bool bad[kFlight];
        uint4* to[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          const int cb = cb0 + 2 * (i % kBlocks);
          bad[i] = false;
          if (kFp8 && cb < 7) {
            if (j0 + i < jobs) bad[i] = e4m3_sixteen(d[i], byte[i], d[i], e[i]);
          } else {
            bad[i] = not_finite(d[i]) || not_finite(e[i]);
            if (bad[i]) d[i] = e[i] = zero;
          }
          marks |= bad[i];
          // the second piece is 16 bytes away (codes) or 64, up or down
          to[i] = piece(max(slot[i], 0), cb, kFp8 && cb < 7 ? 2 * c4 : c4);
        }
        const bool mark = __any_sync(0xffffffffu, marks);
        if (j0 == 0) ready();
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
          if (slot[i] < 0) continue;
          const int turn = kFp8 && cb0 + 2 * (i % kBlocks) < 7 ? 1 : 4;
          *to[i] = d[i];
          *reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(to[i]) ^ (uintptr_t)(16 * turn)) = e[i];
        }
        if (mark) {
#pragma unroll 1
          for (int i = 0; i < kFlight; ++i) {
            const bool b = i == 0 ? bad[0] : i == 1 ? bad[1] : i == 2 ? bad[2] : bad[3];
            const int at = i == 0 ? slot[0] : i == 1 ? slot[1] : i == 2 ? slot[2] : slot[3];
            const uint32_t any = __ballot_sync(0xffffffffu, b);
            if (at < 0 || c4 != 0) continue;
            uint32_t* const word = &sm.bad_cb[cb0 + 2 * (i % kBlocks)][at >> 5];
            if ((any >> lane) & 15u) atomicOr(word, 1u << (at & 31));
            else atomicAnd(word, ~(1u << (at & 31)));
          }
        }
        j0 += kFlight;
      } while (j0 < jobs);
    }
  };
  // Rows of an item out of the cache, by the softmax warps, 8 rows x 4 pieces of 16
  // bytes at a time (whole sectors, and stores without conflicts).  Loops, not
  // straight code: most CTAs come here once, and unrolled it was the fetching of
  // instructions that took the time.
  //
  // bf16, one token a sequence: warp w has groups w and w + 8 of 8 slots, and of the
  // first tokens' channels 64 w ..; the products begin with the first quarter of the
  // channels, while the others are on their way.
  auto quarter_rows = [&](int item) {
    if constexpr (kParts > 1) {
      const uint32_t k = (uint32_t)(item - item0);
      const int par = k & 1, w = warp - 4, r8 = lane >> 2, c4 = lane & 3;
      const Query t = query_of(item);
      // unit u: its group's row of this lane, and where it goes in block 0
      const uint16_t* from[3];
      uint8_t* to[3];
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        const int j = 8 * (u < 2 ? w + 8 * u : 16) + r8;
        const bool is = (u == 2 ? r8 < F : j < W) &&
                        CSA2_IN_BOUNDS(is_window_row(p.w, u == 2 ? t.first + r8 : t.ring + j), err);
        from[u] = is ? p.w.rows + (u == 2 ? t.first + r8 : t.ring + j) * kHeadDim + 8 * c4 : nullptr;
        to[u] = kv + j * 128;
      }
      if (k > 0) ok = ok && mbar_wait(&sm.kv_empty[par ^ 1], ((k - 1) >> 1) & 1, err, wl);
#pragma unroll 1
      for (int cb = 0; cb < 8; ++cb) {
#pragma unroll
        for (int u = 0; u < 3; ++u) {
          if (!from[u] || (u == 2 && cb != w)) continue;
          copy_async(to[u] + cb * kBlk + ((c4 ^ r8) << 4), from[u] + 64 * cb);
          copy_async(to[u] + cb * kBlk + (((4 + c4) ^ r8) << 4), from[u] + 64 * cb + 32);
        }
        if (cb & 1) copy_async_commit();
      }
      ok = whole_warp(ok && mbar_wait(&sm.tab_full, par, err, wl));
      bool there[3];
#pragma unroll
      for (int u = 0; u < 3; ++u) there[u] = sm.slot[par][8 * (u < 2 ? w + 8 * u : 16) + r8] == -2;
#pragma unroll 1
      for (int cb = 0; cb < 8; ++cb) {
        if (cb == 0) copy_async_wait<3>();
        else if (cb == 2) copy_async_wait<2>();
        else if (cb == 4) copy_async_wait<1>();
        else if (cb == 6) copy_async_wait<0>();
#pragma unroll
        for (int u = 0; u < 3; ++u) {
          if (there[u] || (u == 2 && cb != w)) continue;
          *reinterpret_cast<uint4*>(to[u] + cb * kBlk + ((c4 ^ r8) << 4)) = zero;
          *reinterpret_cast<uint4*>(to[u] + cb * kBlk + (((4 + c4) ^ r8) << 4)) = zero;
        }
        if (cb & 1) {
          fence_proxy_async_smem();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(&sm.kv_full[par][cb >> 1]);
        }
      }
    }
  };
  // FP8, and the first item of a tree: warp w has channels 64 w .. 64 w + 63 of all
  // rows, and then of the path's drafts.  bf16 pieces go straight to their places;
  // codes go to the first halves of their rows' places, from where the warp that has
  // brought them takes them again.  (By quarters of the channels the codes take as
  // long: the products slow the warps' own accesses down.)
  auto block_rows = [&](int item) {
    if constexpr (kTree || (kFp8 && !kChunk)) {
      const uint32_t k = (uint32_t)(item - item0);
      const int par = k & 1, cb = warp - 4;
      const Query t = query_of(base_of(item));
      constexpr int kGroups = 17;                        // of 8 slots
      const int r8 = lane >> 2, c4 = lane & 3;
      const bool codes = kFp8 && cb < 7;
      uint8_t* const mine = kv + cb * kBlk + r8 * 128;   // this lane's row of group 0
      uint32_t bad = 0u;         // groups in whose row this lane had an infinity or a NaN
      uint32_t sc[5] = {0u, 0u, 0u, 0u, 0u};             // of slots lane + 32 i
      const bool held = CSA2_IN_BOUNDS(is_window_row(p.w, t.ring) && is_window_row(p.w, t.ring + W - 1) &&
                                           (F == 0 || is_window_row(p.w, t.first + F - 1)), err);
      if (k > 0) ok = ok && mbar_wait(&sm.kv_empty[par ^ 1], ((k - 1) >> 1) & 1, err, wl);
      if (codes) {
        const uint8_t* src = p.w.codes + (t.ring + r8) * 448 + 64 * cb + 16 * c4;
#pragma unroll 1
        for (int j = r8, g = 0; g < 16; ++g, j += 8, src += 8 * 448)
          if (held && j < W) copy_async(mine + g * 1024 + 16 * c4, src);
        if (held && r8 < F)
          copy_async(mine + 16 * 1024 + 16 * c4, p.w.codes + (t.first + r8) * 448 + 64 * cb + 16 * c4);
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          const int j = lane + 32 * i;
          if (held && (i < 4 ? j < W : lane < F))
            sc[i] = ldg_now_u8(p.w.scales + (i < 4 ? t.ring + j : t.first + lane) * 8 + cb);
        }
      } else {
        const int64_t step = kFp8 ? 64 : kHeadDim;
        const uint16_t* base = kFp8 ? p.w.rope + 8 * c4 : p.w.rows + 64 * cb + 8 * c4;
        const uint16_t* src = base + (t.ring + r8) * step;
#pragma unroll 1
        for (int j = r8, g = 0; g < kGroups; ++g, j += 8, src += 8 * step) {
          if (g == 16) src = base + (t.first + r8) * step;
          if (held && (g < 16 ? j < W : r8 < F)) {
            copy_async(mine + g * 1024 + ((c4 ^ r8) << 4), src);
            copy_async(mine + g * 1024 + (((4 + c4) ^ r8) << 4), src + 32);
          }
        }
      }
      copy_async_commit();
      ok = whole_warp(ok && mbar_wait(&sm.tab_full, par, err, wl));
      copy_async_wait<0>();
      __syncwarp();
      if (codes) {
        // the next group's codes on their way while a group's are converted
        auto take = [&](int g) {
          return sm.slot[par][8 * g + r8] == -2 ? *reinterpret_cast<const uint4*>(mine + g * 1024 + 16 * c4) : zero;
        };
        uint4 next = take(0);
#pragma unroll 1
        for (int g = 0; g < kGroups; ++g) {
          const uint32_t byte = __shfl_sync(0xffffffffu, sc[0], 8 * (g & 3) + r8);
          const uint4 v = next;
          if (g + 1 < kGroups) next = take(g + 1);
          uint4 lo, hi;
          if (e4m3_sixteen(v, byte, lo, hi)) bad |= 1u << g;
          __syncwarp();
          uint8_t* const row = mine + g * 1024;
          *reinterpret_cast<uint4*>(row + (((2 * c4) ^ r8) << 4)) = lo;
          *reinterpret_cast<uint4*>(row + (((2 * c4 + 1) ^ r8) << 4)) = hi;
          if ((g & 3) == 3) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[i] = sc[i + 1];
          }
        }
      } else {
#pragma unroll 1
        for (int g = 0; g < kGroups; ++g) {
          uint4* const a = reinterpret_cast<uint4*>(mine + g * 1024 + ((c4 ^ r8) << 4));
          uint4* const b = reinterpret_cast<uint4*>(mine + g * 1024 + (((4 + c4) ^ r8) << 4));
          bool put = sm.slot[par][8 * g + r8] != -2;
          if (kTree && !put && (not_finite(*a) || not_finite(*b))) {
            put = true;
            bad |= 1u << g;
          }
          if (put) *a = *b = zero;
        }
      }
      // Rows of a cache with infinities and NaN are zeros in the products (a
      // probability of 0 times such a value would not be 0): other queries of the
      // tree may not see them.  Those who do answer NaN.
      if (lane < 5) sm.bad_cb[cb][lane] = 0u;
      __syncwarp();
      if (bad) {
        for (int g = 0; g < kGroups; ++g)
          if ((bad >> g) & 1u) atomicOr(&sm.bad_cb[cb][g >> 2], 1u << (8 * (g & 3) + r8));
      }
      __syncwarp();
      if constexpr (kTree) {
        if (ok) listed_rows(t, par, cb, std::integral_constant<int, 1>(), [] {});
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&sm.kv_full[par][kLast]);
    }
  };

  if constexpr (kChunk) {
    // the first item's whole window: 18 blocks in quarters over the ten
    // loading and softmax warps, four quarters in flight
    if ((loader || soft) && item0 < item1) {
      const int64_t g = (p.pos0 + first_token(item0) + tokens_of(item0) - 1) >> 3;
      const int g_mod = (int)(g % kRing);
      constexpr int kJobs = (kRing + 1) * 4, kBatch = 4;
      for (int j0 = lw; j0 < kJobs; j0 += kBatch * kRowWarps) {
        uint4 x[kBatch][4];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int j = j0 + b * kRowWarps;
          if (j < kJobs) chunk_load(g, g_mod, j >> 2, j & 3, x[b]);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int j = j0 + b * kRowWarps;
          if (j < kJobs) chunk_store(j >> 2, j & 3, x[b]);
        }
      }
      fence_proxy_async_smem();
    }
  } else if (warp >= 2) {
    // slots that no row ever takes: read by the products all the same
    for (int i = tid - 64; i < 8 * 8 * 8; i += kThreads - 64)
      *piece(kSlots - 8 + (i & 7), (i >> 3) & 7, i >> 6) = zero;
    fence_proxy_async_smem();
  }
  __syncthreads();

  if (warp == 0) {
    // ------------------------------------------------------------ Q
    if (lane == 0) {
      uint32_t n = 0;
      for (int item = item0; item < item1 && ok; ++item) {
        if (p.withhold && item - item0 >= p.withhold - 1) ok = false;   // tests: all waits run out
        const int now = tokens_of(item) * H / 64;   // boxes of the item: the last may have one
        for (int cb = 0; cb < 8 && ok; ++cb, ++n) {
          const uint32_t s = n % stages, use = n / stages;
          if (use > 0) ok = mbar_wait(&sm.q_empty[s], (use - 1) & 1, err, wl);
          if (!ok) break;
          mbar_arrive_expect_tx(&sm.q_full[s], now * kBox);
          uint8_t* dst = smem + kQOff + s * stage_bytes;
          for (int b = 0; b < now; ++b)
            tma_load_2d(dst + b * kBox, &tm_q, 64 * cb,
                        pair ? query_row(item, b) * H : query_row(item, 0) * H + 64 * b, &sm.q_full[s]);
        }
      }
      // the copies in flight must land before the CTA exits
      if (!ok)
        for (uint32_t k = n > stages ? n - stages : 0; k < n; ++k)
          mbar_wait(&sm.q_full[k % stages], (k / stages) & 1, err, drain_limit(wl));
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_bf16_f32(128, kSlots, false, false);
      const uint32_t id_o = width == 256 ? idesc_bf16_f32(128, 256, false, true) : idesc_bf16_f32(128, 128, false, true);
      const uint64_t d_q = sdesc_sw128(smem_u32(smem + kQOff), 16, 1024);
      const uint64_t d_k = sdesc_sw128(smem_u32(kv), 16, 1024);
      const uint64_t d_v = sdesc_sw128(smem_u32(kv), kBlk, 1024);
      uint32_t n = 0, chunk = 0;
      // channel blocks c0 .. c1 - 1 of an item's S
      auto issue_s = [&](int item, int c0, int c1) {
        const uint32_t j = (uint32_t)(item - item0);
        for (int cb = c0; cb < c1 && ok; ++cb, ++n) {
          const uint32_t s = n % stages;
          if (cb % (8 / kParts) == 0)
            ok = mbar_wait(&sm.kv_full[j & 1][cb / (8 / kParts)], (j >> 1) & 1, err, wl);
          if (ok) ok = mbar_wait(&sm.q_full[s], (n / stages) & 1, err, wl);
          if (!ok) break;
          tc_fence_after();
          for (int k = 0; k < 4; ++k)
            umma_bf16(tmem + kSCol, d_q + ((s * stage_bytes + 32 * k) >> 4),
                      d_k + ((cb * kBlk + 32 * k) >> 4), id_s, (cb | k) ? 1u : 0u);
          umma_commit(&sm.q_empty[s]);
        }
        if (ok && c1 == 8) umma_commit(&sm.s_full);
      };
      auto issue_o = [&](int ch) {
        if (chunk > 0) ok = mbar_wait(&sm.o_empty, (chunk - 1) & 1, err, wl);
        if (!ok) return;
        tc_fence_after();
        for (int ks = 0; ks < kSlots / 16; ++ks)
          umma_bf16_ts(tmem + kOCol, tmem + kPCol + 8 * ks, d_v + ((ch / 64 * kBlk + ks * 2048) >> 4),
                       id_o, ks ? 1u : 0u);
        umma_commit(&sm.o_full);
        ++chunk;
      };
      if (item0 < item1) issue_s(item0, 0, 8);
      for (int item = item0; item < item1 && ok; ++item) {
        const uint32_t k = (uint32_t)(item - item0);
        ok = mbar_wait(&sm.p_full, k & 1, err, wl);
        if (ok) issue_o(ch0);
        // half of the next S while the outputs' first half is read out, where the
        // rows stay as they are
        int c0 = 0;
        if constexpr (kChunk) {
          if (ok && item + 1 < item1 && block_of(item + 1) == block_of(item)) {
            issue_s(item + 1, 0, 4);
            c0 = 4;
          }
        }
        if (ok && split == 1) issue_o(256);
        if (ok) umma_commit(&sm.kv_empty[k & 1]);
        if (ok && item + 1 < item1) issue_s(item + 1, c0, 8);
      }
      griddep_launch();
      if (!ok) {   // the MMAs issued so far must end before the CTA exits
        umma_commit(&sm.end);
        mbar_wait(&sm.end, 0, err, drain_limit(wl));
      }
    }
  } else if (loader) {
    // ------------------------------------------------------------ rows, tables
    int64_t g_have = 0;
    for (int item = item0; item < item1; ++item) {
      const uint32_t k = (uint32_t)(item - item0);
      if constexpr (kChunk) {
        const int64_t g = block_of(item);
        const int a = (int)(g % kRing);
        // at most one new block an item (of at most two tokens)
        const bool fresh = k > 0 && g != g_have;
        g_have = g;
        uint4 x[2][4];
        if (fresh) {
          chunk_load(g, a, a, 2 * lw, x[0]);
          chunk_load(g, a, a, 2 * lw + 1, x[1]);
        }
        // the tables' place was that of the item before the last one; the rows'
        // is needed where one comes in
        if (k > 1) ok = whole_warp(mbar_wait_sleep(&sm.kv_empty[k & 1], ((k - 2) >> 1) & 1, err, wl));
        if (ok) item_tables(item);
        if (fresh) {
          ok = whole_warp(ok && mbar_wait_sleep(&sm.kv_empty[(k - 1) & 1], ((k - 1) >> 1) & 1, err, wl));
          if (ok) {
            chunk_store(a, 2 * lw, x[0]);
            chunk_store(a, 2 * lw + 1, x[1]);
          }
        }
        ok = named_bar_and(3, 32 * kLoadWarps, ok);
        if (!ok) break;
        if (fresh || k == 0) {
          chunk_bad(lw);
          chunk_bad(2 + lw);
          if (lw == 0) chunk_bad(4);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.kv_full[k & 1][0]);
      } else {
        // not before all warps have the last item's: a wait tells neighbouring
        // phases apart only
        if (k > 0) ok = ok && mbar_wait_sleep(&sm.kv_full[(k - 1) & 1][kLast], ((k - 1) >> 1) & 1, err, wl);
        ok = whole_warp(ok);
        if constexpr (kTree) ok = named_bar_and(3, 32 * kLoadWarps, ok);
        if (!ok) break;
        item_tables(item);
        // Of a tree whose rows are here already these warps bring the others, while
        // the softmax warps have the last item's outputs to store.
        if (same_tree(item)) {
          listed_rows(query_of(base_of(item)), k & 1, lw, std::integral_constant<int, 4>(), [&] {
            ok = mbar_wait(&sm.kv_empty[(k - 1) & 1], ((k - 1) >> 1) & 1, err, wl);
          });
          fence_proxy_async_smem();
          ok = whole_warp(ok);
          if (ok && lane < kSoftWarps / kLoadWarps) mbar_arrive(&sm.kv_full[k & 1][0]);
        }
      }
    }
  } else if (soft) {
    // ------------------------------------------------------------ softmax, outputs
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    uint8_t* const box = smem + kOutOff + (warp - 4) * kOutBox;
    uint32_t chunk = 0;
    for (int item = item0; item < item1; ++item) {
      const uint32_t k = (uint32_t)(item - item0), ph = k & 1u;
      // (its last products are done: their outputs are stored)
      if constexpr (kTree) {
        if (!same_tree(item)) block_rows(item);
      } else if constexpr (kParts > 1) {
        quarter_rows(item);
      } else if constexpr (!kChunk) {
        block_rows(item);
      }
      const int n_rows = tokens_of(item) * H;
      const bool live = quad * 32 < n_rows;       // of the warp's rows, all or none
      const int tk = pair ? row >> 6 : 0;
      ok = mbar_wait(&sm.kv_full[ph][kLast], (k >> 1) & 1, err, wl) && ok;
      ok = mbar_wait(&sm.s_full, ph, err, wl) && ok;
      tc_fence_after();
      // a thread has a half of its row: columns 0-79 or 80-143
      const int g0 = half ? 5 : 0, ng = half ? 4 : 5;
      float m = -INFINITY;
      if (live) {
#pragma unroll 1
        for (int g = g0; g < g0 + ng; ++g) {
          uint32_t s[16];
          tmem_ld16(tmem + lanes + kSCol + 16 * g, s);
          const uint32_t v = sm.vis[ph][tk][g >> 1] >> (16 * (g & 1));
#pragma unroll
          for (int i = 0; i < 16; ++i)
            m = fmaxf(m, (v >> i) & 1u ? __uint_as_float(s[i]) * p.scale_log2 : -INFINITY);
        }
        sm.red[half][row] = m;
      }
      // (all of them leave together where a wait ran out)
      ok = named_bar_and(1, 32 * kSoftWarps, ok);
      if (!ok) break;
      if (live) m = fmaxf(m, sm.red[half ^ 1][row]);
      named_bar(1, 32 * kSoftWarps);
      float sum = 0.0f;
      bool bad = false;
      if (live) {
        if constexpr (kChunk) {   // before the next item's masks may come
          uint32_t b = 0;
#pragma unroll
          for (int i = 0; i < 5; ++i) b |= sm.vis[ph][tk][i] & sm.bad[i];
          bad = b != 0;
        }
        if constexpr (kTree || (kFp8 && !kChunk)) {
          uint32_t b = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int w = lane + 32 * i;
            if (w < kSoftWarps * 5) b |= sm.vis[ph][tk][w % 5] & sm.bad_cb[w / 5][w % 5];
          }
          bad = __any_sync(0xffffffffu, b != 0);
        }
        const float m0 = m == -INFINITY ? 0.0f : m;
#pragma unroll 1
        for (int g = g0; g < g0 + ng; ++g) {
          uint32_t s[16], pk[8];
          tmem_ld16(tmem + lanes + kSCol + 16 * g, s);
          const uint32_t v = sm.vis[ph][tk][g >> 1] >> (16 * (g & 1));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float e[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x = fast_exp2(fmaf(__uint_as_float(s[2 * i + h]), p.scale_log2, -m0));
              e[h] = (v >> (2 * i + h)) & 1u ? x : 0.0f;
            }
            const __nv_bfloat162 b2 = __floats2bfloat162_rn(e[0], e[1]);
            pk[i] = *reinterpret_cast<const uint32_t*>(&b2);
            sum += __uint_as_float(pk[i] << 16) + __uint_as_float(pk[i] & 0xFFFF0000u);
          }
          tmem_st8(tmem + lanes + kPCol + 8 * g, pk);
        }
        sm.red[half][row] = sum;
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full);
      if (p.rope_out && half == 1 && (quad & 1) == 0) {
        // sines of the output rotation, by warps with fewer columns: of token
        // quad / 2 (all have left the item before this one)
        const uint64_t turn = (uint64_t)(-sm.at[ph][quad >> 1]) * p.turns[lane];
        float sn, cs;
        sincospif((float)(int64_t)turn * 0x1p-63f, &sn, &cs);
        sm.rope[quad >> 1][lane] = make_float2(cs, sn);
      }
      named_bar(1, 32 * kSoftWarps);
      float inv = 0.0f;
      if (live) {
        const float l = sm.red[0][row] + sm.red[1][row];
        const int h = row & (H - 1);
        const float z = p.sink ? __ldg(p.sink + h) * 1.4426950408889634f : -INFINITY;
        const float M = fmaxf(m, z);
        const float am = m == -INFINITY ? 0.0f : fast_exp2(m - M);
        const float L = l * am + (z == -INFINITY ? 0.0f : fast_exp2(z - M));
        inv = L == 0.0f ? 0.0f : am / L;
        if (bad) inv = NAN;
        if (p.lse && half == 0 && part == 0 && CSA2_IN_BOUNDS(query_row(item, tk) < p.nq, err))
          p.lse[(int64_t)query_row(item, tk) * H + h] =
              inv != inv ? NAN
              : m == -INFINITY ? (p.sink ? __ldg(p.sink + h) : -INFINITY)
                               : (M + log2f(L)) * 0.69314718055994531f;
      }
      // outputs, 32 rows x 32 channels at a time: rounded, turned in the warp's own
      // box so that four lanes have 64 bytes of a row (a lane that stores its own
      // row touches 32 lines an instruction), the next ones on their way
      uint16_t* out = p.out + 8 * (lane & 3);
      if (live) out += ((int64_t)query_row(item, tk) * H + ((32 * quad) & (H - 1)) + (lane >> 2)) * kHeadDim;
      for (int ch = ch0; ch < ch1; ch += width, ++chunk) {
        ok = mbar_wait(&sm.o_full, chunk & 1, err, wl) && ok;
        tc_fence_after();
        const int mine = width / 2 * half;   // this warp's columns of the accumulator: mine ..
        const uint32_t from = tmem + lanes + kOCol + mine;
#pragma unroll 1
        for (int b = 0; b < width / 64; ++b) {
          const int c = ch + mine + 32 * b;       // channel
          uint32_t x[32];
          if (live) tmem_ld32(from + 32 * b, x);
          if (b == width / 64 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.o_empty);
          }
          if (!live) continue;
          if (p.rope_out && c >= 448) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 t = sm.rope[tk][(c - 448) / 2 + i];
              const float u = __uint_as_float(x[2 * i]), v = __uint_as_float(x[2 * i + 1]);
              x[2 * i] = __float_as_uint(fmaf(u, t.x, -(v * t.y)));
              x[2 * i + 1] = __float_as_uint(fmaf(u, t.y, v * t.x));
            }
          }
          __syncwarp();   // the box's last contents are read
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(x[8 * q + 2 * i]) * inv,
                                                              __uint_as_float(x[8 * q + 2 * i + 1]) * inv);
              w[i] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            *reinterpret_cast<uint4*>(box + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
          if (ok && CSA2_IN_BOUNDS(query_row(item, tk) < p.nq && c >= 0 && c + 32 <= kHeadDim, err)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row_ = 8 * i + (lane >> 2);
              *reinterpret_cast<uint4*>(out + 8 * i * kHeadDim + c) = *reinterpret_cast<const uint4*>(
                  box + row_ * 64 + (((lane & 3) ^ ((row_ >> 1) & 3)) << 4));
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <class P, bool kFp8>
cudaError_t launch(const P& p, const CUtensorMap& q, int items, int sms,
                   cudaStream_t s) {
  if (items <= 0) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(
      k_window_attn<P, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // CTAs an item: one sequence takes 11.5 us with four where it takes 13.8 with one,
  // 70 take 12.9 with two (14.6 with one)
  const int split = (int64_t)items * 4 <= sms ? 4 : (int64_t)items * 2 <= sms ? 2 : 1;
  cfg.gridDim = dim3((unsigned)(split > 1 ? items * split : items < sms ? items : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_window_attn<P, kFp8>, p, q, split);
}

}  // namespace

cudaError_t launch_window_decode(const WinDecodeParams& p, const CUtensorMap& q, int sms, cudaStream_t s) {
  return p.w.fp8 ? launch<WinDecodeParams, true>(p, q, p.nq, sms, s)
                 : launch<WinDecodeParams, false>(p, q, p.nq, sms, s);
}

cudaError_t launch_window_tree(const WinTreeParams& p, const CUtensorMap& q, int sms, cudaStream_t s) {
  return p.w.fp8 ? launch<WinTreeParams, true>(p, q, p.n_items, sms < kWinTreeCtas ? sms : kWinTreeCtas, s)
                 : launch<WinTreeParams, false>(p, q, p.n_items, sms < kWinTreeCtas ? sms : kWinTreeCtas, s);
}

cudaError_t launch_window_prefill(const WinPrefillParams& p, const CUtensorMap& q, int sms, cudaStream_t s) {
  return launch<WinPrefillParams, false>(p, q, p.n_heads == 64 ? (p.nq + 1) / 2 : p.nq, sms, s);
}

}  // namespace csa2
