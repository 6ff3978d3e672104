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
// channel blocks of 64; P (bf16) goes from the softmax's registers to tensor
// memory; O is made in two halves of 256 channels, since both halves, S and P
// do not fit the 512 columns together.  A CTA takes neighbouring items: in a
// chunk the rows stay in shared memory as a ring of 17 blocks of 8 positions
// (and one of first tokens), of which one is replaced every 8 tokens.
//
// Roles: warp 0 loads Q (TMA), warp 1 issues the MMAs, warps 2 and 3 load
// rows, warps 4-11 (two for each quadrant of tensor memory lanes) do the
// softmax and the outputs, which leave through shared memory by TMA.
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
constexpr int kChunkFirst = 8 * kRing;  // first tokens, chunks
constexpr int kBlk = kSlots * 128;      // bytes of a 64-channel block of rows
constexpr int kStages = 3;              // Q: 128 rows x 64 channels each
constexpr int kStageBytes = 128 * 128;
constexpr int kLoadWarps = 2, kSoftWarps = 8;
constexpr int kRowWarps = kLoadWarps + kSoftWarps;

constexpr int kKvOff = 0;
constexpr int kQOff = kKvOff + 8 * kBlk;
constexpr int kOutOff = kQOff + kStages * kStageBytes;   // two boxes on their way out
constexpr int kSmallOff = kOutOff + 2 * kStageBytes;
struct Small {
  float red[2][128];            // [half of the columns][row]: maxima, then sums
  float2 rope[2][2][32];        // [item parity][token]: cos, sin of each channel pair
  uint32_t vis[2][5];           // rows that each token sees
  uint32_t bad[5];              // rows that hold an infinity or a NaN (chunks)
  alignas(4) uint8_t bad8[kRing + 1][4];   // the same, 8 rows of each block, by quarter of its loads
  uint8_t path[kRowWarps][64];  // trees: the path's drafts, every loading warp its own
  uint32_t tmem;
  uint64_t q_full[kStages], q_empty[kStages];
  uint64_t kv_full, kv_empty, s_full, p_full, o_full, o_empty, end;
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

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int32_t x,
                                             int32_t y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(x), "r"(y)
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

// Eight E4M3 codes (two words) x sc -> eight bf16, exact.
__device__ __forceinline__ uint4 e4m3_piece(uint32_t w0, uint32_t w1, float sc) {
  const uint32_t w[2] = {w0, w1};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
        (__nv_fp8x2_storage_t)((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * sc, f.y * sc);
    o[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <class P>
constexpr bool kIsChunk = std::is_same<P, WinPrefillParams>::value;
template <class P>
constexpr bool kIsTree = std::is_same<P, WinTreeParams>::value;

template <class P, bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    k_window_attn(const __grid_constant__ P p, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_out) {
  constexpr bool kChunk = kIsChunk<P>, kTree = kIsTree<P>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* kv = smem + kKvOff;
  Small& sm = *reinterpret_cast<Small*>(smem + kSmallOff);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = p.n_heads;
  const bool pair = kChunk && H == 64;    // an item is two tokens
  const int n_items = pair ? (p.nq + 1) / 2 : p.nq;
  const int item0 = (int)((int64_t)n_items * blockIdx.x / gridDim.x);
  const int item1 = (int)((int64_t)n_items * (blockIdx.x + 1) / gridDim.x);
  const int W = p.w.swa, F = p.w.n_first;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.q_full[s], 1);
      mbar_init(&sm.q_empty[s], 1);
    }
    mbar_init(&sm.kv_full, kChunk ? kLoadWarps : kRowWarps);
    mbar_init(&sm.kv_empty, 1);
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.p_full, kSoftWarps);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_empty, kSoftWarps);
    mbar_init(&sm.end, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_out);
  }
  if (warp == 1) { tmem_alloc(&sm.tmem, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  griddep_wait();
  uint32_t* err = p.err;

  // warps that load rows: 0 and 1, and of a cache (and a chunk's first window)
  // 2-9, the softmax's
  const int lw = warp - 2;
  const bool loader = warp == 2 || warp == 3, soft = warp >= 4;

  auto tokens_of = [&](int item) { return pair ? min(2, p.nq - 2 * item) : 1; };
  auto first_token = [&](int item) { return pair ? 2 * item : item; };
  auto piece = [&](int slot, int cb, int k) {
    return reinterpret_cast<uint4*>(kv + cb * kBlk + slot * 128 + ((k ^ (slot & 7)) << 4));
  };

  // ---------------------------------------------------------- rows, chunks
  // Ring block a holds the positions 8 g .. 8 g + 7 of the newest g = a mod 17
  // that is not above g_hi; positions out of the band are zeros.
  auto chunk_block_pos = [&](int64_t g_hi, int a) -> int64_t {
    int64_t d = (g_hi - a) % kRing;
    if (d < 0) d += kRing;
    return 8 * (g_hi - d);
  };
  // A quarter of a block's rows (unit v of 4): four 16-byte pieces a lane, of
  // row lane / 4.  kept in v[]; written by chunk_store.
  auto chunk_load = [&](int64_t g_hi, int a, int v, uint4 (&x)[4]) {
    if constexpr (kChunk) {
      const int r = lane >> 2;
      const uint16_t* src = nullptr;
      if (a < kRing) {
        const int64_t row = chunk_block_pos(g_hi, a) + r - p.band0;
        if (row >= 0 && row < p.n_band) src = p.band + row * kHeadDim;
      } else if (r < F) {
        if (r >= p.band0) {
          if (r - p.band0 < p.n_band) src = p.band + (r - p.band0) * kHeadDim;
        } else if (p.first) {
          src = p.first + r * kHeadDim;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = src ? ldg_now_v4(src + 8 * (4 * (4 * v + i) + (lane & 3))) : make_uint4(0u, 0u, 0u, 0u);
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
      *piece(slot, c >> 3, c & 7) = b ? make_uint4(0u, 0u, 0u, 0u) : x[i];
    }
    const uint32_t any = __ballot_sync(0xffffffffu, bad);
    const uint32_t rows = __ballot_sync(0xffffffffu, lane < 8 && ((any >> (4 * lane)) & 15u));
    if (lane == 0) sm.bad8[a][v] = (uint8_t)rows;
  };

  // ---------------------------------------------------------- rows, cache
  // Ring row j holds position x, the one that is j mod W among the W newest up
  // to `at`; first token f its own.  -1: none.
  auto slot_pos = [&](int64_t at, int at_mod, int j) -> int64_t {
    if (j < W) {
      int d = at_mod - j;
      if (d < 0) d += W;
      const int64_t x = at - d;
      return x >= F ? x : -1;
    }
    const int f = j - kFirstSlot;
    return f >= 0 && f < F && f <= at ? f : -1;
  };
  struct Query {
    int64_t at, pos0;   // its position; positions from pos0 on are drafts'
    int32_t seq, draft0;
    int at_mod;
  };
  auto query_of = [&](int q) -> Query {
    Query t = {};
    if constexpr (kTree) {
      const int tr = p.tree[q];
      t.pos0 = p.pos0[tr];
      t.at = t.pos0 + __popcll(p.path[q]) - 1;
      t.seq = p.seq[tr];
      t.draft0 = p.first[tr];
    } else if constexpr (!kChunk) {
      t.at = p.pos[q];
      t.pos0 = INT64_MAX;
      t.seq = p.identity ? p.seq0 + q : p.seq[q];
    }
    t.at_mod = t.at >= 0 ? (int)(t.at % W) : 0;
    return t;
  };
  // Row of the cache (>= 0) or of a draft (-2 - row) for slot j; -1: none.  A
  // row of the cache counts only if it holds position x.
  auto slot_row = [&](const Query& t, int j, int64_t& x) -> int64_t {
    x = slot_pos(t.at, t.at_mod, j);
    if (x < 0) return -1;
    if constexpr (kTree) {
      if (x >= t.pos0) return -2 - (t.draft0 + (int64_t)sm.path[lw][x - t.pos0]);
    }
    return j < W ? (int64_t)t.seq * W + j : (int64_t)p.w.n_seqs * W + (int64_t)t.seq * F + x;
  };
  // All rows of an item: a warp takes 16 rows x 2 chunks at a time (32-byte
  // pieces of 16 rows: every sector is read once and the swizzled stores have
  // no conflicts), several of them in flight.
  auto cache_load = [&](int item, int w0, int n_warps) {
    if constexpr (!kChunk) {
      const Query t = query_of(item);
      constexpr int kPairs = kFp8 ? 18 : 32;       // chunk pairs of a row
      constexpr int kUnits = kSlots / 16 * kPairs;
      constexpr int kBatch = 7;
      for (int u0 = w0; u0 < kUnits; u0 += kBatch * n_warps) {
        uint4 d[kBatch];
        uint32_t sb[kBatch];
        int64_t tag[kBatch], want[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int u = u0 + b * n_warps;
          d[b] = make_uint4(0u, 0u, 0u, 0u);
          sb[b] = 0;
          tag[b] = want[b] = 0;
          if (u < kUnits) {
            const int j = u / kPairs * 16 + (lane >> 1), c = u % kPairs * 2 + (lane & 1);
            int64_t x;
            int64_t row = slot_row(t, j, x);
            if (row != -1) {
              const uint16_t* rows = p.w.rows;
              const uint8_t* codes = p.w.codes;
              const uint16_t* rope = p.w.rope;
              const uint8_t* scales = p.w.scales;
              bool draft = false;
              if constexpr (kTree) {
                if (row < 0) {
                  draft = true;
                  row = -2 - row;
                  rows = p.d.rows;
                  codes = p.d.codes;
                  rope = p.d.rope;
                  scales = p.d.scales;
                }
              }
              if (!draft) {
                want[b] = x;
                tag[b] = p.w.pos[row];
              }
              if constexpr (kFp8) {
                if (c < 28) {
                  d[b] = ldg_now_v4(codes + row * 448 + 16 * c);
                  sb[b] = ldg_now_u8(scales + row * 8 + (c >> 2));
                } else {
                  d[b] = ldg_now_v4(rope + row * 64 + 8 * (c - 28));
                }
              } else {
                d[b] = ldg_now_v4(rows + row * kHeadDim + 8 * c);
              }
            }
          }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int u = u0 + b * n_warps;
          if (u >= kUnits) break;
          const int j = u / kPairs * 16 + (lane >> 1), c = u % kPairs * 2 + (lane & 1);
          const bool held = tag[b] == want[b];
          if constexpr (kFp8) {
            if (c < 28) {
              const float sc = held ? ue8m0_value(sb[b]) : 0.0f;
              if (!held) d[b] = make_uint4(0u, 0u, 0u, 0u);
              const int cb = c >> 2, k = 2 * (c & 3);
              *piece(j, cb, k) = e4m3_piece(d[b].x, d[b].y, sc);
              *piece(j, cb, k + 1) = e4m3_piece(d[b].z, d[b].w, sc);
            } else {
              *piece(j, 7, c - 28) = held ? d[b] : make_uint4(0u, 0u, 0u, 0u);
            }
          } else {
            *piece(j, c >> 3, c & 7) = held ? d[b] : make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
    }
  };

  // ---------------------------------------------------------- masks, rotation
  // Rows that each token of an item sees (the two loading warps: slots 0-127,
  // then 128-143 by the first), and the sines of the output rotation.
  auto item_tables = [&](int item) {
    const int par = (item - item0) & 1;
    const int n_tok = tokens_of(item), t0 = first_token(item);
    auto bits = [&](int j, int word) {
      bool v0 = false, v1 = false, b = false;
      if constexpr (kChunk) {
        const int64_t at0 = p.pos0 + t0, hi = at0 + n_tok - 1;
        int64_t x = -1;
        bool first = false;
        if (j < kChunkFirst) {
          x = chunk_block_pos(hi >> 3, j >> 3) + (j & 7);
          if (x < F || x < p.band0) x = -1;
        } else {
          first = true;
          x = j - kChunkFirst < F ? j - kChunkFirst : -1;
        }
        v0 = x >= 0 && x <= at0 && (first || x > at0 - W);
        v1 = n_tok > 1 && x >= 0 && x <= hi && (first || x > hi - W);
        const uint32_t q = *reinterpret_cast<const uint32_t*>(sm.bad8[j >> 3]);
        b = ((q | (q >> 8) | (q >> 16) | (q >> 24)) >> (j & 7)) & 1u;
      } else {
        const Query t = query_of(item);
        int64_t x;
        const int64_t row = slot_row(t, j, x);
        v0 = row < -1 || (row >= 0 && p.w.pos[row] == x);
      }
      const uint32_t m0 = __ballot_sync(0xffffffffu, v0), m1 = __ballot_sync(0xffffffffu, v1);
      const uint32_t mb = __ballot_sync(0xffffffffu, b);
      if (lane == 0) {
        sm.vis[0][word] = m0;
        sm.vis[1][word] = m1;
        sm.bad[word] = mb;
      }
    };
    bits(64 * lw + lane, 2 * lw);
    bits(64 * lw + 32 + lane, 2 * lw + 1);
    if (lw == 0) bits(128 + (lane & 15), 4);
    if (p.rope_out) {
      const int tk = lw;
      if (tk < n_tok) {
        int64_t at;
        if constexpr (kChunk) at = p.pos0 + t0 + tk;
        else at = query_of(item).at;
        const uint64_t turn = (uint64_t)(-at) * p.turns[lane];
        float sn, cs;
        sincospif((float)(int64_t)turn * 0x1p-63f, &sn, &cs);
        sm.rope[par][tk][lane] = make_float2(cs, sn);
      }
    }
  };
  auto tree_path = [&](int item) {
    if constexpr (kTree) {
      const uint64_t path = p.path[item];
      __syncwarp();
#pragma unroll
      for (int b = lane; b < 64; b += 32)
        if ((path >> b) & 1ull) sm.path[lw][__popcll(path & ((1ull << b) - 1ull))] = (uint8_t)b;
      __syncwarp();
    }
  };

  bool ok = true;
  if constexpr (kChunk) {
    // the first item's whole window: 18 blocks in quarters over the ten
    // loading and softmax warps, four quarters in flight
    if ((loader || soft) && item0 < item1) {
      const int64_t hi = p.pos0 + first_token(item0) + tokens_of(item0) - 1;
      constexpr int kJobs = (kRing + 1) * 4, kBatch = 4;
      for (int j0 = lw; j0 < kJobs; j0 += kBatch * kRowWarps) {
        uint4 x[kBatch][4];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int j = j0 + b * kRowWarps;
          if (j < kJobs) chunk_load(hi >> 3, j >> 2, j & 3, x[b]);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int j = j0 + b * kRowWarps;
          if (j < kJobs) chunk_store(j >> 2, j & 3, x[b]);
        }
      }
      fence_proxy_async_smem();
    }
    __syncthreads();
  }

  if (warp == 0) {
    // ------------------------------------------------------------ Q
    if (lane == 0) {
      uint32_t n = 0;
      for (int item = item0; item < item1 && ok; ++item) {
        const int boxes = tokens_of(item) * H / 64;
        const int32_t row = first_token(item) * H;
        for (int cb = 0; cb < 8 && ok; ++cb, ++n) {
          const uint32_t s = n % kStages, use = n / kStages;
          if (use > 0) ok = mbar_wait(&sm.q_empty[s], (use - 1) & 1, err);
          if (!ok) break;
          mbar_arrive_expect_tx(&sm.q_full[s], boxes * 8192);
          uint8_t* dst = smem + kQOff + s * kStageBytes;
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(dst + b * 8192, &tm_q, 64 * cb, row + 64 * b, &sm.q_full[s]);
        }
      }
      // the copies in flight must land before the CTA exits
      if (!ok)
        for (uint32_t k = n > kStages ? n - kStages : 0; k < n; ++k)
          mbar_wait(&sm.q_full[k % kStages], (k / kStages) & 1, err, drain_limit(0));
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_bf16_f32(128, kSlots, false, false);
      constexpr uint32_t id_o = idesc_bf16_f32(128, 256, false, true);
      const uint64_t d_q = sdesc_sw128(smem_u32(smem + kQOff), 16, 1024);
      const uint64_t d_k = sdesc_sw128(smem_u32(kv), 16, 1024);
      const uint64_t d_v = sdesc_sw128(smem_u32(kv), kBlk, 1024);
      uint32_t n = 0, chunk = 0;
      for (int item = item0; item < item1 && ok; ++item) {
        const uint32_t ph = (uint32_t)(item - item0) & 1u;
        ok = mbar_wait(&sm.kv_full, ph, err);
        for (int cb = 0; cb < 8 && ok; ++cb, ++n) {
          const uint32_t s = n % kStages;
          ok = mbar_wait(&sm.q_full[s], (n / kStages) & 1, err);
          if (!ok) break;
          tc_fence_after();
          for (int k = 0; k < 4; ++k)
            umma_bf16(tmem + kSCol, d_q + ((s * kStageBytes + 32 * k) >> 4),
                      d_k + ((cb * kBlk + 32 * k) >> 4), id_s, (cb | k) ? 1u : 0u);
          umma_commit(&sm.q_empty[s]);
        }
        if (!ok) break;
        umma_commit(&sm.s_full);
        ok = mbar_wait(&sm.p_full, ph, err);
        for (int h = 0; h < 2 && ok; ++h, ++chunk) {
          if (chunk > 0) ok = mbar_wait(&sm.o_empty, (chunk - 1) & 1, err);
          if (!ok) break;
          tc_fence_after();
          for (int ks = 0; ks < kSlots / 16; ++ks)
            umma_bf16_ts(tmem + kOCol, tmem + kPCol + 8 * ks,
                         d_v + ((4 * h * kBlk + ks * 2048) >> 4), id_o, ks ? 1u : 0u);
          umma_commit(&sm.o_full);
        }
        if (ok) umma_commit(&sm.kv_empty);
      }
      if (!ok) {   // the MMAs issued so far must end before the CTA exits
        umma_commit(&sm.end);
        mbar_wait(&sm.end, 0, err, drain_limit(0));
      }
    }
  } else if (loader) {
    // ------------------------------------------------------------ rows
    int64_t g_have = 0;
    for (int item = item0; item < item1 && ok; ++item) {
      const uint32_t k = (uint32_t)(item - item0);
      if constexpr (kChunk) {
        const int64_t g = (p.pos0 + first_token(item) + tokens_of(item) - 1) >> 3;
        // at most one new block an item (of at most two tokens)
        const bool fresh = k > 0 && g != g_have;
        g_have = g;
        uint4 x[2][4];
        const int a = (int)(g % kRing);
        if (fresh) {
          chunk_load(g, a, 2 * lw, x[0]);
          chunk_load(g, a, 2 * lw + 1, x[1]);
        }
        if (k > 0) ok = mbar_wait_sleep(&sm.kv_empty, (k - 1) & 1, err);
        if (fresh && ok) {
          chunk_store(a, 2 * lw, x[0]);
          chunk_store(a, 2 * lw + 1, x[1]);
        }
        ok = named_bar_and(3, 32 * kLoadWarps, ok);
        if (!ok) break;
        item_tables(item);
      } else {
        if (k > 0) ok = mbar_wait_sleep(&sm.kv_empty, (k - 1) & 1, err);
        if (!ok) break;
        tree_path(item);
        cache_load(item, lw, kRowWarps);
        item_tables(item);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.kv_full);
    }
  } else if (soft) {
    // ------------------------------------------------------------ softmax, outputs
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int row = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const bool issuer = quad == 0 && lane == 0;   // of the half's copies out
    uint8_t* stage = smem + kOutOff + half * kStageBytes;
    uint32_t chunk = 0;
    for (int item = item0; item < item1; ++item) {
      const uint32_t k = (uint32_t)(item - item0), ph = k & 1u;
      if constexpr (!kChunk) {
        if (k > 0) ok = mbar_wait(&sm.kv_empty, (k - 1) & 1, err) && ok;
        tree_path(item);
        cache_load(item, lw, kRowWarps);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.kv_full);
      }
      const int n_rows = tokens_of(item) * H;
      const bool live = quad * 32 < n_rows;       // of the warp's rows, all or none
      const int tk = pair ? row >> 6 : 0;
      ok = mbar_wait(&sm.kv_full, ph, err) && ok;
      ok = mbar_wait(&sm.s_full, ph, err) && ok;
      ok = named_bar_and(1, 32 * kSoftWarps, ok);
      if (!ok) break;
      tc_fence_after();
      // a thread has a half of its row: columns 0-79 or 80-143
      const int g0 = half ? 5 : 0, ng = half ? 4 : 5;
      uint32_t s[5][16];
      float m = -INFINITY;
      if (live) {
#pragma unroll
        for (int g = 0; g < 5; ++g)
          if (g < ng) tmem_ld16_issue(tmem + lanes + kSCol + 16 * (g0 + g), s[g]);
#pragma unroll
        for (int g = 0; g < 5; ++g)
          if (g < ng) tmem_ld16_wait(s[g]);
#pragma unroll
        for (int g = 0; g < 5; ++g) {
          if (g < ng) {
            const uint32_t v = sm.vis[tk][(g0 + g) >> 1] >> (16 * ((g0 + g) & 1));
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float x = (v >> i) & 1u ? __uint_as_float(s[g][i]) * p.scale_log2 : -INFINITY;
              s[g][i] = __float_as_uint(x);
              m = fmaxf(m, x);
            }
          }
        }
        sm.red[half][row] = m;
      }
      named_bar(1, 32 * kSoftWarps);
      if (live) m = fmaxf(m, sm.red[half ^ 1][row]);
      named_bar(1, 32 * kSoftWarps);
      float sum = 0.0f;
      bool bad = false;
      if (live) {
        if constexpr (kChunk) {   // before the next item's masks may come
          uint32_t b = 0;
#pragma unroll
          for (int i = 0; i < 5; ++i) b |= sm.vis[tk][i] & sm.bad[i];
          bad = b != 0;
        }
        const float m0 = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int g = 0; g < 5; ++g) {
          if (g < ng) {
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a = fast_exp2(__uint_as_float(s[g][2 * i]) - m0);
              const float b = fast_exp2(__uint_as_float(s[g][2 * i + 1]) - m0);
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(a, b);
              pk[i] = *reinterpret_cast<const uint32_t*>(&b2);
              sum += __uint_as_float(pk[i] << 16) + __uint_as_float(pk[i] & 0xFFFF0000u);
            }
            tmem_st8(tmem + lanes + kPCol + 8 * (g0 + g), pk);
          }
        }
        sm.red[half][row] = sum;
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full);
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
        if (p.lse && half == 0)
          p.lse[(int64_t)first_token(item) * H + row] =
              inv != inv ? NAN
              : m == -INFINITY ? (p.sink ? __ldg(p.sink + h) : -INFINITY)
                               : (M + log2f(L)) * 0.69314718055994531f;
      }
      const int32_t out_row = first_token(item) * H;
      for (int h = 0; h < 2; ++h, ++chunk) {
        ok = mbar_wait(&sm.o_full, chunk & 1, err) && ok;
        tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
          const int cb = 2 * half + b;            // 64-channel block of the half
          uint32_t w[32];
          if (live) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              uint32_t r[32];
              tmem_ld32(tmem + lanes + kOCol + 64 * cb + 32 * g, r);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float a = __uint_as_float(r[2 * i]) * inv, c = __uint_as_float(r[2 * i + 1]) * inv;
                if (p.rope_out && h == 1 && cb == 3) {
                  const float2 t = sm.rope[ph][tk][16 * g + i];
                  const float a2 = fmaf(a, t.x, -(c * t.y));
                  c = fmaf(a, t.y, c * t.x);
                  a = a2;
                }
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(a, c);
                w[16 * g + i] = *reinterpret_cast<const uint32_t*>(&b2);
              }
            }
          }
          if (b == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.o_empty);
          }
          if (issuer) bulk_wait_read();
          named_bar(4 + half, 16 * kSoftWarps);
          if (live) {
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint4*>(stage + row * 128 + ((c ^ (row & 7)) << 4)) =
                  make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
          }
          fence_proxy_async_smem();
          named_bar(4 + half, 16 * kSoftWarps);
          if (issuer && ok) {
            for (int i = 0; i < n_rows / 64; ++i)
              tma_store_2d(&tm_out, stage + 8192 * i, 64 * (4 * h + cb), out_row + 64 * i);
          }
        }
      }
    }
    if (issuer) bulk_wait_read();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <class P, bool kFp8>
cudaError_t launch(const P& p, const CUtensorMap& q, const CUtensorMap& out, int items, int sms,
                   cudaStream_t s) {
  if (items <= 0) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(
      k_window_attn<P, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < sms ? items : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_window_attn<P, kFp8>, p, q, out);
}

}  // namespace

cudaError_t launch_window_decode(const WinDecodeParams& p, const CUtensorMap& q,
                                 const CUtensorMap& out, int sms, cudaStream_t s) {
  return p.w.fp8 ? launch<WinDecodeParams, true>(p, q, out, p.nq, sms, s)
                 : launch<WinDecodeParams, false>(p, q, out, p.nq, sms, s);
}

cudaError_t launch_window_tree(const WinTreeParams& p, const CUtensorMap& q,
                               const CUtensorMap& out, int sms, cudaStream_t s) {
  return p.w.fp8 ? launch<WinTreeParams, true>(p, q, out, p.nq, sms, s)
                 : launch<WinTreeParams, false>(p, q, out, p.nq, sms, s);
}

cudaError_t launch_window_prefill(const WinPrefillParams& p, const CUtensorMap& q,
                                  const CUtensorMap& out, int sms, cudaStream_t s) {
  return launch<WinPrefillParams, false>(p, q, out, p.n_heads == 64 ? (p.nq + 1) / 2 : p.nq, sms, s);
}

}  // namespace csa2
