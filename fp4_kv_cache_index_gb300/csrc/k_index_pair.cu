// k_index_pair.cu -- index scores of drafted queries over bf16 keys on pairs
// of SMs, for trees whose groups hold up to eight queries (the score and the
// rows' layout of k_index.cu's trees).
//
// Why pairs.  One MMA of k_index.cu is 128 keys x 256 (query, head) columns x
// 16 channels: 4 KB of keys and 8 KB of queries from shared memory, which the
// tensor core fetches at about 64 bytes a cycle, so it takes 195 cycles for
// 128 cycles of arithmetic (128 queries over 2 x 131072 entries: 112 us, the
// MMAs alone 84).  A pair of CTAs issues one MMA of 256 keys x 256 columns
// (cta_group::2): each SM brings 128 keys and half of the queries, 8 KB for
// the same arithmetic, and keeps the accumulator rows of its own keys.
//
// Tiles are 256 keys; CTA r of the pair loads, and forms the scores of, the
// keys 128 r .. 128 r + 127 of each, and holds the query rows 128 r .. of the
// group.  The leader (CTA 0) issues the MMAs.  Barriers: k_full and q_full of
// the leader count the bytes of both CTAs' copies; the MMAs' completion is
// multicast to both CTAs' k_empty, q_empty and acc_full; the epilogue warps of
// both CTAs arrive at the leader's acc_empty.  Every wait is bounded.
//
// Warps: 0 the TMA producer, 1 the MMA issuer (of the leader) and owner of
// tensor memory, 2-17 the epilogue, four per TMEM lane quadrant, each with a
// quarter of the group's queries; its loads of tensor memory run one half row
// (16 heads) ahead of the arithmetic.
#include "csa2_device.cuh"
#include "csa2_kernels.h"

namespace csa2 {
namespace {

constexpr int kEpiThreads = 512;
constexpr int kThreads = 64 + kEpiThreads;
constexpr int kQpg = 8;                                // queries of a group
constexpr int kPairTile = 256;                         // keys of a tile
constexpr int kMyKeys = 128;                           // of which this CTA has these
constexpr int kStageBytes = kMyKeys * kIdxDim * 2;     // 32 KB
constexpr int kStages = 4;
constexpr int kQRows = kQpg * kIdxHeads / 2;           // query rows of this CTA
constexpr int kQBytes = kQRows * kIdxDim * 2;          // 32 KB
constexpr int kN = kQpg * kIdxHeads;                   // accumulator columns
constexpr int kQOff = kStages * kStageBytes;
constexpr int kWOff = kQOff + kQBytes;
constexpr int kHistOff = kWOff + kQpg * kIdxHeads * 4;
constexpr int kBarOff = kHistOff + kQpg * kKeyHistBins * 4;
constexpr int kBars = 2 * kStages + 8;
constexpr int kSmemBytes = kBarOff + kBars * 8 + 16 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory");

// Commit of the pair's MMAs, arriving on the barrier at this place in both
// CTAs (or only in this one).
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void pair_commit_here(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Tiled load into this CTA's shared memory, its bytes counted at `bar` (a
// cluster address: the leader's barrier).
__device__ __forceinline__ void pair_load_2d(void* dst, const CUtensorMap* m, int32_t x, int32_t y,
                                             uint32_t bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2.L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "l"(pol)
      : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    k_index_pair(const __grid_constant__ TreeIndexParams p,
                 const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_q) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* kbuf = smem;
  uint8_t* qbuf = smem + kQOff;
  float* wbuf = reinterpret_cast<float*>(smem + kWOff);
  uint32_t* hs = reinterpret_cast<uint32_t*>(smem + kHistOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
  uint64_t* k_full = bars;                  // [kStages], the leader's
  uint64_t* k_empty = bars + kStages;       // [kStages]
  uint64_t* acc_full = bars + 2 * kStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;       // [2], the leader's
  uint64_t* q_full = acc_full + 4;          // the leader's
  uint64_t* q_empty = q_full + 1;
  uint64_t* drain = q_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) { mbar_init(k_full + i, 1); mbar_init(k_empty + i, 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, 2 * kEpiThreads / 32);   // the epilogue warps of both CTAs
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_q);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  // both CTAs' barriers are set up before either signals the other
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  const long long wl = wait_limit(p.wait_cycles);   // bounded-wait limit (cycles)

  // this pair's tiles; group g holds the tiles [tile_prefix[g], tile_prefix[g + 1])
  const int total = p.tile_prefix[p.n_groups];
  const int pairs = (int)gridDim.x / 2, pair = (int)blockIdx.x / 2;
  const int begin = (int)(((int64_t)total * pair) / pairs);
  const int end = (int)(((int64_t)total * (pair + 1)) / pairs);
  int g0 = 0;
  while (g0 < p.n_groups && p.tile_prefix[g0 + 1] <= begin) ++g0;
  struct Cursor {
    int g, lo, hi;
  };
  auto advance = [&](Cursor& c, int it) {   // to the group of tile `it`
    while (c.hi <= it) {
      ++c.g;
      c.lo = c.hi;
      c.hi = p.tile_prefix[c.g + 1];
    }
  };
  const Cursor c0 = {g0, p.tile_prefix[g0], p.tile_prefix[g0 + 1]};

  if (warp == 0 && lane == 0 && begin < end) {
    // ------------------------------------------------ producer
    const uint64_t pol = l2_policy_evict_first();
    Cursor gc = c0;
    int cur = -1, stage = 0;
    int64_t base = 0;
    uint32_t ph = 0, qph = 0;
    uint32_t armed = 0, armed_ph = 0;   // stages filled at least once, parity of the last fill
    bool ok = true;
    for (int it = begin; it < end && ok; ++it) {
      advance(gc, it);
      if (gc.g != cur) {
        cur = gc.g;
        base = p.entry_base[cur];
        ok = mbar_wait(q_empty, qph ^ 1, p.err, wl);
        if (!ok) break;
        qph ^= 1;
        const int row = p.q_first[cur] * kIdxHeads + rank * kQRows;
        if (leader) mbar_arrive_expect_tx(q_full, 2u * kQBytes);
        const uint32_t bar = dsmem_addr(smem_u32(q_full), 0);
        pair_load_2d(qbuf, &tm_q, 0, row, bar, pol);
        pair_load_2d(qbuf + kQBytes / 2, &tm_q, 64, row, bar, pol);
      }
      ok = mbar_wait(k_empty + stage, ph ^ 1, p.err, wl);
      if (!ok) break;
      if (!(p.inject & kInjectNoKeyLoads)) {   // tests: nothing arrives on k_full
        uint8_t* dst = kbuf + stage * kStageBytes;
        const int32_t row = (int32_t)(base + (int64_t)(it - gc.lo) * kPairTile + rank * kMyKeys);
        if (leader) mbar_arrive_expect_tx(k_full + stage, 2u * kStageBytes);
        const uint32_t bar = dsmem_addr(smem_u32(k_full + stage), 0);
        pair_load_2d(dst, &tm_k, 0, row, bar, pol);
        pair_load_2d(dst + kStageBytes / 2, &tm_k, 64, row, bar, pol);
        armed |= 1u << stage;
        armed_ph = (armed_ph & ~(1u << stage)) | (ph << stage);
      }
      if (++stage == kStages) { stage = 0; ph ^= 1; }
    }
    // no copy may still be writing into either CTA's shared memory (the
    // leader's barriers count both)
    if (leader) {
      for (int s = 0; s < kStages; ++s)
        if (armed & (1u << s)) mbar_wait(k_full + s, (armed_ph >> s) & 1u, p.err, wl);
      if (cur >= 0) mbar_wait(q_full, qph ^ 1, p.err, wl);
    }
  } else if (warp == 1 && lane == 0 && leader && begin < end) {
    // ------------------------------------------------ MMA issuer
    const uint32_t idesc = idesc_bf16_f32(256, kN, false, false);
    const uint64_t adesc0 = sdesc_sw128(smem_u32(kbuf), 16, 1024);
    const uint64_t bdesc0 = sdesc_sw128(smem_u32(qbuf), 16, 1024);
    Cursor gc = c0;
    int cur = -1, stage = 0, acc = 0;
    uint32_t ph = 0, qph = 0, aph = 0;
    bool ok = true;
    for (int it = begin; it < end && ok; ++it) {
      advance(gc, it);
      if (gc.g != cur) {
        cur = gc.g;
        ok = mbar_wait(q_full, qph, p.err, wl);
        if (!ok) break;
        qph ^= 1;
      }
      ok = mbar_wait(k_full + stage, ph, p.err, wl) &&
           mbar_wait_cluster(acc_empty + acc, aph ^ 1, p.err, wl);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem_base + (uint32_t)(acc * kN);
#pragma unroll
      for (int ks = 0; ks < kIdxDim / 16; ++ks) {
        const uint32_t ao = (uint32_t)(stage * kStageBytes + (ks >> 2) * (kStageBytes / 2) + (ks & 3) * 32);
        const uint32_t bo = (uint32_t)((ks >> 2) * (kQBytes / 2) + (ks & 3) * 32);
        pair_mma(d, adesc0 + (ao >> 4), bdesc0 + (bo >> 4), idesc, ks > 0 ? 1u : 0u);
      }
      pair_commit(k_empty + stage);
      pair_commit(acc_full + acc);
      if (it + 1 == end || gc.hi <= it + 1) pair_commit(q_empty);
      if (++stage == kStages) { stage = 0; ph ^= 1; }
      if (++acc == 2) { acc = 0; aph ^= 1; }
    }
    pair_commit_here(drain);
    mbar_wait(drain, 0, p.err, wl);
  } else if (warp >= 2) {
    // ------------------------------------------------ epilogue
    const int quad = warp & 3, row = quad * 32 + lane;
    const int et = threadIdx.x - 64;
    const int j0 = ((warp - 2) >> 2) * 2;          // this warp's queries of the group
    const bool use_hist = p.key_hist != nullptr;
    constexpr int hbins = kQpg * kKeyHistBins;
    auto esync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiThreads) : "memory"); };
    auto flush = [&](int gg) {
      esync();
      const int q0 = p.q_first[gg], q1 = p.q_first[gg + 1];
      for (int i = et; i < hbins; i += kEpiThreads) {
        const uint32_t v = hs[i];
        const int q = q0 + i / kKeyHistBins;
        if (v && q < q1)
          atomicAdd(p.key_hist + (int64_t)q * kKeyHistBins + (i % kKeyHistBins), v);
        hs[i] = 0u;
      }
      esync();
    };
    if (use_hist)
      for (int i = et; i < hbins; i += kEpiThreads) hs[i] = 0u;
    const uint32_t empty0 = dsmem_addr(smem_u32(acc_empty), 0);
    Cursor gc = c0;
    int cur = -1, acc = 0;
    uint32_t aph = 0;
    int mine = 0;                  // live queries of this warp
    int ncom = 0, nvis = 0;        // committed entries, and with the drafts'
    float* out[2] = {nullptr, nullptr};
    uint64_t ents[2] = {0, 0};
    for (int it = begin; it < end; ++it) {
      advance(gc, it);
      const int g = gc.g;
      if (g != cur) {
        if (use_hist && cur >= 0) flush(cur);
        esync();
        const int qg = p.q_first[g], qe = p.q_first[g + 1];
        for (int i = et; i < kQpg * kIdxHeads; i += kEpiThreads) {
          const int q = qg + (i >> 5);
          wbuf[i] = (q < qe) ? __ldg(p.w + (int64_t)q * kIdxHeads + (i & 31)) : 0.0f;
        }
        esync();
        cur = g;
        ncom = p.n_com[g];
        nvis = p.nvis[g];
        mine = max(0, min(2, qe - qg - j0));
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          const int q = min(qg + j0 + jj, p.nq - 1);
          out[jj] = p.scores + (int64_t)q * p.ld;
          ents[jj] = p.ents[q];
        }
      }
      const int e0 = (it - gc.lo) * kPairTile + rank * kMyKeys, e = e0 + row;
      auto store = [&](int jj, float s) {
        int col = e;
        if (e0 + kMyKeys > ncom) {   // the sequence's last tiles
          if (e >= nvis) return;
          if (e >= ncom) {
            // a draft's entry: the path's only, in the order of the path
            const int b = e - ncom;
            if (!((ents[jj] >> b) & 1u)) return;
            col = ncom + __popcll(ents[jj] & ((1ull << b) - 1ull));
          }
        }
        if (!CSA2_IN_BOUNDS(col < p.ld, p.err)) return;
        out[jj][col] = s;
        if (use_hist) atomicAdd(hs + (j0 + jj) * kKeyHistBins + (score_key(s) >> 21), 1u);
      };
      if (!mbar_wait(acc_full + acc, aph, p.err, wl)) break;
      tc_fence_after();
      // the accumulator is free once this warp's last columns are read
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(empty0 + 8u * (uint32_t)acc);
      };
      const uint32_t ta = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(acc * kN + j0 * 32);
      uint32_t ra[16], rb[16];
      if (mine > 0) {
        tmem_ld16_issue(ta, ra);
        tmem_ld16_wait(ra);
      } else {
        release();
      }
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        if (jj >= mine) break;
        const float* w = wbuf + (j0 + jj) * 32;
        uint64_t a = 0, b = 0;
        tmem_ld16_issue(ta + 32 * jj + 16, rb);
        relu_dot_chains(w, ra, 16, a, b);
        tmem_ld16_wait(rb);
        if (jj + 1 < mine) tmem_ld16_issue(ta + 32 * (jj + 1), ra);
        else release();
        relu_dot_chains(w + 16, rb, 16, a, b);
        if (jj + 1 < mine) tmem_ld16_wait(ra);
        store(jj, relu_dot_sum(a, b));
      }
      if (++acc == 2) { acc = 0; aph ^= 1; }
    }
    if (use_hist && cur >= 0) flush(cur);
  }

  tc_fence_before();
  __syncthreads();
  // neither CTA leaves, nor frees its tensor memory, while the other's copies,
  // MMAs or arrivals may still reach it
  cluster_arrive();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem_base)
                 : "memory");
  }
}

}  // namespace

cudaError_t launch_index_pair(const TreeIndexParams& p, const CUtensorMap& tm_k,
                              const CUtensorMap& tm_q, int pairs, cudaStream_t s) {
  if (p.qpg != kQpg || p.tile_keys != kPairTile) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(k_index_pair, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_index_pair, p, tm_k, tm_q);
}

}  // namespace csa2
