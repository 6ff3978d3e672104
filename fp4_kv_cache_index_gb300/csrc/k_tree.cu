// k_tree.cu -- the small kernels around trees of drafted tokens: selected
// score columns back to cache entries, and the accepted path's entries moved
// up behind the committed ones.
#include "csa2_device.cuh"
#include "csa2_kernels.h"

namespace csa2 {
namespace {

// One warp per row.  A row's columns are ascending, and its path's entries
// are the last ones, at most 64 before the padding; every column below n_com
// already is its entry.
__global__ void __launch_bounds__(256) k_tree_map(const __grid_constant__ TreeMapParams p) {
  griddep_wait();
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= p.rows) return;
  const int n_com = p.n_com[row];
  const uint64_t ents = p.ents[row];
  int32_t* idx = p.idx + (int64_t)row * p.k;
  for (int i = lane; i < p.k; i += 32) {
    const int32_t c = idx[i];
    if (c < n_com) continue;
    if (c - n_com >= __popcll(ents)) {   // no column of the row
      idx[i] = -1;
      continue;
    }
    // position of the (c - n_com)-th set bit
    uint64_t m = ents;
    for (int j = c - n_com; j > 0; --j) m &= m - 1;
    idx[i] = n_com + __ffsll((long long)m) - 1;
  }
}

// One block per sequence: at most 64 rows of 256 code bytes, 16 or 32 scale
// bytes and a 256-byte (or 64 + 4 byte) indexer key.  All sources are read
// into registers before anything is written, since the ranges overlap.
constexpr int kAcceptThreads = 512;
__global__ void __launch_bounds__(kAcceptThreads) k_accept(const __grid_constant__ AcceptParams p) {
  const AcceptSeg& g = p.seg[blockIdx.x];
  const int n = __popcll(g.keep);
  const int tid = threadIdx.x;
  __shared__ int32_t src[64];
  if (tid < 64 && ((g.keep >> tid) & 1u)) src[__popcll(g.keep & ((1ull << tid) - 1ull))] = tid;
  if (tid == 0) p.d_len[g.seq] = g.new_len;
  __syncthreads();
  // 16-byte pieces of a row: 16 of codes, 1 or 2 of scales, 16 or 4 of key
  const int ns = p.scale_bytes / 16, nk = p.idxk ? 16 : 4, per = 16 + ns + nk;
  constexpr int kMine = (64 * 34 + kAcceptThreads - 1) / kAcceptThreads;
  uint8_t* const idx_rows = p.idxk ? reinterpret_cast<uint8_t*>(p.idxk) : p.idx_codes;
  auto place = [&](int64_t row, int c) -> uint4* {
    uint8_t* a = c < 16        ? p.codes + row * kCodeBytes + 16 * c
                 : c < 16 + ns ? p.scales + row * p.scale_bytes + 16 * (c - 16)
                               : idx_rows + row * (16 * nk) + 16 * (c - 16 - ns);
    return reinterpret_cast<uint4*>(a);
  };
  uint4 v[kMine];
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int i = tid + k * kAcceptThreads;
    if (i < n * per) v[k] = *place(g.row0 + src[i / per], i % per);
  }
  uint32_t sw = 0;   // MXFP4 keys: the scale word of row tid
  const bool words = !p.idxk && tid < n;
  if (words) sw = reinterpret_cast<const uint32_t*>(p.idx_scales)[g.row0 + src[tid]];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int i = tid + k * kAcceptThreads;
    if (i < n * per) *place(g.row0 + i / per, i % per) = v[k];
  }
  if (words) reinterpret_cast<uint32_t*>(p.idx_scales)[g.row0 + tid] = sw;
}

}  // namespace

cudaError_t launch_tree_map(const TreeMapParams& p, cudaStream_t s) {
  if (p.rows <= 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((p.rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_tree_map, p);
}

cudaError_t launch_accept(const AcceptParams& p, cudaStream_t s) {
  if (p.n_segs <= 0) return cudaSuccess;
  k_accept<<<(unsigned)p.n_segs, kAcceptThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace csa2
