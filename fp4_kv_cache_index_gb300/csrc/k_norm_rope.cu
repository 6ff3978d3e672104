// k_norm_rope.cu -- RMS norm of every head and the position rotation of its
// last channels, in one pass, for several tensors in one launch.
//
//     y = x * rsqrt(mean(x^2) + eps) * weight,
//     (y[r + 2t], y[r + 2t + 1]) rotated by pos * base^(-2t / rope_dim),
// r = dim - rope_dim (the convention of the readout's output rotation, with
// the opposite sign), in fp32, rounded once to the output's type.  The
// reports place it before the attention: queries and KV rows are normed per
// head and rotated on their last 64 channels before the cache quantises them
// (V4.1 report, section 2.4.4; blog reading of the DeepSeek-V4 report,
// section 4.3).
//
// Bound: memory traffic (about 4 flops per element read and written).  A row
// (one head of one token) is held by dim / 16 lanes, 16 channels each in two
// chunks of 8 (chunk l and chunk l + dim / 16), so that every 16-byte access
// of a bf16 row is contiguous over the lanes and the channels stay in
// registers between the sum of squares and the store.  A block takes
// consecutive (token, head) rows of one tensor; it forms the sines and
// cosines of its tokens once, in shared memory, while its rows are in flight.
//
// Angles: pos * f, f in turns per position, is formed modulo one turn in
// 64-bit integer arithmetic (f as a 64-bit fraction: the low 64 bits of the
// product are the fraction of a turn, exact for any position), so far
// positions lose nothing and no 64-bit floating point is needed; sincospif
// then takes an argument in [-1, 1].
#include "csa2_device.cuh"
#include "csa2_kernels.h"

namespace csa2 {
namespace {

constexpr int kNormThreads = 256;
constexpr int kIters = 2;   // row groups of a warp, all loaded before the first is used

__host__ __device__ constexpr int rows_per_block(int dim) {
  return kNormThreads / (dim / 16) * kIters;
}

// Eight channels.  Plain loads, not the read-only path: the output may be
// the input.
__device__ __forceinline__ void load8(const void* base, int64_t i, bool fp32, float (&v)[8]) {
  if (fp32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = s[0], b = s[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ void store8(void* base, int64_t i, bool fp32, const float (&v)[8]) {
  if (fp32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] = float_to_bf16_bits(v[2 * k]) | (float_to_bf16_bits(v[2 * k + 1]) << 16);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int kDim>
__device__ __forceinline__ void norm_rows(const NormParams& p, const NormPart& t, int64_t row0,
                                          float2* tab) {
  constexpr int kLanes = kDim / 16;               // lanes of a row
  constexpr int kRowsIter = kNormThreads / kLanes;
  const int tid = threadIdx.x, l = tid % kLanes;
  const int64_t n_rows = t.n_tokens * t.n_heads;
  const int pairs = t.rope_dim / 2;
  const int64_t tok0 = row0 / t.n_heads;

  float v[kIters][2][8];
  int64_t tok[kIters];
  int head[kIters];
  bool live[kIters];
#pragma unroll
  for (int it = 0; it < kIters; ++it) {
    const int64_t row = row0 + it * kRowsIter + tid / kLanes;
    live[it] = row < n_rows;
    tok[it] = live[it] ? row / t.n_heads : tok0;
    head[it] = live[it] ? (int)(row - tok[it] * t.n_heads) : 0;
    const int64_t at = tok[it] * t.x_token + head[it] * t.x_head;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (live[it]) {
        load8(t.x, at + 8 * (l + c * kLanes), t.x_fp32 != 0, v[it][c]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[it][c][i] = 0.0f;
      }
    }
  }
  if (pairs > 0) {
    // the block's tokens: sine and cosine of every channel pair
    const int64_t last = min(row0 + rows_per_block(kDim), n_rows) - 1;
    const int n = ((int)(last / t.n_heads - tok0) + 1) * pairs;
    for (int i = tid; i < n; i += kNormThreads) {
      const int k = i / pairs;
      const uint64_t turn = (uint64_t)__ldg(t.pos + tok0 + k) * p.turns[t.rope_table][i - k * pairs];
      float sn, cs;
      sincospif((float)(int64_t)turn * 0x1p-63f, &sn, &cs);
      tab[i] = make_float2(cs, sn);
    }
    __syncthreads();
  }
  float wt[2][8];
  if (t.weight) {
#pragma unroll
    for (int c = 0; c < 2; ++c) load8(t.weight, 8 * (l + c * kLanes), true, wt[c]);
  }
#pragma unroll
  for (int it = 0; it < kIters; ++it) {
    float r = 1.0f;
    if (t.norm) {
      auto squares = [&](float s) -> float {
        float ss = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(v[it][c][i] * s, v[it][c][i] * s, ss);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        return ss;
      };
      float ss = squares(1.0f);
      // squares beyond fp32: again with the row scaled by 2^-80 (eps is then
      // far below half a step of the mean)
      const bool big = !(ss < 0x1p120f);
      if (__any_sync(0xffffffffu, big)) {
        const float s2 = squares(0x1p-80f);
        r = big ? rsqrtf(s2 * (1.0f / kDim)) * 0x1p-80f : rsqrtf(fmaf(ss, 1.0f / kDim, p.eps));
      } else {
        r = rsqrtf(fmaf(ss, 1.0f / kDim, p.eps));
      }
    }
    if (!live[it]) continue;
    const int64_t at = tok[it] * t.out_token + head[it] * t.out_head;
    const float2* row_tab = tab + (tok[it] - tok0) * pairs;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int ch = 8 * (l + c * kLanes);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = v[it][c][i] * r;
        if (t.weight) y[i] *= wt[c][i];
      }
      const int pr = (ch - (kDim - t.rope_dim)) / 2;
      if (pairs > 0 && ch >= kDim - t.rope_dim) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 cs = row_tab[pr + i];
          const float a = y[2 * i], b = y[2 * i + 1];
          y[2 * i] = fmaf(a, cs.x, -(b * cs.y));
          y[2 * i + 1] = fmaf(a, cs.y, b * cs.x);
        }
      }
      store8(t.out, at + ch, t.out_fp32 != 0, y);
    }
  }
}

__global__ void __launch_bounds__(kNormThreads) k_norm_rope(const __grid_constant__ NormParams p) {
  extern __shared__ float2 tab[];
  int i = 0;
  while (i + 1 < p.n_parts && p.block0[i + 1] <= (int64_t)blockIdx.x) ++i;
  const NormPart& t = p.part[i];
  const int64_t row0 = ((int64_t)blockIdx.x - p.block0[i]) * rows_per_block(t.dim);
  griddep_wait();
  switch (t.dim) {
    case 512: norm_rows<512>(p, t, row0, tab); break;
    case 256: norm_rows<256>(p, t, row0, tab); break;
    case 128: norm_rows<128>(p, t, row0, tab); break;
    default: norm_rows<64>(p, t, row0, tab); break;
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormParams& p_in, cudaStream_t s) {
  NormParams p = p_in;
  int64_t blocks = 0;
  size_t smem = 0;
  for (int i = 0; i < p.n_parts; ++i) {
    const NormPart& t = p.part[i];
    const int64_t rows = t.n_tokens * t.n_heads, per = rows_per_block(t.dim);
    p.block0[i] = blocks;
    blocks += (rows + per - 1) / per;
    // tokens that a block of `per` rows touches at most
    const int64_t toks = (per + t.n_heads - 2) / t.n_heads + 1;
    const size_t need = (size_t)(toks < per ? toks : per) * (t.rope_dim / 2) * sizeof(float2);
    if (need > smem) smem = need;
  }
  p.block0[p.n_parts] = blocks;
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(k_norm_rope, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kNormThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_norm_rope, p);
}

}  // namespace csa2
