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
// product are the fraction of a turn), so the reduction loses nothing and no
// 64-bit floating point is needed; sincospif then takes an argument in [-1, 1].
// What is left is f's own rounding, a double's (below 2^-51 relative with the
// power and 1 / (2 pi)): an angle is off by less than |pos| * 2^-51 radians,
// below fp32's own steps (2^-24) up to |pos| = 2^27, 2^-20 at 2^31, and no
// longer an angle towards 2^51.
#include <type_traits>

#include "csa2_device.cuh"
#include "csa2_kernels.h"

namespace csa2 {
namespace {

// Blocks and row groups, measured on 8192 tokens of 98 heads in four tensors
// (1.24 GB read and written, 183 us at the measured copy bandwidth): blocks
// of 128 threads, 8 of them an SM at 64 registers, three row groups (96 bytes
// a lane) requested before the first is used: 202 us.  256 threads: 211 us
// (the sine table's barrier idles more warps), 512: 229; two row groups: 216;
// four, with six blocks: 205; streaming hints on the loads: 218, on the
// stores: no change.  The first form of this kernel (fp32 values held in
// registers, 64-bit divisions per row, 3 blocks of 256 threads): 448 us.
constexpr int kNormThreads = 128;
constexpr int kNormBlocks = 8;   // per SM

// Row groups of a warp, all requested before the first is used.
template <bool kF32>
__host__ __device__ constexpr int iters_of() { return kF32 ? 1 : 3; }

__host__ __device__ constexpr int rows_per_block(int dim, bool fp32) {
  return kNormThreads / (dim / 16) * (fp32 ? iters_of<true>() : iters_of<false>());
}

// The sine table of a block stays below the 48 KB that a launch may ask for
// without an attribute of the kernel (which calls from several threads would
// set over each other): at most one token a row, dim / 2 pairs up to 64.
static_assert(rows_per_block(64, false) * 32 * sizeof(float2) <= 48 * 1024, "sine table");
static_assert(rows_per_block(128, false) * kNormMaxPairs * sizeof(float2) <= 48 * 1024, "sine table");

// Eight channels as they are in memory.  Plain loads, not the read-only path:
// the output may be the input.
template <bool kF32>
struct Raw {
  uint4 a[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) +
                                                    i * (kF32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < (kF32 ? 2 : 1); ++k) a[k] = s[k];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < (kF32 ? 2 : 1); ++k) a[k] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < (kF32 ? 2 : 1); ++k) {
      const uint32_t w[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kF32) {
          v[4 * k + i] = __uint_as_float(w[i]);
        } else {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      }
    }
  }
};

__device__ __forceinline__ void store8(void* base, int64_t i, bool fp32, const float (&v)[8]) {
  if (fp32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int kDim, bool kF32>
__device__ __forceinline__ void norm_rows(const NormParams& p, const NormPart& t, uint32_t block,
                                          float2* tab) {
  constexpr int kIters = iters_of<kF32>();
  constexpr int kLanes = kDim / 16;               // lanes of a row
  constexpr int kRowsIter = kNormThreads / kLanes;
  constexpr int kRows = kRowsIter * kIters;
  const uint32_t tid = threadIdx.x, l = tid % kLanes;
  const uint32_t H = (uint32_t)t.n_heads;
  // the block's first row as (token, head); its other rows are few, so their
  // places come from 32-bit arithmetic relative to it
  const int64_t row0 = (int64_t)block * kRows;
  const int64_t tok0 = row0 / H;
  const uint32_t head0 = (uint32_t)(row0 - tok0 * H);
  const int64_t left = t.n_tokens * t.n_heads - row0;
  const uint32_t n_rows = left < kRows ? (uint32_t)left : (uint32_t)kRows;
  const int pairs = t.rope_dim / 2;

  Raw<kF32> x[kIters][2];
#pragma unroll
  for (int it = 0; it < kIters; ++it) {
    const uint32_t r = it * kRowsIter + tid / kLanes, hr = head0 + r, tk = hr / H;
    const int64_t at = (tok0 + tk) * t.x_token + (int64_t)(hr - tk * H) * t.x_head;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (r < n_rows) x[it][c].load(t.x, at + 8 * (l + c * kLanes));
      else x[it][c].zero();
    }
  }
  if (pairs > 0) {
    // sine and cosine of every channel pair of the block's tokens
    const uint32_t n = ((head0 + n_rows - 1) / H + 1) * (uint32_t)pairs;
    for (uint32_t i = tid; i < n; i += kNormThreads) {
      const uint32_t k = i / (uint32_t)pairs;
      const uint64_t turn = (uint64_t)__ldg(t.pos + tok0 + k) * p.turns[t.rope_table][i - k * pairs];
      float sn, cs;
      sincospif((float)(int64_t)turn * 0x1p-63f, &sn, &cs);
      tab[i] = make_float2(cs, sn);
    }
    __syncthreads();
  }
  float scale[kIters];
#pragma unroll
  for (int it = 0; it < kIters; ++it) {
    scale[it] = 1.0f;
    if (t.norm) {
      auto squares = [&](float s) -> float {
        float ss = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float v[8];
          x[it][c].values(v);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(v[i] * s, v[i] * s, ss);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        return ss;
      };
      const float ss = squares(1.0f);
      scale[it] = rsqrtf(fmaf(ss, 1.0f / kDim, p.eps));
      // squares beyond fp32: again with the row scaled by 2^-80 (eps is then
      // far below half a step of the mean)
      const bool big = !(ss < 0x1p120f);
      if (__any_sync(0xffffffffu, big)) {
        const float s2 = squares(0x1p-80f);
        if (big) scale[it] = rsqrtf(s2 * (1.0f / kDim)) * 0x1p-80f;
      }
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int ch = 8 * (int)(l + c * kLanes);
    const int pr = (ch - (kDim - t.rope_dim)) / 2;
    const bool rotate = pairs > 0 && ch >= kDim - t.rope_dim;
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    if (t.weight) {
      const float4* w4 = reinterpret_cast<const float4*>(t.weight + ch);
      const float4 a = __ldg(w4), b = __ldg(w4 + 1);
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
      w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      const uint32_t r = it * kRowsIter + tid / kLanes, hr = head0 + r, tk = hr / H;
      if (r >= n_rows) continue;
      float y[8];
      x[it][c].values(y);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = y[i] * scale[it] * w[i];
      if (rotate) {
        const float4* cs4 = reinterpret_cast<const float4*>(tab + tk * pairs + pr);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 cs = cs4[i];   // (cos, sin) of two pairs
          const float a = y[4 * i], b = y[4 * i + 1], d = y[4 * i + 2], e = y[4 * i + 3];
          y[4 * i] = fmaf(a, cs.x, -(b * cs.y));
          y[4 * i + 1] = fmaf(a, cs.y, b * cs.x);
          y[4 * i + 2] = fmaf(d, cs.z, -(e * cs.w));
          y[4 * i + 3] = fmaf(d, cs.w, e * cs.z);
        }
      }
      store8(t.out, (tok0 + tk) * t.out_token + (int64_t)(hr - tk * H) * t.out_head + ch,
             t.out_fp32 != 0, y);
    }
  }
}

__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
    k_norm_rope(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) float2 tab[];
  int i = 0;
  while (i + 1 < p.n_parts && p.block0[i + 1] <= (int64_t)blockIdx.x) ++i;
  const NormPart& t = p.part[i];
  const uint32_t block = (uint32_t)((int64_t)blockIdx.x - p.block0[i]);
  griddep_wait();
  auto rows = [&](auto dim) {
    constexpr int kDim = decltype(dim)::value;
    if (t.x_fp32) norm_rows<kDim, true>(p, t, block, tab);
    else norm_rows<kDim, false>(p, t, block, tab);
  };
  switch (t.dim) {
    case 512: rows(std::integral_constant<int, 512>()); break;
    case 256: rows(std::integral_constant<int, 256>()); break;
    case 128: rows(std::integral_constant<int, 128>()); break;
    default: rows(std::integral_constant<int, 64>()); break;
  }
}

}  // namespace

cudaError_t launch_norm_rope(const NormParams& p_in, cudaStream_t s) {
  NormParams p = p_in;
  int64_t blocks = 0;
  size_t smem = 0;
  for (int i = 0; i < p.n_parts; ++i) {
    const NormPart& t = p.part[i];
    const int64_t rows = t.n_tokens * t.n_heads, per = rows_per_block(t.dim, t.x_fp32 != 0);
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
