// k_window.cu -- window rows in a cache: rounded as they are written, read
// back in position order, and the rows of an accepted path of drafts.
//
// A row is 512 channels.  In 8 bits (the V4.1 report, section 2.4.4, keeps
// the window's KV in FP8): channels 0-447 as E4M3 codes with one power of two
// per 64 channels, the exponent of their largest magnitude minus 8; channels
// 448-511 as they are.  A code is the nearest E4M3 number (ties to even,
// saturating at 448) of x * 2^-e, a product that is exact; the row read back,
// code * 2^e, is exact in bf16 (4 significant bits).
//
// Bound: memory traffic, and for a decode step the launch.  A warp holds a
// row: lane l has the 16-byte chunks l and l + 32 of 8 channels, so that every
// access is contiguous over the lanes; the 8 lanes of a 64-channel block find
// its largest magnitude by three shuffles of bf16 pairs.  No row is written twice
// by a call (its segments are of different sequences, and a row that a later row of
// its segment replaces is not stored), so there is nothing to order.
//
// Measured: 98000 rows of prompts, rounded into other memory (201 MB) and each
// sequence's last 128 stored: 36.1 us, 5.6 TB/s or 82 % of the copy rate; with 192
// windows read back behind it, 44.7 us.  A chunk of 8192 rows and its window back:
// 5.2 us, 16 single rows and their windows: 3.7 us, two launches each.
#include <cuda_fp16.h>

#include "csa2_device.cuh"
#include "csa2_kernels.h"

namespace csa2 {
namespace {

constexpr int kWarps = 8;   // rows in flight of a block of the three kernels

__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {   // of bf16 pairs
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Eight bf16 of a chunk -> eight E4M3 codes under the scale byte that the
// block's eight lanes agree on.
__device__ __forceinline__ uint2 encode_chunk(const uint4& v, uint32_t& byte) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w}, mag = 0x7FFF7FFFu;
  uint32_t m = larger2(larger2(w[0] & mag, w[1] & mag), larger2(w[2] & mag, w[3] & mag));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = larger2(m, __shfl_xor_sync(0xffffffffu, m, o));
  // a maximum leaves NaN out, but is one where all of its half's channels are
  const uint32_t even = m & 0xFFFFu, odd = m >> 16;
  const uint32_t ex = max(even > 0x7F80u ? 0u : even, odd > 0x7F80u ? 0u : odd) >> 7;
  byte = ex >= 8u ? ex - 8u : 0u;
  // 2^(127 - byte), a normal number: byte is at most 247.  What a product in bf16
  // loses is below 2^-126, where the codes are zeros.
  const uint32_t inv = (254u - byte) * 0x00800080u;
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = bf16x2_mul(w[i], inv);
    c[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(
        make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

__device__ __forceinline__ uint4 decode_chunk(const uint2& c, uint32_t byte) {
  const float sc = ue8m0_value(byte);
  const uint32_t w[2] = {c.x, c.y};
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

// Row of the cache that holds position x of a sequence in the ring, and among
// the first tokens.
__device__ __forceinline__ int64_t ring_row(const WinRows& w, int32_t seq, int64_t x) {
  // x mod swa (at most 128) by 32-bit divisions: 2^32 mod swa times the upper half's
  const uint32_t n = (uint32_t)w.swa, top = (uint32_t)(x >> 32);
  uint32_t m = (uint32_t)x % n;
  if (top) m = (m + (top % n) * ((0xFFFFFFFFu % n + 1u) % n)) % n;
  return (int64_t)seq * w.swa + m;
}
__device__ __forceinline__ int64_t first_row(const WinRows& w, int32_t seq, int64_t x) {
  return (int64_t)w.n_seqs * w.swa + (int64_t)seq * w.n_first + x;
}

// kRows neighbouring rows a warp: with two the search of the segments and the
// latency of the loads are shared, with one a few rows are on more SMs.
template <int kRows>
__global__ void __launch_bounds__(kWarps * 32)
    k_win_append(const __grid_constant__ WinAppendParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t r0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRows;
  if (r0 >= p.n_rows) return;
  int32_t seg = (int32_t)r0;
  if (!p.identity) {
    // the last segment that starts at or before row r0 (empty ones share a
    // start with the one behind them)
    int32_t lo = 0, hi = p.n_segs;
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if (p.first[mid] <= (int32_t)r0) lo = mid;
      else hi = mid;
    }
    seg = lo;
  }
  griddep_wait();
  griddep_launch();
  const WinRows& w = p.w;
  uint4 a[kRows], b[kRows];
  int64_t x[kRows], to_ring[kRows], to_first[kRows];   // its position; rows of the cache, or -1
  bool need[kRows];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t r = r0 + k;
    need[k] = false;
    if (r >= p.n_rows) continue;
    int32_t in_seg = 0, left = 1, seq = p.seq0 + (int32_t)r;
    if (p.identity) {
      seg = (int32_t)r;
    } else {
      while (p.first[seg + 1] <= (int32_t)r) ++seg;   // row r exists: ends
      in_seg = (int32_t)r - p.first[seg];
      left = p.first[seg + 1] - (int32_t)r;
      seq = p.seq[seg];
    }
    const int64_t p0 = p.pos0[seg];
    x[k] = (int64_t)((uint64_t)p0 + (uint64_t)in_seg);
    const bool is = p0 >= 0 && in_seg <= INT64_MAX - p0;   // a position at all
    to_ring[k] = is && left <= w.swa ? ring_row(w, seq, x[k]) : -1;
    to_first[k] = is && x[k] < w.n_first ? first_row(w, seq, x[k]) : -1;
    need[k] = to_ring[k] >= 0 || to_first[k] >= 0 || p.rounded;
    if (!need[k]) continue;
    const uint4* src = reinterpret_cast<const uint4*>(p.rows + r * kHeadDim);
    a[k] = src[lane];   // plain: `rounded` may be `rows`
    b[k] = src[lane + 32];
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (!need[k]) continue;
    uint32_t ba = 0, bb = 0;
    uint2 ca, cb;
    if (w.fp8) {
      ca = encode_chunk(a[k], ba);
      cb = encode_chunk(b[k], bb);   // lanes 24-31: not used
    }
    auto store = [&](int64_t row) {
      if (!CSA2_IN_BOUNDS(is_window_row(w, row), w.err)) return;
      if (w.fp8) {
        uint2* c = reinterpret_cast<uint2*>(w.codes + row * 448);
        c[lane] = ca;
        if (lane < 24) c[lane + 32] = cb;
        else reinterpret_cast<uint4*>(w.rope + row * 64)[lane - 24] = b[k];
        uint8_t* s = w.scales + row * 8;
        if ((lane & 7) == 0) {
          s[lane >> 3] = (uint8_t)ba;
          s[4 + (lane >> 3)] = lane < 24 ? (uint8_t)bb : (uint8_t)0;
        }
      } else {
        uint4* d = reinterpret_cast<uint4*>(w.rows + row * kHeadDim);
        d[lane] = a[k];
        d[lane + 32] = b[k];
      }
      if (lane == 0) w.pos[row] = x[k];
    };
    if (to_ring[k] >= 0) store(to_ring[k]);
    if (to_first[k] >= 0) store(to_first[k]);
    if (p.rounded) {
      uint4* d = reinterpret_cast<uint4*>(p.rounded + (r0 + k) * kHeadDim);
      d[lane] = w.fp8 ? decode_chunk(ca, ba) : a[k];
      d[lane + 32] = w.fp8 && lane < 24 ? decode_chunk(cb, bb) : b[k];
    }
  }
}

// A warp per row: n_rows window rows of a segment, then its first tokens.
__global__ void __launch_bounds__(kWarps * 32)
    k_win_read(const __grid_constant__ WinReadParams p) {
  const int lane = threadIdx.x & 31;
  const WinRows& w = p.w;
  const uint32_t per = (uint32_t)(p.n_rows + (p.first ? w.n_first : 0));
  const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= (int64_t)p.n_segs * per) return;
  const int32_t seg = (int32_t)(i / per), j = (int32_t)(i - (int64_t)seg * per);
  const int32_t seq = p.identity ? p.seq0 + seg : p.seq[seg];
  griddep_wait();
  griddep_launch();
  const int64_t end = p.end[seg];
  const bool first = j >= p.n_rows;
  const int64_t lo = end > p.n_rows ? end - p.n_rows : 0;
  const int64_t x = first ? j - p.n_rows : lo + j;
  const int64_t row = first ? first_row(w, seq, x) : ring_row(w, seq, x);
  if (!CSA2_IN_BOUNDS(is_window_row(w, row) && j < p.n_rows + w.n_first, w.err)) return;
  // the row's tag and the row together: one that is not held is read for nothing
  const int64_t tag = __ldg(w.pos + row);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint2 none = make_uint2(0u, 0u);
  uint4 a = zero, b = zero;
  uint2 ca = none, cb = none, sc = none;
  if (w.fp8) {
    const uint2* c = reinterpret_cast<const uint2*>(w.codes + row * 448);
    ca = __ldg(c + lane);
    if (lane < 24) cb = __ldg(c + lane + 32);
    else b = __ldg(reinterpret_cast<const uint4*>(w.rope + row * 64) + lane - 24);
    sc = __ldg(reinterpret_cast<const uint2*>(w.scales + row * 8));
  } else {
    const uint4* s = reinterpret_cast<const uint4*>(w.rows + row * kHeadDim);
    a = __ldg(s + lane);
    b = __ldg(s + lane + 32);
  }
  const bool held = x < end && tag == x;
  if (!first && p.codes) {
    const int64_t at = (int64_t)seg * p.n_rows + j;
    uint2* d = reinterpret_cast<uint2*>(p.codes + at * 448);
    d[lane] = held ? ca : none;
    if (lane < 24) d[lane + 32] = held ? cb : none;
    else reinterpret_cast<uint4*>(p.rope + at * 64)[lane - 24] = held ? b : zero;
    if (lane == 0) *reinterpret_cast<uint2*>(p.scales + at * 8) = held ? sc : none;
    return;
  }
  if (!held) {
    a = b = zero;
  } else if (w.fp8) {
    a = decode_chunk(ca, (sc.x >> (lane & 24)) & 255u);   // a byte for 8 lanes
    if (lane < 24) b = decode_chunk(cb, (sc.y >> (lane & 24)) & 255u);
  }
  uint16_t* out = first ? p.first + ((int64_t)seg * w.n_first + x) * kHeadDim
                        : p.out + ((int64_t)seg * p.n_rows + j) * kHeadDim;
  uint4* d = reinterpret_cast<uint4*>(out);
  d[lane] = a;
  d[lane + 32] = b;
}

// A block per tree: the accepted path's rows, copied as they are.
__global__ void __launch_bounds__(kWarps * 32)
    k_win_accept(const __grid_constant__ WinAcceptParams p) {
  const int tree = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const WinRows& w = p.w;
  const int32_t first = p.first[tree], n = p.first[tree + 1] - first;
  __shared__ int32_t path[64];   // the path's drafts, the accepted one first
  __shared__ int32_t len_s;
  griddep_wait();
  griddep_launch();
  if (threadIdx.x == 0) {
    int32_t t = p.accepted[tree], len = 0;
    if (t < 0 || t >= n) t = -1;
    for (; t >= 0 && len < 64; t = p.parent[first + t]) path[len++] = t;
    len_s = len;
  }
  __syncthreads();
  const int32_t len = len_s;
  for (int d = warp; d < len; d += kWarps) {
    const int64_t x = p.pos0[tree] + d, src = first + path[len - 1 - d];
    const bool ring = len - d <= w.swa, head = x < w.n_first;
    auto copy = [&](int64_t row) {
      if (!CSA2_IN_BOUNDS(is_window_row(w, row) && src >= first && src < p.first[tree + 1], w.err)) return;
      if (w.fp8) {
        const uint4* c = reinterpret_cast<const uint4*>(p.d.codes + src * 448);
        if (lane < 28) reinterpret_cast<uint4*>(w.codes + row * 448)[lane] = __ldg(c + lane);
        if (lane < 8)
          reinterpret_cast<uint4*>(w.rope + row * 64)[lane] =
              __ldg(reinterpret_cast<const uint4*>(p.d.rope + src * 64) + lane);
        if (lane == 31)
          *reinterpret_cast<uint2*>(w.scales + row * 8) =
              __ldg(reinterpret_cast<const uint2*>(p.d.scales + src * 8));
      } else {
        const uint4* s = reinterpret_cast<const uint4*>(p.d.rows + src * kHeadDim);
        uint4* o = reinterpret_cast<uint4*>(w.rows + row * kHeadDim);
        o[lane] = __ldg(s + lane);
        o[lane + 32] = __ldg(s + lane + 32);
      }
      if (lane == 0) w.pos[row] = x;
    };
    if (ring) copy(ring_row(w, p.seq[tree], x));
    if (head) copy(first_row(w, p.seq[tree], x));
  }
}

template <class P>
cudaError_t launch_rows(void (*kernel)(const P), const P& p, int64_t blocks, cudaStream_t s) {
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1] = {pdl_attribute()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_window_append(const WinAppendParams& p, cudaStream_t s) {
  // two rows a warp from where one a warp fills the GPU's warps several times (98000
  // rows: 37.4 us with one, 36.1 with two, 38.6 with four)
  if (p.n_rows >= 32768) return launch_rows(k_win_append<2>, p, (p.n_rows + 2 * kWarps - 1) / (2 * kWarps), s);
  return launch_rows(k_win_append<1>, p, (p.n_rows + kWarps - 1) / kWarps, s);
}

cudaError_t launch_window_read(const WinReadParams& p, cudaStream_t s) {
  const int64_t rows = (int64_t)p.n_segs * (p.n_rows + (p.first ? p.w.n_first : 0));
  return launch_rows(k_win_read, p, (rows + kWarps - 1) / kWarps, s);
}

cudaError_t launch_window_accept(const WinAcceptParams& p, cudaStream_t s) {
  return launch_rows(k_win_accept, p, p.n_trees, s);
}

}  // namespace csa2
