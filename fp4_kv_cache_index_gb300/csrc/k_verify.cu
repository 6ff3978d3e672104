// k_verify.cu -- which drafts of a tree are kept, and the token that follows
// them: rejection sampling with given random numbers.
//
// At a node of the walk, with p = softmax(target / T) and q = softmax(draft /
// T), child x is accepted if u q(x) < r(x), r = max(p - a q, 0) / b, a = 0 and
// b = 1 at first.  A rejection replaces r by max(r - q, 0) over its sum, which
// is the same form with a + b for a (max(p - a q, 0) / b > q means p > (a + b)
// q) and b = sum max(p - a q, 0): the row that is left is never written, and
// costs a pass over two rows that L2 holds.  The last token is the first
// largest r / noise (of exponential variates it takes token i with probability
// r_i), for which the sum b is not needed.
//
// Bound: reading the rows of the nodes that the walk visits, from HBM.  Which
// those are is known one node after the other, so a walk is a chain of passes
// over a row or two.  A sequence has a cluster of CTAs, each with a share of the
// vocabulary; per pass they join a maximum and a sum through distributed
// shared memory.  Everything that decides where the walk goes is read by the
// cluster's first CTA and taken from its shared memory by all, so that all
// come to the same barriers.
//
// Where the two rows are alike and a child's token is masked in both, it is rejected and
// max(p - a q, 0) is 0 everywhere: a and b then stay as they are.  So that this is seen,
// the two products of a difference are rounded alike, never fused.
//
// Sums and tests in fp32 (64 bits take 64 times as long here).  A test whose two
// sides are nearer to each other than fp32 can tell is made again, with its
// node's sums, in 64 bits.  Of the token's scores fp32 gives bounds, p and a q each a
// few 1e-5 of itself off: if another token's upper bound reaches the best one's lower
// bound (always, where p and a q all but cancel), the node's sums and tests are made
// again in 64 bits, if they were not yet, and all such tokens are scored with those.
// There r is formed by one rejection after the other, each divided by its sum: p - a q
// has lost a token that is left by 1e-9 of p twice.  So the result is the one of 64-bit arithmetic, whatever the order of the sums.
//
// Measured (replayed graphs of one call): 64 sequences of up to 8 drafts over 131072
// tokens, whose walks read 134 MB: 79.6 us.  The SMs are busy for 55 % of that (the longest
// walks have more than twice the average's nodes and no more CTAs), with instructions, of
// which the exponentials are the smaller part, and the joins of a cluster.  One chat
// of 5 drafts over 32000 tokens: 8.4 us; 12 trees of 64 over 100003 tokens of fp32
// without draft logits: 20.4 us.  Twice as many CTAs a sequence take 77 us for the
// mixed batch and a fifth longer for one of equal walks.
#include <type_traits>

#include "csa2_device.cuh"
#include "csa2_kernels.h"

namespace csa2 {
namespace {

// Blocks of 256 threads, two of them an SM, and clusters of up to 16: a batch's walks
// are of very different lengths, and with small shares the long ones have more SMs
// left to them.
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlocks = 2;       // per SM
constexpr int kMaxCluster = 16;

// What a pass gives: merged over a warp's lanes, then over all warps of the cluster.
// `over(n, lane, scale)`: the merge of lanes 0 .. n - 1 (a power of two, the
// others hold nothing), the same bits in each of them.
__device__ __forceinline__ float lanes_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
// Largest logit m of a part of a row, and the sum of exp2((l - m) * scale).  The
// difference of two logits is formed first: it is all but exact, and the
// probabilities that count have small ones (l * scale - m * scale would round
// at the logits' own size).  A NaN or an infinity in the row leaves a NaN in z.
struct Sum {
  float m, z;
  __device__ __forceinline__ void raise(float to, float scale) {
    const float d = m - to;
    // (-inf) - (-inf): nothing in it.  (to is +inf: z is NaN already)
    z *= d == d || z != z ? fast_exp2(d * scale) : 0.0f;
    m = to;
  }
};
struct Sums {
  Sum p, q;
  __device__ __forceinline__ void over(int n, int, float scale) {
    p.raise(lanes_max(p.m), scale);   // lanes without a part hold -inf
    q.raise(lanes_max(q.m), scale);
    for (int o = n / 2; o > 0; o >>= 1) {
      p.z += __shfl_xor_sync(0xffffffffu, p.z, o);
      q.z += __shfl_xor_sync(0xffffffffu, q.z, o);
    }
  }
  // two parts of one lane
  __device__ __forceinline__ void add(Sums b, float scale) {
    const float mp = fmaxf(p.m, b.p.m), mq = fmaxf(q.m, b.q.m);
    p.raise(mp, scale);
    b.p.raise(mp, scale);
    q.raise(mq, scale);
    b.q.raise(mq, scale);
    p.z += b.p.z;
    q.z += b.q.z;
  }
  __device__ static Sums none() { return {{-INFINITY, 0.0f}, {-INFINITY, 0.0f}}; }
};
// (value, index) of the best so far, the lower index of equal values, and the
// value of the second; bad: a NaN or an infinity was seen.
struct Best {
  float v, second;
  int32_t i;
  uint32_t bad;
  __device__ __forceinline__ void add(const Best& b, float) {
    const bool first = v > b.v || (v == b.v && (uint32_t)i < (uint32_t)b.i);
    second = fmaxf(fmaxf(second, b.second), first ? b.v : v);
    if (!first) {
      v = b.v;
      i = b.i;
    }
    bad |= b.bad;
  }
  __device__ __forceinline__ void over(int n, int, float scale) {
    for (int o = n / 2; o > 0; o >>= 1)
      add({__shfl_xor_sync(0xffffffffu, v, o), __shfl_xor_sync(0xffffffffu, second, o),
           __shfl_xor_sync(0xffffffffu, i, o), __shfl_xor_sync(0xffffffffu, bad, o)},
          scale);
  }
  __device__ static Best none() { return {-INFINITY, -INFINITY, -1, 0u}; }
};
// Below the first temperature only the largest logits count (a score in log2 units stays
// a number for logits up to 1e8); above the second one, all alike.
constexpr float kCold = 0x1p-100f, kHot = 0x1p100f;

// Of the scores of what is left at a node: the largest upper bound, whose it is, the
// second largest, and a lower bound of the first one's score.
struct Most {
  float v, second;
  int32_t i;
  float low;
  __device__ __forceinline__ void add(const Most& b, float) {
    const bool first = v > b.v || (v == b.v && (uint32_t)i < (uint32_t)b.i);
    second = fmaxf(fmaxf(second, b.second), first ? b.v : v);
    if (!first) {
      v = b.v;
      i = b.i;
      low = b.low;
    }
  }
  __device__ __forceinline__ void over(int n, int, float scale) {
    for (int o = n / 2; o > 0; o >>= 1)
      add({__shfl_xor_sync(0xffffffffu, v, o), __shfl_xor_sync(0xffffffffu, second, o),
           __shfl_xor_sync(0xffffffffu, i, o), __shfl_xor_sync(0xffffffffu, low, o)},
          scale);
  }
  __device__ static Most none() { return {-INFINITY, -INFINITY, -1, 0.0f}; }
};
template <class Real>
struct Total {
  Real t;
  __device__ __forceinline__ void add(const Total& b, float) { t += b.t; }
  __device__ __forceinline__ void over(int n, int, float) {
    for (int o = n / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  __device__ static Total none() { return {Real(0)}; }
};
struct Sums64 {   // exp2 below the maxima that are known already
  double p, q;
  __device__ __forceinline__ void add(const Sums64& b, float) {
    p += b.p;
    q += b.q;
  }
  __device__ __forceinline__ void over(int n, int, float) {
    for (int o = n / 2; o > 0; o >>= 1) {
      p += __shfl_xor_sync(0xffffffffu, p, o);
      q += __shfl_xor_sync(0xffffffffu, q, o);
    }
  }
  __device__ static Sums64 none() { return {0.0, 0.0}; }
};
struct Exact {   // a score in 64 bits
  double v;
  int32_t i, pad;
  __device__ __forceinline__ void add(const Exact& b, float) {
    if (b.v > v || (b.v == v && (uint32_t)b.i < (uint32_t)i)) *this = b;
  }
  __device__ __forceinline__ void over(int n, int, float scale) {
    for (int o = n / 2; o > 0; o >>= 1)
      add({__shfl_xor_sync(0xffffffffu, v, o), __shfl_xor_sync(0xffffffffu, i, o), 0}, scale);
  }
  __device__ static Exact none() { return {-INFINITY, -1, 0}; }
};

constexpr int kPartWords = 4;
constexpr int kParts = kMaxCluster * kWarps;   // warps of a cluster
struct Kid {       // a child of the node
  int32_t token;
  float u, lp, lq;
};
// What a pass leads to: a sum over what is left is needed, the node's numbers in
// 64 bits, a child is taken, the token is drawn here, or the walk ends without.
enum Action { kSum, kExact, kGo, kToken, kEnd };
// Where the tests of a node stand: what is left is max(p - a q, 0) / b.
template <class Real>
struct Tests {
  Real a, a_prev, b;
  float eps;                 // fp32: what p and a q are good to
  uint64_t todo;             // children that are still to be tested
  bool last;                 // the last one was rejected, what then is left has no sum yet
  int32_t taken;
  int32_t removed[2], n_removed;   // lane r: removed tokens r and r + 32
};
struct Smem {
  // written by the cluster's warps, by pass parity: their parts, and by the
  // first CTA's the node's children
  alignas(16) uint32_t part[2][kParts][kPartWords];
  alignas(16) Kid kid[2][64];
  float temperature;
  int32_t removed[64];       // for the last pass
  double z[2], inv[64][2];   // in 64 bits: the two sums; two factors that are 1 / the sum behind a rejection
  int32_t n_inv, last;       // how many of these, and whether a rejection without follows
};

// 16 bytes or less to `local` of another CTA of the cluster.
template <class T>
__device__ __forceinline__ void st_peer(void* local, uint32_t rank, const T& v) {
  const uint32_t at = dsmem_addr(smem_u32(local), rank);
  if constexpr (sizeof(T) == 16) {
    const uint4 w = *reinterpret_cast<const uint4*>(&v);
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w.x), "r"(w.y),
                 "r"(w.z), "r"(w.w)
                 : "memory");
  } else if constexpr (sizeof(T) == 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(&v);
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(w.x), "r"(w.y) : "memory");
  } else {
    static_assert(sizeof(T) == 4, "words");
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(*reinterpret_cast<const uint32_t*>(&v))
                 : "memory");
  }
}

// A value's bits, asked for now and looked at later.
template <class T>
__device__ __forceinline__ uint32_t bits_now(const T* row, int32_t i) {
  if constexpr (sizeof(T) == 2) return ldg_now_u16(row + i);
  else return ldg_now_u32(row + i);
}
template <class T>
__device__ __forceinline__ float value_of(uint32_t bits) {
  return sizeof(T) == 2 ? bf16_bits_to_float(bits) : __uint_as_float(bits);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 2^x in 64 bits, to their rounding: the Taylor series of e^r, |r| <= ln 2 / 2, to the
// 13th power (the next term is (ln 2 / 2)^14 / 14! = 4e-18).
__device__ __forceinline__ double exp2_64(double x) {
  if (!(x > -1080.0)) return x == x ? 0.0 : x;
  const double n = rint(x), r = (x - n) * 0.693147180559945309;
  double s = 1.0 / 6227020800.0;
  s = fma(s, r, 1.0 / 479001600);
  s = fma(s, r, 1.0 / 39916800);
  s = fma(s, r, 1.0 / 3628800);
  s = fma(s, r, 1.0 / 362880);
  s = fma(s, r, 1.0 / 40320);
  s = fma(s, r, 1.0 / 5040);
  s = fma(s, r, 1.0 / 720);
  s = fma(s, r, 1.0 / 120);
  s = fma(s, r, 1.0 / 24);
  s = fma(s, r, 1.0 / 6);
  s = fma(s, r, 0.5);
  s = fma(s, r, 1.0);
  s = fma(s, r, 1.0);
  // 2^n in two parts, of which both are normal numbers where it is not
  const double low = fmax(n, -1000.0);
  return s * __hiloint2double((int)(1023.0 + fmin(low, 1000.0)) << 20, 0) *
         __hiloint2double((int)(1023.0 + (n - low)) << 20, 0);
}

// Eight neighbouring values of a row as they are in memory.
template <class T>
struct Eight {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* row, int32_t i) {
#pragma unroll
    for (int k = 0; k < (int)(sizeof(T) / 2); ++k) v[k] = ldg_now_v4(row + i + 16 / sizeof(T) * k);
  }
  __device__ __forceinline__ void fill(uint32_t w) {
#pragma unroll
    for (int k = 0; k < (int)(sizeof(T) / 2); ++k) v[k] = make_uint4(w, w, w, w);
  }
  // one by one, `fill` for those outside [0, n)
  __device__ __forceinline__ void gather(const T* row, int32_t i, int32_t n, uint32_t fill) {
    uint32_t w[2 * sizeof(T)];
#pragma unroll
    for (int k = 0; k < (int)(2 * sizeof(T)); ++k) {
      if constexpr (sizeof(T) == 2) {
        const int32_t a = i + 2 * k;
        const uint32_t lo = a >= 0 && a < n ? (uint32_t)__ldg(row + a) : fill;
        const uint32_t hi = a + 1 >= 0 && a + 1 < n ? (uint32_t)__ldg(row + a + 1) : fill;
        w[k] = lo | (hi << 16);
      } else {
        w[k] = i + k >= 0 && i + k < n ? __float_as_uint(__ldg(row + i + k)) : fill;
      }
    }
#pragma unroll
    for (int k = 0; k < (int)(sizeof(T) / 2); ++k)
      v[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  }
  __device__ __forceinline__ float at(int k) const {
    const int j = k * (int)sizeof(T) / 4;
    const uint4& q = v[j >> 2];
    const uint32_t w = (j & 3) == 0 ? q.x : (j & 3) == 1 ? q.y : (j & 3) == 2 ? q.z : q.w;
    if constexpr (sizeof(T) == 2) return __uint_as_float(k & 1 ? w & 0xFFFF0000u : w << 16);
    else return __uint_as_float(w);
  }
  // the largest value (NaN left out)
  __device__ __forceinline__ float max() const {
    if constexpr (sizeof(T) == 2) {
      uint32_t m;
      asm("{\n .reg .b32 a, b;\n max.bf16x2 a, %1, %2;\n max.bf16x2 b, %3, %4;\n"
          " max.bf16x2 %0, a, b;\n}"
          : "=r"(m) : "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w));
      return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
    } else {
      float m = at(0);
#pragma unroll
      for (int k = 1; k < 8; ++k) m = fmaxf(m, at(k));
      return m;
    }
  }
};

// What is left of a token, max(p - a q, 0).  Both products are rounded before they are
// subtracted: where p = a q they are the same bits and nothing is left, as the walk has
// to know.  (These are never contracted; products and sums in pairs were.)
__device__ __forceinline__ float left(float pe, float qe, float ip, float aq) {
  return fmaxf(__fsub_rn(__fmul_rn(pe, ip), __fmul_rn(qe, aq)), 0.0f);
}

// exp2((x - base) * scale) of two values.
__device__ __forceinline__ float2 exps(float x, float y, uint64_t neg_base, uint64_t scale2) {
  const float2 d = unpack2(mul2(add2(pack2(x, y), neg_base), scale2));
  return make_float2(fast_exp2(d.x), fast_exp2(d.y));
}

// Chunks into a thread's sum.
template <class T, int kN>
__device__ __forceinline__ void add_chunks(Sum& s, const Eight<T> (&l)[kN], float scale,
                                           uint64_t scale2) {
  float m = l[0].max();
#pragma unroll
  for (int j = 1; j < kN; ++j) m = fmaxf(m, l[j].max());
  if (m > s.m) {
    s.z *= fast_exp2((s.m - m) * scale);
    s.m = m;
  }
  const float base = s.m == -INFINITY ? 0.0f : s.m;
  const uint64_t nb = pack2(-base, -base);
  uint64_t z[2] = {0, 0};   // zeros
#pragma unroll
  for (int j = 0; j < kN; ++j)
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float2 e = exps(l[j].at(k), l[j].at(k + 1), nb, scale2);
      z[(k >> 1) & 1] = add2(z[(k >> 1) & 1], pack2(e.x, e.y));
    }
  const float2 z2 = unpack2(add2(z[0], z[1]));
  s.z += z2.x + z2.y;
}

// Chunks of two rows that a thread has in flight.  Few where a thread has two in all:
// the code of a pass is then fetched for one use (replayed graphs, bf16 with draft logits:
// 5 drafts over 32000 tokens 8.5 us, with four 9.2; 40 sequences over 1500 tokens 20.2
// and 23.6; 64 sequences over 131072 79.3 with four, 93 with two).
template <class T, bool kSmall>
constexpr int kRows = (kSmall ? 4 : 8) / (int)sizeof(T);

// The CTA's share of one or two rows of logits (and of the noise) in chunks of
// eight elements, kUnroll of them at a time: f(i0, x, y, z), chunk k the elements
// from i0[k] = 8 t - (elements by which the row misses a 16-byte boundary).  A
// row's ends are read element by element, and so is all of a row that misses the
// boundary by another amount than the first; elements outside the row come as
// -inf (noise: 1).  The rows go to L2 ahead of the loads: a thread's loads are
// in flight only between two batches.
template <class T, int kUnroll, bool kNoise, class F>
__device__ __forceinline__ void for_rows(const T* a, const T* b, const float* c, int32_t vocab,
                                         uint32_t rank, uint32_t ctas, F f) {
  constexpr uint32_t kFill = sizeof(T) == 2 ? 0xFF80u : 0xFF800000u;   // -inf
  constexpr uint32_t kFill2 = sizeof(T) == 2 ? 0xFF80FF80u : kFill;
  const int32_t nt = (int32_t)ctas * kThreads, me = (int32_t)rank * kThreads + (int32_t)threadIdx.x;
  const int32_t shift = (int32_t)((reinterpret_cast<uintptr_t>(a) & 15u) / sizeof(T));
  const bool two = b != nullptr;
  const bool alike =
      !two || ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15u) == 0;
  const bool noise_alike =
      kNoise && ((reinterpret_cast<uintptr_t>(c) - 4u * (uintptr_t)shift) & 15u) == 0;
  const int32_t n8 = (vocab + shift + 7) / 8;
  constexpr int kLine = 128 / (8 * (int)sizeof(T));   // chunks of a line
  if (!kNoise && threadIdx.x % kLine == 0)
    for (int32_t t = me + kUnroll * nt; t < n8; t += nt) {
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a + max(8 * t - shift, 0)));
      if (two) asm volatile("prefetch.global.L2 [%0];" ::"l"(b + max(8 * t - shift, 0)));
    }
#pragma unroll 1
  for (int32_t t0 = me; t0 < n8; t0 += kUnroll * nt) {
    Eight<T> x[kUnroll], y[kUnroll];
    Eight<float> z[kNoise ? kUnroll : 1];
    int32_t i0[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const int32_t i = i0[k] = 8 * (t0 + k * nt) - shift;
      const bool inside = i >= 0 && i + 8 <= vocab;
      if (inside) x[k].load(a, i);
      else x[k].fill(kFill2);
      if (inside && alike) y[k].load(two ? b : a, i);
      else y[k].fill(kFill2);
      if constexpr (kNoise) {
        if (inside && noise_alike) z[k].load(c, i);
        else z[k].fill(0x3F800000u);
      }
    }
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      const bool inside = i0[k] >= 0 && i0[k] + 8 <= vocab;
      if (inside && alike && (!kNoise || noise_alike)) continue;
      if (i0[k] >= vocab) continue;
      if (!inside) x[k].gather(a, i0[k], vocab, kFill);
      if (two && !(inside && alike)) y[k].gather(b, i0[k], vocab, kFill);
      if constexpr (kNoise)
        if (!(inside && noise_alike)) z[k].gather(c, i0[k], vocab, 0x3F800000u);
    }
    f(i0, x, y, z);
  }
}

// Logits to log2 units.  A function so that it is not computed ahead, where fp32 will do.
__device__ __noinline__ double scale_64(float temp) { return 1.4426950408889634 / (double)temp; }

// A child's probability, and what is left of both children's behind a rejection (out of
// line as well: in the kernel they cost it registers).
__device__ __noinline__ double probability_64(float l, float m, double scale, double z) {
  return exp2(((double)l - (double)m) * scale) / z;
}
__device__ __noinline__ void left_64(double (&p)[2], const double (&q)[2], double sum) {
  for (int h = 0; h < 2; ++h) p[h] = fmax(p[h] - q[h], 0.0) / sum;
}

// A leaf's p over its noise in 64 bits, in log2 units (as a number it is out of all ranges
// at a small temperature), relative to a token with logit m.
__device__ __noinline__ double exact_leaf(double scale, float l, float m, float e) {
  return ((double)l - (double)m) * scale - log2((double)e);
}
// What is left of p in 64 bits: behind each rejection max(r - q, 0) over its sum; behind
// the last one (`last`) without.  (A sum may be subnormal, where its reciprocal is no
// number: two factors.)
struct Left64 {
  double scale, ip, iq;      // 1 / z of the two rows
  const double (*inv)[2];    // in shared memory
  int32_t n;
  float mp, mq;
  bool two, last;
  __device__ __forceinline__ double of(float l, float d) const {
    double r = __dmul_rn(exp2_64(((double)l - (double)mp) * scale), ip);
    if (two) {
      const double q = __dmul_rn(exp2_64(((double)d - (double)mq) * scale), iq);
      for (int k = 0; k < n; ++k)
        r = __dmul_rn(__dmul_rn(fmax(__dsub_rn(r, q), 0.0), inv[k][0]), inv[k][1]);
      if (last) r = fmax(__dsub_rn(r, q), 0.0);
    }
    return r;
  }
};
__device__ __noinline__ double exact_left(const Left64& n, float l, float d, float e) {
  return n.of(l, d) / (double)e;
}

// The passes over a node's rows, a function each so that each has its own
// registers (inlined into one kernel they spilled).

// Of the logits: maxima and sums.
template <class T, bool kSmall>
__device__ __forceinline__ Sums pass_sums(const T* tr, const T* dr, int32_t V, uint32_t rank,
                                          uint32_t ctas, float scale) {
  const uint64_t scale2 = pack2(scale, scale);
  Sums x = Sums::none();
  for_rows<T, kRows<T, kSmall>, false>(tr, dr, nullptr, V, rank, ctas,
                               [&](auto&, auto& l, auto& d, auto&) {
                                 add_chunks(x.p, l, scale, scale2);
                                 if (dr) add_chunks(x.q, d, scale, scale2);
                               });
  return x;
}

// The first largest logit.
template <class T, bool kSmall>
__device__ __noinline__ Best pass_largest(const T* tr, int32_t V, uint32_t rank, uint32_t ctas) {
  Best x = Best::none();
  for_rows<T, kRows<T, kSmall>, false>(
      tr, static_cast<const T*>(nullptr), nullptr, V, rank, ctas,
      [&](auto& i0, auto& l, auto&, auto&) {
#pragma unroll
        for (int j = 0; j < kRows<T, kSmall>; ++j)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float v = l[j].at(k);
            if (!(v < INFINITY)) x.bad = 1u;
            if (v > x.v) {   // a thread's indices go up
              x.v = v;
              x.i = i0[j] + k;
            }
          }
      });
  return x;
}

// What is left of p, sum max(p - a q, 0).
template <class T, bool kSmall>
__device__ __noinline__ Total<float> pass_total(const T* tr, const T* dr, int32_t V, uint32_t rank,
                                                uint32_t ctas, float scale, Sum sp, Sum sq, float a) {
  Total<float> y = {0.0f};
  const uint64_t bp = pack2(-sp.m, -sp.m), bq = pack2(-sq.m, -sq.m), scale2 = pack2(scale, scale);
  const float ip = 1.0f / sp.z, aq = a / sq.z;
  for_rows<T, kRows<T, kSmall>, false>(
      tr, dr, nullptr, V, rank, ctas, [&](auto&, auto& l, auto& d, auto&) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < kRows<T, kSmall>; ++j)
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 pe = exps(l[j].at(e), l[j].at(e + 1), bp, scale2);
            const float2 qe = exps(d[j].at(e), d[j].at(e + 1), bq, scale2);
            s += left(pe.x, qe.x, ip, aq) + left(pe.y, qe.y, ip, aq);
          }
        y.t += s;
      });
  return y;
}

// The two in 64 bits.
template <class T>
__device__ __noinline__ Sums64 pass_sums64(const T* tr, const T* dr, int32_t V, uint32_t rank,
                                           uint32_t ctas, double scale, float mp, float mq) {
  Sums64 x = {0.0, 0.0};
  for_rows<T, 1, false>(tr, dr, nullptr, V, rank, ctas, [&](auto&, auto& l, auto& d, auto&) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x.p += exp2_64(((double)l[0].at(k) - (double)mp) * scale);
      if (dr) x.q += exp2_64(((double)d[0].at(k) - (double)mq) * scale);
    }
  });
  return x;
}
template <class T>
__device__ __noinline__ Total<double> pass_total64(const T* tr, const T* dr, int32_t V, uint32_t rank,
                                                   uint32_t ctas, const Left64& n) {
  Total<double> y = {0.0};
  for_rows<T, 1, false>(tr, dr, nullptr, V, rank, ctas, [&](auto&, auto& l, auto& d, auto&) {
#pragma unroll
    for (int k = 0; k < 8; ++k) y.t += n.of(l[0].at(k), d[0].at(k));
  });
  return y;
}

// The scores of the last pass.  A leaf's in log2 units (no sum is known), the others'
// as upper bounds of what is left over the noise: p good to a part eps of itself makes
// that p (1 + eps) - a q (1 - eps).
struct Scores {
  float scale;
  bool two;                 // the rest: not of a leaf
  float mp, mq, ip, aq;     // for the upper bound
  float ip_low, aq_high;    // for the lower one
  int32_t n_removed;
  uint32_t removed_bits[2];
  const int32_t* removed;   // in shared memory
  template <bool kLeaf, class T>
  __device__ __forceinline__ void of(int32_t i0, const Eight<T>& l, const Eight<T>& d,
                                     const Eight<float>& e, float (&v)[8], uint32_t& bad) const {
    if constexpr (kLeaf) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float lk = l.at(k);
        if (!(lk < INFINITY)) bad = 1u;
        v[k] = fmaf(lk, scale, -__log2f(e.at(k)));
      }
    } else {
      const uint64_t bp = pack2(-mp, -mp), bq = pack2(-mq, -mq), scale2 = pack2(scale, scale);
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float2 pe = exps(l.at(k), l.at(k + 1), bp, scale2);
        v[k] = pe.x * ip;
        v[k + 1] = pe.y * ip;
        if (two) {
          const float2 qe = exps(d.at(k), d.at(k + 1), bq, scale2);
          v[k] = fmaxf(v[k] - qe.x * aq, 0.0f);
          v[k + 1] = fmaxf(v[k + 1] - qe.y * aq, 0.0f);
        }
        v[k] = __fdividef(v[k], e.at(k));
        v[k + 1] = __fdividef(v[k + 1], e.at(k + 1));
      }
      if (n_removed) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if ((removed_bits[((i0 + k) >> 5) & 1] >> ((i0 + k) & 31)) & 1u)
            for (int r = 0; r < n_removed; ++r)
              if (removed[r] == i0 + k) v[k] = -1.0f;
      }
    }
  }
  // the least that is left of a token
  __device__ __forceinline__ float low(float l, float d, float e) const {
    float s = fast_exp2((l - mp) * scale) * ip_low;
    if (two) s = fmaxf(s - fast_exp2((d - mq) * scale) * aq_high, 0.0f);
    return __fdividef(s, e);
  }
};

// The best score and the value of the second.
template <class T, bool kSmall, bool kLeaf>
__device__ __noinline__ auto pass_token(const T* tr, const T* dr, const float* noise, int32_t V,
                                        uint32_t rank, uint32_t ctas, const Scores& sc) {
  constexpr int kN = kSmall ? 1 : kRows<T, false> / 2;
  std::conditional_t<kLeaf, Best, Most> x = decltype(x)::none();
  uint32_t bad = 0u;
  for_rows<T, kN, true>(
      tr, dr, noise, V, rank, ctas, [&](auto& i0, auto& l, auto& d, auto& e) {
#pragma unroll
        for (int j = 0; j < kN; ++j) {
          float v[8];
          sc.of<kLeaf>(i0[j], l[j], d[j], e[j], v, bad);
          float m = v[0];
#pragma unroll
          for (int k = 1; k < 8; ++k) m = fmaxf(m, v[k]);
          if (m > x.second) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int32_t i = i0[j] + k;
              if (v[k] > x.second && i >= 0 && i < V) {
                if (v[k] > x.v) {
                  x.second = x.v;
                  x.v = v[k];
                  x.i = i;
                } else {
                  x.second = v[k];
                }
              }
            }
          }
        }
      });
  // (the best one's numbers are read again: keeping them took the batch from 80 to 84 us)
  if constexpr (kLeaf) x.bad = bad;
  else if (x.i >= 0)
    x.low = sc.low(value_of<T>(bits_now(tr, x.i)), sc.two ? value_of<T>(bits_now(dr, x.i)) : 0.0f,
                   __ldg(noise + x.i));
  return x;
}

// Again, the candidates from `near` up in 64 bits (of a leaf: with n.scale and n.mp).
template <class T, bool kLeaf>
__device__ __noinline__ Exact pass_near(const T* tr, const T* dr, const float* noise, int32_t V,
                                        uint32_t rank, uint32_t ctas, const Scores& sc, float near,
                                        const Left64& n) {
  Exact best = Exact::none();
  for_rows<T, 1, true>(
      tr, dr, noise, V, rank, ctas, [&](auto& i0, auto& l, auto& d, auto& e) {
        float v[8];
        uint32_t bad;
        sc.of<kLeaf>(i0[0], l[0], d[0], e[0], v, bad);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int32_t i = i0[0] + k;
          if (!(v[k] >= near) || i < 0 || i >= V) continue;
          const double s = kLeaf ? exact_leaf(n.scale, l[0].at(k), n.mp, e[0].at(k))
                                 : exact_left(n, l[0].at(k), d[0].at(k), e[0].at(k));
          best.add({s, i, 0}, 0.0f);
        }
      });
  return best;
}

// fp32's probabilities are good to 2e-6 of themselves (of a token 2^-30 as likely as the
// first; to 1.1e-5 down to 2^-126), b to 2e-6 of 1 + a, and a to the sum of its b's: tests
// with a margin of kEps and, for each rejection, kEpsMore are the right ones, bounds of
// scores the right ones with kEpsLow on top.  A sum is off by half a step for each
// addition that a thread makes in turn: kEpsAdd for those of both rows.
constexpr float kEps = 1e-5f, kEpsMore = 4e-6f, kEpsLow = 1e-5f, kEpsAdd = 0x1p-23f;

// Tests of the children in `todo`, in call order, by a whole warp (every warp of
// the cluster does the same): lane k has what belongs to children k and k + 32;
// `p`, `q`: of their tokens (64 bits, with draft logits: what is left of p).
template <class Real>
__device__ __forceinline__ Action test_children(Tests<Real>& s, bool two, const Kid (&kid)[2],
                                                const Real (&p)[2], const Real (&q)[2], int lane) {
  constexpr bool kFast = sizeof(Real) == 4;
  while (s.todo) {
    const int k = __ffsll((long long)s.todo) - 1, h = k >> 5, l = k & 31;
    s.todo &= s.todo - 1;
    const int32_t t = __shfl_sync(0xffffffffu, h ? kid[1].token : kid[0].token, l);
    if (t < 0) continue;
    const Real pk = __shfl_sync(0xffffffffu, h ? p[1] : p[0], l);
    const Real qk = __shfl_sync(0xffffffffu, h ? q[1] : q[0], l);
    const Real uk = __shfl_sync(0xffffffffu, h ? kid[1].u : kid[0].u, l);
    // certain drafts: nothing is left of a token that was removed
    if (!two && __any_sync(0xffffffffu, s.removed[0] == t || s.removed[1] == t)) continue;
    const Real x = uk * qk * (kFast || !two ? s.b : Real(1)), y = kFast && two ? pk - s.a * qk : pk;
    if (kFast) {
      const float near = two ? (s.a + uk * (1.0f + s.a)) * qk : uk;
      if (fabsf((float)(x - y)) <= s.eps * (float)(pk + near)) return kExact;
    }
    if (x < y) {
      s.taken = k;
      return kGo;
    }
    if (two) {
      s.a_prev = s.a;
      s.a += s.b;
      s.eps += kEpsMore;
      if (s.todo) return kSum;           // else the sum that is left is not needed
      if constexpr (!kFast) s.last = true;
    } else if (s.b - pk > Real(0)) {
      s.b -= pk;
      if (lane == (s.n_removed & 31)) {
        if (s.n_removed < 32) s.removed[0] = t;
        else s.removed[1] = t;
      }
      ++s.n_removed;
    }
  }
  return kToken;
}

template <class T, bool kSmall>
__global__ void __launch_bounds__(kThreads, kBlocks)
    k_verify(const __grid_constant__ VerifyParams p, const int ctas) {
  __shared__ Smem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = (uint32_t)blockIdx.x % (uint32_t)ctas;   // of the cluster
  const int tree = (int)((uint32_t)blockIdx.x / (uint32_t)ctas);
  const int32_t d0 = p.first[tree], n = p.first[tree + 1] - d0, V = p.vocab;
  const T* root = static_cast<const T*>(p.root);
  const T* droot = static_cast<const T*>(p.draft_root);
  const float* noise = p.noise + (int64_t)tree * p.noise_ld;
  // lane k of every warp has the parents of drafts k and k + 32
  int32_t parent[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) parent[h] = lane + 32 * h < n ? p.parent[d0 + lane + 32 * h] : -2;
  const int halves = n > 32 ? 2 : 1;
  griddep_wait();
  // the first CTA's: their tokens and numbers
  int32_t token[2] = {-1, -1};
  float uniform[2] = {0.0f, 0.0f};
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (rank == 0 && lane + 32 * h < n) {
      token[h] = __ldg(p.token + d0 + lane + 32 * h);
      if (p.uniform) uniform[h] = __ldg(p.uniform + d0 + lane + 32 * h);
    }
  if (rank == 0 && tid == 0) {
    const float t = p.temperature ? p.temperature[tree] : 0.0f;
    sm.temperature = t >= kCold ? fminf(t, kHot) : 0.0f;
  }
  // a row's share on its way to L2 while the cluster is not ready to read it
  auto prefetch = [&](const auto* r) {
    constexpr int kLine = 128 / sizeof(*r);
    for (int32_t i = kLine * ((int32_t)rank * kThreads + tid); i < V; i += kLine * ctas * kThreads)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(r + i));
  };
  if (root) prefetch(root + (int64_t)tree * p.ld);
  if (droot) prefetch(droot + (int64_t)tree * p.ld);
  cluster_arrive();
  cluster_wait();
  const float temp = ld_dsmem_f32(dsmem_addr(smem_u32(&sm.temperature), 0));
  const bool greedy = temp == 0.0f;
  const float scale = greedy ? 1.0f : 1.4426950408889634f / temp;   // logits to log2 units
  auto row_of = [&](const void* rows, const T* roots, int node) -> const T* {
    return node < 0 ? (roots ? roots + (int64_t)tree * p.ld : nullptr)
                    : (rows ? static_cast<const T*>(rows) + ((int64_t)d0 + node) * p.ld : nullptr);
  };
  int pass = 0;

  // The threads' parts merged over the cluster, in every thread: each warp
  // sends its own to all CTAs, and after the barrier merges all of them.
  auto join = [&](auto x) {
    using Part = decltype(x);
    static_assert(sizeof(Part) <= 4 * kPartWords, "parts");
    const int par = pass & 1, n_parts = ctas * kWarps;
    ++pass;
    x.over(32, lane, scale);
    if (ctas == 1) {   // (a cluster's barrier takes 500 cycles longer)
      if (lane == 0) *reinterpret_cast<Part*>(sm.part[par][warp]) = x;
      __syncthreads();
    } else {
      if (lane < ctas) st_peer(sm.part[par][rank * kWarps + warp], lane, x);
      cluster_arrive();
      cluster_wait();
    }
    x = lane < n_parts ? *reinterpret_cast<const Part*>(sm.part[par][lane]) : Part::none();
    for (int i = lane + 32; i < n_parts; i += 32) x.add(*reinterpret_cast<const Part*>(sm.part[par][i]), scale);
    x.over(n_parts < 32 ? n_parts : 32, lane, scale);
    // (fewer parts than lanes: lane 0's)
    Part y;
    const uint32_t* from = reinterpret_cast<const uint32_t*>(&x);
    uint32_t* to = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
    for (int k = 0; k < (int)(sizeof(Part) / 4); ++k) to[k] = __shfl_sync(0xffffffffu, from[k], 0);
    return y;
  };

  int node = -1, last = -1;
  int32_t result = -1;
  // the node is gone through again with its numbers in 64 bits, where fp32 cannot tell
  // (the whole of it: nothing is kept for that, and nothing of it computed ahead)
  bool first = true, exact = false;
  const float eps0 = kEps + kEpsAdd * (float)((uint32_t)V / ((uint32_t)ctas * kThreads * 8 * kRows<T, kSmall>));
  if (!root) {
    // the root's only child is the token that the last step has drawn
    if (n > 0) node = last = 0;
  }
  while (root || node >= 0) {
    const uint64_t kids =
        (uint64_t)__ballot_sync(0xffffffffu, parent[0] == node) |
        ((uint64_t)__ballot_sync(0xffffffffu, parent[1] == node) << 32);
    const T* tr = row_of(p.target, root, node);
    const T* dr = kids && !greedy ? row_of(p.draft, droot, node) : nullptr;
    const bool leaf = !kids;
    // the children, by way of the first CTA: its warp r reads their logits and,
    // with its part of the pass, sends them to CTA r
    Kid kid[2] = {{-1, 0.0f, 0.0f, 0.0f}, {-1, 0.0f, 0.0f, 0.0f}};
    const int kid_par = pass & 1;
    uint32_t lp[2], lq[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      lp[h] = lq[h] = 0u;
      if (rank == 0 && h < halves && !leaf && !greedy) {
        const int32_t t = token[h] >= 0 && token[h] < V ? token[h] : 0;
        lp[h] = bits_now(tr, t);
        if (dr) lq[h] = bits_now(dr, t);
      }
    }
    auto send_kids = [&] {
      for (int to = rank == 0 ? warp : ctas; to < ctas; to += kWarps) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (parent[h] == node)
            st_peer(&sm.kid[kid_par][lane + 32 * h], to,
                    Kid{token[h] >= 0 && token[h] < V ? token[h] : -1, uniform[h],
                        value_of<T>(lp[h]), value_of<T>(lq[h])});
      }
    };
    auto take_kids = [&] {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (parent[h] == node) kid[h] = sm.kid[kid_par][lane + 32 * h];
    };

    if (greedy) {
      Best x = pass_largest<T, kSmall>(tr, V, rank, ctas);
      send_kids();
      x = join(x);
      take_kids();
      if (x.bad || x.i < 0) break;
      // the first child with that token
      const uint64_t same =
          (uint64_t)__ballot_sync(0xffffffffu, parent[0] == node && kid[0].token == x.i) |
          ((uint64_t)__ballot_sync(0xffffffffu, parent[1] == node && kid[1].token == x.i) << 32);
      if (!same) {
        result = x.i;
        break;
      }
      node = last = __ffsll((long long)same) - 1;
      continue;
    }

    // what is left at the node
    Sum sp = {0.0f, 1.0f}, sq = {0.0f, 1.0f};
    float left_a = 0.0f, left_a_prev = 0.0f, eps = eps0;
    int32_t n_removed = 0;
    uint32_t removed_bits[2] = {0u, 0u};   // of the removed tokens' last six bits
    if (!leaf) {
      Sums x = pass_sums<T, kSmall>(tr, dr, V, rank, ctas, scale);
      send_kids();
      x = join(x);
      take_kids();
      // the noise is read once, at the walk's end: on its way to L2 meanwhile
      if (first) prefetch(noise);
      first = false;
      if (!(x.p.z < INFINITY && x.p.m > -INFINITY)) break;
      if (dr && !(x.q.z < INFINITY && x.q.m > -INFINITY)) break;
      sp = x.p;
      if (dr) sq = x.q;
      Action action;
      int32_t taken, removed[2];
      if (!exact) {
        Tests<float> s = {0.0f, 0.0f, 1.0f, eps0, kids, false, -1, {-1, -1}, 0};
        float pk[2] = {0.0f, 0.0f}, qk[2] = {0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h >= halves) break;
          pk[h] = __fdividef(exp2f((kid[h].lp - sp.m) * scale), sp.z);
          qk[h] = dr ? __fdividef(exp2f((kid[h].lq - sq.m) * scale), sq.z) : 1.0f;
        }
        while ((action = test_children<float>(s, dr, kid, pk, qk, lane)) == kSum) {
          const Total<float> y =
              join(pass_total<T, kSmall>(tr, dr, V, rank, ctas, scale, sp, sq, s.a));
          s.b = y.t;
          if (!(y.t > s.eps * (1.0f + s.a))) {   // that may be nothing, or a part of it
            action = kExact;
            break;
          }
        }
        taken = s.taken;
        left_a = s.a;
        left_a_prev = s.a_prev;
        eps = s.eps;
        n_removed = s.n_removed;
        removed[0] = s.removed[0];
        removed[1] = s.removed[1];
      } else {
        const double c = scale_64(temp);
        const Sums64 z = join(pass_sums64(tr, dr, V, rank, ctas, c, sp.m, sq.m));
        Tests<double> s = {0.0, 0.0, 1.0, 0.0f, kids, false, -1, {-1, -1}, 0};
        double pk[2], qk[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          pk[h] = probability_64(kid[h].lp, sp.m, c, z.p);
          qk[h] = dr ? probability_64(kid[h].lq, sq.m, c, z.q) : 1.0;
        }
        int32_t n64 = 0;
        while ((action = test_children<double>(s, dr, kid, pk, qk, lane)) == kSum) {
          const Total<double> y = join(pass_total64(
              tr, dr, V, rank, ctas, {c, 1.0 / z.p, 1.0 / z.q, sm.inv, n64, sp.m, sq.m, true, true}));
          if (!(y.t > 0.0)) {   // nothing: as before this rejection
            s.a = s.a_prev;
            continue;
          }
          s.b *= y.t;
          left_64(pk, qk, y.t);
          if (tid == 0) {
            sm.inv[n64][0] = y.t < 0x1p-900 ? 0x1p1000 : 1.0;
            sm.inv[n64][1] = 1.0 / (y.t * sm.inv[n64][0]);
          }
          ++n64;
          __syncthreads();
        }
        taken = s.taken;
        left_a = (float)s.a;
        left_a_prev = (float)s.a_prev;
        n_removed = s.n_removed;
        removed[0] = s.removed[0];
        removed[1] = s.removed[1];
        if (tid == 0) {
          sm.z[0] = z.p;
          sm.z[1] = z.q;
          sm.n_inv = n64;
          sm.last = s.last;
        }
        __syncthreads();
      }
      if (action == kExact) {
        exact = true;
        continue;
      }
      if (action == kGo) {
        node = last = taken;
        exact = false;
        continue;
      }
      if (n_removed) {
        for (int r = 0; r < n_removed; ++r) {
          const int32_t t = __shfl_sync(0xffffffffu, r < 32 ? removed[0] : removed[1], r & 31);
          removed_bits[(t >> 5) & 1] |= 1u << (t & 31);
          if (tid == 0) sm.removed[r] = t;
        }
        __syncthreads();
      }
    }

    // ---- the next token
    Scores sc;
    sc.scale = scale;
    sc.two = dr != nullptr;
    sc.mp = sp.m;
    sc.mq = sq.m;
    sc.n_removed = n_removed;
    sc.removed_bits[0] = removed_bits[0];
    sc.removed_bits[1] = removed_bits[1];
    sc.removed = sm.removed;
    if (leaf) {
      const Best top = join(pass_token<T, kSmall, true>(tr, dr, noise, V, rank, ctas, sc));
      if (top.bad || !(top.v > -INFINITY)) break;
      result = top.i;
      // candidates that the fp32 scores may have in the wrong order: these are off by
      // a few 2^-24 of the logit in log2 units
      const float near = top.v - 2e-6f * (fabsf(top.v) + 256.0f);
      if (top.second >= near) {
        const float base = value_of<T>(bits_now(tr, top.i));
        result = join(pass_near<T, true>(tr, dr, noise, V, rank, ctas, sc, near,
                                         {scale_64(temp), 0.0, 0.0, nullptr, 0, base, 0.0f, false, false})).i;
      }
      break;
    }
    eps += kEpsLow;
    bool again = false;      // nothing is left: as before the last rejection
    while (true) {
      const float ip = 1.0f / sp.z, aq = dr ? (again ? left_a_prev : left_a) / sq.z : 0.0f;
      sc.ip = ip * (1.0f + eps);
      sc.ip_low = ip * (1.0f - eps);
      sc.aq = aq * (1.0f - eps);
      sc.aq_high = aq * (1.0f + eps);
      const Most top = join(pass_token<T, kSmall, false>(tr, dr, noise, V, rank, ctas, sc));
      if (top.low > 0.0f && top.second < top.low) {
        result = top.i;
        break;
      }
      if (dr && !exact) break;
      // (without draft logits the sum is a factor that all have in common)
      const bool last = dr && sm.last && !again;
      const Left64 n = {scale_64(temp), dr ? 1.0 / sm.z[0] : 1.0, dr ? 1.0 / sm.z[1] : 0.0,
                        sm.inv, dr ? sm.n_inv : 0, sp.m, sq.m, dr != nullptr, last};
      const Exact x = join(pass_near<T, false>(tr, dr, noise, V, rank, ctas, sc, top.low, n));
      if (x.v > 0.0) {
        result = x.i;
        break;
      }
      if (!last) break;
      again = true;
    }
    if (result >= 0 || !dr || exact) break;
    exact = true;
  }
  griddep_launch();
  if (rank == 0 && tid == 0) {
    p.accepted[tree] = last;
    p.next_token[tree] = result;
  }
  // no CTA leaves while another may write to its shared memory
  cluster_arrive();
  cluster_wait();
}

template <class T, bool kSmall>
cudaError_t launch(const VerifyParams& p, int cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.n_trees * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2] = {pdl_attribute(), {}};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cluster > 8) {
    const cudaError_t e = cudaFuncSetAttribute(k_verify<T, kSmall>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, k_verify<T, kSmall>, p, cluster);
}

}  // namespace

// CTAs of a sequence's cluster: as many as run at once over the whole GPU, with
// a share of the vocabulary worth a pass each.  Clusters of 16 (8 SMs of one of the
// GPU's processing clusters) with room to spare, since they do not fill those: 8 trees of
// 8 drafts over 131072 tokens take 26.1 us with 16 and 30.0 with 8, one 11.2 and 13.8.
int verify_cluster(int64_t n_trees, int32_t vocab, int sms) {
  int c = 1;
  while (c < kMaxCluster && n_trees * c * (c < 8 ? 2 : 3) <= (int64_t)sms * kBlocks && vocab >= 4096 * c) c *= 2;
  return c;
}

cudaError_t launch_verify(const VerifyParams& p, bool fp32, int cluster, cudaStream_t s) {
  if (p.n_trees <= 0) return cudaSuccess;
  if (cluster < 1 || cluster > kMaxCluster) return cudaErrorInvalidValue;
  if (p.vocab <= 2 * 8 * kThreads * cluster)   // at most two chunks a thread
    return fp32 ? launch<float, true>(p, cluster, s) : launch<uint16_t, true>(p, cluster, s);
  return fp32 ? launch<float, false>(p, cluster, s) : launch<uint16_t, false>(p, cluster, s);
}

}  // namespace csa2
