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
// fp32 on the rows (a sum of 100,000 terms in 4096 partial sums is good to
// about 1e-7), 64 bits on the few numbers that a test compares.  The token: a
// second candidate so near the best that the fp32 scores cannot tell them
// apart is looked for, and if there is one all such are scored again in 64
// bits.
#include "csa2_device.cuh"
#include "csa2_kernels.h"

namespace csa2 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

// (value, index) of the best so far and the value of the second.
struct Best {
  float v, second;
  int32_t i;
};
__device__ __forceinline__ void best_add(Best& b, float v, int32_t i) {
  if (v > b.v || (v == b.v && (uint32_t)i < (uint32_t)b.i)) {
    b.second = b.v;
    b.v = v;
    b.i = i;
  } else if (v > b.second) {
    b.second = v;
  }
}
__device__ __forceinline__ Best best_merge(const Best& a, const Best& b) {
  const bool first = a.v > b.v || (a.v == b.v && (uint32_t)a.i < (uint32_t)b.i);
  Best r = first ? a : b;
  r.second = fmaxf(r.second, first ? b.v : a.v);
  return r;
}
// Largest logit m of a part of a row, and the sum of exp2((l - m) * scale).  The
// difference of two logits is formed first: it is all but exact, and the
// probabilities that count have small ones (l * scale - m * scale would round
// at the logits' own size).
struct Sum {
  float m, z;
};
__device__ __forceinline__ Sum sum_merge(const Sum& a, const Sum& b, float scale) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return {m, 0.0f};
  return {m, a.z * exp2f((a.m - m) * scale) + b.z * exp2f((b.m - m) * scale)};
}

struct Part {      // of a CTA, per pass
  Sum p, q;
  float total;
  uint32_t bad;
  Best best;
  double exact;
  int32_t exact_i;
};
struct Kid {       // a child of the node
  float lp, lq, u;
  int32_t token;   // -1: outside the vocabulary
};
struct Smem {
  Part part[2];        // by pass parity: read by the cluster
  Kid kid[2][64];      // of the cluster's first CTA: read by the cluster
  float temperature;
  Part all;            // of the cluster
  Part warp[kWarps];
  uint64_t kids;       // the node's children
  double pd[64], qd[64];
  int32_t tok[64];
  float u[64];
  // decision of thread 0
  double a, b, a_prev;
  int32_t taken, n_removed;
  int32_t removed[64];
};

__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// A struct of words at `local` in another CTA of the cluster.
template <class T>
__device__ __forceinline__ T ld_peer(const T* local, uint32_t rank) {
  static_assert(sizeof(T) % 4 == 0, "words");
  const uint32_t at = dsmem_addr(smem_u32(local), rank);
  T v;
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int k = 0; k < (int)(sizeof(T) / 4); ++k) w[k] = ld_dsmem_u32(at + 4 * k);
  return v;
}

template <class T>
__device__ __forceinline__ float value_at(const T* row, int64_t i) {
  if constexpr (sizeof(T) == 2) return bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(row) + i));
  else return __ldg(reinterpret_cast<const float*>(row) + i);
}

// Eight values of a row.  vec: neighbours, the row at a 16-byte boundary;
// else a warp's lanes read neighbours, eight rounds of them.
template <class T>
__device__ __forceinline__ void load8(const T* row, int64_t i, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(row) + i));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  } else {
    const float4* s = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(row) + i);
    const float4 a = __ldg(s), b = __ldg(s + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
}

// The CTA's share of rows a, b (nullable) and c (nullable, fp32): f(n, i, x,
// y, z) for eight elements at a time, element k at index i(k); those past the
// end come as `fill`.
template <class T, bool kVec, class F>
__device__ __forceinline__ void for_rows(const T* a, const T* b, const float* c, int32_t vocab,
                                         uint32_t rank, uint32_t ctas, float fill, F f) {
  const int64_t nt = (int64_t)ctas * kThreads, me = (int64_t)rank * kThreads + threadIdx.x;
  const int64_t n8 = ((int64_t)vocab + 7) / 8;
  for (int64_t t = me; t < (kVec ? n8 : (n8 + nt - 1) / nt * nt); t += nt) {
    // kVec: chunk t; else round t / nt of eight strided elements
    const int64_t i0 = kVec ? 8 * t : (t - me) * 8 + me, step = kVec ? 1 : nt;
    float x[8], y[8], z[8];
    if (kVec && i0 + 8 <= vocab) {
      load8<T>(a, i0, x);
      if (b) load8<T>(b, i0, y);
      if (c) load8<float>(reinterpret_cast<const float*>(c), i0, z);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t i = i0 + k * step;
        const bool in = i < vocab;
        x[k] = in ? value_at(a, i) : fill;
        if (b) y[k] = in ? value_at(b, i) : fill;
        if (c) z[k] = in ? __ldg(c + i) : 1.0f;
      }
    }
    f(i0, step, x, y, z);
  }
}

template <class T, bool kVec>
__global__ void __launch_bounds__(kThreads) k_verify(const __grid_constant__ VerifyParams p,
                                                     const int ctas) {
  __shared__ Smem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = (uint32_t)blockIdx.x % (uint32_t)ctas;   // of the cluster
  const int tree = (int)((uint32_t)blockIdx.x / (uint32_t)ctas);
  const int32_t d0 = p.first[tree], n = p.first[tree + 1] - d0, V = p.vocab;
  griddep_wait();
  if (tid == 0) {
    float t = p.temperature ? p.temperature[tree] : 0.0f;
    sm.temperature = t > 0.0f ? t : 0.0f;
  }
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  float temp;
  {
    const uint32_t at = dsmem_addr(smem_u32(&sm.temperature), 0);
    temp = ld_dsmem_f32(at);
  }
  const bool greedy = temp == 0.0f;
  const float scale = greedy ? 1.0f : 1.4426950408889634f / temp;   // logits to log2 units
  const T* root = static_cast<const T*>(p.root);
  const T* droot = static_cast<const T*>(p.draft_root);
  auto row_of = [&](const void* rows, const T* roots, int node) -> const T* {
    return node < 0 ? (roots ? roots + (int64_t)tree * p.ld : nullptr)
                    : (rows ? static_cast<const T*>(rows) + ((int64_t)d0 + node) * p.ld : nullptr);
  };
  int pass = 0;

  // Joins the threads' parts over the cluster into sm.all; `kids`: the
  // children's data of the first CTA into sm.tok / u (and pd, qd: the logits)
  auto join = [&](Part x, bool kids) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Sum yp = {__shfl_xor_sync(0xffffffffu, x.p.m, o), __shfl_xor_sync(0xffffffffu, x.p.z, o)};
      const Sum yq = {__shfl_xor_sync(0xffffffffu, x.q.m, o), __shfl_xor_sync(0xffffffffu, x.q.z, o)};
      const Best yb = {__shfl_xor_sync(0xffffffffu, x.best.v, o),
                       __shfl_xor_sync(0xffffffffu, x.best.second, o),
                       __shfl_xor_sync(0xffffffffu, x.best.i, o)};
      // the lower lane's part first: both lanes get the same sum
      const bool lo = (lane & o) == 0;
      x.p = lo ? sum_merge(x.p, yp, scale) : sum_merge(yp, x.p, scale);
      x.q = lo ? sum_merge(x.q, yq, scale) : sum_merge(yq, x.q, scale);
      x.best = best_merge(x.best, yb);
      x.total += __shfl_xor_sync(0xffffffffu, x.total, o);
      x.bad |= __shfl_xor_sync(0xffffffffu, x.bad, o);
      const double e = __shfl_xor_sync(0xffffffffu, x.exact, o);
      const int32_t ei = __shfl_xor_sync(0xffffffffu, x.exact_i, o);
      if (e > x.exact || (e == x.exact && (uint32_t)ei < (uint32_t)x.exact_i)) {
        x.exact = e;
        x.exact_i = ei;
      }
    }
    auto merge = [&](Part& s, const Part& y) {
      s.p = sum_merge(s.p, y.p, scale);
      s.q = sum_merge(s.q, y.q, scale);
      s.best = best_merge(s.best, y.best);
      s.total += y.total;
      s.bad |= y.bad;
      if (y.exact > s.exact || (y.exact == s.exact && (uint32_t)y.exact_i < (uint32_t)s.exact_i)) {
        s.exact = y.exact;
        s.exact_i = y.exact_i;
      }
    };
    if (lane == 0) sm.warp[warp] = x;
    __syncthreads();
    const int par = pass & 1;
    ++pass;
    if (tid == 0) {
      Part s = sm.warp[0];
      for (int w = 1; w < kWarps; ++w) merge(s, sm.warp[w]);
      sm.part[par] = s;
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    if (tid == 0) {
      Part s = ld_peer(&sm.part[par], 0);
      for (int r = 1; r < ctas; ++r) merge(s, ld_peer(&sm.part[par], r));
      sm.all = s;
    }
    if (kids && tid >= 64 && tid < 128 && ((sm.kids >> (tid - 64)) & 1ull)) {
      const int k = tid - 64;
      const Kid y = ld_peer(&sm.kid[par][k], 0);
      sm.tok[k] = y.token;
      sm.u[k] = y.u;
      sm.pd[k] = y.lp;
      sm.qd[k] = y.lq;
    }
    __syncthreads();
  };
  const Part none = {{-INFINITY, 0.0f}, {-INFINITY, 0.0f}, 0.0f, 0u, {-INFINITY, -INFINITY, -1}, -1.0, -1};

  int node = -1, last = -1;
  int32_t result = -1;
  if (!root) {
    // the root's only child is the token that the last step has drawn
    if (n > 0) node = last = 0;
  }
  while (root || node >= 0) {
    // ---- the node's children
    uint64_t kids = 0;
    {
      const bool kid = tid < 64 && tid < n && p.parent[d0 + tid] == node;
      const uint32_t m = __ballot_sync(0xffffffffu, kid);
      __syncthreads();
      if (warp < 2 && lane == 0) reinterpret_cast<uint32_t*>(&sm.kids)[warp] = m;
      __syncthreads();
      kids = sm.kids;
    }
    const T* tr = row_of(p.target, root, node);
    const T* dr = kids && !greedy ? row_of(p.draft, droot, node) : nullptr;
    if (rank == 0 && tid < 64 && ((kids >> tid) & 1ull)) {
      Kid k = {-INFINITY, -INFINITY, 0.0f, p.token[d0 + tid]};
      if (k.token < 0 || k.token >= V) k.token = -1;
      if (!greedy) {
        k.u = p.uniform[d0 + tid];
        if (k.token >= 0) {
          k.lp = value_at(tr, k.token);
          if (dr) k.lq = value_at(dr, k.token);
        }
      }
      sm.kid[pass & 1][tid] = k;
    }

    if (greedy) {
      Part x = none;
      for_rows<T, kVec>(tr, static_cast<const T*>(nullptr), nullptr, V, rank, ctas, -INFINITY,
                        [&](int64_t i0, int64_t step, const float (&l)[8], const float (&)[8],
                            const float (&)[8]) {
#pragma unroll
                          for (int k = 0; k < 8; ++k) {
                            if (!(l[k] < INFINITY)) x.bad = 1u;
                            if (l[k] > x.best.v) {
                              x.best.v = l[k];
                              x.best.i = (int32_t)(i0 + k * step);
                            }
                          }
                        });
      join(x, true);
      if (sm.all.bad || sm.all.best.i < 0) break;
      const int32_t top = sm.all.best.i;
      int32_t taken = -1;
      for (uint64_t m = kids; m; m &= m - 1) {
        const int k = __ffsll((long long)m) - 1;
        if (sm.tok[k] == top) {
          taken = k;
          break;
        }
      }
      __syncthreads();
      if (taken < 0) {
        result = top;
        break;
      }
      node = last = taken;
      continue;
    }

    // rows p and q of the node for the last pass: p * ip and q * iq
    double a = 0.0, a_prev = 0.0;
    int32_t n_removed = 0;
    Sum sp = {0.0f, 1.0f}, sq = {0.0f, 1.0f};
    if (kids) {
      // ---- maxima and sums of the node's rows
      Part x = none;
      auto add = [&](Sum& s, const float (&l)[8]) {
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (!(l[k] < INFINITY)) x.bad = 1u;
          m = fmaxf(m, l[k]);
        }
        if (m > s.m) {
          s.z *= fast_exp2((s.m - m) * scale);
          s.m = m;
        }
        const float base = s.m == -INFINITY ? 0.0f : s.m;
        float z = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) z += fast_exp2((l[k] - base) * scale);
        s.z += z;
      };
      for_rows<T, kVec>(tr, dr, nullptr, V, rank, ctas, -INFINITY,
                        [&](int64_t, int64_t, const float (&l)[8], const float (&d)[8],
                            const float (&)[8]) {
                          add(x.p, l);
                          if (dr) add(x.q, d);
                        });
      join(x, true);
      sp = sm.all.p;
      sq = sm.all.q;
      if (sm.all.bad || sp.m == -INFINITY || (dr && sq.m == -INFINITY)) break;
      // ---- probabilities of the children's tokens, in 64 bits
      if (tid < 64 && ((kids >> tid) & 1ull)) {
        const double c = 1.4426950408889634 / (double)temp;
        const bool in = sm.tok[tid] >= 0;
        sm.pd[tid] = in ? exp2((sm.pd[tid] - (double)sp.m) * c) / (double)sp.z : 0.0;
        sm.qd[tid] = !in ? 0.0 : dr ? exp2((sm.qd[tid] - (double)sq.m) * c) / (double)sq.z : 1.0;
      }
      __syncthreads();
      // ---- tests, in call order
      double b = 1.0;
      int32_t taken = -1;
      uint64_t m = kids;
      while (m) {
        const int k = __ffsll((long long)m) - 1;
        m &= m - 1;
        const int32_t t = sm.tok[k];
        if (t < 0) continue;
        const double pk = sm.pd[k], qk = sm.qd[k], u = sm.u[k];
        if (dr) {
          if (u * qk * b < pk - a * qk) {
            taken = k;
            break;
          }
          a_prev = a;
          a += b;
          if (!m) break;                 // the sum that is left is not needed
          Part y = none;
          const float ip = 1.0f / sp.z, iq = (float)(a / (double)sq.z);
          for_rows<T, kVec>(tr, dr, nullptr, V, rank, ctas, -INFINITY,
                            [&](int64_t, int64_t, const float (&l)[8], const float (&d)[8],
                                const float (&)[8]) {
                              float s = 0.0f;
#pragma unroll
                              for (int e = 0; e < 8; ++e)
                                s += fmaxf(fast_exp2((l[e] - sp.m) * scale) * ip -
                                               fast_exp2((d[e] - sq.m) * scale) * iq,
                                           0.0f);
                              y.total += s;
                            });
          join(y, false);
          if (sm.all.total > 0.0f) b = sm.all.total;
          else a = a_prev;
          __syncthreads();
        } else {
          bool gone = false;
          for (int r = 0; r < n_removed; ++r) gone |= sm.removed[r] == t;
          if (gone) continue;            // nothing of it is left
          if (u * b < pk) {
            taken = k;
            break;
          }
          if (b - pk > 0.0) {
            b -= pk;
            __syncthreads();
            if (tid == 0) sm.removed[n_removed] = t;
            ++n_removed;
            __syncthreads();
          }
        }
      }
      __syncthreads();
      if (taken >= 0) {
        node = last = taken;
        continue;
      }
    }

    // ---- the next token
    const float* noise = p.noise + (int64_t)tree * p.noise_ld;
    const bool leaf = !kids;
    // scores in log2 units where no sum is needed (a leaf), else probabilities
    // over noise; 64-bit form of element i
    auto exact_score = [&](int32_t i) -> double {
      const double c = 1.4426950408889634 / (double)temp, e = (double)__ldg(noise + i);
      const double l = (double)value_at(tr, i);
      if (leaf) return exp2(l * c - floor((double)sm.all.best.v)) / e;
      const double pv = exp2((l - (double)sp.m) * c) / (double)sp.z;
      if (!dr) return pv / e;
      const double qv = exp2(((double)value_at(dr, i) - (double)sq.m) * c) / (double)sq.z;
      return fmax(pv - a * qv, 0.0) / e;
    };
    bool again = false;
    while (true) {
      const float ip = 1.0f / sp.z, iq = dr ? (float)(a / (double)sq.z) : 0.0f;
      Part x = none;
      auto score = [&](int32_t i, float l, float d, float e) -> float {
        if (leaf) {
          if (!(l < INFINITY)) x.bad = 1u;
          return fmaf(l, scale, -__log2f(e));
        }
        float v = fast_exp2((l - sp.m) * scale) * ip;
        if (dr) v = fmaxf(v - fast_exp2((d - sq.m) * scale) * iq, 0.0f);
        for (int r = 0; r < n_removed; ++r)
          if (sm.removed[r] == i) v = 0.0f;
        return __fdividef(v, e);
      };
      // with the same scores, the candidates within `near` of the best in 64 bits
      auto scan = [&](float near, bool exact) {
        for_rows<T, kVec>(tr, dr, noise, V, rank, ctas, -INFINITY,
                          [&](int64_t i0, int64_t step, const float (&l)[8], const float (&d)[8],
                              const float (&e)[8]) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                              const int64_t i = i0 + k * step;
                              const float v = score((int32_t)i, l[k], dr ? d[k] : 0.0f, e[k]);
                              if (i >= V) continue;
                              if (!exact) {
                                if (v > x.best.second) best_add(x.best, v, (int32_t)i);
                              } else if (v >= near) {
                                const double s = exact_score((int32_t)i);
                                if (s > x.exact || (s == x.exact && (int32_t)i < x.exact_i)) {
                                  x.exact = s;
                                  x.exact_i = (int32_t)i;
                                }
                              }
                            }
                          });
      };
      scan(0.0f, false);
      join(x, false);
      const Part& all = sm.all;
      if (leaf ? (all.bad || !(all.best.v > -INFINITY)) : !(all.best.v > 0.0f)) {
        // a node's row that nothing is left of: as before the last rejection
        if (!leaf && dr && !again && a != a_prev) {
          again = true;
          a = a_prev;
          __syncthreads();
          continue;
        }
        break;
      }
      result = all.best.i;
      const float near = leaf ? all.best.v - 2e-6f * (fabsf(all.best.v) + 256.0f)
                              : all.best.v * (1.0f - 1e-4f);
      if (all.best.second >= near) {
        x = none;
        scan(near, true);
        __syncthreads();
        join(x, false);
        result = sm.all.exact_i;
      }
      break;
    }
    break;
  }
  if (rank == 0 && tid == 0) {
    p.accepted[tree] = last;
    p.next_token[tree] = result;
  }
  // no CTA leaves while another may read its shared memory
  cluster_arrive();
  cluster_wait();
}

template <class T>
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
  return p.vec ? cudaLaunchKernelEx(&cfg, k_verify<T, true>, p, cluster)
               : cudaLaunchKernelEx(&cfg, k_verify<T, false>, p, cluster);
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, bool fp32, int cluster, cudaStream_t s) {
  if (p.n_trees <= 0) return cudaSuccess;
  if (cluster < 1 || cluster > kMaxCluster) return cudaErrorInvalidValue;
  return fp32 ? launch<float>(p, cluster, s) : launch<uint16_t>(p, cluster, s);
}

}  // namespace csa2
