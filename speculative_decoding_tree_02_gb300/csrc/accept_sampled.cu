// accept_sampled: verification of drafted tokens against the target's
// probabilities (temperature, top-k and top-p of each request) from given
// random numbers; include/tv.h states the rule.
//
// Two kernels.  row_kernel takes every node's row of logits at once: a cluster
// of 8 CTAs per row finds its maximum, the truncation's threshold and the mass
// of what is kept, 16 bytes per row.  walk_kernel then needs single logits for
// the accept tests, and passes over a row only for what a rejected draw leaves
// and for the last token.  Rejections only ever turn the distribution into
// max(0, a p - b q) without the tokens that were removed, so two numbers and a
// bit mask stand for it and no row is written.
#include <algorithm>

#include "cluster.cuh"

namespace tv {
namespace {

constexpr int kAsCluster = 8;
constexpr int kAsThreads = 256;
constexpr int kAsWarps = kAsThreads / 32;
constexpr int kAsMaxVocab = 1 << 20;
constexpr int kBins = 32;

// What row_kernel says of a row: p(v) = 2^((l - top) c) inv for l >= floor, else 0;
// greedy rows (inv = -1): floor holds the chosen token.
struct RowStat {
  float top, c, floor, inv;
};

// (l - top) c in [-1e30, 0]: an infinite maximum is given as the largest finite
// number, and NaN and -inf come out at the low end.
__device__ __forceinline__ float log_weight(float l, float top, float c) {
  return fminf(fmaxf((l - top) * c, -1e30f), 0.f);
}
__device__ __forceinline__ float prob(float l, const RowStat& s) {
  return l >= s.floor ? ex2(log_weight(l, s.top, s.c)) * s.inv : 0.f;
}

// Eight consecutive logits; -inf past the end.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int v, int end, bool vec, float (&x)[8]) {
  if (vec && v + 8 <= end) {
    if constexpr (sizeof(T) == 2) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + v));
      x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
      x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
    } else {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + v)), b = __ldg(reinterpret_cast<const float4*>(row + v) + 1);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = -INFINITY;
    if (v + e < end) {
      if constexpr (sizeof(T) == 2) x[e] = bf16_at(reinterpret_cast<const uint16_t*>(row) + v + e);
      else x[e] = row[v + e];
    }
  }
}
template <typename T>
__device__ __forceinline__ float one(const T* row, int v) {
  if constexpr (sizeof(T) == 2) return bf16_at(reinterpret_cast<const uint16_t*>(row) + v);
  else return row[v];
}

// Slice of CTA `rank`: the starts are multiples of 8.
__device__ __forceinline__ int slice_len(int V) { return ((V + kAsCluster - 1) / kAsCluster + 7) / 8 * 8; }

struct RowArgs {
  const void* p;
  const int32_t* node_off;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  RowStat* stat;
  int64_t ld;
  int V, max_nodes, total;
  bool vec;
};

struct RowShared {
  float xf[2][kBins];            // exchanged with the cluster, by parity
  int xi[2][2];
  float tot[kBins];
  float wred[kAsWarps];
  int wred_i[kAsWarps];
};

// Sums over the cluster of up to 32 numbers that lie in sh.xf[e & 1] of each
// CTA; every CTA adds them in the order of the ranks.
__device__ __forceinline__ void cluster_sums(RowShared& sh, int e, int n) {
  cl::sync();
  if (threadIdx.x < n) {
    float t = 0.f;
    for (uint32_t c = 0; c < kAsCluster; ++c) t += cl::peek(&sh.xf[e & 1][threadIdx.x], c);
    sh.tot[threadIdx.x] = t;
  }
  __syncthreads();
}

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}

// The bin in which the running sum over tot[0], tot[1], .. reaches `target`
// (the last one with anything in it, if none does), and the sum before it.
__device__ __forceinline__ int crossing(const float* tot, float target, float before, float& above) {
  int at = 0;
  float run = before;
  above = before;
  for (int b = 0; b < kBins; ++b) {
    const float t = tot[b];
    if (t > 0.f) {
      at = b;
      above = run;
      if (run + t >= target) break;
    }
    run += t;
  }
  return at;
}

template <typename T, bool kTrunc>
__global__ void __cluster_dims__(kAsCluster, 1, 1) __launch_bounds__(kAsThreads) row_kernel(const RowArgs a) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ RowShared sh;
  griddep_wait();
  griddep_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cl::rank();
  const int r = blockIdx.y, i = blockIdx.x / kAsCluster;
  const int n0 = max(a.node_off[r], 0);
  if (i >= a.node_off[r + 1] - n0 || n0 + i >= a.total) return;      // (the whole cluster)
  const int64_t row = n0 + i;
  const T* p = static_cast<const T*>(a.p) + row * a.ld;
  const int V = a.V, S = slice_len(V);
  const int v0 = min(V, static_cast<int>(rank) * S), v1 = min(V, v0 + S);
  const float temp = a.temperature ? a.temperature[r] : 1.f;
  const bool greedy = !(temp > 0.f);
  const float c = fminf(kLog2e / temp, 1e30f);
  int k = kTrunc && a.top_k ? a.top_k[r] : 0;
  if (k >= V) k = 0;
  const float nucleus = kTrunc && a.top_p ? a.top_p[r] : 1.f;
  const bool by_k = !greedy && k > 0, by_p = !greedy && nucleus < 1.f;
  T* xs = reinterpret_cast<T*>(dyn);              // the slice, each thread's own eighths

  // maximum (and its first place); the slice into shared memory where passes follow
  float m = -INFINITY, s = 0.f;
  int at = 0x7fffffff;
  const bool stage = by_k || by_p;
  for (int v = v0 + 8 * tid; v < v1; v += 8 * kAsThreads) {
    float x[8];
    load8(p, v, v1, a.vec, x);
    float m8 = x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) m8 = fmaxf(m8, x[e]);
    if (greedy) {
      if (m8 > m) {
        m = m8;
#pragma unroll
        for (int e = 7; e >= 0; --e)
          if (x[e] == m8) at = v + e;
      }
      continue;
    }
    if (stage) {
      m = fmaxf(m, m8);
      if constexpr (kTrunc) {
        if constexpr (sizeof(T) == 2) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = (__float_as_uint(x[2 * e]) >> 16) | (__float_as_uint(x[2 * e + 1]) & 0xffff0000u);
          *reinterpret_cast<uint4*>(xs + (v - v0)) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          *reinterpret_cast<float4*>(xs + (v - v0)) = make_float4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<float4*>(xs + (v - v0) + 4) = make_float4(x[4], x[5], x[6], x[7]);
        }
      }
      continue;
    }
    if (m8 > 3.402823466e38f) m8 = 3.402823466e38f;
    if (m8 > m) {                                 // running maximum and sum
      s *= ex2(fmaxf((m - m8) * c, -1e30f));
      m = m8;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s += ex2(log_weight(x[e], m, c));
  }
  int e = 0;
  // over the cluster: the maximum, its first place or the sum
  const float wm = warp_max(m);
  if (lane == 0) sh.wred[warp] = wm;
  const int wi = __reduce_min_sync(0xffffffffu, m == wm && greedy ? at : 0x7fffffff);
  if (lane == 0) sh.wred_i[warp] = wi;
  __syncthreads();
  float top = sh.wred[0];
  for (int w = 1; w < kAsWarps; ++w) top = fmaxf(top, sh.wred[w]);
  if (tid == 0) {
    int first = 0x7fffffff;
    for (int w = 0; w < kAsWarps; ++w)
      if (sh.wred[w] == top) first = min(first, sh.wred_i[w]);
    sh.xf[e & 1][0] = top;
    sh.xi[e & 1][0] = first;
  }
  cl::sync();
  float all = -INFINITY;
  int first = 0x7fffffff;
  for (uint32_t q = 0; q < kAsCluster; ++q) {
    const float t = cl::peek(&sh.xf[e & 1][0], q);
    const int f = cl::peek(&sh.xi[e & 1][0], q);
    if (t > all) { all = t; first = f; }          // (ranks in index order: the first of equals stays)
  }
  ++e;
  RowStat out;
  out.c = c;
  out.floor = -INFINITY;
  if (greedy) {
    out.top = all;
    out.floor = __int_as_float(first == 0x7fffffff ? -1 : first);
    out.inv = -1.f;
    if (rank == 0 && tid == 0) a.stat[row] = out;
    cl::sync();                                   // no CTA leaves while another may read its shared memory
    return;
  }
  const float mine = m;
  top = fminf(all, 3.402823466e38f);
  out.top = top;
  float mass = 0.f;
  if (!stage) {
    if (mine == -INFINITY) s = 0.f;
    else s *= ex2(fmaxf((mine - top) * c, -1e30f));
    s = warp_sum(s);
    if (lane == 0) sh.wred[warp] = s;
    __syncthreads();
    if (tid == 0) {
      float t = 0.f;
      for (int w = 0; w < kAsWarps; ++w) t += sh.wred[w];
      sh.xf[e & 1][0] = t;
    }
    cluster_sums(sh, e++, 1);
    mass = sh.tot[0];
  }
  if constexpr (kTrunc) {
    if (stage && all > -INFINITY) {
      float* hist = reinterpret_cast<float*>(dyn + ((static_cast<size_t>(S) * sizeof(T) + 15) & ~static_cast<size_t>(15)));
      // fn(l) of every staged logit of this thread
      auto each = [&](auto&& fn) {
        for (int v = 8 * tid; v < v1 - v0; v += 8 * kAsThreads) {
          if constexpr (sizeof(T) == 2) {
            const uint4 w = *reinterpret_cast<const uint4*>(xs + v);
            fn(bf16_lo(w.x)); fn(bf16_hi(w.x)); fn(bf16_lo(w.y)); fn(bf16_hi(w.y));
            fn(bf16_lo(w.z)); fn(bf16_hi(w.z)); fn(bf16_lo(w.w)); fn(bf16_hi(w.w));
          } else {
            const float4 w = *reinterpret_cast<const float4*>(xs + v), y = *reinterpret_cast<const float4*>(xs + v + 4);
            fn(w.x); fn(w.y); fn(w.z); fn(w.w);
            fn(y.x); fn(y.y); fn(y.z); fn(y.w);
          }
        }
      };
      // sums of fn's values per bin over the cluster, into sh.tot: every thread adds in a column of its own
      auto bins = [&](auto&& add) {
#pragma unroll
        for (int b = 0; b < kBins; ++b) hist[b * kAsThreads + tid] = 0.f;
        each(add);
        __syncthreads();
        for (int b = warp; b < kBins; b += kAsWarps) {
          float t = 0.f;
#pragma unroll
          for (int u = 0; u < kAsThreads / 32; ++u) t += hist[b * kAsThreads + 32 * u + lane];
          t = warp_sum(t);
          if (lane == 0) sh.xf[e & 1][b] = t;
        }
        cluster_sums(sh, e++, kBins);
      };
      // Threshold: the lowest logit whose class is needed so that tokens
      // counted (or weighed) from the top reach the target; the first pass
      // bins by powers of two of the weight, the others by five bits of the
      // ordered bits of the logits of one bin.
      float floor_ = -INFINITY;
      auto search = [&](bool weigh, float part) {
        auto value = [&](float x) { return weigh ? ex2(x) : 1.f; };
        bins([&](float l) {
          if (l >= floor_) {
            const float x = log_weight(l, top, c);
            hist[min(kBins - 1, static_cast<int>(fminf(-x, 1e6f))) * kAsThreads + tid] += value(x);
          }
        });
        float target = part;
        if (weigh) {
          float t = 0.f;
          for (int b = 0; b < kBins; ++b) t += sh.tot[b];
          target = part * t;
        }
        float above;
        const int bin = crossing(sh.tot, target, 0.f, above);
        auto inside = [&](float l) {
          return l >= floor_ && min(kBins - 1, static_cast<int>(fminf(-log_weight(l, top, c), 1e6f))) == bin;
        };
        uint32_t lo = 0xffffffffu, hi = 0;
        each([&](float l) {
          if (inside(l)) {
            const uint32_t q = order_key(l);
            lo = min(lo, q);
            hi = max(hi, q);
          }
        });
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) { sh.wred[warp] = __uint_as_float(lo); sh.wred_i[warp] = static_cast<int>(hi); }
        __syncthreads();
        if (tid == 0) {
          for (int w = 1; w < kAsWarps; ++w) {
            lo = min(lo, __float_as_uint(sh.wred[w]));
            hi = max(hi, static_cast<uint32_t>(sh.wred_i[w]));
          }
          sh.xi[e & 1][0] = static_cast<int>(lo);
          sh.xi[e & 1][1] = static_cast<int>(hi);
        }
        cl::sync();
        lo = 0xffffffffu;
        hi = 0;
        for (uint32_t q = 0; q < kAsCluster; ++q) {
          lo = min(lo, static_cast<uint32_t>(cl::peek(&sh.xi[e & 1][0], q)));
          hi = max(hi, static_cast<uint32_t>(cl::peek(&sh.xi[e & 1][1], q)));
        }
        ++e;
        // keys in [lo, hi]; bits above `bits` are the same in both
        int bits = 32 - __clz(static_cast<int>(lo ^ hi));
        float cls = sh.tot[bin];                  // (what a single class weighs, once bits is 0)
        while (bits > 0) {
          const int sh_ = max(0, bits - 5);
          const uint32_t base = bits >= 32 ? 0u : lo >> bits << bits;
          bins([&](float l) {
            const uint32_t q = order_key(l);
            if (l >= floor_ && q >= lo && q <= hi)
              hist[(kBins - 1 - static_cast<int>((q - base) >> sh_)) * kAsThreads + tid] += value(log_weight(l, top, c));
          });
          const float before = above;
          const int d = kBins - 1 - crossing(sh.tot, target, before, above);
          cls = sh.tot[kBins - 1 - d];
          const uint32_t l2 = base + (static_cast<uint32_t>(d) << sh_), h2 = l2 + ((1u << sh_) - 1u);
          lo = max(lo, l2);
          hi = min(hi, h2);
          bits = sh_;
        }
        floor_ = key_value(lo);
        mass = above + cls;
      };
      if (by_k) search(false, static_cast<float>(k));
      if (by_p) {
        search(true, nucleus);
      } else {                                    // the mass of the k highest
        float t = 0.f;
        each([&](float l) { t += l >= floor_ ? ex2(log_weight(l, top, c)) : 0.f; });
        t = warp_sum(t);
        if (lane == 0) sh.wred[warp] = t;
        __syncthreads();
        if (tid == 0) {
          t = 0.f;
          for (int w = 0; w < kAsWarps; ++w) t += sh.wred[w];
          sh.xf[e & 1][0] = t;
        }
        cluster_sums(sh, e++, 1);
        mass = sh.tot[0];
      }
      out.floor = floor_;
    }
  }
  out.inv = mass > 0.f ? 1.f / mass : 0.f;
  if (rank == 0 && tid == 0) a.stat[row] = out;
  cl::sync();                                     // no CTA leaves while another may read its shared memory
}

struct WalkArgs {
  const int32_t* parent;
  const int32_t* tok;
  const void* p;
  const float* q;
  const uint8_t* drawn;
  const int32_t* node_off;
  const float* u_node;
  const float* race;
  const RowStat* stat;
  int32_t* accept_len;
  int32_t* best_node;
  int32_t* path;
  int32_t* bonus;
  int64_t ld, ldq, ldr;
  int V, max_nodes, max_depth, total;
  bool vec_p, vec_q, vec_r;
};

struct WalkShared {
  int16_t first[TV_MAX_NODES], next[TV_MAX_NODES];   // child lists in index order
  int32_t tok[TV_MAX_NODES], kills[TV_MAX_NODES];
  float px[TV_MAX_NODES], qx[TV_MAX_NODES], u[TV_MAX_NODES];
  uint8_t flag[TV_MAX_NODES];                         // 1: drawn, 2: token removed
  float xf[2];
  int xi[2];
  float wred[kAsWarps];
  int wred_i[kAsWarps];
};

// A cluster of 8 CTAs walks one request's tree, all taking the same decisions.
template <typename T>
__global__ void __cluster_dims__(kAsCluster, 1, 1) __launch_bounds__(kAsThreads) walk_kernel(const WalkArgs a) {
  extern __shared__ uint32_t gone[];              // a bit per token of the slice: removed
  __shared__ WalkShared sh;
  griddep_wait();
  griddep_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cl::rank();
  const int r = blockIdx.x / kAsCluster;
  const int n0 = max(a.node_off[r], 0);
  const int n = max(0, min(min(a.node_off[r + 1], a.total) - n0, a.max_nodes));
  const int V = a.V, S = slice_len(V);
  const int v0 = min(V, static_cast<int>(rank) * S), v1 = min(V, v0 + S);
  const bool scribe = rank == 0 && tid == 0;
  if (rank == 0)
    for (int d = tid; d <= a.max_depth; d += kAsThreads)
      a.path[static_cast<int64_t>(r) * (a.max_depth + 1) + d] = d == 0 && n > 0 ? 0 : -1;
  if (n == 0) {                                   // (the whole cluster)
    if (scribe) { a.accept_len[r] = -1; a.best_node[r] = -1; a.bonus[r] = -1; }
    return;
  }
  const T* pl = static_cast<const T*>(a.p);
  for (int w = tid; w < (S + 31) / 32; w += kAsThreads) gone[w] = 0;
  for (int i = tid; i < n; i += kAsThreads) { sh.first[i] = -1; sh.next[i] = -1; }
  // both probabilities of every node's token at its parent
  for (int i = tid; i < n; i += kAsThreads) {
    const int par = a.parent[n0 + i], x = a.tok[n0 + i];
    float px = 0.f, qx = 0.f;
    uint8_t flag = 0;
    if (i > 0 && par >= 0 && par < i && x >= 0 && x < V) {
      const int64_t row = n0 + par;
      const RowStat s = a.stat[row];
      px = s.inv < 0.f ? 0.f : prob(one(pl + row * a.ld, x), s);
      if (a.q) qx = a.q[row * a.ldq + x];
    }
    if (a.q && (!a.drawn || a.drawn[n0 + i])) flag = 1;
    sh.px[i] = px;
    sh.qx[i] = qx;
    sh.tok[i] = x;
    sh.flag[i] = flag;
    sh.u[i] = a.u_node[n0 + i];
  }
  __syncthreads();
  if (tid == 0) {
    for (int i = n - 1; i >= 1; --i) {
      const int p = a.parent[n0 + i];
      if (p >= 0 && p < i) { sh.next[i] = sh.first[p]; sh.first[p] = static_cast<int16_t>(i); }
    }
  }
  __syncthreads();

  int cur = 0, depth = 0, e = 0, kills = 0;
  auto revive = [&]() {                           // no token is removed any more
    __syncthreads();
    for (int j = tid; j < kills; j += kAsThreads) {
      const int x = sh.kills[j];
      if (x >= v0 && x < v1) gone[(x - v0) >> 5] = 0;
    }
    kills = 0;
    __syncthreads();
  };
  for (;;) {
    const int64_t row = n0 + cur;
    const RowStat st = a.stat[row];
    const T* prow = pl + row * a.ld;
    const float* qrow = a.q ? a.q + row * a.ldq : nullptr;
    const bool greedy = st.inv < 0.f;
    // what is left of the distribution: max(0, fa p - fb q), removed tokens apart; its mass (-1: not known)
    float fa = 1.f, fb = 0.f, left = 1.f;
    // eight tokens of it
    auto rest8 = [&](int v, float (&x)[8]) {
      load8(prow, v, v1, a.vec_p, x);
      float q[8];
      if (fb > 0.f) load8(qrow, v, v1, a.vec_q, q);
      const uint32_t dead = kills ? gone[(v - v0) >> 5] >> ((v - v0) & 31) : 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = prob(x[j], st);
        if (fb > 0.f) x[j] = fmaxf(0.f, fmaf(fa, x[j], -fb * q[j]));
        if (dead & (1u << j) || v + j >= v1) x[j] = 0.f;
      }
    };
    auto reset = [&]() {
      fa = 1.f;
      fb = 0.f;
      left = 1.f;
      if (kills) revive();
      for (int i = tid; i < n; i += kAsThreads) sh.flag[i] &= 1;
      __syncthreads();
    };
    int next = -1;
    for (int ch = sh.first[cur]; ch >= 0; ch = sh.next[ch]) {
      const int x = sh.tok[ch];
      if (greedy) {
        if (x == __float_as_int(st.floor)) { next = ch; break; }
        continue;
      }
      if (left < 0.f) {                           // after a rejected draw
        float z = 0.f;
        for (int v = v0 + 8 * tid; v < v1; v += 8 * kAsThreads) {
          float y[8];
          rest8(v, y);
          z += ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
        }
        z = warp_sum(z);
        if (lane == 0) sh.wred[warp] = z;
        __syncthreads();
        if (tid == 0) {
          z = 0.f;
          for (int w = 0; w < kAsWarps; ++w) z += sh.wred[w];
          sh.xf[e & 1] = z;
        }
        cl::sync();
        left = 0.f;
        for (uint32_t c = 0; c < kAsCluster; ++c) left += cl::peek(&sh.xf[e & 1], c);
        ++e;
      }
      if (!(left > 0.f)) reset();                 // nothing left (rounding only): the target's own again
      const bool is_drawn = sh.flag[ch] & 1;
      const float have = sh.flag[ch] & 2 ? 0.f : fmaxf(0.f, fmaf(fa, sh.px[ch], -fb * sh.qx[ch]));
      if (sh.u[ch] * (is_drawn ? sh.qx[ch] : 1.f) < have / left) { next = ch; break; }
      if (is_drawn) {
        fa /= left;
        fb = fb / left + 1.f;
        left = -1.f;
      } else if (x >= 0 && x < V && !(sh.flag[ch] & 2)) {
        left -= have;
        __syncthreads();                          // (every thread has read its flags)
        if (tid == 0) {
          sh.kills[kills] = x;
          if (x >= v0 && x < v1) gone[(x - v0) >> 5] |= 1u << ((x - v0) & 31);
        }
        ++kills;
        for (int i = tid; i < n; i += kAsThreads)
          if (sh.tok[i] == x) sh.flag[i] |= 2;    // (of nodes under other parents too: cleared at the next node)
        __syncthreads();
      }
    }
    if (next >= 0) {
      cur = next;
      ++depth;
      if (scribe && depth <= a.max_depth) a.path[static_cast<int64_t>(r) * (a.max_depth + 1) + depth] = cur;
      if (kills) reset();
      continue;
    }
    int token = greedy ? __float_as_int(st.floor) : -1;
    if (!greedy) {
      const float* race = a.race + static_cast<int64_t>(r) * a.ldr;
      for (int turn = 0; turn < 2 && token < 0; ++turn) {
        if (turn == 1) reset();                   // (nothing left: the target's own)
        float best = 0.f;
        int at = 0x7fffffff;
        for (int v = v0 + 8 * tid; v < v1; v += 8 * kAsThreads) {
          float y[8], t[8];
          load8(race, v, v1, a.vec_r, t);
          rest8(v, y);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (y[j] > 0.f) {
              const float f = y[j] / t[j];
              if (f > best) { best = f; at = v + j; }
            }
          }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          const float f = __shfl_xor_sync(0xffffffffu, best, o);
          const int i = __shfl_xor_sync(0xffffffffu, at, o);
          if (better(f, i, best, at)) { best = f; at = i; }
        }
        if (lane == 0) { sh.wred[warp] = best; sh.wred_i[warp] = at; }
        __syncthreads();
        if (tid == 0) {
          for (int w = 1; w < kAsWarps; ++w)
            if (better(sh.wred[w], sh.wred_i[w], best, at)) { best = sh.wred[w]; at = sh.wred_i[w]; }
          sh.xf[e & 1] = best;
          sh.xi[e & 1] = at;
        }
        cl::sync();
        best = 0.f;
        for (uint32_t c = 0; c < kAsCluster; ++c) {
          const float f = cl::peek(&sh.xf[e & 1], c);
          const int i = cl::peek(&sh.xi[e & 1], c);
          if (f > best) { best = f; token = i; }  // (ranks in token order: the first of equals stays)
        }
        ++e;
      }
    }
    if (scribe) {
      a.accept_len[r] = depth;
      a.best_node[r] = cur;
      a.bonus[r] = token;
    }
    cl::sync();                                   // no CTA leaves while another may read its shared memory
    return;
  }
}

template <typename T>
int run(const RowArgs& ra, const WalkArgs& wa, int B, cudaStream_t st) {
  const bool trunc = ra.top_k || ra.top_p;
  const int S = ((ra.V + kAsCluster - 1) / kAsCluster + 7) / 8 * 8;
  const dim3 rows(static_cast<unsigned>(kAsCluster) * ra.max_nodes, B);
  int rc;
  if (trunc) {
    const size_t smem = ((static_cast<size_t>(S) * sizeof(T) + 15) & ~static_cast<size_t>(15)) + kBins * kAsThreads * 4;
    if (smem > 220 << 10) return TV_EUNSUPPORTED;
    if (!smem_limit(row_kernel<T, true>, 220 << 10)) return TV_ECUDA;
    rc = launch_pdl(row_kernel<T, true>, rows, dim3(kAsThreads), smem, st, ra);
  } else {
    rc = launch_pdl(row_kernel<T, false>, rows, dim3(kAsThreads), 0, st, ra);
  }
  if (rc != TV_OK) return rc;
  return launch_pdl(walk_kernel<T>, dim3(static_cast<unsigned>(kAsCluster) * B), dim3(kAsThreads),
                    static_cast<size_t>(S + 31) / 32 * 4, st, wa);
}

}  // namespace
}  // namespace tv

using namespace tv;

TV_API size_t accept_sampled_workspace_size(int B, int total_nodes, int V) {
  if (B <= 0 || total_nodes <= 0 || V <= 0) return 0;
  return static_cast<size_t>(total_nodes) * sizeof(RowStat);
}

TV_API int accept_sampled(const int32_t* parent, const int32_t* tok, const void* p_logits, int dtype, int V, int64_t ld,
                          const float* q_prob, int64_t ldq, const uint8_t* drawn, const int32_t* node_off, int B,
                          int max_nodes, int total_nodes, int max_depth, const float* temperature, const int32_t* top_k,
                          const float* top_p, const float* u_node, const float* race, int64_t ldr, int32_t* accept_len,
                          int32_t* best_node, int32_t* path, int32_t* bonus, void* ws, size_t ws_bytes,
                          tv_stream_t stream) {
  if (dtype != TV_F32 && dtype != TV_BF16) return TV_EINVAL;
  if (B < 0 || max_nodes < 0 || total_nodes < 0 || max_depth < 0 || V <= 0 || ld < V || ldr < V) return TV_EINVAL;
  if (q_prob && ldq < V) return TV_EINVAL;
  if (drawn && !q_prob) return TV_EINVAL;
  if (max_nodes > TV_MAX_NODES || V > kAsMaxVocab || B > 65535) return TV_EUNSUPPORTED;
  if (B == 0) return TV_OK;
  if (!node_off || !accept_len || !best_node || !path || !bonus) return TV_EINVAL;
  if (total_nodes > 0 && max_nodes > 0) {
    if (!parent || !tok || !p_logits || !u_node || !race) return TV_EINVAL;
    if (!ws || ws_bytes < accept_sampled_workspace_size(B, total_nodes, V) || !aligned(ws, 16)) return TV_EWORKSPACE;
  }
  const bool bf = dtype == TV_BF16;
  const bool vec_p = aligned(p_logits, 16) && ld % (bf ? 8 : 4) == 0;
  const bool vec_q = aligned(q_prob, 16) && ldq % 4 == 0, vec_r = aligned(race, 16) && ldr % 4 == 0;
  const RowArgs ra{p_logits, node_off, temperature, top_k, top_p, static_cast<RowStat*>(ws), ld, V,
                   std::max(max_nodes, 1), total_nodes, vec_p};
  const WalkArgs wa{parent, tok, p_logits, q_prob, drawn, node_off, u_node, race, static_cast<const RowStat*>(ws),
                    accept_len, best_node, path, bonus, ld, ldq, ldr, V, max_nodes, max_depth, total_nodes, vec_p, vec_q,
                    vec_r};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return bf ? run<uint16_t>(ra, wa, B, st) : run<float>(ra, wa, B, st);
}
