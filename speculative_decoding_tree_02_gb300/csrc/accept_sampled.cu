// accept_sampled: verification of drafted tokens against the target's
// probabilities (temperature, top-k and top-p of each request) from given
// random numbers; include/tv.h states the rule.
//
// Two kernels.  row_kernel takes the nodes' rows of logits side by side: a
// cluster of 8 CTAs per row finds its maximum, the truncation's threshold and
// the mass of what is kept, 16 bytes per row; rows that the walk turns out not
// to reach while others are still waiting are left out.  walk_kernel then needs
// single logits for the accept tests, and passes over a row only for what a
// rejected draw leaves and for the last token.  Rejections only ever turn the
// distribution into max(0, a p - b q) without the tokens that were removed, so
// two numbers and a bit mask stand for it and no row is written.
#include <cuda_bf16.h>

#include <algorithm>

#include "cluster.cuh"

namespace tv {
namespace {

constexpr int kAsCluster = 8;
constexpr int kAsThreads = 256;
constexpr int kAsWarps = kAsThreads / 32;
constexpr int kAsMaxVocab = 1 << 20;
constexpr int kMaxSlice = 220 << 10;   // shared memory of a CTA that stages its slice of a row
constexpr int kBins = 16;

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

// Eight consecutive logits as loaded.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> raw8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.v[i] = ldg_stream(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
__device__ __forceinline__ void widen8(const Raw8<uint16_t>& r, float (&x)[8]) {
  const uint4 w = r.v[0];
  x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z); x[5] = bf16_hi(w.z); x[6] = bf16_lo(w.w); x[7] = bf16_hi(w.w);
}
__device__ __forceinline__ void widen8(const Raw8<float>& r, float (&x)[8]) {
  const uint4 a = r.v[0], b = r.v[1];
  x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y); x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
  x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y); x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
}
// Eight consecutive numbers, whatever their alignment; -inf past the end.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int v, int end, bool vec, float (&x)[8]) {
  if (vec && v + 8 <= end) {
    widen8(raw8(row + v), x);
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
// The same as they are stored.
template <typename T>
__device__ __forceinline__ Raw8<T> tail8(const T* row, int v, int end) {
  float x[8];
  load8(row, v, end, false, x);
  Raw8<T> r;
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = (__float_as_uint(x[2 * e]) >> 16) | (__float_as_uint(x[2 * e + 1]) & 0xffff0000u);
    r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    r.v[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    r.v[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
  }
  return r;
}
// fn(v, eight) for the eights of [v0, v1) that a thread owns (v = v0 + 8 tid,
// then kThreads eights further), kAhead of them on their way at a time.
template <int kThreads, int kAhead, typename T, typename F>
__device__ __forceinline__ void sweep(const T* row, int v0, int v1, bool vec, F&& fn) {
  int v = v0 + 8 * static_cast<int>(threadIdx.x);
  if (vec) {
    for (; v + 8 <= v1; v += 8 * kThreads * kAhead) {
      Raw8<T> w[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (v + 8 * kThreads * u + 8 <= v1) w[u] = raw8(row + v + 8 * kThreads * u);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (v + 8 * kThreads * u + 8 <= v1) fn(v + 8 * kThreads * u, w[u]);
    }
    const int tail = v0 + (v1 - v0) / 8 * 8;      // a last, shorter one
    if (tail < v1 && (tail - v0) / 8 % kThreads == static_cast<int>(threadIdx.x)) fn(tail, tail8(row, tail, v1));
    return;
  }
  for (; v < v1; v += 8 * kThreads) fn(v, tail8(row, v, v1));
}
// Their maximum.
__device__ __forceinline__ float max8(const Raw8<uint16_t>& r) {
  const uint4 w = r.v[0];
  const __nv_bfloat162 m = __hmax2(__hmax2(*reinterpret_cast<const __nv_bfloat162*>(&w.x), *reinterpret_cast<const __nv_bfloat162*>(&w.y)),
                                   __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&w.z), *reinterpret_cast<const __nv_bfloat162*>(&w.w)));
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float max8(const Raw8<float>& r) {
  float x[8];
  widen8(r, x);
  return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
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
  // for leaving out rows that the walk cannot reach; dead NULL: none are
  int32_t* dead;
  const int32_t* parent;
  const int32_t* tok;
  const float* q;
  const uint8_t* drawn;
  const float* u_node;
  int64_t ldq;
};

// Mass left after a refused proposal is what was left less its probability,
// until less than this part of the last sum is: a difference of nearly equal
// numbers is off by the whole's rounding, so the remainder is then summed.
constexpr float kResum = 0.25f;

// A node's token is accepted: u q < p' for a drawn one, u < p' otherwise.
__device__ __forceinline__ bool accepted(float u, bool drawn, float q, float have, float left) {
  return u * (drawn ? q : 1.f) < have / left;
}

constexpr int kList = 256;         // listed logits of a warp
constexpr int kCompare = 1024;     // listed logits of a row that are compared with one another, at most
constexpr float kCut = 12.f;       // the first list goes down to 2^-kCut of the highest weight
constexpr int kCutPick = 4;        // or, for k up to 64 kCutPick, to a cut found among the threads' maxima
constexpr float kWorth = 8192.f;   // logits of a bin, at most, that are listed before they are told apart further
constexpr int kScratch = kBins * kAsThreads * 4;
static_assert(kScratch >= TV_MAX_NODES * 3, "see judge_children");
static_assert(kScratch / 2 == kAsWarps * kList * 4, "the lists fill the second half of the scratch");

struct RowShared {
  float xf[2][kBins];              // exchanged with the cluster, by parity
  float tot[kBins];
  float wred[kAsWarps];
  float wmax[kAsWarps], wcut[kAsWarps], wz[kAsWarps], wzl[kAsWarps];   // per warp, read by the cluster, written once
  int wfirst[kAsWarps];
  int listed[kAsWarps];            // logits that passed the list's condition, per warp
  float scan[kAsWarps];
  int hit;                         // rows that the walk cannot reach: what the first CTA saw
  float out;                       // what the first CTA found
};

// Sums over the cluster of up to kBins numbers that lie in sh.xf[e & 1] of each
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
__device__ __forceinline__ int crossing(const float* tot, int n, float target, float before, float& above) {
  int at = 0;
  float run = before;
  above = before;
  for (int b = 0; b < n; ++b) {
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

// Eight staged logits, free of NaN and +inf.
template <typename T>
__device__ __forceinline__ Raw8<T> staged8(const T* xs) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.v[i] = reinterpret_cast<const uint4*>(xs)[i];
  return r;
}
// Stages eight logits (NaN as -inf, +inf as the largest number); their maximum.
__device__ __forceinline__ float stage8(uint16_t* xs, Raw8<uint16_t> r) {
  const __nv_bfloat162 lo = __halves2bfloat162(__ushort_as_bfloat16(0xff80), __ushort_as_bfloat16(0xff80));
  const __nv_bfloat162 hi = __halves2bfloat162(__ushort_as_bfloat16(0x7f7f), __ushort_as_bfloat16(0x7f7f));
  uint32_t* w[4] = {&r.v[0].x, &r.v[0].y, &r.v[0].z, &r.v[0].w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 v = __hmin2(__hmax2(*reinterpret_cast<const __nv_bfloat162*>(w[e]), lo), hi);
    *w[e] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(xs) = r.v[0];
  return max8(r);
}
__device__ __forceinline__ float stage8(float* xs, const Raw8<float>& r) {
  float x[8], m = -INFINITY;
  widen8(r, x);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = fminf(fmaxf(x[e], -INFINITY), 3.402823466e38f);
    m = fmaxf(m, x[e]);
  }
  *reinterpret_cast<float4*>(xs) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(xs + 4) = make_float4(x[4], x[5], x[6], x[7]);
  return m;
}

// Room that a CTA needs to leave out rows: the nodes' parents, and a mark per node.
constexpr int kPruneBytes = TV_MAX_NODES * 3;

// What is certain about the children of node i, whose row's stat is known: the
// walk's own tests in its order and arithmetic, as far as they need nothing
// but single probabilities, up to the first acceptance, the first rejection that
// leaves a mass to be summed (a draw's, or one below kResum) or the 32nd child.  Rejected children and
// those behind an accepted one cannot be reached, nor can their descendants:
// all of these get a.dead = 1.  By a CTA, `room` being shared memory.
template <typename T>
__device__ __forceinline__ void judge_children(const RowArgs& a, int n0, int nodes, int i, const RowStat& st, uint8_t* room) {
  int16_t* par = reinterpret_cast<int16_t*>(room);
  uint8_t* mark = room + 2 * TV_MAX_NODES;
  const int tid = threadIdx.x, lane = tid & 31;
  __syncthreads();
  for (int j = i + 1 + tid; j < nodes; j += blockDim.x) {
    const int p = a.parent[n0 + j];
    par[j] = static_cast<int16_t>(p >= 0 && p < j ? p : -1);
    mark[j] = 0;
  }
  __syncthreads();
  if (tid < 32) {
    const T* p = static_cast<const T*>(a.p) + static_cast<int64_t>(n0 + i) * a.ld;
    int mine = -1, found = 0;                     // lane l: the l-th child
    int stop = nodes;                             // first node that was not looked at
    for (int j0 = i + 1; j0 < nodes; j0 += 32) {
      const unsigned b = __ballot_sync(0xffffffffu, j0 + lane < nodes && par[j0 + lane] == i);
      if (found + __popc(b) > 32) { stop = j0; break; }
      for (unsigned m = b; m; m &= m - 1u, ++found)
        if (lane == found) mine = j0 + __ffs(static_cast<int>(m)) - 1;
    }
    float px = 0.f, qx = 0.f, u = 0.f;
    int x = -1;
    bool drawn = false, in = false;
    if (mine >= 0) {
      x = a.tok[n0 + mine];
      in = x >= 0 && x < a.V;
      if (in && st.inv >= 0.f) px = prob(one(p, x), st);
      if (in && a.q) qx = a.q[static_cast<int64_t>(n0 + i) * a.ldq + x];
      u = a.u_node[n0 + mine];
      drawn = a.q && (!a.drawn || a.drawn[n0 + mine]);
    }
    float left = 1.f;
    unsigned dead = 0;
    for (int ch = 0; ch < found; ++ch) {
      const int xc = __shfl_sync(0xffffffffu, x, ch);
      const float pc = __shfl_sync(0xffffffffu, px, ch), qc = __shfl_sync(0xffffffffu, qx, ch),
                  uc = __shfl_sync(0xffffffffu, u, ch);
      const bool dc = __shfl_sync(0xffffffffu, drawn, ch), inc = __shfl_sync(0xffffffffu, in, ch);
      bool yes;
      if (st.inv < 0.f) {
        yes = xc >= 0 && xc == __float_as_int(st.floor);
      } else {
        // (a token that a rejected sibling had is removed)
        const bool twice = __any_sync(0xffffffffu, in && x == xc && (dead >> lane & 1u));
        const float have = twice ? 0.f : pc;
        yes = accepted(uc, dc, qc, have, left);
        if (!yes && dc) {
          dead |= 1u << ch;
          break;
        }
        if (!yes && inc && !twice) {
          left -= have;
          if (!(left >= kResum)) {
            dead |= 1u << ch;
            break;
          }
        }
      }
      if (yes) {                                  // the others behind it
        dead |= ch < 31 ? ~0u << (ch + 1) : 0u;
        for (int j = stop + lane; j < nodes; j += 32)
          if (par[j] == i) mark[j] = 1;
        break;
      }
      dead |= 1u << ch;
    }
    if (mine >= 0 && (dead >> lane & 1u)) mark[mine] = 1;
  }
  __syncthreads();
  for (int j = i + 1 + tid; j < nodes; j += blockDim.x) {
    int x = j;                                    // the child of i that j descends from, if any
    while (par[x] > i) x = par[x];
    if (par[x] == i && mark[x]) a.dead[n0 + j] = 1;
  }
}

// One row of logits: a cluster of 8 CTAs.  The slice of a CTA is staged in
// shared memory and read once from there in most calls: the highest logit is
// known by then, so one pass sums the weights and lists those above 2^-12 of
// the highest, a handful in a peaked distribution (top-k: those above a cut
// that the warps' maxima give); the first CTA compares the listed logits with
// one another, which gives each what lies above it, while the others leave.
// Where the list does not reach the threshold (flat distributions, large k)
// or overflows, the logits are binned by powers of two of the weight, the
// threshold's bin by parts of it, listed as soon as the lists hold it, until it
// is short enough to be compared; ties beyond that are told apart by four bits
// of the ordered bits at a time.  All sums have a fixed order.
// A row of 151936 bf16 logits takes a cluster 11.4 us (5.4 until the maximum is
// known, 4.0 for the list, 2 for comparing); 76 clusters run at a time.  Bound by
// these latencies: 64 chains of 16 nodes 84 us of 105.  Where the list falls short
// every level of the search is a pass, and 1000 listed logits take some 100 us to
// compare: the same chains at T = 1 take 199 us (top-p 0.95) and 636 (0.99).
template <typename T, bool kTrunc>
__global__ void __cluster_dims__(kAsCluster, 1, 1) __launch_bounds__(kAsThreads, 4) row_kernel(const RowArgs a) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ RowShared sh;
  griddep_wait();
  griddep_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cl::rank();
  const int r = blockIdx.x / kAsCluster, i = blockIdx.y;
  const int n0 = max(a.node_off[r], 0);
  const int nodes = min(min(a.node_off[r + 1], a.total) - n0, a.max_nodes);
  if (i >= nodes) return;                         // (the whole cluster)
  const int64_t row = n0 + i;
  if (a.dead && i > 0) {
    // one CTA looks, so that all do the same
    if (rank == 0 && tid == 0) sh.hit = *reinterpret_cast<volatile const int32_t*>(a.dead + row);
    cl::sync();
    const bool gone = cl::peek(&sh.hit, 0) != 0;
    cl::arrive();                                 // (the first CTA stays until all have looked)
    if (gone) {
      cl::wait();
      return;
    }
  }
  const T* p = static_cast<const T*>(a.p) + row * a.ld;
  const int V = a.V, S = slice_len(V);
  const int v0 = min(V, static_cast<int>(rank) * S), v1 = min(V, v0 + S);
  const float temp = a.temperature ? a.temperature[r] : 1.f;
  const bool greedy = !(temp > 0.f);
  const float c = fmaxf(fminf(kLog2e / temp, 1e30f), 1e-30f);
  int k = kTrunc && a.top_k ? a.top_k[r] : 0;
  if (k >= V) k = 0;
  const float nucleus = kTrunc && a.top_p ? (a.top_p[r] < 0.f ? 0.f : a.top_p[r]) : 1.f;
  const bool by_k = !greedy && k > 0, by_p = !greedy && nucleus < 1.f;
  T* xs = reinterpret_cast<T*>(dyn);              // the slice, each thread's own eighths

  // maximum (and its first place); the slice into shared memory where passes follow
  float m = -INFINITY, s = 0.f;
  int at = 0x7fffffff;
  const bool stage = by_k || by_p;
  if constexpr (kTrunc) {
    if (stage) {
      if (a.vec) {                                // all of them on their way at once
        for (int v = v0 + 8 * tid; v + 8 <= v1; v += 8 * kAsThreads) {
          const auto to = static_cast<uint32_t>(__cvta_generic_to_shared(xs + (v - v0)));
#pragma unroll
          for (int u = 0; u < static_cast<int>(sizeof(T) / 2); ++u)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 16u * u), "l"(p + v + 16 / sizeof(T) * u)
                         : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (int v = v0 + 8 * tid; v < v1; v += 8 * kAsThreads)
          m = fmaxf(m, stage8(xs + (v - v0), v + 8 <= v1 ? staged8(xs + (v - v0)) : tail8(p, v, v1)));
      } else {
        sweep<kAsThreads, 5>(p, v0, v1, false, [&](int v, const Raw8<T>& w) { m = fmaxf(m, stage8(xs + (v - v0), w)); });
      }
    }
  }
  if (!stage) sweep<kAsThreads, 5>(p, v0, v1, a.vec, [&](int v, const Raw8<T>& w) {
    float x[8], m8 = max8(w);
    widen8(w, x);
    if (greedy) {
      if (m8 > m) {
        m = m8;
#pragma unroll
        for (int e = 7; e >= 0; --e)
          if (x[e] == m8) at = v + e;
      }
      return;
    }
    if (m8 > 3.402823466e38f) m8 = 3.402823466e38f;
    if (m8 > m) {                                 // running maximum and sum
      s *= ex2(fmaxf((m - m8) * c, -1e30f));
      m = m8;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s += ex2(log_weight(x[e], m, c));
  });
  if (a.dead && i > 0) cl::wait();
  int e = 0;
  // every warp's maximum and its first place; for top-k also the j-th highest
  // of its lanes' maxima, 64 j >= k
  const int pick = (k + kAsCluster * kAsWarps - 1) / (kAsCluster * kAsWarps);
  const bool by_cut = kTrunc && by_k && pick <= kCutPick;
  {
    const float wm = warp_max(m);
    const int wi = greedy ? __reduce_min_sync(0xffffffffu, m == wm ? at : 0x7fffffff) : 0;
    if (lane == 0) { sh.wmax[warp] = wm; sh.wfirst[warp] = wi; }
    if (by_cut) {
      float x = m, y = wm;
      for (int t = 1; t < pick; ++t) {
        if (lane == __ffs(static_cast<int>(__ballot_sync(0xffffffffu, x == y))) - 1) x = -INFINITY;
        y = warp_max(x);
      }
      if (lane == 0) sh.wcut[warp] = y;
    }
  }
  // lane l: the numbers of warps l and l + 32 of the cluster's 64
  auto of64 = [&](const auto* v, auto& c0, auto& c1) {
    c0 = cl::peek(v + (lane & 7), lane >> 3);
    c1 = cl::peek(v + (lane & 7), 4 + (lane >> 3));
  };
  cl::sync();
  float all, cut = -INFINITY;
  int first = 0x7fffffff;
  {
    float c0, c1;
    of64(sh.wmax, c0, c1);
    all = warp_max(fmaxf(c0, c1));
    if (greedy) {
      int f0, f1;
      of64(sh.wfirst, f0, f1);
      first = __reduce_min_sync(0xffffffffu, min(c0 == all ? f0 : 0x7fffffff, c1 == all ? f1 : 0x7fffffff));
    }
    if (by_cut) {                                 // the highest number that enough warps reach for k logits
      of64(sh.wcut, c0, c1);
      const int warps = (k + pick - 1) / pick;
      int a0 = 0, a1 = 0;
#pragma unroll 8
      for (int t = 0; t < 32; ++t) {
        const float x = __shfl_sync(0xffffffffu, c0, t), y = __shfl_sync(0xffffffffu, c1, t);
        a0 += (x > c0 ? 1 : 0) + (y > c0 ? 1 : 0);
        a1 += (x > c1 ? 1 : 0) + (y > c1 ? 1 : 0);
      }
      cut = -warp_max(fmaxf(a0 < warps ? -c0 : -INFINITY, a1 < warps ? -c1 : -INFINITY));
    }
  }
  // by the first CTA: the row is done
  auto publish = [&](const RowStat& st) {
    if (tid == 0) a.stat[row] = st;
    if (a.dead) judge_children<T>(a, n0, nodes, i, st, dyn);    // (no pass over the slice follows)
  };
  RowStat out;
  out.c = c;
  out.floor = -INFINITY;
  if (greedy) {
    out.top = all;
    out.floor = __int_as_float(first == 0x7fffffff ? -1 : first);
    out.inv = -1.f;
    if (rank == 0) publish(out);
    cl::sync();                                   // no CTA leaves while another may read its shared memory
    return;
  }
  const float top = fminf(all, 3.402823466e38f);
  out.top = top;
  float mass = 0.f;
  // sum of a number per thread over the cluster
  auto total = [&](float x) {
    x = warp_sum(x);
    if (lane == 0) sh.wred[warp] = x;
    __syncthreads();
    if (tid == 0) {
      x = 0.f;
      for (int w = 0; w < kAsWarps; ++w) x += sh.wred[w];
      sh.xf[e & 1][0] = x;
    }
    cluster_sums(sh, e++, 1);
    return sh.tot[0];
  };
  if (!stage) {
    if (m == -INFINITY) s = 0.f;
    else s *= ex2(fmaxf((m - top) * c, -1e30f));
    mass = total(s);
  }
  if constexpr (kTrunc) {
    if (stage && all > -INFINITY) {
      float* hist = reinterpret_cast<float*>(dyn + ((static_cast<size_t>(S) * sizeof(T) + 15) & ~static_cast<size_t>(15)));
      float* list = hist + kScratch / 8;          // second half: a run for each warp
      const int n = v1 - v0, rounds = (n + 8 * kAsThreads - 1) / (8 * kAsThreads);
      auto weight = [&](float l) { return ex2((l - top) * c); };
      // fn(l) of every staged logit of this thread
      auto each = [&](auto&& fn) {
        for (int v = 8 * tid; v < n; v += 8 * kAsThreads) {
          float x[8];
          widen8(staged8(xs + v), x);
#pragma unroll
          for (int j = 0; j < 8; ++j) fn(x[j]);
        }
      };
      // Lists the logits in [lo, hi], warp by warp, in a fixed order; adds
      // the weights of all logits to z and of the listed ones to zl, if asked.
      auto make_list = [&](float lo, float hi, bool sum, float& z, float& zl) {
        int cnt = 0;
        for (int q = 0; q < rounds; ++q) {
          const int v = 8 * (q * kAsThreads + tid);
          Raw8<T> raw{};
          float x[8], m8 = -INFINITY;
          if (v < n) {
            raw = staged8(xs + v);
            m8 = max8(raw);
            if (sum) {
              float y[8];
              widen8(raw, x);
#pragma unroll
              for (int j = 0; j < 8; ++j) y[j] = weight(x[j]);
              z += ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
            }
          }
          if (!__any_sync(0xffffffffu, m8 >= lo) || cnt > kList) continue;
          uint32_t in = 0;
          if (v < n && m8 >= lo) {                // (lo may be -inf, as m8 is behind the slice)
            widen8(raw, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) in |= (x[j] >= lo && x[j] <= hi ? 1u : 0u) << j;
          }
          for (unsigned lanes = __ballot_sync(0xffffffffu, in != 0u); lanes; lanes &= lanes - 1u) {
            const int src = __ffs(static_cast<int>(lanes)) - 1;
            const int more = __popc(__shfl_sync(0xffffffffu, in, src));
            if (lane == src) {
              int to = cnt;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (in >> j & 1u) {
                  if (to < kList) list[warp * kList + to] = x[j];
                  ++to;
                  if (sum) zl += weight(x[j]);
                }
            }
            cnt += more;
          }
        }
        if (lane == 0) sh.listed[warp] = cnt;
      };
      // After a cluster barrier: logits on the cluster's lists, -1 when one overflowed, -2 when they are too many to compare.
      int c0, c1;                                 // lane l: the counts of segments l and l + 32 of the 64
      auto usable = [&]() {
        of64(sh.listed, c0, c1);
        const bool over = __any_sync(0xffffffffu, c0 > kList || c1 > kList);
        const int sum = __reduce_add_sync(0xffffffffu, min(c0, kList) + min(c1, kList));
        return over ? -1 : sum > kCompare ? -2 : sum;
      };
      // The first CTA copies the lists of all to the start of its scratch: warp w the segments of CTA w.
      auto copy = [&]() {
        int at[8], end = 0;
        const int before = __reduce_add_sync(0xffffffffu, ((lane >> 3) < warp ? c0 : 0) + (4 + (lane >> 3) < warp ? c1 : 0));
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          at[q] = end;
          end += __shfl_sync(0xffffffffu, warp < 4 ? c0 : c1, 8 * (warp & 3) + q);
        }
        for (int t = lane; t < end; t += 32) {
          int q = 0, o = 0;
#pragma unroll
          for (int u = 1; u < 8; ++u)
            if (t >= at[u]) { q = u; o = at[u]; }
          hist[before + t] = cl::peek(&list[q * kList + t - o], warp);
        }
      };
      // Sum over the CTA, by all of its threads.
      auto cta_sum = [&](float x) {
        x = warp_sum(x);
        __syncthreads();
        if (lane == 0) sh.wred[warp] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int w = 0; w < kAsWarps; ++w) x += sh.wred[w];
        return x;
      };
      // Of the copied list: how many logits are higher than each and what these
      // weigh, which tells what top-k (of `left` tokens; 0: off) and top-p (up to
      // the mass `target`, or its share of z; below 0: off) keep, whole classes as
      // equals get equal numbers.  Sets out.floor and mass, `above` included.
      auto settle = [&](int cnt, int left, float above, float target, float share) {
        constexpr int kOwn = kCompare / kAsThreads;
        float* ws = hist + kCompare;                 // weights
        const int pad = (cnt + 31) / 32 * 32;
        for (int q = tid; q < pad; q += kAsThreads) {
          if (q >= cnt) hist[q] = -INFINITY;
          ws[q] = q < cnt ? weight(hist[q]) : 0.f;
        }
        __syncthreads();
        float own[kOwn], mine[kOwn];
        bool keep[kOwn];
        float z = 0.f, low = INFINITY;
#pragma unroll
        for (int u = 0; u < kOwn; ++u) {
          const int q = tid + u * kAsThreads;
          own[u] = q < cnt ? hist[q] : INFINITY;
          mine[u] = 0.f;
          int more = 0;
          if (u * kAsThreads + 32 * warp < cnt) { // (for the warp as a whole)
            // (sums of 32 at a time: one sum of all would lose the small weights behind a large one)
            for (int j0 = 0; j0 < pad; j0 += 32) {
              float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 l = *reinterpret_cast<const float4*>(hist + j0 + j), w = *reinterpret_cast<const float4*>(ws + j0 + j);
                if (l.x > own[u]) { ++more; part[0] += w.x; }
                if (l.y > own[u]) { ++more; part[1] += w.y; }
                if (l.z > own[u]) { ++more; part[2] += w.z; }
                if (l.w > own[u]) { ++more; part[3] += w.w; }
              }
              mine[u] += (part[0] + part[1]) + (part[2] + part[3]);
            }
          }
          keep[u] = q < cnt && (left == 0 || more < left);
          if (keep[u]) { z += ws[q]; low = fminf(low, own[u]); }
        }
        if (left > 0) z = cta_sum(z);
        if (share >= 0.f) target = share * z;
        if (target >= 0.f) {
          z = 0.f;
          low = INFINITY;
#pragma unroll
          for (int u = 0; u < kOwn; ++u) {
            keep[u] = keep[u] && (above + mine[u] < target || mine[u] == 0.f);      // (the highest class always)
            if (keep[u]) { z += ws[tid + u * kAsThreads]; low = fminf(low, own[u]); }
          }
          z = cta_sum(z);
        }
        mass = above + z;
        low = -warp_max(-low);
        if (lane == 0) sh.scan[warp] = low;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kAsWarps; ++w) low = fminf(low, sh.scan[w]);
        out.floor = low;
      };
      // The lists hold every logit that matters: the first CTA finds the
      // threshold, the others are done.
      auto finish = [&](int cnt, float z) {
        if (rank == 0) copy();
        cl::sync();
        if (rank != 0) return;
        settle(cnt, by_k ? k : 0, 0.f, by_p && !by_k ? nucleus * z : -1.f, by_p && by_k ? nucleus : -1.f);
        out.inv = mass > 0.f ? 1.f / mass : 0.f;
        publish(out);
      };

      // ---- the highest, listed while all are summed
      // (all of them, if the list has room for a whole row)
      float z = 0.f, zl = 0.f;
      const float lowest = -3.402823466e38f;
      make_list(V <= kCompare ? lowest : fmaxf(by_cut ? cut : top - kCut / c, lowest), INFINITY, !by_k, z, zl);
      z = warp_sum(z);
      zl = warp_sum(zl);
      if (lane == 0) { sh.wz[warp] = z; sh.wzl[warp] = zl; }
      cl::sync();
      if (!by_k) {
        float x, y;
        of64(sh.wz, x, y);
        z = warp_sum(x + y);
        of64(sh.wzl, x, y);
        zl = warp_sum(x + y);
      }
      int cnt = usable();
      if (cnt > 0 && (by_k ? k <= cnt : zl >= nucleus * z)) {
        finish(cnt, z);
        return;
      }

      // ---- bins of y = (top - l) c, then of a part of them
      // sums of values per bin over the cluster, into sh.tot: every thread adds in a column of its own
      auto sum_bins = [&](int nb) {
        __syncthreads();
        for (int b = warp; b < nb; b += kAsWarps) {
          float t = 0.f;
#pragma unroll
          for (int u = 0; u < kAsThreads / 32; ++u) t += hist[b * kAsThreads + 32 * u + lane];
          t = warp_sum(t);
          if (lane == 0) sh.xf[e & 1][b] = t;
        }
        cluster_sums(sh, e++, nb);
      };
      auto bins = [&](int nb, auto&& add) {
        for (int b = 0; b < nb; ++b) hist[b * kAsThreads + tid] = 0.f;
        each(add);
        sum_bins(nb);
      };
      float floor_ = -INFINITY;                   // what top-k leaves
      // The lowest logit that is needed for the tokens counted (or weighed)
      // from the top to reach the target; bins from y0 on, 1 / inv wide.  true: this CTA has nothing left to do.
      auto search = [&](bool weigh, float part, float y0, float inv) {
        float lo = floor_, hi = INFINITY, above = 0.f, target = part;
        bool listed = false;                      // the lists hold all of [lo, hi]
        for (int level = 0; level < 5; ++level) {
          const int nb = listed ? kBins / 2 : kBins;    // (the lists keep their half of the scratch)
          auto bin_of = [&](float l) { return static_cast<int>(fminf(fmaxf(((top - l) * c - y0) * inv, 0.f), nb - 1.f)); };
          if (listed) {
            for (int b = 0; b < nb; ++b) hist[b * kAsThreads + tid] = 0.f;
            for (int q = lane; q < sh.listed[warp]; q += 32) {
              const float l = list[warp * kList + q];
              hist[bin_of(l) * kAsThreads + tid] += weigh ? weight(l) : 1.f;
            }
            sum_bins(nb);
          } else if (weigh) {
            bins(nb, [&](float l) {
              if (l >= lo && l <= hi) hist[bin_of(l) * kAsThreads + tid] += weight(l);
            });
          } else {
            bins(nb, [&](float l) {
              if (l >= lo && l <= hi) hist[bin_of(l) * kAsThreads + tid] += 1.f;
            });
          }
          if (weigh && level == 0) {
            float t = 0.f;
            for (int b = 0; b < nb; ++b) t += sh.tot[b];
            target = part * t;
          }
          const int bin = crossing(sh.tot, nb, target, above, above);
          // at most so many logits in the bin, and down to it
          float most = 0.f, whole = 0.f;
          for (int b = 0; b <= bin; ++b) {
            most = weigh ? sh.tot[b] * exp2f(y0 + (b + 1) / inv) : sh.tot[b];
            whole += most;
          }
          // the bin's lowest and highest number, by bisection of the ordered bits
          if (warp == 0) {
            const bool low = lane == 0;
            uint32_t k0 = order_key(-3.402823466e38f), k1 = order_key(top);
            while (k0 < k1) {
              const uint32_t mid = k0 + (k1 - k0 + (low ? 0u : 1u)) / 2u;
              const int b = bin_of(key_value(mid));
              if (low) {
                if (b <= bin) k1 = mid;
                else k0 = mid + 1u;
              } else {
                if (b >= bin) k0 = mid;
                else k1 = mid - 1u;
              }
            }
            if (lane == 0) sh.scan[0] = bin == nb - 1 && level == 0 ? -INFINITY : key_value(k0);
            if (lane == 1) sh.scan[1] = bin == 0 && level == 0 ? INFINITY : key_value(k0);
          }
          __syncthreads();
          lo = fmaxf(lo, sh.scan[0]);
          hi = fminf(hi, sh.scan[1]);
          __syncthreads();
          // top-k whose few logits are worth listing as a whole: top-p then needs no search of its own
          if (level == 0 && !weigh && whole <= kCompare && bin < nb - 1) {
            float u0, u1;
            make_list(lo, INFINITY, false, u0, u1);
            cl::sync();
            cnt = usable();
            if (cnt > 0) {
              finish(cnt, 0.f);
              return true;
            }
          } else if (listed) {                    // what of the lists is in the bin
            int kept = 0;
            const int had = sh.listed[warp];
            for (int q = 0; q < had; q += 32) {
              const float l = q + lane < had ? list[warp * kList + q + lane] : NAN;
              const bool in = l >= lo && l <= hi;
              const unsigned m = __ballot_sync(0xffffffffu, in);
              if (in) list[warp * kList + kept + __popc(m & ((1u << lane) - 1u))] = l;
              kept += __popc(m);
              __syncwarp();
            }
            if (lane == 0) sh.listed[warp] = kept;
            cl::sync();
            cnt = usable();
          } else if (most <= kWorth) {
            float u0, u1;
            make_list(lo, hi, false, u0, u1);
            cl::sync();
            cnt = usable();
            listed = cnt != -1;
          } else {
            cnt = -1;
          }
          if (listed && cnt > 0) {
            if (rank == 0) copy();
            cl::sync();                           // (this and the next: sh.out is written between two barriers)
            if (rank == 0) {
              if (weigh) {
                settle(cnt, 0, above, target, -1.f);
                out.inv = mass > 0.f ? 1.f / mass : 0.f;
                publish(out);
              } else {
                settle(cnt, max(1, static_cast<int>(target - above)), 0.f, -1.f, -1.f);
                if (tid == 0) sh.out = out.floor;
              }
            }
            if (weigh) return true;
            cl::sync();
            floor_ = cl::peek(&sh.out, 0);
            return false;
          }
          y0 += bin / inv;
          inv *= listed ? kBins / 2 : kBins;
        }
        // flat to the last: by four bits of the ordered bits; keys in [klo, khi], those above `bits` the same in both
        uint32_t klo = order_key(lo), khi = order_key(fminf(hi, top));
        int bits = 32 - __clz(static_cast<int>(klo ^ khi));
        float cls = 0.f;
        do {
          const int low = max(0, bits - 4);
          const uint32_t base = bits >= 32 ? 0u : klo >> bits << bits;
          bins(16, [&](float l) {
            const uint32_t q = order_key(l);
            if (q >= klo && q <= khi)
              hist[(15 - static_cast<int>((q - base) >> low)) * kAsThreads + tid] += weigh ? weight(l) : 1.f;
          });
          const int d = 15 - crossing(sh.tot, 16, target, above, above);
          cls = sh.tot[15 - d];
          const uint32_t l2 = base + (static_cast<uint32_t>(d) << low), h2 = l2 + ((1u << low) - 1u);
          klo = max(klo, l2);
          khi = min(khi, h2);
          bits = low;
        } while (bits > 0);
        floor_ = key_value(klo);
        mass = above + cls;
        return false;
      };
      const bool below = !by_k && cnt > 0;         // the list was complete, the threshold lies below it
      if (by_k && search(false, static_cast<float>(k), 0.f, 1.f)) return;
      if (by_p) {
        if (search(true, nucleus, below ? kCut : 0.f, below ? 2.f : 1.f)) return;
      } else {                                    // the mass of the k highest
        float t = 0.f;
        each([&](float l) { t += l >= floor_ ? weight(l) : 0.f; });
        mass = total(t);
      }
      out.floor = floor_;
    }
  }
  out.inv = mass > 0.f ? 1.f / mass : 0.f;
  if (rank == 0) publish(out);
  cl::sync();                                     // no CTA leaves while another may read its shared memory
}

constexpr int kWalkThreads = 256;
constexpr int kWalkWarps = kWalkThreads / 32;

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
  int16_t par[TV_MAX_NODES];                          // -1: none, or not before the node
  int32_t tok[TV_MAX_NODES], kills[TV_MAX_NODES];
  float px[TV_MAX_NODES], qx[TV_MAX_NODES], u[TV_MAX_NODES];
  uint8_t flag[TV_MAX_NODES];                         // 1: drawn, 2: token removed
  float xf[2];
  int xi[2];
  float wred[kWalkWarps];
  int wred_i[kWalkWarps];
};

// A cluster of 8 CTAs walks one request's tree, all taking the same decisions.
// Latency bound: 9 us (2 for both probabilities of all nodes, 4..5 for the pass for
// the last token, 2 for its maximum over the cluster), 20 us for 64 requests. Four
// CTAs to an SM hold it at 64 registers; 312 bytes of a thread are spilled in bf16, 536 in fp32.
template <typename T>
__global__ void __cluster_dims__(kAsCluster, 1, 1) __launch_bounds__(kWalkThreads, 4) walk_kernel(const WalkArgs a) {
  extern __shared__ __align__(16) RowStat stats[];    // the nodes' rows
  uint32_t* gone = reinterpret_cast<uint32_t*>(stats + a.max_nodes);   // a bit per token of the slice: removed
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
    for (int d = tid; d <= a.max_depth; d += kWalkThreads)
      a.path[static_cast<int64_t>(r) * (a.max_depth + 1) + d] = d == 0 && n > 0 ? 0 : -1;
  if (n == 0) {                                   // (the whole cluster)
    if (scribe) { a.accept_len[r] = -1; a.best_node[r] = -1; a.bonus[r] = -1; }
    return;
  }
  const T* pl = static_cast<const T*>(a.p);
  for (int w = tid; w < (S + 31) / 32; w += kWalkThreads) gone[w] = 0;
  // both probabilities of every node's token at its parent
  for (int i = tid; i < n; i += kWalkThreads) {
    const int par = a.parent[n0 + i], x = a.tok[n0 + i];
    float px = 0.f, qx = 0.f;
    uint8_t flag = 0;
    stats[i] = a.stat[n0 + i];
    if (i > 0 && par >= 0 && par < i && x >= 0 && x < V) {
      const int64_t row = n0 + par;
      const float l = one(pl + row * a.ld, x);
      if (a.q) qx = a.q[row * a.ldq + x];
      const RowStat s = a.stat[row];
      px = s.inv < 0.f ? 0.f : prob(l, s);
    }
    if (a.q && (!a.drawn || a.drawn[n0 + i])) flag = 1;
    sh.par[i] = static_cast<int16_t>(i > 0 && par >= 0 && par < i ? par : -1);
    sh.px[i] = px;
    sh.qx[i] = qx;
    sh.tok[i] = x;
    sh.flag[i] = flag;
    sh.u[i] = a.u_node[n0 + i];
  }
  __syncthreads();
  // the first child of node c from index j on, -1: none
  auto child = [&](int c, int j) {
    for (; j < n; j += 32) {
      const unsigned b = __ballot_sync(0xffffffffu, j + lane < n && sh.par[j + lane] == c);
      if (b) return j + __ffs(static_cast<int>(b)) - 1;
    }
    return -1;
  };

  int cur = 0, depth = 0, e = 0, kills = 0;
  auto revive = [&]() {                           // no token is removed any more
    __syncthreads();
    for (int j = tid; j < kills; j += kWalkThreads) {
      const int x = sh.kills[j];
      if (x >= v0 && x < v1) gone[(x - v0) >> 5] = 0;
    }
    kills = 0;
    __syncthreads();
  };
  for (;;) {
    const int64_t row = n0 + cur;
    const RowStat st = stats[cur];
    const T* prow = pl + row * a.ld;
    const float* qrow = a.q ? a.q + row * a.ldq : nullptr;
    const bool greedy = st.inv < 0.f;
    // what is left of the distribution: max(0, fa p - fb q), removed tokens apart; its mass (-1: not known), and the
    // least that a difference may leave of it
    float fa = 1.f, fb = 0.f, left = 1.f, least = kResum;
    // what is left at eight tokens from v on, w their logits
    auto rest8 = [&](int v, const Raw8<T>& w, float (&y)[8]) {
      float q[8], x[8];
      widen8(w, x);
      if (fb > 0.f) load8(qrow, v, v1, a.vec_q, q);
      const uint32_t dead = kills ? gone[(v - v0) >> 5] >> ((v - v0) & 31) : 0u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = prob(x[j], st);
        if (fb > 0.f) y[j] = fmaxf(0.f, fmaf(fa, y[j], -fb * q[j]));
        if (dead & (1u << j) || v + j >= v1) y[j] = 0.f;
      }
    };
    auto reset = [&]() {
      fa = 1.f;
      fb = 0.f;
      left = 1.f;
      least = kResum;
      if (kills) revive();
      for (int i = tid; i < n; i += kWalkThreads) sh.flag[i] &= 1;
      __syncthreads();
    };
    int next = -1;
    for (int ch = child(cur, cur + 1); ch >= 0; ch = child(cur, ch + 1)) {
      const int x = sh.tok[ch];
      if (greedy) {
        if (x >= 0 && x == __float_as_int(st.floor)) { next = ch; break; }
        continue;
      }
      if (left < 0.f) {                           // after a rejected draw, or with little left
        float z = 0.f;
        sweep<kWalkThreads, 3>(prow, v0, v1, a.vec_p, [&](int v, const Raw8<T>& w) {
          if (!(max8(w) >= st.floor)) return;     // (none of them is kept)
          float y[8];
          rest8(v, w, y);
          z += ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
        });
        z = warp_sum(z);
        if (lane == 0) sh.wred[warp] = z;
        __syncthreads();
        if (tid == 0) {
          z = 0.f;
          for (int w = 0; w < kWalkWarps; ++w) z += sh.wred[w];
          sh.xf[e & 1] = z;
        }
        cl::sync();
        left = 0.f;
        for (uint32_t c = 0; c < kAsCluster; ++c) left += cl::peek(&sh.xf[e & 1], c);
        ++e;
        least = kResum * left;
      }
      if (!(left > 0.f)) reset();                 // nothing left (rounding only): the target's own again
      const bool is_drawn = sh.flag[ch] & 1;
      const float have = sh.flag[ch] & 2 ? 0.f : fb > 0.f ? fmaxf(0.f, fmaf(fa, sh.px[ch], -fb * sh.qx[ch])) : fa * sh.px[ch];
      if (accepted(sh.u[ch], is_drawn, sh.qx[ch], have, left)) { next = ch; break; }
      if (is_drawn) {
        fa /= left;
        fb = fb / left + 1.f;
        left = -1.f;
      } else if (x >= 0 && x < V && !(sh.flag[ch] & 2)) {
        left -= have;
        if (!(left >= least)) left = -1.f;
        __syncthreads();                          // (every thread has read its flags)
        if (tid == 0) {
          sh.kills[kills] = x;
          if (x >= v0 && x < v1) gone[(x - v0) >> 5] |= 1u << ((x - v0) & 31);
        }
        ++kills;
        for (int i = tid; i < n; i += kWalkThreads)
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
        sweep<kWalkThreads, 3>(prow, v0, v1, a.vec_p, [&](int v, const Raw8<T>& w) {
          if (!(max8(w) >= st.floor)) return;     // (none of them is kept)
          float y[8], t[8];
          load8(race, v, v1, a.vec_r, t);
          rest8(v, w, y);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (y[j] > 0.f) {
              const float f = y[j] / t[j];
              if (f > best) { best = f; at = v + j; }
            }
          }
        });
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          const float f = __shfl_xor_sync(0xffffffffu, best, o);
          const int i = __shfl_xor_sync(0xffffffffu, at, o);
          if (better(f, i, best, at)) { best = f; at = i; }
        }
        if (lane == 0) { sh.wred[warp] = best; sh.wred_i[warp] = at; }
        __syncthreads();
        if (tid == 0) {
          for (int w = 1; w < kWalkWarps; ++w)
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
  // nodes in the order of their index, the requests' side by side: a row's
  // descendants come late enough to be left out when it ends the walk
  const dim3 rows(static_cast<unsigned>(kAsCluster) * B, ra.max_nodes);
  const bool some = ra.max_nodes > 0 && ra.total > 0;     // (else no array but the offsets and outputs is there)
  const size_t row_smem =
      trunc ? ((static_cast<size_t>(S) * sizeof(T) + 15) & ~static_cast<size_t>(15)) + kScratch : kPruneBytes;
  if (row_smem > kMaxSlice) return TV_EUNSUPPORTED;
  if (trunc && !smem_limit(row_kernel<T, true>, kMaxSlice)) return TV_ECUDA;
  if (ra.dead && cudaMemsetAsync(ra.dead, 0, static_cast<size_t>(ra.total) * 4, st) != cudaSuccess) {
    cudaGetLastError();
    return TV_ECUDA;
  }
  const int rc = !some   ? TV_OK
                 : trunc ? launch_pdl(row_kernel<T, true>, rows, dim3(kAsThreads), row_smem, st, ra)
                         : launch_pdl(row_kernel<T, false>, rows, dim3(kAsThreads), row_smem, st, ra);
  if (rc != TV_OK) return rc;
  const size_t smem = static_cast<size_t>(wa.max_nodes) * sizeof(RowStat) + static_cast<size_t>(S + 31) / 32 * 4;
  if (smem > 20 << 10 && !smem_limit(walk_kernel<T>, 40 << 10)) return TV_ECUDA;
  return launch_pdl(walk_kernel<T>, dim3(static_cast<unsigned>(kAsCluster) * B), dim3(kWalkThreads), smem, st, wa);
}

}  // namespace
}  // namespace tv

using namespace tv;

TV_API size_t accept_sampled_workspace_size(int B, int total_nodes, int V) {
  if (B <= 0 || total_nodes <= 0 || V <= 0) return 0;
  return static_cast<size_t>(total_nodes) * (sizeof(RowStat) + 4);
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
  // Rows that cannot be reached are left out where there are more than twice
  // what runs at a time (four CTAs to an SM).
  const bool prune = static_cast<int64_t>(B) * max_nodes * kAsCluster > 8ll * sm_count() && total_nodes > 0;
  auto* stat = static_cast<RowStat*>(ws);
  const RowArgs ra{p_logits, node_off, temperature, top_k, top_p, stat, ld, V, max_nodes, total_nodes, vec_p,
                   prune ? reinterpret_cast<int32_t*>(stat + total_nodes) : nullptr, parent, tok, q_prob, drawn, u_node,
                   ldq};
  const WalkArgs wa{parent, tok, p_logits, q_prob, drawn, node_off, u_node, race, static_cast<const RowStat*>(ws),
                    accept_len, best_node, path, bonus, ld, ldq, ldr, V, max_nodes, max_depth, total_nodes, vec_p, vec_q,
                    vec_r};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return bf ? run<uint16_t>(ra, wa, B, st) : run<float>(ra, wa, B, st);
}
