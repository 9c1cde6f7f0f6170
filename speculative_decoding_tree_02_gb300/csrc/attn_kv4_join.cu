// tree_verify_attn_kv4: what the two tensor-core kernels share on the side —
// the extents of row tiles whose keys do not follow from the lengths alone,
// the joining of units that were cut, and the report of an expired wait.
#include <cstdlib>

#include "kv4_device.cuh"

namespace tv {
namespace kv4 {
namespace {

// One warp per entry (request x row tile of nq nodes), lanes = nodes.
__global__ void __launch_bounds__(128) extent_kernel(const AttnArgs a, int nq, int tiles, int4* out) {
  griddep_wait();
  griddep_release();
  const int e = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (e >= a.B * tiles) return;
  const int r = e / tiles, first = e % tiles * nq;
  const Span s = node_span(a, r);
  const int len = prefix_len(a, r), last = min(first + nq, s.cnt);
  int vis = 0, lo = 1 << 30, hi = -1;           // 64-node words of the masks that are not empty
  for (int i = first + lane; i < last; i += 32) {
    vis = max(vis, a.vis_prefix ? min(max(a.vis_prefix[s.n0 + i], 0), len) : len);
    const uint64_t* row = a.anc + static_cast<int64_t>(s.n0 + i) * a.anc_words;
    for (int w0 = 0; w0 < a.anc_words; w0 += 8) {
      uint64_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = w0 + k < a.anc_words ? row[w0 + k] : 0ull;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (v[k]) {
          lo = min(lo, w0 + k);
          hi = max(hi, w0 + k);
        }
    }
  }
  vis = __reduce_max_sync(0xffffffffu, vis);
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  const bool live = first < s.cnt;
  // at least one tile for a live entry: its rows are written even if they see nothing
  const int top = live ? (s.cnt - 1) / kTreeTile : 0;
  const int t0 = min(lo / (kTreeTile / 64), top);
  const int nt = live ? max(0, min(hi / (kTreeTile / 64), top) - t0) + 1 : 0;
  if (lane == 0) out[e] = make_int4(live ? vis : 0, t0, nt, 0);
}

// A wait ran out: units are missing, so every row of the call reports it, not what the memory held.
template <int D>
__device__ __noinline__ void fail_rows(const AttnArgs& a) {
  const int ctas = static_cast<int>(gridDim.x * gridDim.y), cta = static_cast<int>(blockIdx.y * gridDim.x + blockIdx.x);
  if (cta == 0 && threadIdx.x == 0 && a.err) *a.err = 1;
  for (int r = cta; r < a.B; r += ctas) {
    const Span s = node_span(a, r);
    const int64_t row0 = static_cast<int64_t>(s.n0) * a.Hq, rows = static_cast<int64_t>(s.cnt) * a.Hq;
    for (int64_t i = threadIdx.x; i < rows * D; i += blockDim.x) static_cast<uint16_t*>(a.out)[row0 * D + i] = 0x7fc0;
    if (a.lse)
      for (int64_t i = threadIdx.x; i < rows; i += blockDim.x) a.lse[row0 + i] = __uint_as_float(0x7fc00000u);
  }
}

// Piece 0 of a cut unit is slot 1 of the run where the unit starts, piece i
// slot 0 of the i-th run after it.  CTA = (starting run, eight rows), warp =
// row, lane = D / 32 dims; the pieces are taken in run order, eight loads in
// flight.  Bound by the latency of those loads: 12 us for the 304 runs of 64
// chains of 64 rows, 6 us for the runs of 64 single tokens (cold caches).
template <int D>
__global__ void __launch_bounds__(256, 4) join_kernel(const AttnArgs a, const Pieces p, const int* status, int R,
                                                   int nq) {
  griddep_wait();
  griddep_release();
  const int4 d = p.desc[blockIdx.x];             // pieces, request, row tile, KV head
  if (__builtin_expect(*status != 0, 0)) {
    fail_rows<D>(a);
    return;
  }
  if (d.x < 2) return;
  const int g = a.Hq / a.Hkv, lane = threadIdx.x & 31;
  const Span s = node_span(a, d.y);
  const int rows = min(nq, s.cnt - d.z * nq) * g;
  constexpr int kV = D / 32, kAhead = 8;
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (r < rows) {
    auto slot = [&](int i) {
      return static_cast<int64_t>(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * R + r;
    };
    float M = kLow, sum = 0.f, acc[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) acc[k] = 0.f;
    for (int i0 = 0; i0 < d.x; i0 += kAhead) {
      float2 ml[kAhead];
      float o[kAhead][kV];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        ml[i] = make_float2(kLow, 0.f);
        if (i0 + i < d.x) {
          ml[i] = p.ml[slot(i0 + i)];
#pragma unroll
          for (int k = 0; k < kV; ++k) o[i][k] = p.o[slot(i0 + i) * D + 32 * k + lane];
        }
      }
      const float old = M;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) M = fmaxf(M, ml[i].x);
      const float keep = ex2(old - M);
      sum *= keep;
#pragma unroll
      for (int k = 0; k < kV; ++k) acc[k] *= keep;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (ml[i].y == 0.f) continue;            // nothing seen in this piece
        const float w = ex2(ml[i].x - M);
        sum = fmaf(w, ml[i].y, sum);
#pragma unroll
        for (int k = 0; k < kV; ++k) acc[k] = fmaf(w, o[i][k], acc[k]);
      }
    }
    const int64_t row = static_cast<int64_t>(s.n0 + d.z * nq + r / g) * a.Hq + d.w * g + r % g;
    const float f = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int k = 0; k < kV; ++k)
      static_cast<uint16_t*>(a.out)[row * D + 32 * k + lane] = static_cast<uint16_t>(tc::pack_bf16(acc[k] * f, 0.f));
    if (lane == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
  }
}

}  // namespace

int attn_extents(const AttnArgs& a, int nq, int tiles, int4* out, cudaStream_t st) {
  return launch_pdl(extent_kernel, dim3((a.B * tiles + 3) / 4), dim3(128), 0, st, a, nq, tiles, out);
}

int attn_join(const AttnArgs& a, const Pieces& p, const int* status, int runs, int R, int nq, cudaStream_t st) {
  return a.d == 128 ? launch_pdl(join_kernel<128>, dim3(runs, R / 8), dim3(256), 0, st, a, p, status, R, nq)
                    : launch_pdl(join_kernel<64>, dim3(runs, R / 8), dim3(256), 0, st, a, p, status, R, nq);
}

int initial_status() {
  static const int planted = [] {
    const char* e = std::getenv("TV_TEST_ATTN_KV4_STATUS");
    return e ? std::atoi(e) : 0;
  }();
  return planted;
}

size_t pieces_bytes(int runs, int R, int d) {
  return align256(static_cast<size_t>(runs) * sizeof(int4)) + align256(2ull * runs * R * sizeof(float2)) +
         2ull * runs * R * d * sizeof(float);
}
Pieces pieces_at(char* base, int runs, int R) {
  Pieces p;
  p.desc = reinterpret_cast<int4*>(base);
  base += align256(static_cast<size_t>(runs) * sizeof(int4));
  p.ml = reinterpret_cast<float2*>(base);
  p.o = reinterpret_cast<float*>(base + align256(2ull * runs * R * sizeof(float2)));
  return p;
}

}  // namespace kv4
}  // namespace tv
