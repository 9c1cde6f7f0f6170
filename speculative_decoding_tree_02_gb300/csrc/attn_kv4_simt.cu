// tree_verify_attn_kv4, CUDA-core path: fp32 rows (bf16 rows run on the
// tensor cores).  CTA = (query head, node, request), four warps; the warps
// take the keys in turn, 32 at a time:
//   score: lane = key; the lane walks its key's code words (or its tree row)
//          against q in shared memory, so a score needs no reduction;
//   value: lane = dims; the 32 weights are broadcast by shuffles and each
//          lane adds its D/32 dims of every value.
// Each warp keeps its own running maximum and sum (softmax in one pass); the
// four partial rows are joined in warp order at the end, so the result does
// not depend on timing.  Bound by issue slots: 4 d multiply-adds per key and
// head, each behind a nibble extraction.  60 nodes x 4 heads of 64 over 128
// tokens: see the launch's note below.
#include "kv4.cuh"

namespace tv {
namespace kv4 {

template <int D>
__global__ void __launch_bounds__(128) attn_simt_kernel(const AttnArgs a) {
  constexpr int kDl = D / 32;            // dims per lane of the value product
  __shared__ float sq[D];
  __shared__ float so[4][D];
  __shared__ float2 sml[4];
  griddep_wait();
  griddep_release();
  const int r = blockIdx.z, ln = blockIdx.y, hq = blockIdx.x;
  const Span sp = node_span(a, r);
  if (ln >= sp.cnt) return;
  const int gn = sp.n0 + ln, h = hq / (a.Hq / a.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = prefix_len(a, r);
  const int vis = a.vis_prefix ? min(max(a.vis_prefix[gn], 0), len) : len;
  const float* q = static_cast<const float*>(a.q) + gn * a.ldq + static_cast<int64_t>(hq) * D;
  for (int i = threadIdx.x; i < D; i += 128) sq[i] = q[i];
  __syncthreads();
  const float c2 = a.scale * kLog2e;
  float m = -INFINITY, l = 0.f, o[kDl];
#pragma unroll
  for (int i = 0; i < kDl; ++i) o[i] = 0.f;

  // joins 32 scores (base-2 units; -inf: not visible) to the running softmax; returns the lane's weight
  auto weigh = [&](float x, bool seen) {
    float mx = seen ? x : -INFINITY;
    mx = fmaxf(m, warp_max(mx));
    const float base = mx == -INFINITY ? 0.f : mx;
    const float corr = m == -INFINITY ? 0.f : ex2(m - base);
    const float p = seen ? ex2(x - base) : 0.f;
    l = l * corr + warp_sum(p);
#pragma unroll
    for (int i = 0; i < kDl; ++i) o[i] *= corr;
    m = mx;
    return p;
  };

  for (int k0 = warp * 32; k0 < vis; k0 += 128) {
    const int key = k0 + lane;
    bool seen = key < vis;
    const uint8_t* blk = nullptr;
    int slot = 0;
    if (seen) {
      const int page = a.block_table[static_cast<int64_t>(r) * a.table_ld + key / a.page_size];
      slot = key % a.page_size;
      if (page >= 0 && page < a.n_pages) {
        blk = a.cache + (static_cast<int64_t>(page) * a.Hkv + h) * block_bytes(a.page_size, D);
      } else {
        seen = false;
        if (a.err) *a.err = 1;
      }
    }
    float x = 0.f, sv = 0.f;
    if (seen) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(blk + k_word(a.page_size, slot, 32 * c));
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 32; ++i) x = fmaf(decode(ww[i >> 3], i & 7), sq[32 * c + i], x);
      }
      x *= bf16_at(reinterpret_cast<const uint16_t*>(blk + k_scale(a.page_size, D, slot))) * c2;
      sv = bf16_at(reinterpret_cast<const uint16_t*>(blk + v_scale(a.page_size, D, slot)));
    }
    const float p = weigh(x, seen);
    const float pv = seen ? p * sv : 0.f;
    // two 16-token groups; the page is the same for all tokens of a group
#pragma unroll
    for (int gr = 0; gr < 2; ++gr) {
      const unsigned mask = __ballot_sync(0xffffffffu, seen) >> (16 * gr) & 0xffffu;
      if (!mask) continue;
      const int src = 16 * gr + __ffs(static_cast<int>(mask)) - 1;
      const uint64_t b = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(blk), src);
      const int group = (k0 + 16 * gr) % a.page_size / 16;
      uint2 w[kDl];
#pragma unroll
      for (int i = 0; i < kDl; ++i)
        w[i] = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(b) +
                                               v_group(a.page_size, D, group, lane + 32 * i));
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        const float pt = __shfl_sync(0xffffffffu, pv, 16 * gr + t);
#pragma unroll
        for (int i = 0; i < kDl; ++i) o[i] = fmaf(pt, decode(t < 8 ? w[i].x : w[i].y, t & 7), o[i]);
      }
    }
  }
  // the node's ancestors, 32 nodes of the request at a time
  for (int j0 = warp * 32; j0 < sp.cnt && j0 < 64 * a.anc_words; j0 += 128) {
    const int j = j0 + lane;
    const uint64_t word = a.anc[static_cast<int64_t>(gn) * a.anc_words + (j0 >> 6)];
    const unsigned bits = static_cast<unsigned>(word >> (j0 & 63));
    if (!bits) continue;
    const bool seen = ((bits >> lane) & 1u) && j < sp.cnt;
    float x = 0.f;
    if (seen) {
      const float* kr = static_cast<const float*>(a.k_tree) + (sp.n0 + j) * a.ldk + static_cast<int64_t>(h) * D;
      for (int i = 0; i < D; ++i) x = fmaf(kr[i], sq[i], x);
      x *= c2;
    }
    const float p = weigh(x, seen);
    unsigned todo = __ballot_sync(0xffffffffu, seen);
    while (todo) {   // only visible rows are read: a masked row may hold anything
      const int t = __ffs(static_cast<int>(todo)) - 1;
      todo &= todo - 1;
      const float pt = __shfl_sync(0xffffffffu, p, t);
      const float* vr = static_cast<const float*>(a.v_tree) + (sp.n0 + j0 + t) * a.ldv + static_cast<int64_t>(h) * D;
#pragma unroll
      for (int i = 0; i < kDl; ++i) o[i] = fmaf(pt, vr[lane + 32 * i], o[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kDl; ++i) so[warp][lane + 32 * i] = o[i];
  if (lane == 0) sml[warp] = make_float2(m, l);
  __syncthreads();
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < 4; ++w) M = fmaxf(M, sml[w].x);
  float f[4], L = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    // an unused warp has l = 0; a warp whose scores are NaN has m = -inf and l = NaN
    f[w] = sml[w].x == -INFINITY ? (sml[w].y == 0.f ? 0.f : sml[w].y) : ex2(sml[w].x - M);
    L += f[w] * sml[w].y;
  }
  const int64_t at = static_cast<int64_t>(gn) * a.Hq + hq;
  for (int i = threadIdx.x; i < D; i += 128) {
    float acc = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) acc = fmaf(f[w], so[w][i], acc);
    acc = L == 0.f ? 0.f : acc / L;
    static_cast<float*>(a.out)[at * D + i] = acc;
  }
  if (threadIdx.x == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

int attn_simt(const AttnArgs& a, cudaStream_t st) {
  const dim3 grid(a.Hq, a.max_nodes, a.B);
  return a.d == 128 ? launch_pdl(attn_simt_kernel<128>, grid, dim3(128), 0, st, a)
                    : launch_pdl(attn_simt_kernel<64>, grid, dim3(128), 0, st, a);
}

}  // namespace kv4
}  // namespace tv
