// tree_verify_attn_kv4, CUDA-core path: fp32 rows (bf16 rows run on the
// tensor cores).  CTA = (R rows = nodes x heads of one KV head, that head,
// request), four warps; the warps take the keys in turn, 32 at a time:
//   score: lane = key; the lane walks its key's code words (or its tree row)
//          against the rows' q in shared memory, so a score needs no reduction;
//   value: lane = dims; the 32 weights of every row are read back from shared
//          memory and each lane adds its D/32 dims of every value.
// Each warp keeps its own running maxima and sums (softmax in one pass); the
// four partial rows are joined in warp order at the end, so the result does
// not depend on timing.  Bound by issue slots: 4 d multiply-adds per key and
// row; the nibble extractions before them are shared by the R rows.  60 nodes
// x 4 heads of 64 over 128 tokens (R = 1) 10.7 us, 4 requests of 64 nodes x 32
// heads of 128 over 1000 tokens (R = 8) 210 us = 20 TFLOP/s.
#include "kv4.cuh"

namespace tv {
namespace kv4 {

template <int D, int R>
__global__ void __launch_bounds__(128) attn_simt_kernel(const AttnArgs a, int* status) {
  constexpr int kDl = D / 32;            // dims per lane of the value product
  __shared__ __align__(16) float sq[R][D];
  __shared__ __align__(16) float sp_w[4][32][R];   // a warp's weights
  __shared__ float so[4][R][D];
  __shared__ float2 sml[4][R];
  griddep_wait();
  griddep_release();
  if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) *status = 0;   // (nothing waits here)
  const int r = blockIdx.z, h = blockIdx.y, g = a.Hq / a.Hkv;
  const Span sp = node_span(a, r);
  const int row0 = blockIdx.x * R, rows = min(R, sp.cnt * g - row0);   // row = node g + head of the group
  if (rows <= 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = prefix_len(a, r);
  int vis[R], most = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    vis[i] = i < rows ? len : 0;
    if (i < rows && a.vis_prefix) vis[i] = min(max(a.vis_prefix[sp.n0 + (row0 + i) / g], 0), len);
    most = max(most, vis[i]);
  }
  for (int i = threadIdx.x; i < R * D; i += 128) {
    const int row = row0 + i / D;
    sq[i / D][i % D] = i / D < rows ? static_cast<const float*>(a.q)[(sp.n0 + row / g) * a.ldq +
                                                                     static_cast<int64_t>(h * g + row % g) * D + i % D]
                                    : 0.f;
  }
  __syncthreads();
  const float c2 = a.scale * kLog2e;
  float m[R], l[R], o[R][kDl];           // l: this lane's share
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < kDl; ++j) o[i][j] = 0.f;
  }

  // joins 32 scores (base-2 units; not seen: no weight) to row i's running softmax; returns the lane's weight
  auto weigh = [&](int i, float x, bool seen) {
    const float mx = fmaxf(m[i], warp_max(seen ? x : -INFINITY));
    const float base = mx == -INFINITY ? 0.f : mx;
    if (mx != m[i]) {
      const float corr = m[i] == -INFINITY ? 0.f : ex2(m[i] - base);
      l[i] *= corr;
#pragma unroll
      for (int j = 0; j < kDl; ++j) o[i][j] *= corr;
      m[i] = mx;
    }
    const float p = seen ? ex2(x - base) : 0.f;
    l[i] += p;
    return p;
  };

  for (int k0 = warp * 32; k0 < most; k0 += 128) {
    const int key = k0 + lane;
    bool there = key < most;
    const uint8_t* blk = nullptr;
    int slot = 0;
    if (there) {
      const int page = a.block_table[static_cast<int64_t>(r) * a.table_ld + key / a.page_size];
      slot = key % a.page_size;
      if (page >= 0 && page < a.n_pages) {
        blk = a.cache + (static_cast<int64_t>(page) * a.Hkv + h) * block_bytes(a.page_size, D);
      } else {
        there = false;
        if (a.err) *a.err = 1;
      }
    }
    float x[R], sv = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = 0.f;
    if (there) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(blk + k_word(a.page_size, slot, 32 * c));
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float n[4] = {decode(ww[e >> 3], e & 7), decode(ww[e >> 3], (e & 7) + 1), decode(ww[e >> 3], (e & 7) + 2),
                              decode(ww[e >> 3], (e & 7) + 3)};
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const float4 q = *reinterpret_cast<const float4*>(&sq[i][32 * c + e]);
            x[i] = fmaf(n[3], q.w, fmaf(n[2], q.z, fmaf(n[1], q.y, fmaf(n[0], q.x, x[i]))));
          }
        }
      }
      const float sk = bf16_at(reinterpret_cast<const uint16_t*>(blk + k_scale(a.page_size, D, slot))) * c2;
#pragma unroll
      for (int i = 0; i < R; ++i) x[i] *= sk;
      sv = bf16_at(reinterpret_cast<const uint16_t*>(blk + v_scale(a.page_size, D, slot)));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const bool seen = there && key < vis[i];
      const float p = weigh(i, x[i], seen);
      sp_w[warp][lane][i] = seen ? p * sv : 0.f;
    }
    __syncwarp();
    // two 16-token groups; the page is the same for all tokens of a group
#pragma unroll
    for (int gr = 0; gr < 2; ++gr) {
      const unsigned mask = __ballot_sync(0xffffffffu, there) >> (16 * gr) & 0xffffu;
      if (!mask) continue;
      const int src = 16 * gr + __ffs(static_cast<int>(mask)) - 1;
      const uint64_t b = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(blk), src);
      const int group = (k0 + 16 * gr) % a.page_size / 16;
      uint2 w[kDl];
#pragma unroll
      for (int j = 0; j < kDl; ++j)
        w[j] = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(b) +
                                               v_group(a.page_size, D, group, lane + 32 * j));
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        float n[kDl];
#pragma unroll
        for (int j = 0; j < kDl; ++j) n[j] = decode(t < 8 ? w[j].x : w[j].y, t & 7);
        float pt[R];
        if constexpr (R % 4 == 0) {
#pragma unroll
          for (int i = 0; i < R; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(&sp_w[warp][16 * gr + t][i]);
            pt[i] = v.x; pt[i + 1] = v.y; pt[i + 2] = v.z; pt[i + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < R; ++i) pt[i] = sp_w[warp][16 * gr + t][i];
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < kDl; ++j) o[i][j] = fmaf(pt[i], n[j], o[i][j]);
      }
    }
  }
  // the nodes' ancestors, 32 nodes of the request at a time
  for (int j0 = warp * 32; j0 < sp.cnt && j0 < 64 * a.anc_words; j0 += 128) {
    const int j = j0 + lane;
    unsigned bits[R], any = 0u;          // the nodes that row i sees
#pragma unroll
    for (int i = 0; i < R; ++i) {
      bits[i] = 0u;
      if (i < rows)
        bits[i] = static_cast<unsigned>(a.anc[static_cast<int64_t>(sp.n0 + (row0 + i) / g) * a.anc_words + (j0 >> 6)] >>
                                        (j0 & 63));
      if (sp.cnt - j0 < 32) bits[i] &= (1u << (sp.cnt - j0)) - 1u;
      any |= bits[i];
    }
    if (!any) continue;
    float x[R];
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = 0.f;
    if ((any >> lane) & 1u) {
      const float* kr = static_cast<const float*>(a.k_tree) + (sp.n0 + j) * a.ldk + static_cast<int64_t>(h) * D;
      for (int e = 0; e < D; e += 4) {
        const float4 n = *reinterpret_cast<const float4*>(kr + e);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(&sq[i][e]);
          x[i] = fmaf(n.w, q.w, fmaf(n.z, q.z, fmaf(n.y, q.y, fmaf(n.x, q.x, x[i]))));
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < R; ++i) sp_w[warp][lane][i] = weigh(i, x[i] * c2, (bits[i] >> lane) & 1u);
    __syncwarp();
    while (any) {   // only visible rows are read, and added to the rows that see them: others may hold anything
      const int t = __ffs(static_cast<int>(any)) - 1;
      any &= any - 1;
      const float* vr = static_cast<const float*>(a.v_tree) + (sp.n0 + j0 + t) * a.ldv + static_cast<int64_t>(h) * D;
      float n[kDl];
#pragma unroll
      for (int k = 0; k < kDl; ++k) n[k] = vr[lane + 32 * k];
#pragma unroll
      for (int i = 0; i < R; ++i)
        if ((bits[i] >> t) & 1u) {
          const float pt = sp_w[warp][t][i];
#pragma unroll
          for (int k = 0; k < kDl; ++k) o[i][k] = fmaf(pt, n[k], o[i][k]);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
#pragma unroll
    for (int j = 0; j < kDl; ++j) so[warp][i][lane + 32 * j] = o[i][j];
    const float sum = warp_sum(l[i]);
    if (lane == 0) sml[warp][i] = make_float2(m[i], sum);
  }
  __syncthreads();
  for (int x = threadIdx.x; x < rows * D; x += 128) {
    const int i = x / D, dim = x % D;
    float M = -INFINITY, f[4], L = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, sml[w][i].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      // an unused warp has l = 0; a warp whose scores are NaN has m = -inf and l = NaN
      f[w] = sml[w][i].x == -INFINITY ? (sml[w][i].y == 0.f ? 0.f : sml[w][i].y) : ex2(sml[w][i].x - M);
      L += f[w] * sml[w][i].y;
      acc = fmaf(f[w], so[w][i][dim], acc);
    }
    const int64_t at = static_cast<int64_t>(sp.n0 + (row0 + i) / g) * a.Hq + h * g + (row0 + i) % g;
    static_cast<float*>(a.out)[at * D + dim] = L == 0.f ? 0.f : acc / L;
    if (dim == 0 && a.lse) a.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
  }
}

template <int D, int R>
int launch(const AttnArgs& a, void* ws, cudaStream_t st) {
  const dim3 grid((a.max_nodes * (a.Hq / a.Hkv) + R - 1) / R, a.Hkv, a.B);
  return launch_pdl(attn_simt_kernel<D, R>, grid, dim3(128), 0, st, a, static_cast<int*>(ws));
}

int attn_simt(const AttnArgs& a, void* ws, cudaStream_t st) {
  // Eight rows to a CTA once that gives every SM one, else one row: 256 CTAs of eight 74 us against 114 with a row
  // each (64 nodes x 32 heads of 128, 1000 tokens), 1024 of them 73 against 123 (64 heads of 64); 128 of them 45
  // against 41, 32 of them 64 against 27.
  const int64_t groups = static_cast<int64_t>((a.max_nodes * (a.Hq / a.Hkv) + 7) / 8) * a.Hkv * a.B;
  if (groups >= sm_count()) return a.d == 128 ? launch<128, 8>(a, ws, st) : launch<64, 8>(a, ws, st);
  return a.d == 128 ? launch<128, 1>(a, ws, st) : launch<64, 1>(a, ws, st);
}

}  // namespace kv4
}  // namespace tv
