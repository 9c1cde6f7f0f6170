// tree_verify_attn_kv4 for few query rows (bf16; at most 16 rows = nodes x
// heads of one KV head: single tokens, short drafts), d = 64 or 128.
//
// Every warp works by itself: it walks its own run of 64-token chunks, with
// the codes of the next chunk on their way into its half of shared memory, and
// keeps queries, weights and outputs in registers.  The products are taken
// transposed, so that the dequantised operand is the 16-row A of mma.sync and
// eight query rows are its 8 columns:
//   S^T [16 keys x 8 rows]  = K Q^T     a thread owns code word t of keys g, g + 8
//   O^T [16 dims x 8 rows] += V^T P^T   a thread owns dims 2g, 2g + 1, tokens 2t, 2t + 1 (+ 8)
// (g = lane / 4, t = lane % 4).  A code word holds exactly the operand pairs
// that its thread needs: (w >> 4i) & 0x000f000f | 0x43004300 are two bf16
// numbers 128 + code, minus 136 the values n, exact.  The order of the dims
// within the contraction is free, so q's fragment is 16 consecutive bytes of
// a row.  S^T's accumulators, packed to bf16 and transposed by movmatrix, are
// P^T's operand.
//
// Why not the tcgen05 kernel: with so few rows the work is the dequantisation
// (2.75 instructions for two codes, whatever the path) and the reading of 132
// bytes per token and head; mma.sync's 1024 multiply-adds per cycle and SM
// (measured) take 256 of the 720 cycles that 128 tokens take at the measured
// copy rate, and there is no hand-over between warps to wait for.
//
// The list of all units (request, KV head), in chunks, is cut into runs of equal
// cost, one per warp; a unit that a run's end cuts leaves fp32 partials that
// attn_join joins in run order.
//
// Bound by issue slots: 1400 instructions to a warp and chunk for 8 rows, 56%
// of the slots taken, with the three warps per scheduler that 160 registers
// leave.  64 requests of 32 heads of 128 over 512..4096 tokens: one token each
// 50 us (3.1 TB/s, 46% of the measured copy rate), 16 rows per KV head 76 us.
// One request over 2048 tokens 14.5 us with its joining.
#include <algorithm>

#include "kv4.cuh"
#include "kv4_device.cuh"

namespace tv {
namespace kv4 {
namespace {

constexpr int kChunk = 64;     // tokens per chunk
// What a unit costs beside its chunks, in chunks: 64 single tokens 51.5 us without it, 50.4 at 1, 51.9 at 2, 53 at 3;
// 16 rows per KV head 79, 76, 73, 75 (8 KV heads of 128; other geometries take the same number untimed).
constexpr int kUnitCost = 1;

template <int D, int NB>
struct Lay {
  static constexpr int kWarps = NB == 1 ? 12 : 8;
  static constexpr uint32_t kStage = kChunk * (D + 4);
  static constexpr uint32_t kQ = 2 * kStage;                     // [NB][D / 32][32 lanes][16 B]
  static constexpr uint32_t kWarp = kQ + NB * (D / 32) * 512;    // bytes of one warp
  static constexpr uint32_t kBars = kWarps * kWarp;              // two mbarriers per warp
  static constexpr uint32_t kMisc = kBars + 16 * kWarps;         // abort flag, entry sums
  static constexpr uint32_t kBytes = kMisc + 16 + 8 * kWarps;
  static_assert(kWarp % 128 == 0 && kBytes <= 232448, "layout");
};

struct MmaArgs {
  AttnArgs a;
  int* status;
  int status0;            // its first value
  Pieces pieces;          // runs = workers, 8 NB rows
  const int4* extents;    // [B] x = visible prefix (per-node prefixes), or NULL
  int workers;
  uint32_t magic;         // kMagic
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Chunks of request e (one KV head): its prefix, then its nodes.
struct Unit {
  int len, np, nb;        // visible prefix, prefix chunks, chunks
};
__device__ __forceinline__ Unit unit_of(const MmaArgs& p, int e) {
  Unit u;
  const bool live = node_span(p.a, e).cnt > 0;
  u.len = p.extents ? p.extents[e].x : prefix_len(p.a, e);
  u.np = live ? (u.len + kChunk - 1) / kChunk : 0;
  u.nb = u.np + (live ? 1 : 0);
  return u;
}

template <int D, int NB>
__global__ void __launch_bounds__(32 * Lay<D, NB>::kWarps, 1) mma_kernel(const __grid_constant__ MmaArgs p) {
  using L = Lay<D, NB>;
  constexpr int kC = D / 32, kDm = D / 16, R = 8 * NB;
  constexpr int M = kChunk / 16;                 // blocks of 16 keys; the nodes fit in one, being no more than the rows
  extern __shared__ __align__(128) uint8_t sm[];
  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  const int g = a.Hq / a.Hkv;
  uint8_t* mine = sm + warp * L::kWarp;
  const uint32_t mine_s = tc::smem_u32(mine);
  const uint32_t bars = tc::smem_u32(sm + L::kBars) + 16 * warp;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kMisc);
  long long* sums = reinterpret_cast<long long*>(sm + L::kMisc + 16);
  if (lane == 0) {
    tc::mbar_init(bars, 1);
    tc::mbar_init(bars + 8, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x == 0) *abort_flag = 0;
  griddep_wait();
  griddep_release();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = p.status0;   // an expired wait writes it seconds later

  // ---- this warp's run: [w0, w1) of the list of all units, each kUnitCost places and then its chunks
  const int per = ((a.B + L::kWarps - 1) / L::kWarps + 31) / 32 * 32;   // entries (requests) per warp
  auto cost_of = [&](int e, int end) {
    const int nb = e < end ? unit_of(p, e).nb : 0;
    return nb ? static_cast<long long>(nb + kUnitCost) * a.Hkv : 0ll;
  };
  {
    const int lo = min(warp * per, a.B), hi = min(lo + per, a.B);
    long long s = 0;
    for (int e = lo; e < hi; e += 32) s += cost_of(e + lane, hi);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sums[warp] = s;
  }
  __syncthreads();
  long long W = 0;
  for (int w = 0; w < L::kWarps; ++w) W += sums[w];
  // Runs of one place while two warps to an SM take them all (one request over 2048 tokens 14.5 us, with two places
  // 16.5), else of two at least (one request over 8192 tokens 20.5 us, with one place 24.5: its units' many pieces are
  // joined one after another; 16 rows, 16 requests over 500 tokens 20.6 and 22.7).
  const long long G = min(static_cast<long long>(p.workers), max((W + 1) / 2, min(W, 2ll * gridDim.x)));
  const int worker = static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) * warp;   // neighbours on other SMs
  if (lane == 0) p.pieces.desc[worker] = make_int4(0, 0, 0, 0);
  if (worker >= G) return;
  const long long w0 = worker * W / G, w1 = (worker + 1) * W / G;
  int e = 0;
  long long before = 0;                          // places before entry e
  {
    int w = 0;
    while (before + sums[w] <= w0) before += sums[w++];
    const int hi = min(w * per + per, a.B);
    for (e = w * per;; e += 32) {
      const long long c = cost_of(e + lane, hi);
      long long x = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + x > w0);
      if (past) {
        const int at = __ffs(static_cast<int>(past)) - 1;
        e += at;
        before += __shfl_sync(0xffffffffu, x - c, at);
        break;
      }
      before += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  Unit u = unit_of(p, e);
  const int skip = static_cast<int>(w0 - before), at = skip % (u.nb + kUnitCost);
  int h = skip / (u.nb + kUnitCost), blk = max(0, at - kUnitCost);
  int left = static_cast<int>(w1 - w0) + at;     // places from the start of the unit to the end of the run
  // (a chunk is in the run while kUnitCost + its index < left)

  // ---- the loads run two chunks ahead, their page numbers three
  const int P = a.page_size, Pe = min(P, kChunk), shift = 31 - __clz(Pe);
  const uint32_t blk_e = Pe * (D + 4);           // bytes of a staged page
  // a block of 16 keys lies in one staged page; offset of its page and its first slot
  int pg[4], sl[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    pg[m] = ((16 * m) >> shift) * blk_e;
    sl[m] = (16 * m) & (Pe - 1);
  }
  const int page_shift = 31 - __clz(P);
  int le = e, lh = h, lblk = blk, lpage = -1;    // next chunk to load, this lane's page of it
  Unit lu = u;
  int lleft = left, lnext = 0;                                 // chunks loaded
  auto look = [&]() {                            // the page numbers of the next chunk to load
    lpage = -1;
    if (lblk == lu.nb) {
      lblk = 0;
      lleft -= lu.nb + kUnitCost;
      if (kUnitCost >= lleft) return;
      if (++lh == a.Hkv) {
        lh = 0;
        do lu = unit_of(p, ++le);
        while (lu.nb == 0 && le + 1 < a.B);
      }
    }
    if (kUnitCost + lblk >= lleft) return;
    const int key = lblk * kChunk + (P > kChunk ? 0 : lane << shift);
    if (lblk < lu.np && (P > kChunk ? lane <= kC + 2 : lane < kChunk >> shift) && key < lu.len)
      lpage = a.block_table[static_cast<int64_t>(le) * a.table_ld + (key >> page_shift)];
  };
  unsigned good = 0u;                            // staged pages of the two stages, 8 bits each
  auto load = [&](int st) {
    if (kUnitCost + lblk >= lleft) return;
    const bool wanted = lpage != -1;
    const bool ok = wanted && lpage >= 0 && lpage < a.n_pages;
    // a lane that wants no page has -1 too: entries of -1 are told by the token they should hold
    const int key = lblk * kChunk + (P > kChunk ? 0 : lane << shift);
    const bool needs = lblk < lu.np && (P > kChunk ? lane == 0 : lane < kChunk >> shift) && key < lu.len;
    if (needs && !ok && a.err) *a.err = 1;
    const unsigned have = __ballot_sync(0xffffffffu, ok);
    good = st ? (good & 0x00ffu) | (have << 8) : (good & 0xff00u) | have;
    const uint32_t bar = bars + 8 * st, dst = mine_s + st * L::kStage;
    const uint32_t bytes = P > kChunk ? (have ? L::kStage : 0u) : __popc(have) * blk_e;
    if (lane == 0) {
      if (bytes) tc::mbar_expect_tx(bar, bytes);
      else tc::mbar_arrive(bar);
    }
    __syncwarp();
    if (ok) {
      const uint8_t* src = a.cache + (static_cast<int64_t>(lpage) * a.Hkv + lh) * block_bytes(P, D);
      if (P <= kChunk) {
        bulk_load(dst + lane * blk_e, src, blk_e, bar);
      } else {                                   // half of a 128-token page, staged as a page of 64
        const int half = lblk & 1;
        if (lane < kC) bulk_load(dst + lane * 1024, src + lane * (P * 16) + half * 1024, 1024, bar);
        else if (lane == kC) bulk_load(dst + 32 * D, src + (P / 2) * D + half * 32 * D, 32 * D, bar);
        else bulk_load(dst + kChunk * D + (lane - kC - 1) * 128, src + P * D + (lane - kC - 1) * 2 * P + half * 128, 128, bar);
      }
    }
    ++lblk;
    ++lnext;
  };
  // ---- state of the running unit
  uint64_t nm[NB], l[NB];                        // rows 8 nb + 2t, + 1: negated references, sums
  uint32_t unset = 0;                            // bit 2 nb + i: that row has no reference yet
  uint32_t live = 0;
  int vis[2 * NB], low_vis = 0;
  float o[kDm][NB][4];
  bool dirty = false;
  int n0 = 0, cnt = 0;
  const float c2 = a.scale * kLog2e;
  const uint32_t magic = p.magic;
  int seg_blk = blk;
  bool fresh = true;
  auto row_at = [&](int r) { return static_cast<int64_t>(n0 + r / g) * a.Hq + h * g + r % g; };   // output row

  look();
  for (int it = -2;;) {
    load(it & 1);                                // the chunk after next (before the first chunk: the first two)
    look();
    if (++it < 0) continue;
    const int st = it & 1;
    if (blk == u.nb) {                           // next unit
      left -= u.nb + kUnitCost;
      if (kUnitCost >= left) break;
      blk = seg_blk = 0;
      fresh = true;
      if (++h == a.Hkv) {
        h = 0;
        do u = unit_of(p, ++e);
        while (u.nb == 0 && e + 1 < a.B);
      }
    }
    if (kUnitCost + blk >= left) break;
    if (fresh) {
      fresh = false;
      const Span sp = node_span(a, e);
      n0 = sp.n0;
      cnt = sp.cnt;
      const int rows = cnt * g;
      __syncwarp();
#pragma unroll 1
      for (int nb = 0; nb < NB; ++nb) {          // eight rows' loads in one latency
        const int r = 8 * nb + gq;
        const uint16_t* row = static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(n0 + min(r, rows - 1) / g) * a.ldq +
                              static_cast<int64_t>(h * g + min(r, rows - 1) % g) * D + 8 * tq;
        uint4 v[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) v[c] = *reinterpret_cast<const uint4*>(row + 32 * c);
#pragma unroll
        for (int c = 0; c < kC; ++c)
          *reinterpret_cast<uint4*>(mine + L::kQ + (nb * kC + c) * 512 + lane * 16) =
              r < rows ? v[c] : make_uint4(0u, 0u, 0u, 0u);
      }
      live = 0;
      low_vis = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < 2 * NB; ++i) {
        const int r = 8 * (i >> 1) + 2 * tq + (i & 1);
        vis[i] = 0x7fffffff;
        if (r < rows) {
          live |= 1u << i;
          if (a.vis_prefix) vis[i] = a.vis_prefix[n0 + r / g];
        }
        low_vis = min(low_vis, vis[i]);
      }
      low_vis = __reduce_min_sync(0xffffffffu, low_vis);
      unset = (1u << (2 * NB)) - 1u;
      dirty = false;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        nm[i] = 0ull;
        l[i] = 0ull;
      }
#pragma unroll
      for (int d = 0; d < kDm; ++d)
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[d][i][k] = 0.f;
      __syncwarp();
    }
    // (a warp may leave by itself: no barrier of the CTA follows)
    if (!warp_wait(bars + 8 * st, (it >> 1) & 1, abort_flag, p.status, 61)) break;
    const uint8_t* stage = mine + st * L::kStage;
    const bool tree = blk == u.np;
    const int key0 = blk * kChunk, nkeys = tree ? cnt : min(kChunk, u.len - key0);
    const unsigned pages = (good >> (8 * st)) & 0xffu;

    // ---- S^T = K Q^T
    float s[M][NB][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[m][i][k] = 0.f;
    if (!tree) {
      const uint8_t* kp[M];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        kp[m] = stage + pg[m] + 16 * sl[m] + gq * 16 + tq * 4;
      }
#pragma unroll 1
      for (int c = 0; c < kC; ++c) {
        uint4 q[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) q[i] = *reinterpret_cast<const uint4*>(mine + L::kQ + (i * kC + c) * 512 + lane * 16);
#pragma unroll
        for (int m = 0; m < M; ++m) {
          uint32_t x[4], y[4];
          decode8(*reinterpret_cast<const uint32_t*>(kp[m]), x, magic);         // key g
          decode8(*reinterpret_cast<const uint32_t*>(kp[m] + 128), y, magic);   // key g + 8: the same page
          kp[m] += Pe * 16;
          const uint32_t f0[4] = {x[0], y[0], x[1], y[1]}, f1[4] = {x[2], y[2], x[3], y[3]};
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            mma16816(s[m][i], f0, q[i].x, q[i].y);
            mma16816(s[m][i], f1, q[i].z, q[i].w);
          }
        }
      }
    } else {
      // the nodes' own keys, at most 16 (beyond the last: that one again, masked below)
      {
        uint4 x[2][kC];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint16_t* row = static_cast<const uint16_t*>(a.k_tree) +
                                static_cast<int64_t>(n0 + min(gq + 8 * b, cnt - 1)) * a.ldk +
                                static_cast<int64_t>(h) * D + 8 * tq;
#pragma unroll
          for (int c = 0; c < kC; ++c) x[b][c] = *reinterpret_cast<const uint4*>(row + 32 * c);
        }
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          const uint32_t f0[4] = {x[0][c].x, x[1][c].x, x[0][c].y, x[1][c].y};
          const uint32_t f1[4] = {x[0][c].z, x[1][c].z, x[0][c].w, x[1][c].w};
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const uint4 q = *reinterpret_cast<const uint4*>(mine + L::kQ + (i * kC + c) * 512 + lane * 16);
            mma16816(s[0][i], f0, q.x, q.y);
            mma16816(s[0][i], f1, q.z, q.w);
          }
        }
      }
    }

    // ---- scores in base-2 units over the references: keys 16 m + g, + 8, rows 2t, 2t + 1
    uint64_t y[M][NB][2];
    float sv[M][2];
    const bool full = !tree && nkeys == kChunk && key0 + kChunk <= low_vis &&
                      (P > kChunk ? pages != 0 : pages == (1u << (kChunk >> shift)) - 1u);
    uint32_t seen = 0u;                          // bit 4 (M i + m) + k: that score counts
    {
#pragma unroll
      for (int m = 0; m < M; ++m) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float sk = c2;
          sv[m][b] = 1.f;
          if (!tree) {
            const uint8_t* at = stage + pg[m] + 2 * sl[m] + Pe * D + 2 * gq + 16 * b;
            sk = c2 * bf16_at(reinterpret_cast<const uint16_t*>(at));
            sv[m][b] = bf16_at(reinterpret_cast<const uint16_t*>(at + 2 * Pe));
          }
          const uint64_t sk2 = pair(sk, sk);
#pragma unroll
          for (int i = 0; i < NB; ++i) y[m][i][b] = fma2(pair(s[m][i][2 * b], s[m][i][2 * b + 1]), sk2, nm[i]);
        }
      }
      if (__builtin_expect(!full, 0)) {
        uint32_t anc[2 * NB];
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) {
          const int r = 8 * (i >> 1) + 2 * tq + (i & 1);
          anc[i] = 0u;
          if (tree && ((live >> i) & 1u))
            anc[i] = static_cast<uint32_t>(a.anc[static_cast<int64_t>(n0 + r / g) * a.anc_words]);
        }
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int k = 16 * m + gq + 8 * b;
            const bool there = k < nkeys && (tree || (P > kChunk ? pages != 0 : (pages >> (k >> shift)) & 1u));
            if (!there) sv[m][b] = 0.f;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
              bool sees[2];
              float v[2];
              split(y[m][i][b], v[0], v[1]);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                sees[q] = there && (tree ? (anc[2 * i + q] >> (k & 31)) & 1u : key0 + k < vis[2 * i + q]);
                if (sees[q]) seen |= 1u << (4 * M * i + 4 * m + 2 * b + q);
                else v[q] = -INFINITY;
              }
              y[m][i][b] = pair(v[0], v[1]);
            }
          }
      }
    }
    bool grow = __any_sync(0xffffffffu, (unset & live) != 0u);
    if (!grow) {
      float mx = -INFINITY;
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float v0, v1;
            split(y[m][i][b], v0, v1);
            mx = max3(mx, v0, v1);
          }
      grow = __any_sync(0xffffffffu, mx > 8.f);
    }
    if (__builtin_expect(grow, 0)) {
      // new references: the rows' maxima so far
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        float top[2] = {-INFINITY, -INFINITY}, sh[2], corr[2], old[2];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float v0, v1;
            split(y[m][i][b], v0, v1);
            top[0] = fmaxf(top[0], v0);
            top[1] = fmaxf(top[1], v1);
          }
        split(nm[i], old[0], old[1]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top[q] = fmaxf(top[q], __shfl_xor_sync(0xffffffffu, top[q], x));
          const uint32_t bit = 1u << (2 * i + q);
          const bool none = unset & bit;
          sh[q] = none ? (top[q] == -INFINITY ? 0.f : top[q]) : fmaxf(top[q], 0.f);
          corr[q] = none ? 0.f : ex2(-sh[q]);
          if (top[q] != -INFINITY) unset &= ~bit;
        }
        const uint64_t shift2 = pair(-sh[0], -sh[1]), corr2 = pair(corr[0], corr[1]);
        nm[i] = add2(nm[i], shift2);
        l[i] = mul2(l[i], corr2);
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int b = 0; b < 2; ++b) y[m][i][b] = add2(y[m][i][b], shift2);
#pragma unroll
        for (int d = 0; d < kDm; ++d) {
          o[d][i][0] *= corr[0];
          o[d][i][1] *= corr[1];
          o[d][i][2] *= corr[0];
          o[d][i][3] *= corr[1];
        }
      }
    }
    // ---- weights, times the value's scale, as P^T's operand: keys 16 m + 2t, + 1 (+ 8), row g
    uint32_t pb[M][NB][2];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint64_t sv2 = pair(sv[m][b], sv[m][b]);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          float v0, v1;
          split(y[m][i][b], v0, v1);
          const uint64_t w = pair(ex2(v0), ex2(v1));
          l[i] = add2(l[i], w);
          split(mul2(w, sv2), v0, v1);
          pb[m][i][b] = tc::pack_bf16(v0, v1);
        }
      }
    if (__builtin_expect(!full, 0)) {
      // zero weights times the scale of a value row that was not finite are NaN: rows that do not see it stay clean
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const uint32_t two = seen >> (4 * M * i + 4 * m + 2 * b);
            pb[m][i][b] &= (two & 1u ? 0x0000ffffu : 0u) | (two & 2u ? 0xffff0000u : 0u);
          }
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int b = 0; b < 2; ++b) pb[m][i][b] = transpose8x8(pb[m][i][b]);

    // ---- O^T += V^T P^T
    if (!tree) {
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const uint8_t* vg = stage + pg[m] + sl[m] * (D / 2) + Pe * (D / 2) +
                            gq * 16;
#pragma unroll
        for (int d = 0; d < kDm; ++d) {
          const uint4 w = *reinterpret_cast<const uint4*>(vg + d * 128);   // dims 16 d + 2g, + 1: tokens 0-7, 8-15
          const uint32_t f[4] = {decode_pair(w.x >> (4 * tq), magic), decode_pair(w.z >> (4 * tq), magic),
                                 decode_pair(w.y >> (4 * tq), magic), decode_pair(w.w >> (4 * tq), magic)};
#pragma unroll
          for (int i = 0; i < NB; ++i) mma16816(o[d][i], f, pb[m][i][0], pb[m][i][1]);
        }
      }
    } else {
      // the nodes' own values; one that is not finite must not meet the zero weights of rows that do not see it:
      // it is taken out here and added at the end to the rows that see it
      {
        const uint16_t* rows[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          rows[k] = static_cast<const uint16_t*>(a.v_tree) +
                    static_cast<int64_t>(n0 + min(2 * tq + (k & 1) + 8 * (k >> 1), cnt - 1)) * a.ldv +
                    static_cast<int64_t>(h) * D + 2 * gq;
#pragma unroll
        for (int d0 = 0; d0 < kDm; d0 += 4) {    // four blocks' loads in one latency
          uint32_t w[4][4];
#pragma unroll
          for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int k = 0; k < 4; ++k) w[d][k] = *reinterpret_cast<const uint32_t*>(rows[k] + 16 * (d0 + d));
#pragma unroll
          for (int d = 0; d < 4; ++d) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t& e = w[d][k];
              if (2 * tq + (k & 1) + 8 * (k >> 1) >= cnt) e = 0u;
              if ((e & 0x7f80u) == 0x7f80u) { e &= 0xffff0000u; dirty = true; }
              if ((e & 0x7f800000u) == 0x7f800000u) { e &= 0x0000ffffu; dirty = true; }
            }
            const uint32_t f[4] = {__byte_perm(w[d][0], w[d][1], 0x5410), __byte_perm(w[d][0], w[d][1], 0x7632),
                                   __byte_perm(w[d][2], w[d][3], 0x5410), __byte_perm(w[d][2], w[d][3], 0x7632)};
#pragma unroll
            for (int i = 0; i < NB; ++i) mma16816(o[d0 + d][i], f, pb[0][i][0], pb[0][i][1]);
          }
        }
      }
    }

    __syncwarp();                                // the stage was read
    if (blk != u.nb - 1 && kUnitCost + blk + 1 < left) {
      ++blk;
      continue;
    }

    // ---- end of the unit's run here
    const bool whole = seg_blk == 0 && blk == u.nb - 1;
    const int64_t slot = 2 * worker + (seg_blk == 0 ? 1 : 0);
    if (seg_blk == 0 && blk != u.nb - 1 && lane == 0) {
      const long long u1 = w1 - left + kUnitCost + u.nb;  // place after the unit
      const long long k = (u1 * G + W - 1) / W - 1;       // run of its last chunk
      p.pieces.desc[worker] = make_int4(static_cast<int>(k) - worker + 1, e, 0, h);
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      float sum[2], m[2];
      split(l[i], sum[0], sum[1]);
      split(nm[i], m[0], m[1]);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], x);
        const int r = 8 * i + 2 * tq + q;
        if (!((live >> (2 * i + q)) & 1u)) continue;
        const float f = sum[q] == 0.f ? 0.f : 1.f / sum[q];
        if (whole) {
          const int64_t row = row_at(r);
          if (gq == 0 && a.lse) a.lse[row] = sum[q] == 0.f ? -INFINITY : (log2f(sum[q]) - m[q]) * kLn2;
          uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + row * D + 2 * gq);
#pragma unroll
          for (int d = 0; d < kDm; ++d) out[8 * d] = tc::pack_bf16(o[d][i][q] * f, o[d][i][2 + q] * f);
        } else {
          if (gq == 0) p.pieces.ml[slot * R + r] = make_float2(sum[q] == 0.f ? kLow : -m[q], sum[q]);
          float2* out = reinterpret_cast<float2*>(p.pieces.o + (slot * R + r) * D + 2 * gq);
#pragma unroll
          for (int d = 0; d < kDm; ++d) out[8 * d] = make_float2(o[d][i][q], o[d][i][2 + q]);
        }
      }
    }
    if (__builtin_expect(__any_sync(0xffffffffu, dirty), 0)) {
      // tree values that are not finite, added to the rows that see them
      __syncwarp();
      const int rows = cnt * g;
#pragma unroll 1
      for (int j = 0; j < cnt; ++j)
#pragma unroll 1
        for (int dim = lane; dim < D; dim += 32) {
          const uint32_t v = static_cast<const uint16_t*>(a.v_tree)[static_cast<int64_t>(n0 + j) * a.ldv +
                                                                    static_cast<int64_t>(h) * D + dim];
          if ((v & 0x7f80u) != 0x7f80u) continue;
#pragma unroll 1
          for (int r = 0; r < rows; ++r) {
            if (!((a.anc[static_cast<int64_t>(n0 + r / g) * a.anc_words] >> j) & 1ull)) continue;
            if (whole) {
              uint16_t* o16 = static_cast<uint16_t*>(a.out) + row_at(r) * D + dim;
              *o16 = static_cast<uint16_t>(tc::pack_bf16(bf16_at(o16) + __uint_as_float(v << 16), 0.f));
            } else {
              p.pieces.o[(slot * R + r) * D + dim] += __uint_as_float(v << 16);
            }
          }
        }
      __syncwarp();
    }
    ++blk;
  }
  // after an expired wait: copies in flight land before the CTA ends
  if (*abort_flag) {
    for (int it = max(0, lnext - 2); it < lnext; ++it) drain(bars + 8 * (it & 1), (it >> 1) & 1);
  }
}

int blocks_of(int max_nodes, int g) {            // blocks of eight rows
  const int rows = max_nodes * g;
  return rows <= 8 ? 1 : 2;
}
int warps_of(int nb) { return nb == 1 ? Lay<128, 1>::kWarps : Lay<128, 2>::kWarps; }

template <int D, int NB>
int launch(const MmaArgs& p, cudaStream_t st) {
  using L = Lay<D, NB>;
  if (!smem_limit(mma_kernel<D, NB>, static_cast<int>(L::kBytes))) return TV_ECUDA;
  const int rc = launch_pdl(mma_kernel<D, NB>, dim3(p.workers / L::kWarps), dim3(32 * L::kWarps), L::kBytes, st, p);
  if (rc != TV_OK) return rc;
  return attn_join(p.a, p.pieces, p.status, p.workers, 8 * NB, p.a.max_nodes, st);
}

}  // namespace

// [status word (256 B)] [extents] [pieces of cut units]
size_t attn_mma_workspace(int B, int max_nodes, int Hq, int Hkv, int d) {
  const int nb = blocks_of(max_nodes, Hq / Hkv);
  return 256 + align256(static_cast<size_t>(B) * sizeof(int4)) + pieces_bytes(sm_count() * warps_of(nb), 8 * nb, d);
}

int attn_mma(const AttnArgs& a, void* ws, cudaStream_t st) {
  MmaArgs p{};
  p.a = a;
  p.magic = kMagic;
  const int nb = blocks_of(a.max_nodes, a.Hq / a.Hkv);
  p.workers = sm_count() * warps_of(nb);
  char* base = static_cast<char*>(ws);
  p.status = reinterpret_cast<int*>(base);
  p.status0 = initial_status();
  int4* extents = reinterpret_cast<int4*>(base + 256);
  p.pieces = pieces_at(base + 256 + align256(static_cast<size_t>(a.B) * sizeof(int4)), p.workers, 8 * nb);
  if (a.vis_prefix) {
    const int rc = attn_extents(a, a.max_nodes, 1, extents, st);
    if (rc != TV_OK) return rc;
    p.extents = extents;
  }
  if (a.d == 128) return nb == 1 ? launch<128, 1>(p, st) : launch<128, 2>(p, st);
  return nb == 1 ? launch<64, 1>(p, st) : launch<64, 2>(p, st);
}

}  // namespace kv4
}  // namespace tv
