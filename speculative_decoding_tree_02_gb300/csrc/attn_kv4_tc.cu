// tree_verify_attn_kv4, tensor-core path (bf16 rows, d = 64 or 128).
//
// The products are taken transposed, so that the 128 tensor-memory lanes of an
// MMA are keys and dims, not query rows:
//   S^T [keys x rows] = K Q^T          A = K   (lanes: keys, 32-bit columns: dim pairs)
//   O^T [dims x rows] += V^T (s_v P)^T A = V^T (lanes: dims, columns: key pairs)
// A tile then costs N = 16, 32 or 64 columns for its query rows (nodes x the
// heads of one KV head): a single token pays for 16, not for 128 rows.  Both A
// operands are tensor-memory operands that the dequantising warps write
// straight from registers: a thread owns one key (or one dim), reads its code
// words from the staged block, turns each into four bf16 pairs
//   n = bf16x2((w >> 4i) & 0x000f000f | 0x43004300) - 136      (128 + code - 136)
// and stores them; shared memory carries the codes once (132 bytes per token)
// and the small B operands.  n is exact in bf16, the scales are applied in
// fp32: s_k to the scores, s_v to the weights before their rounding to bf16.
//
// Softmax: a thread owns one key of the tile, so its s_k, s_v and visibility
// are scalars; row maxima run across lanes, which a tile only pays for when a
// score exceeds the row's running reference by 2^8 (then every weight is
// rescaled); one vote per tile decides.  Row sums stay in registers, one per
// thread and row, until the end of the unit.
//
// Work: a unit is (request, row tile, KV head); its key tiles of 128 (cached
// tokens, then the tree's nodes) follow one another, and the list of all units
// is cut into equal runs, one per CTA (one CTA per SM).  A unit cut by a run's
// end leaves fp32 partials that a second kernel joins in run order, so results
// do not depend on timing.
//
// Roles: warps 0-3 keys, 4-7 values, then one or two softmax warpgroups (up to
// 32 rows each), one MMA issuer, one producer (bulk copies of whole (page,
// head) blocks into a ring).  K, V, S and P are double-buffered.
//
// Every wait is bounded (2 s): on expiry the CTA records an error code in the
// workspace status word and stops; tensor memory is always released.
#include <algorithm>

#include "kv4.cuh"
#include "kv4_device.cuh"

namespace tv {
namespace kv4 {
namespace {

using namespace tc;

constexpr int kKeys = 128;        // keys per tile
constexpr int kStages = 6;        // staged tiles

enum Bar { RAW_FULL = 0, RAW_EMPTY = RAW_FULL + kStages, K_FULL = RAW_EMPTY + kStages, V_FULL = K_FULL + 2,
           S_FULL = V_FULL + 2, S_FREE = S_FULL + 2, P_FULL = S_FREE + 2, PV_DONE = P_FULL + 2, DRAIN = PV_DONE + 2,
           N_BARS = DRAIN + 1 };

// What the producer says about a staged tile.
struct alignas(16) Tile {
  int flags;         // kFirst ..
  int key0, nkeys;   // first token (node) of the tile, how many
  int groups;        // bit i: the page of tokens 16 i .. 16 i + 15 of the tile is staged
  int r, t, h;       // request, row tile, KV head
  int seg;           // running number of the unit in this CTA
  int n0, cnt;       // first node of the request, nodes
  int slot;          // -1: the whole unit is here; else its partial slot
};
enum { kFirst = 1, kLast = 2, kTree = 4, kEnd = 8 };   // first, last tile of its unit's run here; tree nodes; no more

template <int D, int N>
struct Lay {
  static constexpr int kGroups = N > 32 ? 2 : 1;              // softmax warpgroups
  static constexpr int kCols = N / kGroups;                   // rows per softmax warpgroup
  static constexpr int kSoft0 = 8;                            // first softmax warp
  static constexpr int kMma = kSoft0 + 4 * kGroups;
  static constexpr int kProd = kMma + 1;
  static constexpr int kWarps = kProd + 1;
  static constexpr int kThreads = 32 * kWarps;
  // Registers a thread: the compiler's share at launch (65536 over warps that
  // come four to a scheduler), what the dequantising warps give up and what
  // the softmax warps take.
  static constexpr int kLaunchRegs = kWarps <= 16 ? 128 : 96;
  static constexpr int kConvRegs = kWarps <= 16 ? 80 : 56;
  static constexpr int kSoftRegs = kWarps <= 16 ? 192 : 136;
  static_assert(8 * kConvRegs + 4 * kGroups * kSoftRegs + 2 * kLaunchRegs <= kWarps * kLaunchRegs, "register split");
  static constexpr uint32_t kStage = kKeys * (D + 4);
  static constexpr uint32_t kQHalf = N * 128;                 // N rows x 64 dims
  static constexpr uint32_t kQ = 0;                           // two buffers
  static constexpr uint32_t kQBytes = (D / 64) * kQHalf;
  static constexpr uint32_t kP = kQ + 2 * kQBytes;            // two buffers of 128 keys x 64 rows
  static constexpr uint32_t kPBytes = kKeys * 128;
  static constexpr uint32_t kRaw = kP + 2 * kPBytes;
  static constexpr uint32_t kTiles = kRaw + kStages * kStage;             // Tile per stage
  static constexpr uint32_t kBars = kTiles + kStages * 64;
  static constexpr uint32_t kMisc = kBars + 8 * 32;                       // tmem slot, abort, start, dirty
  static constexpr uint32_t kRef = kMisc + 64;                            // float [2][N] running references
  static constexpr uint32_t kCorr = kRef + 8 * N;                         // float [N]
  static constexpr uint32_t kInv = kCorr + 4 * N;                         // float [N]
  static constexpr uint32_t kVis = kInv + 4 * N;                          // int [N]
  static constexpr uint32_t kRow = kVis + 4 * N;                          // int [N] output row, -1: none
  static constexpr uint32_t kAnc = kRow + 4 * N;                          // u32 [4][N]
  static constexpr uint32_t kWarpMax = kAnc + 16 * N;                     // [groups][4][32]
  static constexpr uint32_t kSums = kWarpMax + 512 * kGroups;             // long long [kWarps]
  static constexpr uint32_t kBytes = kSums + 8 * kWarps + 1024;           // + alignment slack
  static_assert(sizeof(Tile) == 48 && N_BARS <= 32 && kRef % 16 == 0 && kSums % 8 == 0, "layout");
  // tensor memory: K0 K1 V0 V1 (64 columns each), S0 S1 (N each), O (N)
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t tK = 0, tV = 128, tS = 256, tO = 256 + 2 * N;
};

struct TcArgs {
  AttnArgs a;
  int* status;
  int4* desc;        // [grid] pieces of the unit that starts in a CTA and ends in another
  float2* ml;        // [2 grid][N]
  float* o;          // [2 grid][N][D]
  const int4* extents;   // [B * tiles] from extent_kernel, or NULL
  int nq, tiles, grid;
  uint32_t magic;        // kMagic
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16]) { tmem_st16(taddr, r); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[32]) { tmem_st32(taddr, r); }
// Barrier of one softmax warpgroup, and the same with an OR over its threads.
__device__ __forceinline__ void wg_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool wg_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(p))
      : "memory");
  return r != 0;
}
// Key tiles of a row tile (entry = request x row tile): prefix tiles over the
// tokens that any of its rows sees, then tree tiles from the lowest visible
// node on.  They follow from the lengths alone unless nodes have prefixes of
// their own or the tree spans several key tiles; then extent_kernel works them
// out first.
struct Extent {
  int len, np, t0, nt;    // visible prefix, prefix tiles, first tree tile, tree tiles
};
__device__ __forceinline__ Extent extent_of(const TcArgs& p, int e) {
  if (p.extents) {
    const int4 v = p.extents[e];
    return Extent{v.x, (v.x + kKeys - 1) / kKeys, v.y, v.z};
  }
  const int r = e / p.tiles;
  const bool live = e % p.tiles * p.nq < node_span(p.a, r).cnt;
  const int len = prefix_len(p.a, r);
  return Extent{len, live ? (len + kKeys - 1) / kKeys : 0, 0, live ? 1 : 0};
}
// One warp per entry, lanes = nodes.
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
  const int top = live ? (s.cnt - 1) / kKeys : 0;
  const int t0 = min(lo / 2, top), nt = live ? max(0, min(hi / 2, top) - t0) + 1 : 0;
  if (lane == 0) out[e] = make_int4(live ? vis : 0, t0, nt, 0);
}
// Tiles of entry e, all KV heads; 0 past the end.
__device__ __forceinline__ long long entry_tiles(const TcArgs& p, int e, int end) {
  if (e >= end) return 0;
  const Extent x = extent_of(p, e);
  return static_cast<long long>(x.np + x.nt) * p.a.Hkv;
}
__device__ __forceinline__ long long warp_sum_ll(long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D, int N>
__global__ void __launch_bounds__(Lay<D, N>::kThreads, 1) attn_kernel(const __grid_constant__ TcArgs p) {
  using L = Lay<D, N>;
  constexpr int C = L::kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(sm);
  const AttnArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = a.Hq / a.Hkv;
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sm + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kMisc + 4);
  volatile int* dirty = reinterpret_cast<volatile int*>(sm + L::kMisc + 32);   // [4] seg + 1 of a unit with non-finite values
  long long* sums = reinterpret_cast<long long*>(sm + L::kSums);
  long long* start = reinterpret_cast<long long*>(sm + L::kMisc + 8);          // [2]: entry, tiles before it
  auto bar = [&](int i) { return sb + L::kBars + 8u * i; };
  if (threadIdx.x == 0) {
    for (int i = 0; i < N_BARS; ++i) {
      uint32_t c = 1;
      if (i >= RAW_EMPTY && i < RAW_EMPTY + kStages) c = 8 + 4 * L::kGroups + 1;
      if ((i >= K_FULL && i < K_FULL + 2) || (i >= V_FULL && i < V_FULL + 2)) c = 4;
      if ((i >= S_FREE && i < S_FREE + 2) || (i >= P_FULL && i < P_FULL + 2)) c = 4 * L::kGroups;
      mbar_init(bar(i), c);
    }
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) dirty[i] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  griddep_wait();
  griddep_release();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = 0;   // an expired wait writes it seconds later
  if (warp == L::kMma) {
    __syncwarp();
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sb + L::kMisc),
                 "r"(L::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // ---- this CTA's run: tiles [w0, w1) of the list of all units
  const int E = a.B * p.tiles;
  const int per = ((E + L::kWarps - 1) / L::kWarps + 31) / 32 * 32;     // entries per warp
  const int e_lo = min(warp * per, E), e_hi = min(e_lo + per, E);
  {
    long long s = 0;
    for (int e = e_lo; e < e_hi; e += 32) s += entry_tiles(p, e + lane, e_hi);
    s = warp_sum_ll(s);
    if (lane == 0) sums[warp] = s;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  long long W = 0, before = 0;
  for (int w = 0; w < L::kWarps; ++w) {
    if (w == warp) before = W;
    W += sums[w];
  }
  const long long G = min(static_cast<long long>(p.grid), W);
  const long long w0 = G > 0 ? blockIdx.x * W / G : 0, w1 = G > 0 ? (blockIdx.x + 1) * W / G : 0;
  const bool work = blockIdx.x < G;
  if (work && w0 >= before && w0 < before + sums[warp]) {   // this warp's entries hold the first tile
    long long at = before;
    for (int e = e_lo; e < e_hi; e += 32) {
      const long long c = entry_tiles(p, e + lane, e_hi);
      long long x = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const long long mine = at + x - c;
      if (w0 >= mine && w0 < mine + c) {
        start[0] = e + lane;
        start[1] = mine;
      }
      at += __shfl_sync(0xffffffffu, x, 31);
      if (at > w0) break;
    }
  }
  if (threadIdx.x == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  __syncthreads();

  int* err = p.status;
  uint8_t* raw = sm + L::kRaw;
  auto tile_at = [&](int st) -> const Tile& { return *reinterpret_cast<const Tile*>(sm + L::kTiles + 64 * st); };
  const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  const int own = 32 * (warp & 3) + lane;        // key (or dim) of a thread of the four-warp roles
  const uint32_t blk_bytes = static_cast<uint32_t>(a.page_size) * (D + 4);
  const int ps_shift = 31 - __clz(a.page_size);

  if (!work) {
    // nothing to do
  } else if (warp == L::kProd) {
    // ================= producer
    int e = static_cast<int>(start[0]);
    long long pos = w0;
    Extent x = extent_of(p, e);
    int nb = x.np + x.nt;
    const long long off = w0 - start[1];
    int h = static_cast<int>(off / nb), blk = static_cast<int>(off % nb);
    int seg = 0, seg_blk = blk;                  // first tile of the running unit in this CTA
    const int per_tile = kKeys >> ps_shift;      // pages of a tile
    int issued = 0;
    // Pass it works out tile it and asks for its pages' numbers, then issues
    // tile it - 1, whose numbers have arrived meanwhile.
    Tile cur, nx;
    int page = -1, npage = -1;
    cur.flags = nx.flags = 0;
    for (int it = 0;; ++it) {
      if (!(nx.flags & kEnd)) {
        npage = -1;
        if (pos >= w1) {
          nx.flags = kEnd;
        } else {
          if (blk == nb) {                       // next unit
            blk = seg_blk = 0;
            ++seg;
            if (++h == a.Hkv) {
              h = 0;
              do {
                x = extent_of(p, ++e);
                nb = x.np + x.nt;
              } while (nb == 0 && e + 1 < E);
            }
          }
          nx.r = e / p.tiles;
          nx.t = e % p.tiles;
          const Span sp = node_span(a, nx.r);
          const bool tree = blk >= x.np;
          nx.h = h;
          nx.n0 = sp.n0;
          nx.cnt = sp.cnt;
          nx.seg = seg;
          const bool last = blk == nb - 1 || pos == w1 - 1;
          const bool whole = seg_blk == 0 && pos + (nb - 1 - blk) < w1;
          nx.flags = (blk == seg_blk ? kFirst : 0) | (last ? kLast : 0) | (tree ? kTree : 0);
          nx.slot = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (seg_blk == 0 ? 1 : 0);
          if (!tree) {
            nx.key0 = blk * kKeys;
            nx.nkeys = min(kKeys, x.len - nx.key0);
            if (lane < per_tile && (lane << ps_shift) < nx.nkeys)
              npage = a.block_table[static_cast<int64_t>(nx.r) * a.table_ld + (nx.key0 >> ps_shift) + lane];
          } else {
            nx.key0 = (x.t0 + blk - x.np) * kKeys;
            nx.nkeys = min(kKeys, sp.cnt - nx.key0);
          }
          if (last && blk != nb - 1 && seg_blk == 0 && lane == 0) {
            // a unit that starts here and goes on: its pieces, for the joining kernel
            const long long u1 = pos + (nb - blk);           // position after the unit
            const long long k = (u1 * G + W - 1) / W - 1;    // CTA of its last tile
            p.desc[blockIdx.x] = make_int4(static_cast<int>(k) - static_cast<int>(blockIdx.x) + 1, nx.r, nx.t, h);
          }
          ++blk;
          ++pos;
        }
      }
      if (it > 0) {
        const int i = it - 1, st = i % kStages;
        if (i >= kStages && !warp_wait(bar(RAW_EMPTY + st), ((i / kStages) - 1) & 1, abort_flag, err, 41)) break;
        const bool wanted = !(cur.flags & (kTree | kEnd)) && lane < per_tile && (lane << ps_shift) < cur.nkeys;
        const bool good = wanted && page >= 0 && page < a.n_pages;
        if (wanted && !good && a.err) *a.err = 1;
        const unsigned have = __ballot_sync(0xffffffffu, good);
        if (lane == 0) {
          Tile* t = reinterpret_cast<Tile*>(sm + L::kTiles + 64 * st);
          cur.groups = 0;
          for (int gr = 0; gr < 8; ++gr) cur.groups |= ((have >> ((16 * gr) >> ps_shift)) & 1) << gr;
          *t = cur;
          if (have)
            mbar_expect_tx(bar(RAW_FULL + st), __popc(have) * blk_bytes);
          else
            mbar_arrive(bar(RAW_FULL + st));
        }
        __syncwarp();
        if (good)
          bulk_load(sb + L::kRaw + st * L::kStage + lane * blk_bytes,
                    a.cache + (static_cast<int64_t>(page) * a.Hkv + cur.h) * blk_bytes, blk_bytes, bar(RAW_FULL + st));
        issued = it;
        if (cur.flags & kEnd) break;
      }
      cur = nx;
      page = npage;
    }
    // after an expired wait: copies in flight land before the CTA ends
    if (*abort_flag) {
      for (int it = max(0, issued - kStages); it < issued; ++it) {
        const long long t0 = clock64();
        while (!mbar_try(bar(RAW_FULL + it % kStages), (it / kStages) & 1) && clock64() - t0 < kWaitClocks) {
        }
      }
    }
  } else if (warp == L::kMma) {
    // ================= MMA issuer (event loop)
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16(128, N, 0);
      constexpr uint32_t idO = idesc_bf16(128, N, 1);
      int ns = 0, npv = 0, total = -1;
      uint32_t firsts = 0;                       // bit j & 7: tile j is the first of its unit
      uint32_t idle = 0;                         // polls without progress
      long long since = 0;
      bool ok = true;
      while (ok && (total < 0 || npv < total)) {
        bool prog = false;
        if (total < 0 && mbar_test(bar(RAW_FULL + ns % kStages), (ns / kStages) & 1)) {
          const Tile& t = tile_at(ns % kStages);
          if (t.flags & kEnd) {
            total = ns;
            prog = true;
          } else if (mbar_test(bar(K_FULL + (ns & 1)), (ns >> 1) & 1) &&
                     (ns < 2 || mbar_test(bar(S_FREE + (ns & 1)), ((ns >> 1) - 1) & 1))) {
            tc_fence_after();
            const uint32_t q = sb + L::kQ + (t.seg & 1) * L::kQBytes;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_bf16_ts(tmem + L::tS + N * (ns & 1), tmem + L::tK + 64 * (ns & 1) + 8 * kk,
                           sdesc(q + (kk >> 2) * L::kQHalf + (kk & 3) * 32, 16, 1024), idS, kk > 0);
            umma_commit(bar(S_FULL + (ns & 1)));
            firsts = (firsts & ~(1u << (ns & 7))) | (static_cast<uint32_t>(t.flags & kFirst) << (ns & 7));
            mbar_arrive(bar(RAW_EMPTY + ns % kStages));
            ++ns;
            prog = true;
          }
        }
        if (npv < ns && mbar_test(bar(P_FULL + (npv & 1)), (npv >> 1) & 1) &&
            mbar_test(bar(V_FULL + (npv & 1)), (npv >> 1) & 1)) {
          tc_fence_after();
          const uint32_t pb = sb + L::kP + (npv & 1) * L::kPBytes;
          const uint32_t first = (firsts >> (npv & 7)) & 1u;
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            umma_bf16_ts(tmem + L::tO, tmem + L::tV + 64 * (npv & 1) + 8 * kk, sdesc(pb + kk * 2048, L::kPBytes, 1024),
                         idO, (first && kk == 0) ? 0u : 1u);
          umma_commit(bar(PV_DONE + (npv & 1)));
          ++npv;
          prog = true;
        }
        if (prog) {
          idle = 0;
        } else if ((++idle & 255) == 0) {
          if (idle == 256) since = clock64();
          if (*abort_flag) {
            ok = false;
          } else if (clock64() - since > kWaitClocks) {
            *abort_flag = 1;
            atomicExch(err, 42);
            ok = false;
          }
        }
      }
      umma_commit(bar(DRAIN));
      if (!mbar_try(bar(DRAIN), 0)) wait_slow(bar(DRAIN), 0, abort_flag, err, 43);
    }
  } else if (warp < 4) {
    // ================= keys: thread = key
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kConvRegs));
    for (int it = 0;; ++it) {
      const int st = it % kStages, b = it & 1;
      if (!warp_wait(bar(RAW_FULL + st), (it / kStages) & 1, abort_flag, err, 44)) break;
      const Tile& t = tile_at(st);
      const int flags = t.flags;
      if (flags & kEnd) break;
      // S(it - 2) has read this K buffer, and every S of the unit before last its Q buffer
      if (it >= 2 &&
          !warp_wait(bar(S_FULL + b), ((it >> 1) - 1) & 1, abort_flag, err, 45))
        break;
      tc_fence_after();
      if (flags & kFirst) {
        uint8_t* qs = sm + L::kQ + (t.seg & 1) * L::kQBytes;
        const int node0 = t.t * p.nq, rows = min(p.nq, t.cnt - node0) * g;
#pragma unroll 2
        for (int i = threadIdx.x; i < N * (D / 8); i += 128) {
          const int rr = i / (D / 8), c = i % (D / 8);
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (rr < rows)
            v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                static_cast<int64_t>(t.n0 + node0 + rr / g) * a.ldq +
                                                static_cast<int64_t>(t.h * g + rr % g) * D + 8 * c);
          *reinterpret_cast<uint4*>(qs + (c >> 3) * L::kQHalf + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = v;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      const uint32_t dst = tmem + L::tK + 64 * b + lane_off;
      if (!(flags & kTree)) {
        const uint8_t* blk = raw + st * L::kStage + (own >> ps_shift) * blk_bytes;
        const int slot = own & (a.page_size - 1);
        const uint4* from = reinterpret_cast<const uint4*>(blk + slot * 16);
        uint4 w = *from;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {       // rolled: the roles share the instruction caches
          uint32_t r[16];
          const uint4 now = w;
          from += a.page_size;
          if (c + 1 < D / 32) w = *from;
          decode8(now.x, r, p.magic);
          decode8(now.y, r + 4, p.magic);
          decode8(now.z, r + 8, p.magic);
          decode8(now.w, r + 12, p.magic);
          tmem_st16(dst + 16 * c, r);
        }
      } else {
        const bool live = own < t.nkeys;
        const uint16_t* row = static_cast<const uint16_t*>(a.k_tree) +
                              static_cast<int64_t>(t.n0 + t.key0 + (live ? own : 0)) * a.ldk +
                              static_cast<int64_t>(t.h) * D;
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint32_t r[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 w = live ? *reinterpret_cast<const uint4*>(row + 64 * c + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
            r[4 * i] = w.x; r[4 * i + 1] = w.y; r[4 * i + 2] = w.z; r[4 * i + 3] = w.w;
          }
          tmem_st32(dst + 32 * c, r);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(K_FULL + b));
        mbar_arrive(bar(RAW_EMPTY + st));
      }
    }
  } else if (warp < 8) {
    // ================= values: thread = dim
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kConvRegs));
    for (int it = 0;; ++it) {
      const int st = it % kStages, b = it & 1;
      if (!warp_wait(bar(RAW_FULL + st), (it / kStages) & 1, abort_flag, err, 46)) break;
      const Tile& t = tile_at(st);
      const int flags = t.flags;
      if (flags & kEnd) break;
      if (it >= 2 &&
          !warp_wait(bar(PV_DONE + b), ((it >> 1) - 1) & 1, abort_flag, err, 47))
        break;
      tc_fence_after();
      const uint32_t dst = tmem + L::tV + 64 * b + lane_off;
      if (32 * (warp & 3) < D) {                 // d = 64: the upper lanes' results are not used
        if (!(flags & kTree)) {
          const uint8_t* base = raw + st * L::kStage + a.page_size * (D / 2) + own * 8;
          const int gshift = ps_shift - 4;       // groups of 16 tokens per page
          auto word = [&](int gr) {
            return *reinterpret_cast<const uint2*>(base + (gr >> gshift) * blk_bytes +
                                                   (gr & ((1 << gshift) - 1)) * (D * 8));
          };
          uint2 w0 = word(0), w1 = word(1);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t r[16];
            const uint2 a0 = w0, a1 = w1;
            if (c < 3) {
              w0 = word(2 * c + 2);
              w1 = word(2 * c + 3);
            }
            decode8(a0.x, r, p.magic);
            decode8(a0.y, r + 4, p.magic);
            decode8(a1.x, r + 8, p.magic);
            decode8(a1.y, r + 12, p.magic);
            tmem_st16(dst + 16 * c, r);
          }
        } else {
          // a value that is not finite must not meet the zero weights of rows that do not see it: it is taken
          // out here and added at the end to the rows that see it
          const int nk = t.nkeys;
          const uint16_t* col = static_cast<const uint16_t*>(a.v_tree) +
                                static_cast<int64_t>(t.n0 + t.key0) * a.ldv + static_cast<int64_t>(t.h) * D + own;
          bool bad = false;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t r[16];
            const uint16_t* from = col + static_cast<int64_t>(32 * c) * a.ldv;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int k0 = 32 * c + 2 * i;
              uint32_t lo = 0u, hi = 0u;         // (a part without nodes is stored as zeros)
              if (k0 < nk) lo = *from;
              from += a.ldv;
              if (k0 + 1 < nk) hi = *from;
              from += a.ldv;
              if ((lo & 0x7f80u) == 0x7f80u) { lo = 0u; bad = true; }
              if ((hi & 0x7f80u) == 0x7f80u) { hi = 0u; bad = true; }
              r[i] = lo | (hi << 16);
            }
            tmem_st16(dst + 16 * c, r);
          }
          if (bad) dirty[t.seg & 3] = t.seg + 1;
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(V_FULL + b));
        mbar_arrive(bar(RAW_EMPTY + st));
      }
    }
  } else {
    // ================= softmax: thread = key, columns = rows c0 .. c0 + C - 1 of the row tile
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kSoftRegs));
    const int wg = (warp - L::kSoft0) >> 2, wid = 1 + wg;
    const int c0 = wg * C;
    const float c2 = a.scale * kLog2e;
    // a row's reference (what its scores are taken over) is kept negated; -0 (and a row sum of 0): none yet
    float* nref = reinterpret_cast<float*>(sm + L::kRef) + c0;
    float* shift_s = nref + N;
    float* corr_s = reinterpret_cast<float*>(sm + L::kCorr) + c0;
    float* inv_s = reinterpret_cast<float*>(sm + L::kInv) + c0;
    int* vis_s = reinterpret_cast<int*>(sm + L::kVis) + c0;
    int* row_s = reinterpret_cast<int*>(sm + L::kRow) + c0;
    uint32_t* anc_s = reinterpret_cast<uint32_t*>(sm + L::kAnc) + c0;   // [4][N]
    int* wmax = reinterpret_cast<int*>(sm + L::kWarpMax) + wg * 128;
    const int tid = threadIdx.x - 32 * L::kSoft0 - 128 * wg;    // 0..127 in the warpgroup
    uint64_t l[C / 2];                                          // this key's share of the rows' sums
#pragma unroll
    for (int c = 0; c < C / 2; ++c) l[c] = 0ull;
    bool force = false;                                         // a row of the unit has no reference yet
    for (int it = 0;; ++it) {
      const int st = it % kStages, b = it & 1;
      if (!warp_wait(bar(RAW_FULL + st), (it / kStages) & 1, abort_flag, err, 48)) break;
      const Tile t = tile_at(st);
      if (t.flags & kEnd) break;
      const bool first = t.flags & kFirst, last = t.flags & kLast, tree = t.flags & kTree;
      float sk = c2, sv = 1.f;
      bool valid = own < t.nkeys;
      if (!tree) {
        valid = valid && ((t.groups >> (own >> 4)) & 1);
        const uint8_t* blk = raw + st * L::kStage + (own >> ps_shift) * blk_bytes;
        const int slot = own & (a.page_size - 1);
        sk = valid ? c2 * bf16_at(reinterpret_cast<const uint16_t*>(blk + k_scale(a.page_size, D, slot))) : 0.f;
        sv = valid ? bf16_at(reinterpret_cast<const uint16_t*>(blk + v_scale(a.page_size, D, slot))) : 0.f;
      }
      const int key = valid && !tree ? t.key0 + own : 0x7fffffff;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(RAW_EMPTY + st));
      if (first || tree) {
        wg_sync(wid);                            // the unit (tile) before is done with these arrays
        if (tid < C) {
          const int rr = c0 + tid, ln = t.t * p.nq + rr / g;
          const bool live = rr < p.nq * g && ln < t.cnt;
          const int gn = t.n0 + ln;
          if (first) {
            nref[tid] = -0.f;
            row_s[tid] = live ? gn * a.Hq + t.h * g + rr % g : -1;
            vis_s[tid] = live ? (a.vis_prefix ? a.vis_prefix[gn] : 0x7fffffff) : 0;
          }
          if (tree) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int word = (t.key0 >> 6) + w;
              const uint64_t v = live && word < a.anc_words ? a.anc[static_cast<int64_t>(gn) * a.anc_words + word] : 0ull;
              anc_s[(2 * w) * N + tid] = static_cast<uint32_t>(v);
              anc_s[(2 * w + 1) * N + tid] = static_cast<uint32_t>(v >> 32);
            }
          }
        }
        wg_sync(wid);
      }
      if (!warp_wait(bar(S_FULL + b), (it >> 1) & 1, abort_flag, err, 49)) break;
      tc_fence_after();
      // scores in base-2 units over the rows' references, two rows to a register pair; -inf: not seen
      uint64_t y[C / 2];
      {
        uint32_t x[C];
        tmem_ld(tmem + L::tS + N * b + c0 + lane_off, x);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < C; ++c) pin(x[c]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(S_FREE + b));
        const uint64_t sk2 = pair(sk, sk);
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(nref + c);
          y[c / 2] = fma2(pair(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sk2, m.x);
          y[c / 2 + 1] = fma2(pair(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sk2, m.y);
        }
      }
      if (__builtin_expect(tree || a.vis_prefix != nullptr || !__all_sync(0xffffffffu, valid), 0)) {
        const uint32_t* words = anc_s + (warp & 3) * N;
#pragma unroll
        for (int c = 0; c < C; c += 2) {
          float lo, hi;
          split(y[c / 2], lo, hi);
          const bool s0 = tree ? valid && ((words[c] >> lane) & 1u) : key < vis_s[c];
          const bool s1 = tree ? valid && ((words[c + 1] >> lane) & 1u) : key < vis_s[c + 1];
          y[c / 2] = pair(s0 ? lo : -INFINITY, s1 ? hi : -INFINITY);
        }
      }
      bool slow = first || force;
      if (!slow) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < C / 2; ++c) {
          float lo, hi;
          split(y[c], lo, hi);
          mx[c & 1] = max3(mx[c & 1], lo, hi);
        }
        slow = wg_any(wid, fmaxf(mx[0], mx[1]) > 8.f);
      }
      if (__builtin_expect(slow, 0)) {
        // new references: the rows' maxima so far
        int mine = static_cast<int>(0x80000000);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float lo, hi;
          split(y[c / 2], lo, hi);
          int v = __float_as_int(c & 1 ? hi : lo);
          v ^= (v >> 31) & 0x7fffffff;           // order of floats as order of integers
          v = __reduce_max_sync(0xffffffffu, v);
          if ((lane & (C - 1)) == c) mine = v;
        }
        if (lane < C) wmax[(warp & 3) * 32 + lane] = mine;
        wg_sync(wid);
        bool none = false;
        float sh = 0.f, next = 0.f;
        if (lane < C) {                          // every warp works out the same
          int v = wmax[lane];
#pragma unroll
          for (int w = 1; w < 4; ++w) v = max(v, wmax[32 * w + lane]);
          v ^= (v >> 31) & 0x7fffffff;
          const float top = __int_as_float(v), old = nref[lane];
          const bool unset = __float_as_uint(old) == 0x80000000u;
          sh = unset ? (top == -INFINITY ? 0.f : top) : fmaxf(top, 0.f);
          if (top != top) sh = top;
          next = unset && top == -INFINITY ? -0.f : old - sh;
          none = row_s[lane] >= 0 && unset && top == -INFINITY;
          corr_s[lane] = unset ? 0.f : ex2(-sh);
          shift_s[lane] = -sh;
        }
        force = __any_sync(0xffffffffu, none);
        wg_sync(wid);                            // all have read the old references
        if (lane < C) nref[lane] = next;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(shift_s + c);
          const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(corr_s + c);
          y[c / 2] = add2(y[c / 2], m.x);
          y[c / 2 + 1] = add2(y[c / 2 + 1], m.y);
          l[c / 2] = mul2(l[c / 2], f.x);
          l[c / 2 + 1] = mul2(l[c / 2 + 1], f.y);
        }
        if (!first) {
          if (!warp_wait(bar(PV_DONE + (b ^ 1)), ((it - 1) >> 1) & 1, abort_flag, err, 50)) break;
          tc_fence_after();
          uint32_t o[C];
          tmem_ld(tmem + L::tO + c0 + lane_off, o);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < C; ++c) {
            pin(o[c]);
            o[c] = __float_as_uint(__uint_as_float(o[c]) * corr_s[c]);
          }
          tmem_st(tmem + L::tO + c0 + lane_off, o);
          tmem_st_wait();
          tc_fence_before();
        }
      }
      // weights
      uint32_t pk[C / 2];
      const uint64_t sv2 = pair(sv, sv);
#pragma unroll
      for (int c = 0; c < C / 2; ++c) {
        float lo, hi;
        split(y[c], lo, hi);
        const uint64_t e = pair(ex2(lo), ex2(hi));
        l[c] = add2(l[c], e);
        split(mul2(e, sv2), lo, hi);
        pk[c] = pack_bf16(lo, hi);
      }
      if (__builtin_expect(sv != sv && a.vis_prefix != nullptr, 0)) {
        // a value row that was not finite: zero weights times its scale are NaN, rows that do not see it stay clean
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (key >= vis_s[c]) pk[c >> 1] &= c & 1 ? 0x0000ffffu : 0xffff0000u;
      }
      if (it >= 2 && !warp_wait(bar(PV_DONE + b), ((it >> 1) - 1) & 1, abort_flag, err, 51)) break;
      uint8_t* prow = sm + L::kP + b * L::kPBytes + own * 128;
#pragma unroll
      for (int c = 0; c < C / 8; ++c)
        *reinterpret_cast<uint4*>(prow + (((c0 / 8 + c) ^ (own & 7)) << 4)) =
            make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      // the value warps' note on non-finite tree rows, read at the end of the unit (V's phase cannot move on
      // before P is given away)
      if (last && tree && !warp_wait(bar(V_FULL + b), (it >> 1) & 1, abort_flag, err, 53)) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(P_FULL + b));
      if (__builtin_expect(!last, 1)) continue;

      // ---- end of the unit's run here: sums over the keys' threads, then O^T
      float ls[C];
#pragma unroll
      for (int c = 0; c < C / 2; ++c) {
        split(l[c], ls[2 * c], ls[2 * c + 1]);
        l[c] = 0ull;
      }
      force = false;
      // reduce-scatter over the lanes: lane i ends with column i % C
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        if (o >= C) {
#pragma unroll
          for (int c = 0; c < C; ++c) ls[c] += __shfl_xor_sync(0xffffffffu, ls[c], o);
        } else {
          const bool up = lane & o;
#pragma unroll
          for (int c = 0; c < o; ++c) {
            const float keep = up ? ls[c + o] : ls[c], give = up ? ls[c] : ls[c + o];
            ls[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
      }
      if (lane < C) wmax[(warp & 3) * 32 + lane] = __float_as_int(ls[0]);
      wg_sync(wid);
      if (lane < C) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) sum += __int_as_float(wmax[32 * w + lane]);
        inv_s[lane] = t.slot >= 0 ? 1.f : (sum == 0.f ? 0.f : 1.f / sum);   // partials stay unnormalised
        if ((warp & 3) == 0) {
          const float m = -nref[lane];
          if (t.slot >= 0) {
            p.ml[static_cast<int64_t>(t.slot) * N + c0 + lane] = make_float2(sum == 0.f ? kLow : m, sum);
          } else if (a.lse && row_s[lane] >= 0) {
            a.lse[row_s[lane]] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
          }
        }
      }
      __syncwarp();
      if (!warp_wait(bar(PV_DONE + b), (it >> 1) & 1, abort_flag, err, 52)) break;
      tc_fence_after();
      uint32_t o[C];
      tmem_ld(tmem + L::tO + c0 + lane_off, o);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < C; ++c) pin(o[c]);
      tc_fence_before();                         // O was read: the next unit's first PV may overwrite it
      if (own < D) {
        if (t.slot >= 0) {
          float* po = p.o + (static_cast<int64_t>(t.slot) * N + c0) * D + own;
#pragma unroll
          for (int c = 0; c < C; ++c)
            if (row_s[c] >= 0) po[c * D] = __uint_as_float(o[c]);
        } else {
          uint16_t* out = static_cast<uint16_t*>(a.out) + own;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int row = row_s[c];
            if (row >= 0) {
              const float f = __uint_as_float(o[c]) * inv_s[c];
              out[static_cast<int64_t>(row) * D] = static_cast<uint16_t>(pack_bf16(f, 0.f));
            }
          }
        }
        if (__builtin_expect(dirty[t.seg & 3] == t.seg + 1, 0)) {
          // tree values that are not finite, added to the rows that see them (this thread wrote these elements)
          const uint16_t* col = static_cast<const uint16_t*>(a.v_tree) + static_cast<int64_t>(t.n0) * a.ldv +
                                static_cast<int64_t>(t.h) * D + own;
#pragma unroll 1
          for (int j = 0; j < min(t.cnt, 64 * a.anc_words); ++j) {
            const uint32_t v = col[static_cast<int64_t>(j) * a.ldv];
            if ((v & 0x7f80u) != 0x7f80u) continue;
#pragma unroll 1
            for (int c = 0; c < C; ++c) {
              const int row = row_s[c];
              if (row < 0) continue;
              const uint64_t word = a.anc[static_cast<int64_t>(row / a.Hq) * a.anc_words + (j >> 6)];
              if (!((word >> (j & 63)) & 1ull)) continue;
              const float f = __uint_as_float(v << 16);
              if (t.slot >= 0) {
                p.o[(static_cast<int64_t>(t.slot) * N + c0 + c) * D + own] += f;
              } else {
                uint16_t* o16 = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(row) * D + own;
                *o16 = static_cast<uint16_t>(pack_bf16(bf16_at(o16) + f, 0.f));
              }
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == L::kMma) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(L::kTmemCols) : "memory");
  }
}

// Joins the pieces of a unit that was cut: piece 0 is slot 1 of the CTA where
// the unit starts, piece i slot 0 of the i-th CTA after it.  CTA = (starting
// CTA, eight rows), thread = four dims of a row.
template <int D>
__global__ void __launch_bounds__(2 * D) join_kernel(const TcArgs p, int N) {
  griddep_wait();
  griddep_release();
  const int4 d = p.desc[blockIdx.x];
  if (d.x < 2) return;
  const AttnArgs& a = p.a;
  const int g = a.Hq / a.Hkv, c = blockIdx.y * 8 + threadIdx.x / (D / 4), dim = threadIdx.x % (D / 4) * 4;
  const Span s = node_span(a, d.y);
  if (c >= min(p.nq, s.cnt - d.z * p.nq) * g) return;
  auto slot = [&](int i) {
    return static_cast<int64_t>(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * N + c;
  };
  float M = kLow, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kAhead = 4;                      // pieces whose loads are in flight together
  for (int i0 = 0; i0 < d.x; i0 += kAhead) {
    float2 ml[kAhead];
    float4 o[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      ml[k] = make_float2(kLow, 0.f);
      if (i0 + k < d.x) {
        ml[k] = p.ml[slot(i0 + k)];
        o[k] = *reinterpret_cast<const float4*>(p.o + slot(i0 + k) * D + dim);
      }
    }
    const float old = M;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) M = fmaxf(M, ml[k].x);
    const float keep = ex2(old - M);
    sum *= keep;
    acc.x *= keep; acc.y *= keep; acc.z *= keep; acc.w *= keep;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (ml[k].y == 0.f) continue;              // nothing seen in this piece
      const float w = ex2(ml[k].x - M);
      sum = fmaf(w, ml[k].y, sum);
      acc.x = fmaf(w, o[k].x, acc.x);
      acc.y = fmaf(w, o[k].y, acc.y);
      acc.z = fmaf(w, o[k].z, acc.z);
      acc.w = fmaf(w, o[k].w, acc.w);
    }
  }
  const int64_t row = static_cast<int64_t>(s.n0 + d.z * p.nq + c / g) * a.Hq + d.w * g + c % g;
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * D + dim) =
      make_uint2(pack_bf16(acc.x * f, acc.y * f), pack_bf16(acc.z * f, acc.w * f));
  if (dim == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
}

constexpr int kRows = 64;   // query rows of a unit

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <int D, int N>
int launch(const TcArgs& p, cudaStream_t st) {
  using L = Lay<D, N>;
  if (!smem_limit(attn_kernel<D, N>, static_cast<int>(L::kBytes))) return TV_ECUDA;
  const int rc = launch_pdl(attn_kernel<D, N>, dim3(p.grid), dim3(L::kThreads), L::kBytes, st, p);
  if (rc != TV_OK) return rc;
  return launch_pdl(join_kernel<D>, dim3(p.grid, N / 8), dim3(2 * D), 0, st, p, N);
}

bool wants_extents(const AttnArgs& a) { return a.vis_prefix != nullptr || a.max_nodes > kKeys; }

}  // namespace

int attn_extents(const AttnArgs& a, int nq, int tiles, int4* out, cudaStream_t st) {
  return launch_pdl(extent_kernel, dim3((a.B * tiles + 3) / 4), dim3(128), 0, st, a, nq, tiles, out);
}

// [status word (256 B)] [extents] [pieces of cut units] [partial (m, l)] [partial o]
size_t attn_tc_workspace(int B, int max_nodes, int Hq, int Hkv, int d) {
  const size_t G = sm_count(), N = kRows, nq = N / (Hq / Hkv);
  const size_t entries = static_cast<size_t>(B) * ((max_nodes + nq - 1) / nq);
  return 256 + align256(entries * sizeof(int4)) + align256(G * sizeof(int4)) + align256(2 * G * N * sizeof(float2)) +
         2 * G * N * d * sizeof(float);
}

int attn_tc(const AttnArgs& a, void* ws, cudaStream_t st) {
  TcArgs p{};
  p.a = a;
  p.magic = kMagic;
  const int g = a.Hq / a.Hkv, N = kRows;
  p.grid = sm_count();
  p.nq = N / g;
  p.tiles = (a.max_nodes + p.nq - 1) / p.nq;
  const int entries = a.B * p.tiles;
  char* base = static_cast<char*>(ws);
  p.status = reinterpret_cast<int*>(base);
  base += 256;
  int4* extents = reinterpret_cast<int4*>(base);
  base += align256(static_cast<size_t>(entries) * sizeof(int4));
  p.desc = reinterpret_cast<int4*>(base);
  base += align256(p.grid * sizeof(int4));
  p.ml = reinterpret_cast<float2*>(base);
  base += align256(2ull * p.grid * N * sizeof(float2));
  p.o = reinterpret_cast<float*>(base);
  if (wants_extents(a)) {
    const int rc = attn_extents(a, p.nq, p.tiles, extents, st);
    if (rc != TV_OK) return rc;
    p.extents = extents;
  }
  return a.d == 128 ? launch<128, kRows>(p, st) : launch<64, kRows>(p, st);
}

}  // namespace kv4
}  // namespace tv
