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
#include "tc_common.cuh"

namespace tv {
namespace kv4 {
namespace {

using namespace tc;

constexpr int kKeys = 128;        // keys per tile
constexpr int kStages = 6;        // staged tiles
constexpr float kLow = -3.3895314e38f;   // reference of a row that has seen nothing

enum Bar { RAW_FULL = 0, RAW_EMPTY = RAW_FULL + kStages, K_FULL = RAW_EMPTY + kStages, V_FULL = K_FULL + 2,
           S_FULL = V_FULL + 2, S_FREE = S_FULL + 2, P_FULL = S_FREE + 2, PV_DONE = P_FULL + 2, DRAIN = PV_DONE + 2,
           N_BARS = DRAIN + 1 };

// What the producer says about a staged tile.
struct Tile {
  int kind;          // kPrefix, kTree, kEnd
  int flags;         // 1: first of its unit's run, 2: last
  int r, t, h;       // request, row tile, KV head
  int n0, cnt;       // first node of the request, nodes
  int key0, nkeys;   // first token (node) of the tile, how many
  int groups;        // bit i: the page of tokens 16 i .. 16 i + 15 of the tile is staged
  int seg;           // running number of the unit in this CTA
  int slot;          // -1: the whole unit is here; else its partial slot
};
enum { kPrefix = 0, kTree = 1, kEnd = 2 };

template <int D, int N>
struct Lay {
  static constexpr int kGroups = N > 32 ? 2 : 1;              // softmax warpgroups
  static constexpr int kCols = N / kGroups;                   // rows per softmax warpgroup
  static constexpr int kSoft0 = 8;                            // first softmax warp
  static constexpr int kMma = kSoft0 + 4 * kGroups;
  static constexpr int kProd = kMma + 1;
  static constexpr int kWarps = kProd + 1;
  static constexpr int kThreads = 32 * kWarps;
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
  static_assert(sizeof(Tile) <= 64 && N_BARS <= 32 && kRef % 16 == 0 && kSums % 8 == 0, "layout");
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
  int nq, tiles, grid;
  int by_node;       // a unit's key range depends on its nodes (per-node prefixes, several tree tiles)
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
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
// Eight codes -> four bf16 pairs (items 2i, 2i + 1) of n = code - 8, exact.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t* r) {
  const uint32_t bias = 0x43084308u;   // bf16 136, 136
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;   // bf16 128 + code
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                     *reinterpret_cast<const __nv_bfloat162*>(&bias));
    r[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// Key tiles of a unit: prefix tiles over the tokens that any of its rows sees,
// then tree tiles from the lowest visible ancestor on.
struct Extent {
  int n0, cnt, len;       // nodes of the request, visible prefix of the row tile
  int np, t0, nt;         // prefix tiles, first tree tile, tree tiles
};
__device__ __forceinline__ Extent extent_plain(const TcArgs& p, int e) {
  Extent x;
  const int r = e / p.tiles, t = e % p.tiles;
  const Span s = node_span(p.a, r);
  x.n0 = s.n0;
  x.cnt = s.cnt;
  x.len = prefix_len(p.a, r);
  const bool live = t * p.nq < s.cnt;
  x.np = live ? (x.len + kKeys - 1) / kKeys : 0;
  x.t0 = 0;
  x.nt = live ? 1 : 0;
  return x;
}
// One entry by a whole warp, lanes = nodes.
__device__ __forceinline__ Extent extent_by_node(const TcArgs& p, int e, int lane) {
  Extent x;
  const int r = e / p.tiles, t = e % p.tiles;
  const Span s = node_span(p.a, r);
  x.n0 = s.n0;
  x.cnt = s.cnt;
  const int len = prefix_len(p.a, r);
  const int first = t * p.nq, last = min(first + p.nq, s.cnt);
  int vis = 0, lo = 1 << 30, hi = -1;           // 64-node words of the masks that are not empty
  for (int i = first + lane; i < last; i += 32) {
    vis = max(vis, p.a.vis_prefix ? min(max(p.a.vis_prefix[s.n0 + i], 0), len) : len);
    const uint64_t* row = p.a.anc + static_cast<int64_t>(s.n0 + i) * p.a.anc_words;
    for (int w0 = 0; w0 < p.a.anc_words; w0 += 8) {
      uint64_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = w0 + k < p.a.anc_words ? row[w0 + k] : 0ull;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (v[k]) {
          lo = min(lo, w0 + k);
          hi = max(hi, w0 + k);
        }
    }
  }
  x.len = __reduce_max_sync(0xffffffffu, vis);
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  const bool live = first < s.cnt;
  x.np = live ? (x.len + kKeys - 1) / kKeys : 0;
  // at least one tile for a live unit: its rows are written even if they see nothing
  const int top = live ? (s.cnt - 1) / kKeys : 0;
  x.t0 = min(lo / 2, top);
  x.nt = live ? max(0, min(hi / 2, top) - x.t0) + 1 : 0;
  return x;
}
__device__ __forceinline__ Extent extent_of(const TcArgs& p, int e, int lane) {
  return p.by_node ? extent_by_node(p, e, lane) : extent_plain(p, e);
}
// Tiles of entries e0 + lane (all KV heads of each), 0 past the end.
__device__ __forceinline__ long long entry_tiles(const TcArgs& p, int e0, int end, int lane) {
  long long mine = 0;
  if (!p.by_node) {
    if (e0 + lane < end) {
      const Extent x = extent_plain(p, e0 + lane);
      mine = x.np + x.nt;
    }
  } else {
    for (int i = 0; i < 32 && e0 + i < end; ++i) {
      const Extent x = extent_by_node(p, e0 + i, lane);
      if (lane == i) mine = x.np + x.nt;
    }
  }
  return mine * p.a.Hkv;
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
  const int per = p.by_node ? (E + L::kWarps - 1) / L::kWarps           // entries per warp
                            : ((E + L::kWarps - 1) / L::kWarps + 31) / 32 * 32;
  const int e_lo = min(warp * per, E), e_hi = min(e_lo + per, E);
  {
    long long s = 0;
    for (int e = e_lo; e < e_hi; e += 32) s += entry_tiles(p, e, e_hi, lane);
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
      const long long c = entry_tiles(p, e, e_hi, lane);
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
    Extent x = extent_of(p, e, lane);
    int nb = x.np + x.nt;
    long long off = w0 - start[1];
    int h = static_cast<int>(off / nb), blk = static_cast<int>(off % nb);
    int seg = 0, seg_blk = blk;                  // first tile of the running unit in this CTA
    const int per_tile = kKeys >> ps_shift;      // pages of a tile
    const int end_of_list = E;
    int issued = 0;
    bool ok = true;
    // the next tile, and this lane's page of it
    Tile nx;
    int npage;
    auto gen = [&]() {
      npage = -1;
      if (pos >= w1) {
        nx.kind = kEnd;
        nx.flags = 0;
        return;
      }
      while (blk == nb) {                        // next unit
        blk = 0;
        ++seg;
        if (++h == a.Hkv) {
          h = 0;
          do {
            ++e;
            x = extent_of(p, e, lane);
            nb = x.np + x.nt;
          } while (nb == 0 && e + 1 < end_of_list);
        }
        seg_blk = 0;
      }
      nx.kind = blk < x.np ? kPrefix : kTree;
      nx.r = e / p.tiles;
      nx.t = e % p.tiles;
      nx.h = h;
      nx.n0 = x.n0;
      nx.cnt = x.cnt;
      nx.seg = seg;
      const bool last = blk == nb - 1 || pos == w1 - 1;
      const bool whole = seg_blk == 0 && pos + (nb - 1 - blk) < w1;
      nx.flags = (blk == seg_blk ? 1 : 0) | (last ? 2 : 0);
      nx.slot = whole ? -1 : 2 * static_cast<int>(blockIdx.x) + (seg_blk == 0 ? 1 : 0);
      if (nx.kind == kPrefix) {
        nx.key0 = blk * kKeys;
        nx.nkeys = min(kKeys, x.len - nx.key0);
        if (lane < per_tile && (lane << ps_shift) < nx.nkeys)
          npage = a.block_table[static_cast<int64_t>(nx.r) * a.table_ld + (nx.key0 >> ps_shift) + lane];
      } else {
        nx.key0 = (x.t0 + blk - x.np) * kKeys;
        nx.nkeys = min(kKeys, x.cnt - nx.key0);
      }
      if (blk == nb - 1 || pos == w1 - 1) {
        // the unit that starts here and goes on: its pieces, for the joining kernel
        if (seg_blk == 0 && blk != nb - 1 && lane == 0) {
          const long long u1 = pos + (nb - blk);            // position after the unit
          const long long k = (u1 * G + W - 1) / W - 1;     // CTA of its last tile
          p.desc[blockIdx.x] = make_int4(static_cast<int>(k) - static_cast<int>(blockIdx.x) + 1, nx.r, nx.t, h);
        }
      }
      ++blk;
      ++pos;
    };
    gen();
    for (int it = 0; ok; ++it) {
      const Tile cur = nx;
      const int page = npage;
      if (cur.kind != kEnd) gen();
      const int st = it % kStages;
      if (it >= kStages)
        ok = __all_sync(0xffffffffu, mbar_wait(bar(RAW_EMPTY + st), ((it / kStages) - 1) & 1, abort_flag, err, 41));
      if (!ok) break;
      const bool wanted = cur.kind == kPrefix && lane < per_tile && (lane << ps_shift) < cur.nkeys;
      const bool good = wanted && page >= 0 && page < a.n_pages;
      if (wanted && !good && a.err) *a.err = 1;
      const unsigned have = __ballot_sync(0xffffffffu, good);
      if (lane == 0) {
        Tile* t = reinterpret_cast<Tile*>(sm + L::kTiles + 64 * st);
        *t = cur;
        int groups = 0;
        for (int i = 0; i < 8; ++i) groups |= ((have >> ((16 * i) >> ps_shift)) & 1) << i;
        t->groups = groups;
        if (have)
          mbar_expect_tx(bar(RAW_FULL + st), __popc(have) * blk_bytes);
        else
          mbar_arrive(bar(RAW_FULL + st));
      }
      __syncwarp();
      if (good)
        bulk_load(sb + L::kRaw + st * L::kStage + lane * blk_bytes,
                  a.cache + (static_cast<int64_t>(page) * a.Hkv + cur.h) * blk_bytes, blk_bytes, bar(RAW_FULL + st));
      issued = it + 1;
      if (cur.kind == kEnd) break;
    }
    // after an expired wait: copies in flight land before the CTA ends
    if (*abort_flag) {
      for (int it = max(0, issued - kStages); it < issued; ++it) {
        const uint64_t t0 = gtime();
        while (!mbar_try(bar(RAW_FULL + it % kStages), (it / kStages) & 1) && gtime() - t0 < kTimeoutNs) {
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
      uint64_t since = 0;
      bool ok = true;
      while (ok && (total < 0 || npv < total)) {
        bool prog = false;
        if (total < 0 && mbar_test(bar(RAW_FULL + ns % kStages), (ns / kStages) & 1)) {
          const Tile& t = tile_at(ns % kStages);
          if (t.kind == kEnd) {
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
            firsts = (firsts & ~(1u << (ns & 7))) | (static_cast<uint32_t>(t.flags & 1) << (ns & 7));
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
        if (prog) since = 0;
        else if (!still_waiting(since, abort_flag, err, 42)) ok = false;
      }
      umma_commit(bar(DRAIN));
      mbar_wait(bar(DRAIN), 0, abort_flag, err, 43);
    }
  } else if (warp < 4) {
    // ================= keys: thread = key
    for (int it = 0;; ++it) {
      const int st = it % kStages, b = it & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(RAW_FULL + st), (it / kStages) & 1, abort_flag, err, 44))) break;
      const Tile& t = tile_at(st);
      const int kind = t.kind;
      if (kind == kEnd) break;
      const bool first = t.flags & 1;
      // S(it - 2) has read this K buffer, and every S of the unit before last its Q buffer
      if (it >= 2 &&
          !__all_sync(0xffffffffu, mbar_wait(bar(S_FULL + b), ((it >> 1) - 1) & 1, abort_flag, err, 45)))
        break;
      tc_fence_after();
      if (first) {
        uint8_t* qs = sm + L::kQ + (t.seg & 1) * L::kQBytes;
        const int node0 = t.t * p.nq, rows = min(p.nq, t.cnt - node0) * g;
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
      if (kind == kPrefix) {
        const uint8_t* blk = raw + st * L::kStage + (own >> ps_shift) * blk_bytes;
        const int slot = own & (a.page_size - 1);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t r[32];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 w = *reinterpret_cast<const uint4*>(blk + ((2 * c + i) * a.page_size + slot) * 16);
            decode8(w.x, r + 16 * i);
            decode8(w.y, r + 16 * i + 4);
            decode8(w.z, r + 16 * i + 8);
            decode8(w.w, r + 16 * i + 12);
          }
          tmem_st32(dst + 32 * c, r);
        }
      } else {
        const bool live = own < t.nkeys;
        const uint16_t* row = static_cast<const uint16_t*>(a.k_tree) +
                              static_cast<int64_t>(t.n0 + t.key0 + (live ? own : 0)) * a.ldk +
                              static_cast<int64_t>(t.h) * D;
#pragma unroll
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
    for (int it = 0;; ++it) {
      const int st = it % kStages, b = it & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(RAW_FULL + st), (it / kStages) & 1, abort_flag, err, 46))) break;
      const Tile& t = tile_at(st);
      const int kind = t.kind;
      if (kind == kEnd) break;
      if (it >= 2 &&
          !__all_sync(0xffffffffu, mbar_wait(bar(PV_DONE + b), ((it >> 1) - 1) & 1, abort_flag, err, 47)))
        break;
      tc_fence_after();
      const uint32_t dst = tmem + L::tV + 64 * b + lane_off;
      if (32 * (warp & 3) < D) {                 // d = 64: the upper lanes' results are not used
        if (kind == kPrefix) {
          const uint8_t* base = raw + st * L::kStage + a.page_size * (D / 2) + own * 8;
          const int gshift = ps_shift - 4;       // groups of 16 tokens per page
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t r[32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int gr = 4 * c + i;
              const uint2 w = *reinterpret_cast<const uint2*>(base + (gr >> gshift) * blk_bytes +
                                                              (gr & ((1 << gshift) - 1)) * (D * 8));
              decode8(w.x, r + 8 * i);
              decode8(w.y, r + 8 * i + 4);
            }
            tmem_st32(dst + 32 * c, r);
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
              uint32_t lo = 0u, hi = 0u;
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
    const int wg = (warp - L::kSoft0) >> 2, wid = 1 + wg;
    const int c0 = wg * C;
    const float c2 = a.scale * kLog2e;
    float* ref = reinterpret_cast<float*>(sm + L::kRef);        // [2][N]
    float* corr_s = reinterpret_cast<float*>(sm + L::kCorr);
    float* inv_s = reinterpret_cast<float*>(sm + L::kInv);
    int* vis_s = reinterpret_cast<int*>(sm + L::kVis);
    int* row_s = reinterpret_cast<int*>(sm + L::kRow);
    uint32_t* anc_s = reinterpret_cast<uint32_t*>(sm + L::kAnc);   // [4][N]
    int* wmax = reinterpret_cast<int*>(sm + L::kWarpMax) + wg * 128;
    const int tid = threadIdx.x - 32 * L::kSoft0 - 128 * wg;    // 0..127 in the warpgroup
    int par = 0;                                                // ref[par] is current
    float l[C];
#pragma unroll
    for (int c = 0; c < C; ++c) l[c] = 0.f;
    for (int it = 0;; ++it) {
      const int st = it % kStages, b = it & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(RAW_FULL + st), (it / kStages) & 1, abort_flag, err, 48))) break;
      const Tile t = tile_at(st);
      if (t.kind == kEnd) break;
      const bool first = t.flags & 1, last = t.flags & 2, tree = t.kind == kTree;
      float sk = c2, sv = 1.f;
      bool valid = own < t.nkeys;
      if (!tree) {
        valid = valid && ((t.groups >> (own >> 4)) & 1);
        const uint8_t* blk = raw + st * L::kStage + (own >> ps_shift) * blk_bytes;
        const int slot = own & (a.page_size - 1);
        sk = valid ? c2 * bf16_at(reinterpret_cast<const uint16_t*>(blk + k_scale(a.page_size, D, slot))) : 0.f;
        sv = valid ? bf16_at(reinterpret_cast<const uint16_t*>(blk + v_scale(a.page_size, D, slot))) : 0.f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(RAW_EMPTY + st));
      if (first || tree) {
        wg_sync(wid);                            // the unit (tile) before is done with these arrays
        if (tid < C) {
          const int rr = c0 + tid, ln = t.t * p.nq + rr / g;
          const bool live = rr < p.nq * g && ln < t.cnt;
          const int gn = t.n0 + ln;
          if (first) {
            ref[par * N + rr] = kLow;
            row_s[rr] = live ? gn * a.Hq + t.h * g + rr % g : -1;
            vis_s[rr] = live ? (a.vis_prefix ? a.vis_prefix[gn] : 0x7fffffff) : 0;
          }
          if (tree) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int word = (t.key0 >> 6) + w;
              const uint64_t v = live && word < a.anc_words ? a.anc[static_cast<int64_t>(gn) * a.anc_words + word] : 0ull;
              anc_s[(2 * w) * N + rr] = static_cast<uint32_t>(v);
              anc_s[(2 * w + 1) * N + rr] = static_cast<uint32_t>(v >> 32);
            }
          }
        }
        wg_sync(wid);
      }
      if (!__all_sync(0xffffffffu, mbar_wait(bar(S_FULL + b), (it >> 1) & 1, abort_flag, err, 49))) break;
      tc_fence_after();
      const uint32_t tS = tmem + L::tS + N * b + c0 + lane_off;
      uint32_t x[C];
      // scores of this key in base-2 units, minus the rows' references; -inf where the row does not see the key
      auto scores = [&](bool sub) {
        tmem_ld(tS, x);
        tmem_ld_wait();
        const uint32_t* words = anc_s + (warp & 3) * N + c0;
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(ref + par * N + c0 + c);
          const float m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            pin(x[c + i]);
            x[c + i] = __float_as_uint(fmaf(__uint_as_float(x[c + i]), sk, sub ? -m[i] : 0.f));
          }
        }
        if (tree) {
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const uint4 w4 = *reinterpret_cast<const uint4*>(words + c);
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!(valid && ((w[i] >> lane) & 1u))) x[c + i] = __float_as_uint(-INFINITY);
          }
        } else if (a.vis_prefix) {
          const int key = valid ? t.key0 + own : 0x7fffffff;
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const int4 v4 = *reinterpret_cast<const int4*>(vis_s + c0 + c);
            const int v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key >= v[i]) x[c + i] = __float_as_uint(-INFINITY);
          }
        } else if (!__all_sync(0xffffffffu, valid)) {
          if (!valid) {
#pragma unroll
            for (int c = 0; c < C; ++c) x[c] = __float_as_uint(-INFINITY);
          }
        }
      };
      bool slow = first;
      if (!first) {
        scores(true);
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < C; ++c) mx[c & 1] = fmaxf(mx[c & 1], __uint_as_float(x[c]));
        slow = wg_any(wid, fmaxf(mx[0], mx[1]) > 8.f);
      }
      if (slow) {
        // new references: the rows' maxima so far
        scores(false);
        int mine = static_cast<int>(0x80000000);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          int v = static_cast<int>(x[c]);
          v ^= (v >> 31) & 0x7fffffff;           // order of floats as order of integers
          v = __reduce_max_sync(0xffffffffu, v);
          if ((lane & (C - 1)) == c) mine = v;
        }
        if (lane < C) wmax[(warp & 3) * 32 + lane] = mine;
        wg_sync(wid);
        if (lane < C) {                          // every warp writes the same values
          int v = wmax[lane];
#pragma unroll
          for (int w = 1; w < 4; ++w) v = max(v, wmax[32 * w + lane]);
          v ^= (v >> 31) & 0x7fffffff;
          const float old = ref[par * N + c0 + lane];
          const float now = fmaxf(old, __int_as_float(v));
          ref[(par ^ 1) * N + c0 + lane] = now;
          corr_s[c0 + lane] = ex2(old - now);
        }
        __syncwarp();
        par ^= 1;
        if (first) {
#pragma unroll
          for (int c = 0; c < C; ++c) l[c] = 0.f;
        } else {
          if (!__all_sync(0xffffffffu,
                          mbar_wait(bar(PV_DONE + (b ^ 1)), ((it - 1) >> 1) & 1, abort_flag, err, 50)))
            break;
          tc_fence_after();
          uint32_t o[C];
          tmem_ld(tmem + L::tO + c0 + lane_off, o);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < C; c += 4) {
            const float4 f4 = *reinterpret_cast<const float4*>(corr_s + c0 + c);
            const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              pin(o[c + i]);
              o[c + i] = __float_as_uint(__uint_as_float(o[c + i]) * f[i]);
              l[c + i] *= f[i];
            }
          }
          tmem_st(tmem + L::tO + c0 + lane_off, o);
          tmem_st_wait();
        }
        scores(true);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(S_FREE + b));
      // weights
      uint32_t pk[C / 2];
#pragma unroll
      for (int c = 0; c < C; c += 2) {
        const float e0 = ex2(__uint_as_float(x[c])), e1 = ex2(__uint_as_float(x[c + 1]));
        l[c] += e0;
        l[c + 1] += e1;
        pk[c >> 1] = pack_bf16(e0 * sv, e1 * sv);
      }
      if (it >= 2 &&
          !__all_sync(0xffffffffu, mbar_wait(bar(PV_DONE + b), ((it >> 1) - 1) & 1, abort_flag, err, 51)))
        break;
      uint8_t* prow = sm + L::kP + b * L::kPBytes + own * 128;
#pragma unroll
      for (int c = 0; c < C / 8; ++c)
        *reinterpret_cast<uint4*>(prow + (((c0 / 8 + c) ^ (own & 7)) << 4)) =
            make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      // the value warps' note on non-finite tree rows, read at the end of the unit (V's phase cannot move on
      // before P is given away)
      if (last && tree &&
          !__all_sync(0xffffffffu, mbar_wait(bar(V_FULL + b), (it >> 1) & 1, abort_flag, err, 53)))
        break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(P_FULL + b));
      if (!last) continue;

      // ---- end of the unit's run here: sums over the keys' threads, then O^T
      if (!__all_sync(0xffffffffu, mbar_wait(bar(PV_DONE + b), (it >> 1) & 1, abort_flag, err, 52))) break;
      tc_fence_after();
      // reduce-scatter over the lanes: lane i ends with column i % C
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        if (o >= C) {
#pragma unroll
          for (int c = 0; c < C; ++c) l[c] += __shfl_xor_sync(0xffffffffu, l[c], o);
        } else {
          const bool up = lane & o;
#pragma unroll
          for (int c = 0; c < o; ++c) {
            const float keep = up ? l[c + o] : l[c], give = up ? l[c] : l[c + o];
            l[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
      }
      if (lane < C) wmax[(warp & 3) * 32 + lane] = __float_as_int(l[0]);
      wg_sync(wid);
      float lsum = 0.f;
      if (lane < C) {
#pragma unroll
        for (int w = 0; w < 4; ++w) lsum += __int_as_float(wmax[32 * w + lane]);
        inv_s[c0 + lane] = t.slot >= 0 ? 1.f : (lsum == 0.f ? 0.f : 1.f / lsum);   // partials stay unnormalised
        if ((warp & 3) == 0) {
          const float m = ref[par * N + c0 + lane];
          if (t.slot >= 0) {
            p.ml[static_cast<int64_t>(t.slot) * N + c0 + lane] = make_float2(m, lsum);
          } else if (a.lse && row_s[c0 + lane] >= 0) {
            a.lse[row_s[c0 + lane]] = lsum == 0.f ? -INFINITY : (m + log2f(lsum)) * kLn2;
          }
        }
      }
      __syncwarp();
      uint32_t o[C];
      tmem_ld(tmem + L::tO + c0 + lane_off, o);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < C; ++c) pin(o[c]);
      if (own < D) {
        if (dirty[t.seg & 3] == t.seg + 1) {
          // non-finite tree values, added to the rows that see them
          const uint16_t* col = static_cast<const uint16_t*>(a.v_tree) + static_cast<int64_t>(t.n0) * a.ldv +
                                static_cast<int64_t>(t.h) * D + own;
          for (int j = 0; j < t.cnt; ++j) {
            const uint32_t v = col[static_cast<int64_t>(j) * a.ldv];
            if ((v & 0x7f80u) != 0x7f80u || (j >> 6) >= a.anc_words) continue;
#pragma unroll
            for (int c = 0; c < C; ++c) {
              const int row = row_s[c0 + c];
              if (row < 0) continue;
              const uint64_t word = a.anc[static_cast<int64_t>(row / a.Hq) * a.anc_words + (j >> 6)];
              if ((word >> (j & 63)) & 1ull) o[c] = __float_as_uint(__uint_as_float(o[c]) + __uint_as_float(v << 16));
            }
          }
        }
        if (t.slot >= 0) {
          float* po = p.o + static_cast<int64_t>(t.slot) * N * D + c0 * D + own;
#pragma unroll
          for (int c = 0; c < C; ++c)
            if (row_s[c0 + c] >= 0) po[c * D] = __uint_as_float(o[c]);
        } else {
          uint16_t* out = static_cast<uint16_t*>(a.out) + own;
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const int row = row_s[c0 + c];
            if (row >= 0) {
              const float f = __uint_as_float(o[c]) * inv_s[c0 + c];
              out[static_cast<int64_t>(row) * D] = static_cast<uint16_t>(pack_bf16(f, 0.f));
            }
          }
        }
      }
      tc_fence_before();                         // O was read: the next unit's first PV may overwrite it
#pragma unroll
      for (int c = 0; c < C; ++c) l[c] = 0.f;
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
// CTA, share of the rows), thread = dim.
template <int D>
__global__ void __launch_bounds__(D) join_kernel(const TcArgs p, int N) {
  griddep_wait();
  griddep_release();
  const int4 d = p.desc[blockIdx.x];
  if (d.x < 2) return;
  const AttnArgs& a = p.a;
  const int g = a.Hq / a.Hkv;
  const Span s = node_span(a, d.y);
  auto slot = [&](int i) { return static_cast<int64_t>(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)); };
  const int rows = min(p.nq, s.cnt - d.z * p.nq) * g;
  for (int c = blockIdx.y; c < rows; c += gridDim.y) {
    float M = -INFINITY;
    for (int i = 0; i < d.x; ++i) M = fmaxf(M, p.ml[slot(i) * N + c].x);
    float acc = 0.f, sum = 0.f;
#pragma unroll 4
    for (int i = 0; i < d.x; ++i) {
      const float2 ml = p.ml[slot(i) * N + c];
      const float o = p.o[(slot(i) * N + c) * D + threadIdx.x];
      if (ml.y == 0.f) continue;                 // nothing seen in this piece
      const float w = ex2(ml.x - M);
      sum = fmaf(w, ml.y, sum);
      acc = fmaf(w, o, acc);
    }
    const int64_t row = static_cast<int64_t>(s.n0 + d.z * p.nq + c / g) * a.Hq + d.w * g + c % g;
    const float f = sum == 0.f ? 0.f : acc / sum;
    static_cast<uint16_t*>(a.out)[row * D + threadIdx.x] = static_cast<uint16_t>(pack_bf16(f, 0.f));
    if (threadIdx.x == 0 && a.lse) a.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
  }
}

int rows_of(int max_nodes, int g) {
  const long long rows = static_cast<long long>(max_nodes) * g;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <int D, int N>
int launch(const TcArgs& p, cudaStream_t st) {
  using L = Lay<D, N>;
  if (!smem_limit(attn_kernel<D, N>, static_cast<int>(L::kBytes))) return TV_ECUDA;
  const int rc = launch_pdl(attn_kernel<D, N>, dim3(p.grid), dim3(L::kThreads), L::kBytes, st, p);
  if (rc != TV_OK) return rc;
  return launch_pdl(join_kernel<D>, dim3(p.grid, 4), dim3(D), 0, st, p, N);
}

}  // namespace

size_t attn_tc_workspace(int max_nodes, int Hq, int Hkv, int d) {
  const size_t G = sm_count(), N = rows_of(max_nodes, Hq / Hkv);
  return 256 + align256(G * sizeof(int4)) + align256(2 * G * N * sizeof(float2)) + 2 * G * N * d * sizeof(float);
}

int attn_tc(const AttnArgs& a, void* ws, cudaStream_t st) {
  TcArgs p{};
  p.a = a;
  const int g = a.Hq / a.Hkv, N = rows_of(a.max_nodes, g);
  p.grid = sm_count();
  p.nq = N / g;
  p.tiles = (a.max_nodes + p.nq - 1) / p.nq;
  p.by_node = a.vis_prefix != nullptr || a.max_nodes > kKeys;
  char* base = static_cast<char*>(ws);
  p.status = reinterpret_cast<int*>(base);
  base += 256;
  p.desc = reinterpret_cast<int4*>(base);
  base += align256(p.grid * sizeof(int4));
  p.ml = reinterpret_cast<float2*>(base);
  base += align256(2ull * p.grid * N * sizeof(float2));
  p.o = reinterpret_cast<float*>(base);
  if (a.d == 128) return N == 16 ? launch<128, 16>(p, st) : N == 32 ? launch<128, 32>(p, st) : launch<128, 64>(p, st);
  return N == 16 ? launch<64, 16>(p, st) : N == 32 ? launch<64, 32>(p, st) : launch<64, 64>(p, st);
}

}  // namespace kv4
}  // namespace tv
