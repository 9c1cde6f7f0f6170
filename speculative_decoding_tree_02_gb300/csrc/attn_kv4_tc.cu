// tree_verify_attn_kv4, tcgen05 path (bf16 rows, d = 64 or 128, row tiles of
// up to 64 query rows = nodes x the heads of one KV head).
//
// The products are taken transposed, so that the 128 tensor-memory lanes of an
// MMA are keys and dims, not query rows:
//   S^T [keys x rows] = K Q^T            A = K   (lanes: keys, 32-bit columns: dim pairs)
//   O^T [dims x rows] += V^T (s_v P)^T   A = V^T (lanes: dims, columns: key pairs)
// A tile of 128 keys then costs 64 columns for its rows instead of a 128-row
// tile, and both A operands are tensor-memory operands that the threads write
// straight from registers: a thread owns one key (then one dim) of the tile,
// reads its code words from the staged block and turns each into four bf16
// pairs (see decode_pair); shared memory carries the codes once, 132 bytes per
// token, and the small B operands Q and P.  The values n are exact in bf16;
// the scales are applied in fp32, s_k to the scores, s_v to the weights before
// their rounding to bf16.
//
// Softmax: a thread owns one key of the tile, so its scales and visibility
// are scalars; row maxima run across lanes, which a tile only pays for when a
// score exceeds the row's running reference by 2^8 (then everything is
// rescaled); one vote per tile decides.  Row sums stay in registers, one per
// thread and row, until the end of the unit.
//
// A CTA is two teams of two warpgroups that share nothing but the SM: each
// team walks its own run of the list of all units (request, row tile, KV head;
// a unit's tiles of 128 cached tokens, then of 128 nodes, follow one another),
// so that one dequantises while the other takes its softmax; runs are of equal
// cost (kUnitCost).  In a team each
// warpgroup writes half of K's columns, then, beside S, half of V^T's; then
// both take the softmax of 32 rows each, write P, and PV runs beside the next
// tile's K.  A unit cut by a run's end leaves fp32 partials that
// attn_join joins in run order.
//
// Bound by issue slots and by the serial chain of a tile: 128 tokens cost a
// team 4400 cycles (700 instructions to each of its 8 warps, 64% of the slots
// of the two teams), of which the issue of S and of PV, by a lane whose
// warpgroup waits for it, are 500 each.  64 chains of 16 nodes x 32 heads over
// 512..4096 tokens 105 us (25% of the measured copy rate counted in the 132
// bytes per token and head, 19% of the measured matrix rate), 8 requests of
// 452 rows per KV head over 8192 tokens 309 us (20% of the matrix rate).
// Tried on the 64 chains, against 120..154 us of the teams at those times: dequantising, softmax and MMA issue in warps of
// their own that hand tiles over through barriers 185 us (most issue slots
// went to instruction fetches of five kinds of code and to the polls of
// waiting warps); one warpgroup doing everything for its tile 203 us (two
// warps to a scheduler do not fill it); loads and MMA issue moved to two more
// warps 159 us (112 registers are left to the others, which spill); the words
// shared out unevenly to spare the issuing warps 148 us (loops in place of
// straight code).
//
// Every wait is bounded (2 s). A warp whose wait expires records an error code
// in the workspace status word, raises its team's abort flag and goes on with
// whatever is there (addresses follow from the lengths and tables alone, so
// all accesses stay in bounds) up to the team's vote before PV, which sends the
// whole team out of the loop at once: no barrier ever counts a warp that has
// left. The team then waits, bounded again, for its MMAs and copies in flight;
// tensor memory is always released.
#include <algorithm>

#include "kv4.cuh"
#include "kv4_device.cuh"

namespace tv {
namespace kv4 {
namespace {

using namespace tc;

constexpr int kKeys = 128;        // keys per tile
constexpr int kRowsT = 64;        // rows per tile
constexpr int kCols = 32;         // rows per warpgroup in the softmax
constexpr int kStages = 4;        // staged tiles per team
// What a unit costs beside its tiles, in tiles: its queries, its first tile's references, its tile of nodes, its output.
// A tree of 512 units of 1 to 33 tiles 172 us without it, 115 at 2, 104 at 3, 105 at 6; 64 chains 122, 107, 105, 109
// (both of 8 KV heads of 128; other geometries take the same number untimed).
constexpr int kUnitCost = 3;

template <int D>
struct Lay {
  static constexpr uint32_t kStage = kKeys * (D + 4);
  static constexpr uint32_t kQHalf = kRowsT * 128;            // 64 rows x 64 dims
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kP = (D / 64) * kQHalf;           // 128 keys x 64 rows
  static constexpr uint32_t kRaw = kP + kKeys * 128;
  static constexpr uint32_t kRef = kRaw + kStages * kStage;   // float [64] negated references
  static constexpr uint32_t kShift = kRef + 256;              // float [64]
  static constexpr uint32_t kCorr = kShift + 256;             // float [64]
  static constexpr uint32_t kInv = kCorr + 256;               // float [64]
  static constexpr uint32_t kVis = kInv + 256;                // int [64]
  static constexpr uint32_t kRow = kVis + 256;                // int [64] output row, -1: none
  static constexpr uint32_t kWarpMax = kRow + 256;            // float [2][4][32]
  static constexpr uint32_t kPages = kWarpMax + 1024;         // u8 [kStages][8] page i of the tile is staged; dirty, low_vis, abort flag
  static constexpr uint32_t kBars = kPages + 48;              // RAW [kStages], S, PV
  static constexpr uint32_t kTeam = (kBars + 64 + 1023) / 1024 * 1024;    // bytes of a team
  static constexpr uint32_t kMisc = 2 * kTeam;                // tensor memory address, entry sums
  static constexpr uint32_t kBytes = kMisc + 192 + 1024;      // + alignment slack
  static_assert(kBytes <= 232448, "shared memory");
  // tensor memory of a team (256 columns): K, V, S, O
  static constexpr uint32_t tK = 0, tV = 64, tS = 128, tO = 192;
};

struct TcArgs {
  AttnArgs a;
  int* status;
  int status0;            // its first value
  Pieces pieces;          // runs = 2 grid
  const int4* extents;    // [B * tiles] from attn_extents, or NULL
  int nq, tiles, grid;
  uint32_t magic;         // kMagic
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Maximum over a warp, NaN when a value is.
__device__ __forceinline__ float redux_max(float x) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
  return r != 0;
}
// Barriers of a team and of a warpgroup, and with an OR over their threads.
__device__ __forceinline__ void team_sync(int id) { asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void wg_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
template <int kThreads>
__device__ __forceinline__ bool any_of(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"(static_cast<uint32_t>(p)), "n"(kThreads)
      : "memory");
  return r != 0;
}

// By a whole warp: until the phase is over or the wait has expired, which the abort flag then tells; the warp goes on
// either way. The slow part is a call, so that the tile's registers need not meet its own (in line: 3% slower).
__device__ __noinline__ void slow_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int code) {
  bounded_wait(bar, parity, abort_flag, err, code);
}
__device__ __forceinline__ void team_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int code) {
  if (__builtin_expect(__all_sync(0xffffffffu, mbar_test(bar, parity)), 1)) return;
  slow_wait(bar, parity, abort_flag, err, code);
  __syncwarp();
}

// Key tiles of an entry (request x row tile): prefix tiles over the tokens
// that any of its rows sees, then tree tiles from the lowest visible node on.
struct Extent {
  int len, np, t0, nb;    // visible prefix, prefix tiles, first tree tile, all tiles
};
__device__ __forceinline__ Extent extent_of(const TcArgs& p, int e) {
  if (p.extents) {
    const int4 v = p.extents[e];
    const int np = (v.x + kKeys - 1) / kKeys;
    return Extent{v.x, np, v.y, np + v.z};
  }
  const int r = e / p.tiles;
  const bool live = e % p.tiles * p.nq < node_span(p.a, r).cnt;
  const int len = prefix_len(p.a, r), np = live ? (len + kKeys - 1) / kKeys : 0;
  return Extent{len, np, 0, np + (live ? 1 : 0)};
}

template <int D>
__global__ void __launch_bounds__(512, 1) attn_kernel(const __grid_constant__ TcArgs p) {
  using L = Lay<D>;
  static_assert(kTreeTile == kKeys, "tree tiles");
  extern __shared__ uint8_t smem_raw[];
  // aligned by an offset, so that the compiler still knows the pointer to be one to shared memory
  uint8_t* sm0 = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const AttnArgs& a = p.a;
  // the warp's number by a shuffle, so that the compiler knows all that follows from it to be uniform
  const int warp16 = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int team = warp16 >> 3, half = (warp16 >> 2) & 1;   // warpgroup of the team
  const int tid = threadIdx.x & 127, warp = warp16 & 3, lane = tid & 31, c0 = kCols * half;
  const int tbar = 1 + team, wid = 3 + 2 * team + half;
  const int g = a.Hq / a.Hkv;
  uint8_t* sm = sm0 + team * L::kTeam;
  const uint32_t sb = smem_u32(sm);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sm0 + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kPages + 44);
  long long* sums = reinterpret_cast<long long*>(sm0 + L::kMisc + 16);
  auto raw_bar = [&](int st) { return sb + L::kBars + 8u * st; };
  const uint32_t s_bar = sb + L::kBars + 8 * kStages, pv_bar = s_bar + 8;
  const uint32_t blk_bytes = static_cast<uint32_t>(a.page_size) * (D + 4);
  const int ps_shift = 31 - __clz(a.page_size), per_tile = kKeys >> ps_shift;
  if (tid == 0 && half == 0) {
    for (int i = 0; i < kStages + 2; ++i) mbar_init(sb + L::kBars + 8 * i, i < kStages ? per_tile : 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  griddep_wait();
  griddep_release();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = p.status0;   // an expired wait writes it seconds later
  if (threadIdx.x < 32) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(sm0 + L::kMisc)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }

  // ---- this team's run: [w0, w1) of the list of all units, each kUnitCost places and then its tiles
  const int E = a.B * p.tiles;
  const int per = ((E + 15) / 16 + 31) / 32 * 32;  // entries per warp
  auto cost_of = [&](int e, int end) {
    const int nb = e < end ? extent_of(p, e).nb : 0;
    return nb ? static_cast<long long>(nb + kUnitCost) * a.Hkv : 0ll;
  };
  {
    const int w16 = warp16, lo = min(w16 * per, E), hi = min(lo + per, E);
    long long s = 0;
    for (int e = lo; e < hi; e += 32) s += cost_of(e + lane, hi);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sums[w16] = s;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0) + 256 * team;
  long long W = 0;
  for (int w = 0; w < 16; ++w) W += sums[w];
  const long long G = min(2ll * p.grid, W);
  const int run = static_cast<int>(blockIdx.x) + p.grid * team;
  if (tid == 0 && half == 0) p.pieces.desc[run] = make_int4(0, 0, 0, 0);

  if (run < G) {
    const long long w0 = run * W / G, w1 = (run + 1) * W / G;
    int e = 0;
    long long before = 0;                        // places before entry e
    {
      int w = 0;
      while (before + sums[w] <= w0) before += sums[w++];
      const int hi = min(w * per + per, E);
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
    Extent x = extent_of(p, e);
    const int skip = static_cast<int>(w0 - before), at = skip % (x.nb + kUnitCost);
    int h = skip / (x.nb + kUnitCost), blk = max(0, at - kUnitCost);
    int left = static_cast<int>(w1 - w0) + at;   // places from the start of the unit to the end of the run
    // (a tile is in the run while kUnitCost + its index < left)

    // ---- loads: page i of a tile by the team's warp 7 - i, kStages tiles ahead, its number one more
    const int page_i = 7 - (warp16 & 7);
    const bool loader = page_i < per_tile;
    volatile uint8_t* staged = sm + L::kPages;
    int le = e, lh = h, lblk = blk, lleft = left, lnext = 0, lpage = -1, lr = e / p.tiles, lt = e % p.tiles;
    Extent lx = x;
    auto look = [&]() {                          // this warp's page of the next tile to load
      lpage = -1;
      if (lblk == lx.nb) {
        lblk = 0;
        lleft -= lx.nb + kUnitCost;
        if (kUnitCost >= lleft) return;
        if (++lh == a.Hkv) {
          lh = 0;
          do {
            lx = extent_of(p, ++le);
            if (++lt == p.tiles) { lt = 0; ++lr; }
          } while (lx.nb == 0 && le + 1 < E);
        }
      }
      if (kUnitCost + lblk >= lleft) return;
      const int key = lblk * kKeys + (page_i << ps_shift);
      if (lblk < lx.np && key < lx.len)
        lpage = a.block_table[static_cast<int64_t>(lr) * a.table_ld + (key >> ps_shift)];
    };
    // What the start of a unit and its tile of nodes read, on its way into L1 some tiles ahead.
    auto announce = [&]() {
      const Span sp = node_span(a, lr);
      const int node0 = lt * p.nq, nodes = min(p.nq, sp.cnt - node0);
      for (int i = lane; i < nodes * g; i += 32) {
        const uint16_t* row = static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(sp.n0 + node0 + i / g) * a.ldq +
                              static_cast<int64_t>(lh * g + i % g) * D;
        asm volatile("prefetch.global.L1 [%0];" ::"l"(row));
        if (D == 128) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + 64));
      }
    };
    auto load = [&](int st) {
      if (kUnitCost + lblk >= lleft) return;
      if (page_i == 0 && lblk == 0 && lnext > 0) announce();
      const bool wanted = lblk < lx.np && lblk * kKeys + (page_i << ps_shift) < lx.len;
      const int page = __shfl_sync(0xffffffffu, lpage, 0);
      const bool ok = wanted && page >= 0 && page < a.n_pages;
      if (elect()) {
        staged[8 * st + page_i] = ok;
        if (ok) {
          mbar_expect_tx(raw_bar(st), blk_bytes);
          bulk_load(sb + L::kRaw + st * L::kStage + page_i * blk_bytes,
                    a.cache + (static_cast<int64_t>(page) * a.Hkv + lh) * blk_bytes, blk_bytes, raw_bar(st));
        } else {
          mbar_arrive(raw_bar(st));
          if (wanted && a.err) *a.err = 1;
        }
      }
      __syncwarp();
      ++lblk;
      ++lnext;
    };
    if (loader) {
      look();
#pragma unroll 1
      for (int st = 0; st < kStages; ++st) {
        load(st);
        look();
      }
    }

    // ---- per thread: a key, then a dim, of each tile (half of its words)
    const uint32_t lane_off = static_cast<uint32_t>(32 * warp) << 16;
    const int slot = tid & (a.page_size - 1), page_off = (tid >> ps_shift) * static_cast<int>(blk_bytes);
    const int chunk_step = a.page_size * 16, key_off = page_off + slot * 16 + half * (D / 64) * chunk_step;
    const int scale_off = page_off + k_scale(a.page_size, D, slot);
    int group_off[4];                            // groups of 16 tokens of this half in the staged pages, at this dim
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k0 = 64 * half + 16 * i;
      group_off[i] = (k0 >> ps_shift) * static_cast<int>(blk_bytes) + a.page_size * (D / 2) +
                     (k0 & (a.page_size - 1)) * (D / 2) + tid * 8;
    }
    const int inv_g = 65536 / g + 1;             // row / g = row inv_g / 2^16 for the 64 rows and g <= 64
    auto node_of = [&](int row) { return row * inv_g >> 16; };
    const float c2 = a.scale * kLog2e;
    // a row's reference (what its scores are taken over) is kept negated; 0 while it has none
    float* nref = reinterpret_cast<float*>(sm + L::kRef) + c0;
    float* shift_s = reinterpret_cast<float*>(sm + L::kShift) + c0;
    float* corr_s = reinterpret_cast<float*>(sm + L::kCorr) + c0;
    float* inv_s = reinterpret_cast<float*>(sm + L::kInv) + c0;
    int* vis_s = reinterpret_cast<int*>(sm + L::kVis) + c0;
    int* row_s = reinterpret_cast<int*>(sm + L::kRow) + c0;
    float* wmax = reinterpret_cast<float*>(sm + L::kWarpMax) + 128 * half;   // [4][32]
    uint64_t l[kCols / 2];                       // this key's share of the rows' sums
#pragma unroll
    for (int c = 0; c < kCols / 2; ++c) l[c] = 0ull;
    volatile int* dirty = reinterpret_cast<volatile int*>(sm + L::kPages + 32);   // non-finite tree values met
    volatile int* low_vis = reinterpret_cast<volatile int*>(sm + L::kPages + 36);  // [2] prefix that all rows see
    bool force = false, fresh = true;            // a row without reference; a new unit
    // Threads 0 .. 31 of a warpgroup: row c0 + tid has no reference yet. Kept apart from its value: any number can be one
    // (a row of zeros has the reference 0).
    bool unset = true;
    bool aborted = false;                        // the team's vote ended the loop
    int seg_blk = blk, unit_e = -1, r = 0, t = 0, n0 = 0, cnt = 0;
    int st = 0, turn = 0, it = 0;
    for (;; ++it) {
      if (blk == x.nb) {                         // next unit
        left -= x.nb + kUnitCost;
        if (kUnitCost >= left) break;
        blk = seg_blk = 0;
        fresh = true;
        if (++h == a.Hkv) {
          h = 0;
          do x = extent_of(p, ++e);
          while (x.nb == 0 && e + 1 < E);
        }
      }
      if (kUnitCost + blk >= left) break;
      const bool first = fresh;
      if (fresh) {
        // the unit's queries, K-major with the 128-byte swizzle; its rows (all MMAs of the unit before have completed)
        fresh = false;
        if (e != unit_e) {                       // (else another KV head of the same rows)
          unit_e = e;
          r = e / p.tiles;
          t = e % p.tiles;
          const Span sp = node_span(a, r);
          n0 = sp.n0;
          cnt = sp.cnt;
        }
        const int node0 = t * p.nq, rows = min(p.nq, cnt - node0) * g;
#pragma unroll 4
        for (int i = tid + 128 * half; i < kRowsT * (D / 8); i += 256) {
          const int rr = i / (D / 8), c = i % (D / 8);
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (rr < rows)
            v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                static_cast<int64_t>(n0 + node0 + node_of(rr)) * a.ldq +
                                                static_cast<int64_t>(h * g + rr - node_of(rr) * g) * D + 8 * c);
          *reinterpret_cast<uint4*>(sm + L::kQ + (c >> 3) * L::kQHalf + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) = v;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (tid < kCols) {
          const int rr = c0 + tid, gn = n0 + node0 + node_of(rr);
          nref[tid] = 0.f;
          row_s[tid] = rr < rows ? gn * a.Hq + h * g + rr - node_of(rr) * g : -1;
          const int vis = rr < rows ? (a.vis_prefix ? a.vis_prefix[gn] : 0x7fffffff) : 0;
          vis_s[tid] = vis;
          const int lowest = __reduce_min_sync(0xffffffffu, rr < rows ? vis : 0x7fffffff);
          if (tid == 0) low_vis[half] = lowest;
        }
        force = false;
        unset = true;
        if (tid == 0 && half == 0) *dirty = 0;
        team_sync(tbar);
      }
      const bool tree = blk >= x.np, last = blk == x.nb - 1 || kUnitCost + blk + 1 >= left;
      const int key0 = (tree ? x.t0 + blk - x.np : blk) * kKeys;
      const int nkeys = min(kKeys, (tree ? cnt : x.len) - key0);
      team_wait(raw_bar(st), turn, abort_flag, p.status, 41);
      const uint8_t* raw = sm + L::kRaw + st * L::kStage;

      // ---- K: thread = key, half of the dims
      bool valid = tid < nkeys;
      uint32_t see = 0u;                         // tree tiles: this row's nodes, then this node's rows
      if (!tree) {
        uint4 w[D / 64];
#pragma unroll
        for (int c = 0; c < D / 64; ++c) w[c] = *reinterpret_cast<const uint4*>(raw + key_off + c * chunk_step);
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t v[16];
          decode8(w[c].x, v, p.magic);
          decode8(w[c].y, v + 4, p.magic);
          decode8(w[c].z, v + 8, p.magic);
          decode8(w[c].w, v + 12, p.magic);
          tmem_st16(tmem + L::tK + lane_off + half * (D / 4) + 16 * c, v);
        }
      } else {
        const uint16_t* row = static_cast<const uint16_t*>(a.k_tree) +
                              static_cast<int64_t>(n0 + key0 + min(tid, nkeys - 1)) * a.ldk + static_cast<int64_t>(h) * D +
                              half * (D / 2);   // (places without nodes: the last one, masked below)
        uint32_t v[D / 4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint4 w = *reinterpret_cast<const uint4*>(row + 8 * i);
          v[4 * i] = w.x; v[4 * i + 1] = w.y; v[4 * i + 2] = w.z; v[4 * i + 3] = w.w;
        }
        // the mask of row c0 + lane over the 32 nodes of this warp
        const int node0 = t * p.nq, node = node0 + node_of(c0 + lane), word = (key0 >> 6) + (warp >> 1);
        if (c0 + lane < min(p.nq, cnt - node0) * g && word < a.anc_words)
          see = reinterpret_cast<const uint32_t*>(a.anc + static_cast<int64_t>(n0 + node) * a.anc_words + word)[warp & 1];
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t u[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) u[i] = v[16 * c + i];
          tmem_st16(tmem + L::tK + lane_off + half * (D / 4) + 16 * c, u);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      team_sync(tbar);
      if (half == 0 && warp == 0 && elect()) {
        tc_fence_after();
        constexpr uint32_t idS = idesc_bf16(128, kRowsT, 0);
        const uint64_t qdesc = sdesc(sb + L::kQ, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)      // descriptors count 16 bytes
          umma_bf16_ts(tmem + L::tS, tmem + L::tK + 8 * kk, qdesc + ((kk >> 2) * L::kQHalf + (kk & 3) * 32) / 16, idS, kk > 0);
        umma_commit(s_bar);
      }
      __syncwarp();

      // ---- V^T: thread = dim, half of the tokens, once PV of the tile before has read the last one
      if (it > 0) team_wait(pv_bar, (it - 1) & 1, abort_flag, p.status, 42);
      tc_fence_after();
      if (32 * warp < D) {                       // d = 64: the upper lanes' results are not used
        if (!tree) {
          uint2 w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint2*>(raw + group_off[i]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t v[16];
            decode8(w[2 * c].x, v, p.magic);
            decode8(w[2 * c].y, v + 4, p.magic);
            decode8(w[2 * c + 1].x, v + 8, p.magic);
            decode8(w[2 * c + 1].y, v + 12, p.magic);
            tmem_st16(tmem + L::tV + lane_off + 32 * half + 16 * c, v);
          }
        } else {
          // a value that is not finite must not meet the zero weights of rows that do not see it: it is taken
          // out here and added at the end to the rows that see it
          bool bad = false;
          // lanes 2j, 2j + 1 read dims 2j, 2j + 1 of an even and of the next token and swap a half
          const uint16_t* rows = static_cast<const uint16_t*>(a.v_tree) + static_cast<int64_t>(n0 + key0) * a.ldv +
                                 static_cast<int64_t>(h) * D + (tid & ~1);
          const int ldv = static_cast<int>(a.ldv);
#pragma unroll 1
          for (int c = 2 * half; c < 2 * half + 2; ++c) {
            uint32_t v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0u;   // places without nodes are zeros
            if (32 * c < nkeys) {
              // all loads first (beyond the last node: that node again), in one latency
              const int k0 = 32 * c + (tid & 1);
              uint32_t odd = 0u;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                v[i] = *reinterpret_cast<const uint32_t*>(rows + static_cast<int64_t>(min(k0 + 2 * i, nkeys - 1)) * ldv);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                if (k0 + 2 * i >= nkeys) v[i] = 0u;
                odd |= (v[i] & 0x7f807f80u) + 0x00800080u;   // bits 15 and 31: an exponent of ones
              }
              if (__any_sync(0xffffffffu, odd & 0x80008000u)) {
                bad = true;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  if ((v[i] & 0x7f80u) == 0x7f80u) v[i] &= 0xffff0000u;
                  if ((v[i] & 0x7f800000u) == 0x7f800000u) v[i] &= 0x0000ffffu;
                }
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, v[i], 1);
                v[i] = tid & 1 ? __byte_perm(other, v[i], 0x7632) : __byte_perm(v[i], other, 0x5410);
              }
            }
            tmem_st16(tmem + L::tV + lane_off + 16 * c, v);
          }
          if (bad) *dirty = 1;
        }
      }
      // this key's scales
      float sk = c2, sv = 1.f;
      if (!tree) {
        valid = valid && staged[8 * st + (tid >> ps_shift)];
        sk = valid ? c2 * bf16_at(reinterpret_cast<const uint16_t*>(raw + scale_off)) : 0.f;
        sv = valid ? bf16_at(reinterpret_cast<const uint16_t*>(raw + scale_off + 2 * a.page_size)) : 0.f;
      }
      const int key = valid && !tree ? key0 + tid : 0x7fffffff;
      if (loader && it > 0) {                    // the stage of the tile before, which all have read
        load(st == 0 ? kStages - 1 : st - 1);
        look();
      }
      tmem_st_wait();

      if (tree) {                                // transpose the warp's 32 x 32 mask bits
        uint32_t low = 0x0000ffffu;
#pragma unroll
        for (int j = 16; j; j >>= 1, low ^= low << j) {
          const uint32_t w = __shfl_xor_sync(0xffffffffu, see, j);
          see = lane & j ? (see & ~low) | ((w >> j) & low) : (see & low) | ((w << j) & ~low);
        }
      }

      // ---- softmax: thread = key; scores in base-2 units over the rows' references, two rows to a register pair
      team_wait(s_bar, it & 1, abort_flag, p.status, 43);
      tc_fence_after();
      uint64_t y[kCols / 2];
      for (bool slow = first || force;;) {
      {
        const uint64_t sk2 = pair(sk, sk);
        uint32_t v[kCols];
        tmem_ld32(tmem + L::tS + lane_off + c0, v);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(nref + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) pin(v[c + i]);
          y[c / 2] = fma2(pair(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), sk2, m.x);
          y[c / 2 + 1] = fma2(pair(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])), sk2, m.y);
        }
      }
      if (__builtin_expect(tree || low_vis[half] < min(key0 + kKeys, x.len), 0)) {
        if (!tree) {
          see = 0u;
#pragma unroll 1
          for (int c = 0; c < kCols; c += 4) {
            const int4 q = *reinterpret_cast<const int4*>(vis_s + c);
            see |= ((key < q.x ? 1u : 0u) | (key < q.y ? 2u : 0u) | (key < q.z ? 4u : 0u) | (key < q.w ? 8u : 0u)) << c;
          }
        }
        if (!valid) see = 0u;
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) {
          float lo, hi;
          split(y[c], lo, hi);
          if (!((see >> (2 * c)) & 1u)) lo = -INFINITY;
          if (!((see >> (2 * c + 1)) & 1u)) hi = -INFINITY;
          y[c] = pair(lo, hi);
        }
      } else if (!__all_sync(0xffffffffu, valid)) {   // every row sees every valid key
        const uint64_t none = pair(-INFINITY, -INFINITY);
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) y[c] = valid ? y[c] : none;
      }
      if (__builtin_expect(slow, 0)) {
        // new references: the rows' maxima so far
        float mine = 0.f;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          float lo, hi;
          split(y[c / 2], lo, hi);
          const float v = redux_max(c & 1 ? hi : lo);
          if (lane == c) mine = v;
        }
        wmax[warp * kCols + lane] = mine;
        wg_sync(wid);
        bool none = false;
        if (tid < kCols) {
          const float top = max_nan(max_nan(wmax[tid], wmax[kCols + tid]), max_nan(wmax[2 * kCols + tid], wmax[3 * kCols + tid]));
          const float old = nref[tid];
          const bool empty = unset && top == -INFINITY;
          float sh = unset ? (empty ? 0.f : top) : fmaxf(top, 0.f);
          if (top != top) sh = top;
          nref[tid] = old - sh;                  // (none: old = 0, and sh = 0 if the row is still empty)
          none = row_s[tid] >= 0 && empty;
          corr_s[tid] = unset ? 0.f : ex2(-sh);
          shift_s[tid] = -sh;
          unset = empty;
        }
        force = any_of<128>(wid, none);
#pragma unroll
        for (int c = 0; c < kCols; c += 4) {
          const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(shift_s + c);
          const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(corr_s + c);
          y[c / 2] = add2(y[c / 2], m.x);
          y[c / 2 + 1] = add2(y[c / 2 + 1], m.y);
          l[c / 2] = mul2(l[c / 2], f.x);
          l[c / 2 + 1] = mul2(l[c / 2 + 1], f.y);
        }
        if (!first) {                            // (PV of the tile before has completed: waited for above)
#pragma unroll 1
          for (int c = 0; c < kCols; c += 16) {
            uint32_t o[16];
            tmem_ld16(tmem + L::tO + lane_off + c0 + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              pin(o[i]);
              o[i] = __float_as_uint(__uint_as_float(o[i]) * corr_s[c + i]);
            }
            tmem_st16(tmem + L::tO + lane_off + c0 + c, o);
          }
          tmem_st_wait();
        }
      }
      // ---- weights, times the value's scale -> P, one 128-byte swizzled row per key
      float mx[2] = {-INFINITY, -INFINITY};
      {
        const uint64_t sv2 = pair(sv, sv);
        uint8_t* prow = sm + L::kP + tid * 128;
        const bool bad = sv != sv && a.vis_prefix != nullptr;
#pragma unroll
        for (int c8 = 0; c8 < kCols / 8; ++c8) {
          uint32_t pk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 4 * c8 + i;
            float lo, hi;
            split(y[c], lo, hi);
            mx[i & 1] = max3(mx[i & 1], lo, hi);
            y[c] = pair(ex2(lo), ex2(hi));
            split(mul2(y[c], sv2), lo, hi);
            pk[i] = pack_bf16(lo, hi);
          }
          if (__builtin_expect(bad, 0)) {
            // a value row that was not finite: zero weights times its scale are NaN, rows that do not see it stay clean
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (key >= vis_s[8 * c8 + i]) pk[i >> 1] &= i & 1 ? 0x0000ffffu : 0xffff0000u;
          }
          *reinterpret_cast<uint4*>(prow + (((c8 + c0 / 8) ^ (tid & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_fence_before();
      // a score beyond a reference by 2^8: the same again over new references; a wait that expired: out of the loop
      slow = any_of<256>(tbar, *abort_flag != 0 || (!slow && fmaxf(mx[0], mx[1]) > 8.f));
      if (__builtin_expect(!slow, 1)) break;
      // The same for all threads: whoever raised it did so before the vote, there being no wait between two votes.
      aborted = *abort_flag != 0;
      if (aborted) break;
      }
      if (__builtin_expect(aborted, 0)) break;
      if (half == 1 && warp == 0 && elect()) {
        tc_fence_after();
        constexpr uint32_t idO = idesc_bf16(128, kRowsT, 1);
        const uint64_t pdesc = sdesc(sb + L::kP, 1024, 1024);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          umma_bf16_ts(tmem + L::tO, tmem + L::tV + 8 * kk, pdesc + kk * (2048 / 16), idO, kk > 0 || !first);
        umma_commit(pv_bar);
      }
      __syncwarp();
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) l[c] = add2(l[c], y[c]);
      if (++st == kStages) { st = 0; turn ^= 1; }
      ++blk;
      if (__builtin_expect(!last, 1)) continue;

      // ---- end of the unit's run here: sums over the keys' threads, then O^T
      const bool whole = seg_blk == 0 && blk == x.nb;
      const int64_t piece = 2 * run + (seg_blk == 0 ? 1 : 0);
      if (seg_blk == 0 && !whole && tid == 0 && half == 0) {
        const long long u1 = w1 - left + kUnitCost + x.nb;  // place after the unit
        const long long k = (u1 * G + W - 1) / W - 1;       // run of its last tile
        p.pieces.desc[run] = make_int4(static_cast<int>(k) - run + 1, r, t, h);
      }
      // reduce-scatter over the lanes: lane i ends with column i
      float ls[kCols];
#pragma unroll
      for (int c = 0; c < kCols / 2; ++c) {
        split(l[c], ls[2 * c], ls[2 * c + 1]);
        l[c] = 0ull;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int c = 0; c < o; ++c) {
          const float keep = up ? ls[c + o] : ls[c], give = up ? ls[c] : ls[c + o];
          ls[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
      }
      wmax[warp * kCols + lane] = ls[0];
      wg_sync(wid);
      if (tid < kCols) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) sum += wmax[w * kCols + tid];
        inv_s[tid] = sum == 0.f ? 0.f : 1.f / sum;
        const float m = -nref[tid];
        if (!whole) {
          p.pieces.ml[piece * kRowsT + c0 + tid] = make_float2(sum == 0.f ? kLow : m, sum);
        } else if (a.lse && row_s[tid] >= 0) {
          a.lse[row_s[tid]] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
        }
      }
      wg_sync(wid);
      team_wait(pv_bar, it & 1, abort_flag, p.status, 44);   // (expired: the next tile waits for the same phase)
      tc_fence_after();
      if (32 * warp < D) {
#pragma unroll 1
        for (int c = 0; c < kCols; c += 16) {
          uint32_t o[16];
          tmem_ld16(tmem + L::tO + lane_off + c0 + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) pin(o[i]);
          if (whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int row = row_s[c + i];
              const uint16_t f = static_cast<uint16_t>(pack_bf16(__uint_as_float(o[i]) * inv_s[c + i], 0.f));
              if (row >= 0) static_cast<uint16_t*>(a.out)[static_cast<int64_t>(row) * D + tid] = f;
            }
          } else {
            float* po = p.pieces.o + (piece * kRowsT + c0 + c) * D + tid;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (row_s[c + i] >= 0) po[i * D] = __uint_as_float(o[i]);
          }
        }
        if (__builtin_expect(*dirty, 0)) {
          // tree values that are not finite, added to the rows that see them (this thread wrote these elements)
          const uint16_t* col = static_cast<const uint16_t*>(a.v_tree) + static_cast<int64_t>(n0) * a.ldv +
                                static_cast<int64_t>(h) * D + tid;
#pragma unroll 1
          for (int j = 0; j < min(cnt, 64 * a.anc_words); ++j) {
            const uint32_t v = col[static_cast<int64_t>(j) * a.ldv];
            if ((v & 0x7f80u) != 0x7f80u) continue;
#pragma unroll 1
            for (int c = 0; c < kCols; ++c) {
              const int row = row_s[c];
              if (row < 0) continue;
              const uint64_t word = a.anc[static_cast<int64_t>(row / a.Hq) * a.anc_words + (j >> 6)];
              if (!((word >> (j & 63)) & 1ull)) continue;
              const float f = __uint_as_float(v << 16);
              if (whole) {
                uint16_t* o16 = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(row) * D + tid;
                *o16 = static_cast<uint16_t>(pack_bf16(bf16_at(o16) + f, 0.f));
              } else {
                p.pieces.o[(piece * kRowsT + c0 + c) * D + tid] += f;
              }
            }
          }
        }
      }
      tc_fence_before();
      team_sync(tbar);                           // all have read O and the rows' arrays: the next unit may begin
    }
    // All that was issued has been waited for, but after an expired wait: then PV of the tile before, S of the tile whose
    // vote ended the loop, and the copies of the staged tiles may be in flight still, and end before the CTA does.
    if (*abort_flag) {
      if (tid == 0) {
        if (it > 0) drain(pv_bar, (it - 1) & 1);
        if (aborted) drain(s_bar, it & 1);
      }
      if (loader)
        for (int i = max(0, lnext - kStages); i < lnext; ++i) drain(raw_bar(i % kStages), (i / kStages) & 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x < 32) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(misc[0]), "r"(512) : "memory");
  }
}

template <int D>
int launch(const TcArgs& p, cudaStream_t st) {
  if (!smem_limit(attn_kernel<D>, static_cast<int>(Lay<D>::kBytes))) return TV_ECUDA;
  const int rc = launch_pdl(attn_kernel<D>, dim3(p.grid), dim3(512), Lay<D>::kBytes, st, p);
  return rc != TV_OK ? rc : attn_join(p.a, p.pieces, p.status, 2 * p.grid, kRowsT, p.nq, st);
}

}  // namespace

// [status word (256 B)] [extents] [pieces of cut units]
size_t attn_tc_workspace(int B, int max_nodes, int Hq, int Hkv, int d) {
  const int nq = kRowsT / (Hq / Hkv);
  const size_t entries = static_cast<size_t>(B) * ((max_nodes + nq - 1) / nq);
  return 256 + align256(entries * sizeof(int4)) + pieces_bytes(2 * sm_count(), kRowsT, d);
}

int attn_tc(const AttnArgs& a, void* ws, cudaStream_t st) {
  TcArgs p{};
  p.a = a;
  p.magic = kMagic;
  p.grid = sm_count();
  p.nq = kRowsT / (a.Hq / a.Hkv);
  p.tiles = (a.max_nodes + p.nq - 1) / p.nq;
  char* base = static_cast<char*>(ws);
  p.status = reinterpret_cast<int*>(base);
  p.status0 = initial_status();
  int4* extents = reinterpret_cast<int4*>(base + 256);
  p.pieces = pieces_at(base + 256 + align256(static_cast<size_t>(a.B) * p.tiles * sizeof(int4)), 2 * p.grid, kRowsT);
  if (a.vis_prefix || a.max_nodes > kKeys) {
    const int rc = attn_extents(a, p.nq, p.tiles, extents, st);
    if (rc != TV_OK) return rc;
    p.extents = extents;
  }
  return a.d == 128 ? launch<128>(p, st) : launch<64>(p, st);
}

}  // namespace kv4
}  // namespace tv
