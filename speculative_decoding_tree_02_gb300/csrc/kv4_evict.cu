// Eviction from the paged 4-bit cache: kv4_evict_select chooses the tokens that
// a request keeps by their accumulated weights, kv4_compact moves them
// together.  Every KV head keeps tokens of its own, all heads of a request the
// same number.
#include <algorithm>

#include "cluster.cuh"
#include "kv4.cuh"

namespace tv {
namespace kv4 {
namespace {

// -------------------------------------------------------------------- select
struct SelectArgs {
  const float* score;
  const int32_t* cache_len;
  const int32_t* budget;
  int32_t* idx;
  float* score_out;
  int32_t* new_len;
  int32_t* err;
  int64_t score_ld, idx_ld, out_ld;
  int n_sink, n_recent, Hkv, max_len, slice;
};

// Order of the scores as unsigned integers: zeros alike, NaN below all.
__device__ __forceinline__ uint32_t score_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return x == x ? b ^ (b >> 31 ? 0xffffffffu : 0x80000000u) : 0u;
}

constexpr int kBins = 2048;
constexpr int kPick = 512;             // candidates that are compared directly

// A cluster of up to 8 CTAs = one (request, KV head); each CTA stages a slice
// of the row of scores in shared memory, so that the row is read once and
// score_out may be the same array.  The threshold is found by counting digits
// of the keys, 11 bits at a time (8 where the counts are added over a cluster,
// for fewer remote reads: 8 x 131072 scores 24 us against 35), until the digit
// that it lies in has at most 512 tokens, which are listed and compared with one
// another: one count for a few thousand scores.  Then kept tokens get their
// places from counts in index order, ties included.  512 threads, 1024 in a
// cluster of 8.  Latency bound: 64 x 8 rows of 512..4096 scores 16.7 us (8 at the
// median row, 16 on SMs with four of the longest), 8 rows of 131072 22.7 us.
template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs a, const uint32_t csize) {
  constexpr int kSelWarps = kSelThreads / 32;
  extern __shared__ __align__(16) float xs[];
  __shared__ uint32_t hist[2][kBins];
  __shared__ __align__(16) uint32_t cand[kPick];       // this CTA's candidates
  __shared__ __align__(16) uint32_t each[kPick];       // the cluster's
  __shared__ uint32_t n_cand;
  __shared__ uint32_t pub[2][2];                       // kept-for-sure and tied tokens of this CTA's slice
  __shared__ uint32_t wsum[kSelWarps][2];
  __shared__ uint32_t s_key, s_need, s_left;
  griddep_wait();
  griddep_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cl::rank();
  const int r = blockIdx.z, h = blockIdx.y;
  const int64_t row = static_cast<int64_t>(r) * a.Hkv + h;
  const int len = a.cache_len[r], want = a.budget[r];
  const bool bad = len < 0 || len > a.max_len;
  int n = bad ? 0 : min(len, max(want, 0));
  const bool cut = n > a.idx_ld;
  if (cut) n = static_cast<int>(a.idx_ld);
  if (rank == 0 && h == 0 && tid == 0) {
    a.new_len[r] = bad ? len : n;
    if ((bad || cut || want < 0) && a.err) *a.err = 1;
  }
  int32_t* idx = a.idx + row * a.idx_ld;
  for (int64_t j = n + static_cast<int64_t>(rank) * kSelThreads + tid; j < a.idx_ld;
       j += static_cast<int64_t>(csize) * kSelThreads)
    idx[j] = -1;
  if (n == 0) return;                                  // (the same in all CTAs of the cluster)

  // forced tokens: [0, ms) and [len - mr, len); of those between, `rest`
  const int ms = min(a.n_sink, n), mr = min(a.n_recent, n - ms);
  const int mid0 = ms, mid1 = len - mr, rest = n - ms - mr;
  const int i0 = min(len, static_cast<int>(rank) * a.slice), i1 = min(len, i0 + a.slice);
  const float* src = a.score + row * a.score_ld;
  // all on their way at once; slices start at multiples of 4
  const uint32_t xs0 = static_cast<uint32_t>(__cvta_generic_to_shared(xs));
  const bool vec = reinterpret_cast<uintptr_t>(src) % 16 == 0;
  const int i4 = vec ? i0 + (i1 - i0) / 4 * 4 : i0;
  for (int i = i0 + 4 * tid; i < i4; i += 4 * kSelThreads)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(xs0 + 4u * (i - i0)), "l"(src + i) : "memory");
  for (int i = i4 + tid; i < i1; i += kSelThreads)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(xs0 + 4u * (i - i0)), "l"(src + i) : "memory");
  asm volatile("cp.async.wait_all;" ::: "memory");

  // the `rest`-th highest key between, and how many of its equals are taken
  uint32_t key = 0, need = 0xffffffffu;                // everything between
  if (rest < mid1 - mid0) {
    if (rest == 0) {
      key = 0xffffffffu;                               // (above every key)
      need = 0;
    } else {
      uint32_t left = rest, known = 0;                 // bits of the key that are known, from the top
      const int j0 = max(i0, mid0), j1 = min(i1, mid1);
      key = 0;
      for (int b = tid; b < kBins; b += kSelThreads) hist[0][b] = 0;
      if (tid == 0) n_cand = 0;
      __syncthreads();
      const int own = csize > 1 ? 1 : 4;               // digits of a thread
      for (int pass = 0;; ++pass) {
        const int bits = min(csize > 1 ? 8 : 11, 32 - static_cast<int>(known)), down = 32 - static_cast<int>(known) - bits;
        uint32_t* hs = hist[pass & 1];
        for (int i = j0 + tid; i < j1; i += kSelThreads) {
          const uint32_t k = score_key(xs[i - i0]);
          if (known == 0 || (k ^ key) >> (32 - known) == 0) atomicAdd(&hs[(k >> down) & ((1u << bits) - 1u)], 1u);
        }
        if (csize > 1) cl::sync();
        else __syncthreads();
        // digits from the highest, `own` to a thread
        const int top = (1 << bits) - 1 - own * tid;
        uint32_t v[4] = {0, 0, 0, 0}, mine = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (u >= own || top < u) break;
          if (csize > 1) {
#pragma unroll
            for (uint32_t c = 0; c < 8; ++c)
              if (c < csize) v[u] += cl::peek(&hs[top - u], c);
          } else {
            v[u] = hs[top - u];
          }
          mine += v[u];
        }
        for (int b = tid; b < (1 << bits); b += kSelThreads) hist[(pass & 1) ^ 1][b] = 0;   // (its readers passed this barrier)
        uint32_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        if (lane == 31) wsum[warp][0] = inc;
        __syncthreads();
        uint32_t before = inc - mine;
        for (int w = 0; w < warp; ++w) before += wsum[w][0];
        if (before < left && left <= before + mine) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            if (before < left && left <= before + v[u]) {
              s_key = key | (static_cast<uint32_t>(top - u) << down);
              s_need = left - before;
              s_left = v[u];
            }
            before += v[u];
          }
        }
        __syncthreads();
        key = s_key;
        left = s_need;
        known += bits;
        if (known == 32 || s_left <= kPick) break;
      }
      if (known < 32) {                                // few candidates: each compares itself with all
        for (int i = j0 + tid; i < j1; i += kSelThreads) {
          const uint32_t k = score_key(xs[i - i0]);
          if ((k ^ key) >> (32 - known) == 0) cand[atomicAdd(&n_cand, 1u)] = k;
        }
        const uint32_t n_all = s_left;
        if (csize > 1) cl::sync();
        else __syncthreads();
        uint32_t to = 0;
        for (uint32_t c = 0; c < csize; ++c) {
          const uint32_t m = csize > 1 ? cl::peek(&n_cand, c) : n_cand;
          if (tid < static_cast<int>(m)) each[to + tid] = csize > 1 ? cl::peek(&cand[tid], c) : cand[tid];
          to += m;
        }
        if (tid < 4 && n_all + tid < kPick) each[n_all + tid] = 0;   // (pads the last four; key 0 is below or equal to all)
        __syncthreads();
        const uint32_t k = tid < static_cast<int>(n_all) ? each[tid] : 0;
        uint32_t more = 0, same = 0;
        if (32 * warp < static_cast<int>(n_all))
          for (uint32_t j = 0; j < n_all; j += 4) {
            const uint4 o = *reinterpret_cast<const uint4*>(&each[j]);
            more += (o.x > k) + (o.y > k) + (o.z > k) + (o.w > k);
            same += (o.x == k) + (o.y == k) + (o.z == k) + (o.w == k);
          }
        if (tid < static_cast<int>(n_all) && more < left && left <= more + same) {
          s_key = k;
          s_need = left - more;
        }
        __syncthreads();
        key = s_key;
        left = s_need;
      }
      need = left;
    }
  }
  __syncthreads();

  // places: a warp owns a run of the slice
  const int run = ((i1 - i0 + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(i1, i0 + warp * run), w1 = min(i1, w0 + run);
  auto sure = [&](int i, uint32_t k) { return i < mid0 || i >= mid1 || k > key; };
  uint32_t n_sure = 0, n_tie = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = score_key(xs[i - i0]);
    const bool s = sure(i, k);
    n_sure += s;
    n_tie += !s && k == key;
  }
  n_sure = __reduce_add_sync(0xffffffffu, n_sure);
  n_tie = __reduce_add_sync(0xffffffffu, n_tie);
  if (lane == 0) { wsum[warp][0] = n_sure; wsum[warp][1] = n_tie; }
  __syncthreads();
  uint32_t at_sure = 0, at_tie = 0;
  for (int w = 0; w < warp; ++w) { at_sure += wsum[w][0]; at_tie += wsum[w][1]; }
  if (csize > 1) {
    if (tid == 0) {
      uint32_t s = 0, t = 0;
      for (int w = 0; w < kSelWarps; ++w) { s += wsum[w][0]; t += wsum[w][1]; }
      pub[0][0] = s;
      pub[0][1] = t;
    }
    cl::sync();                                        // (also: every score is staged before one is written)
    for (uint32_t c = 0; c < rank; ++c) { at_sure += cl::peek(&pub[0][0], c); at_tie += cl::peek(&pub[0][1], c); }
  }
  float* out = a.score_out ? a.score_out + row * a.out_ld : nullptr;
  for (int b = w0; b < w1; b += 32) {
    const int i = b + lane;
    const bool in = i < w1;
    const float x = in ? xs[i - i0] : 0.f;
    const uint32_t k = score_key(x);
    const bool s = in && sure(i, k), t = in && !s && k == key;
    const unsigned ms_ = __ballot_sync(0xffffffffu, s), mt = __ballot_sync(0xffffffffu, t);
    const unsigned below = (1u << lane) - 1u;
    const uint32_t ties = at_tie + __popc(mt & below);
    if (s || (t && ties < need)) {
      const uint32_t j = at_sure + __popc(ms_ & below) + min(ties, need);
      idx[j] = i;
      if (out) out[j] = x;
    }
    at_sure += __popc(ms_);
    at_tie += __popc(mt);
  }
  if (csize > 1) cl::sync();                           // no CTA leaves while another may read its shared memory
}

// ------------------------------------------------------------------- compact
struct CompactArgs {
  uint8_t* cache;
  const int32_t* block_table;
  const int32_t* dst_table;     // NULL: in place
  const int32_t* cache_len;
  const int32_t* new_len;
  const int32_t* idx;
  int32_t* err;
  int64_t idx_ld;
  int n_pages, P, table_ld, dst_ld, Hkv, max_keep;
};

constexpr int kWin = 64;        // tokens that D threads move at a time

// What a window's threads share: where its tokens come from and its groups go.
struct Window {
  int4 v[kWin];                 // address of the token's value word at dim 0, rotation that brings its nibble to bit 0
  int64_t block[kWin];          // byte offset of its source block, -1: does not move
  int slot[kWin];
  int64_t to[kWin / 16];        // byte offset of the destination block of 16 tokens, -1: none
  uint32_t live[kWin / 32];     // tokens that move
};

// D threads move a window of 64 kept tokens of one (request, KV head): keys
// and scales token by token in 16-byte units, values dim by dim (thread = dim):
// the 16 nibbles of a destination word are picked from the words of their
// source groups, each rotated into place.  A group of the destination belongs
// to one window, so words are written whole; nibbles of tokens that do not move
// are kept.
//   kInPlace: the windows of a (request, KV head) are taken in order by one
//   cluster, blockDim.y windows to a CTA at a time.  Kept tokens only move
//   towards the front, so what one round writes lies before all that later
//   rounds read; one cluster barrier between a round's reads and its writes
//   makes that hold inside the round too.
//   else: every window is a CTA of its own.
// Kept tokens among others that go cost whole sectors: 24341 of 72097 tokens of 8
// heads of 128 (25.7 MB) read 75 MB.  27.6 us from cold caches, 36% of the DRAM's
// peak; waits for memory (resolving a token is three dependent loads).
template <int D, bool kInPlace>
__global__ void __launch_bounds__(kInPlace ? 4 * D : D) compact_kernel(const CompactArgs a) {
  __shared__ Window win[kInPlace ? 4 : 1];
  griddep_wait();
  griddep_release();
  const int dim = threadIdx.x, y = threadIdx.y;
  Window& sh = win[kInPlace ? y : 0];
  const int r = blockIdx.z, h = blockIdx.y;
  const int len = a.cache_len[r];
  int n = a.new_len[r];
  const int64_t cap = static_cast<int64_t>(a.table_ld) * a.P;
  const int32_t* table = a.block_table + static_cast<int64_t>(r) * a.table_ld;
  const int32_t* dtable = kInPlace ? table : a.dst_table + static_cast<int64_t>(r) * a.dst_ld;
  const int dld = kInPlace ? a.table_ld : a.dst_ld;
  const int32_t* idx = a.idx + (static_cast<int64_t>(r) * a.Hkv + h) * a.idx_ld;
  const int ps = 31 - __clz(a.P);
  if (n > a.max_keep || n < 0) {
    if (blockIdx.x == 0 && h == 0 && dim == 0 && y == 0 && a.err) *a.err = 1;
    n = max(0, min(n, a.max_keep));
  }
  constexpr int kUnits = kWin * (D / 32) / D;   // 16-byte units of keys per thread: 2
  for (int w = kInPlace ? (blockIdx.x * blockDim.y) : blockIdx.x;; w += gridDim.x * blockDim.y) {
    // a CTA of a cluster stays for the barriers as long as any of its CTAs has a window
    if ((kInPlace ? w - static_cast<int>(blockIdx.x * blockDim.y) : w) * kWin >= n) return;
    const int j0 = (w + y) * kWin;
    bool bad = false;
    if (dim < kWin) {
      const int j = j0 + dim;
      int64_t blk = -1;
      int slot = 0;
      if (j < n) {
        const int t = idx[j];
        bad = true;
        if (t >= 0 && t < len && t < cap) {
          const int page = table[t >> ps];
          if (page >= 0 && page < a.n_pages) {
            bad = false;
            slot = t & (a.P - 1);
            if (!kInPlace || t != j) blk = (static_cast<int64_t>(page) * a.Hkv + h) * block_bytes(a.P, D);
          }
        }
      }
      int64_t to = -1;
      if (dim % 16 == 0 && j < n) {
        const int page = (j >> ps) < dld ? dtable[j >> ps] : -1;
        if (page >= 0 && page < a.n_pages) to = (static_cast<int64_t>(page) * a.Hkv + h) * block_bytes(a.P, D);
        else bad = true;
        sh.to[dim / 16] = to;
      }
      to = __shfl_sync(0xffffffffu, to, dim & 16);
      if (to < 0) blk = -1;                     // nowhere to go
      sh.block[dim] = blk;
      sh.slot[dim] = slot;
      const uint64_t at = reinterpret_cast<uint64_t>(a.cache) +
                          (blk >= 0 ? blk + v_group(a.P, D, slot >> 4, 0) + ((slot >> 3) & 1) * 4 : 0);
      sh.v[dim] = make_int4(static_cast<int>(at), static_cast<int>(at >> 32), 32 - 4 * nibble_of(slot & 7), 0);
      const unsigned live = __ballot_sync(0xffffffffu, blk >= 0);
      if ((dim & 31) == 0) sh.live[dim >> 5] = live;
    }
    __syncthreads();
    // reads
    uint4 kc[kUnits];
    uint2 vw[kWin / 16];
    uint16_t sc[2 * kWin / D];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int unit = u * D + dim, i = unit % kWin, c = unit / kWin;
      const int64_t blk = sh.block[i];
      if (blk >= 0) kc[u] = *reinterpret_cast<const uint4*>(a.cache + blk + k_word(a.P, sh.slot[i], 32 * c));
    }
#pragma unroll
    for (int u = 0; u < 2 * kWin / D; ++u) {
      const int unit = u * D + dim, i = unit % kWin;
      const int64_t blk = sh.block[i];
      if (blk >= 0)
        sc[u] = *reinterpret_cast<const uint16_t*>(
            a.cache + blk + (unit < kWin ? k_scale(a.P, D, sh.slot[i]) : v_scale(a.P, D, sh.slot[i])));
    }
#pragma unroll
    for (int q = 0; q < kWin / 16; ++q) {
      vw[q] = make_uint2(0u, 0u);
      if (((sh.live[q >> 1] >> (16 * (q & 1))) & 0xffffu) == 0u) continue;
      uint32_t word[16];
      int turn[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {            // (tokens that do not move: some word, masked when it is stored)
        const int4 t = sh.v[16 * q + e];
        const uint64_t at = static_cast<uint32_t>(t.x) | static_cast<uint64_t>(static_cast<uint32_t>(t.y)) << 32;
        word[e] = *reinterpret_cast<const uint32_t*>(at + 8u * dim);
        turn[e] = t.z;
      }
      uint32_t v[2] = {0u, 0u};
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int to = 4 * nibble_of(e & 7);
        v[e >> 3] |= __funnelshift_l(word[e], word[e], turn[e] + to) & (15u << to);
      }
      vw[q] = make_uint2(v[0], v[1]);
    }
    if constexpr (kInPlace) cl::sync();
    // writes
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int unit = u * D + dim, i = unit % kWin, c = unit / kWin;
      if (sh.block[i] < 0) continue;
      *reinterpret_cast<uint4*>(a.cache + sh.to[i >> 4] + k_word(a.P, (j0 + i) & (a.P - 1), 32 * c)) = kc[u];
    }
#pragma unroll
    for (int u = 0; u < 2 * kWin / D; ++u) {
      const int unit = u * D + dim, i = unit % kWin, slot = (j0 + i) & (a.P - 1);
      if (sh.block[i] < 0) continue;
      *reinterpret_cast<uint16_t*>(a.cache + sh.to[i >> 4] + (unit < kWin ? k_scale(a.P, D, slot) : v_scale(a.P, D, slot))) =
          sc[u];
    }
#pragma unroll
    for (int q = 0; q < kWin / 16; ++q) {
      const uint32_t live = (sh.live[q >> 1] >> (16 * (q & 1))) & 0xffffu;
      if (live == 0u) continue;
      uint2* dst = reinterpret_cast<uint2*>(a.cache + sh.to[q] + v_group(a.P, D, ((j0 + 16 * q) & (a.P - 1)) >> 4, dim));
      uint2 v = vw[q];
      if (live != 0xffffu) {
        uint32_t m[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (live >> e & 1u) m[e >> 3] |= 15u << (4 * nibble_of(e & 7));
        const uint2 old = *dst;
        v.x = (v.x & m[0]) | (old.x & ~m[0]);
        v.y = (v.y & m[1]) | (old.y & ~m[1]);
      }
      *dst = v;
    }
    if (bad && a.err) *a.err = 1;
    if constexpr (!kInPlace) return;
    __syncthreads();                                   // (the next round rewrites the window)
  }
}

}  // namespace
}  // namespace kv4
}  // namespace tv

using namespace tv;

namespace {
// CTAs of a cluster of select_kernel: as many as leave each a slice of at most
// 4096 scores, at most 8.
constexpr int kSlice = 4096, kMaxSlice = 49152;
int select_cluster(int max_len) {
  int c = 1;
  while (c < 8 && (max_len + c - 1) / c > kSlice) c *= 2;
  return c;
}
}  // namespace

TV_API int kv4_evict_select(const float* score, int64_t score_ld, const int32_t* cache_len, const int32_t* budget,
                            int n_sink, int n_recent, int B, int Hkv, int max_len, int32_t* idx, int64_t idx_ld,
                            float* score_out, int64_t score_out_ld, int32_t* new_len, int32_t* err,
                            tv_stream_t stream) {
  if (B < 0 || Hkv <= 0 || max_len < 0 || n_sink < 0 || n_recent < 0 || idx_ld < 0 || score_ld < max_len)
    return TV_EINVAL;
  if (score_out && score_out_ld < std::min<int64_t>(idx_ld, max_len)) return TV_EINVAL;
  if (B > 65535 || Hkv > 65535 || max_len > 8 * kMaxSlice) return TV_EUNSUPPORTED;
  if (B == 0) return TV_OK;
  if (!cache_len || !budget || !new_len || new_len == cache_len || new_len == budget) return TV_EINVAL;
  if ((max_len > 0 && !score) || (idx_ld > 0 && !idx)) return TV_EINVAL;
  if (score_out && score_out == score && score_out_ld != score_ld) return TV_EINVAL;
  const int c = select_cluster(max_len), slice = ((max_len + c - 1) / c + 3) / 4 * 4;
  const int bytes = std::max(slice, 4) * 4;
  if (bytes > 24 << 10 && !smem_limit(kv4::select_kernel<512>, kMaxSlice * 4)) return TV_ECUDA;
  if (c == 8 && !smem_limit(kv4::select_kernel<1024>, kMaxSlice * 4)) return TV_ECUDA;
  const kv4::SelectArgs a{score, cache_len, budget, idx, score_out, new_len, err, score_ld, idx_ld, score_out_ld,
                          n_sink, n_recent, Hkv, max_len, slice};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(c, Hkv, B);
  const auto cs = static_cast<uint32_t>(c);
  return c == 8 ? cl::launch_pdl(kv4::select_kernel<1024>, c, grid, dim3(1024), bytes, st, a, cs)
                : cl::launch_pdl(kv4::select_kernel<512>, c, grid, dim3(512), bytes, st, a, cs);
}

TV_API int kv4_compact(void* cache, int n_pages, int page_size, const int32_t* block_table, int table_ld,
                       const int32_t* cache_len, const int32_t* idx, int64_t idx_ld, const int32_t* new_len, int B,
                       int max_keep, const int32_t* dst_table, int dst_ld, int Hkv, int d, int32_t* err,
                       tv_stream_t stream) {
  if (B < 0 || max_keep < 0 || n_pages < 0 || table_ld < 0 || dst_ld < 0 || Hkv <= 0 || page_size <= 0 || idx_ld < 0)
    return TV_EINVAL;
  if (!kv4::page_size_ok(page_size) || (d != 64 && d != 128)) return TV_EUNSUPPORTED;
  if (B > 65535 || Hkv > 65535 || static_cast<int64_t>(table_ld) * page_size > 0x7fffffffll ||
      static_cast<int64_t>(dst_ld) * page_size > 0x7fffffffll || max_keep > 0x7fffffff - 4096)
    return TV_EUNSUPPORTED;
  if (max_keep > idx_ld) return TV_EINVAL;
  if (B == 0 || max_keep == 0) return TV_OK;
  if ((n_pages > 0 && !cache) || (table_ld > 0 && !block_table) || !cache_len || !idx || !new_len || !aligned(cache, 16))
    return TV_EINVAL;
  if (dst_table == block_table) dst_table = nullptr;    // in place
  const kv4::CompactArgs a{static_cast<uint8_t*>(cache), block_table, dst_table, cache_len, new_len, idx, err, idx_ld,
                           n_pages, page_size, table_ld, dst_ld, Hkv, max_keep};
  const int windows = (max_keep + kv4::kWin - 1) / kv4::kWin;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dst_table)
    return d == 128 ? launch_pdl(kv4::compact_kernel<128, false>, dim3(windows, Hkv, B), dim3(128), 0, st, a)
                    : launch_pdl(kv4::compact_kernel<64, false>, dim3(windows, Hkv, B), dim3(64), 0, st, a);
  // in place: four windows to a CTA, clusters large enough that the (request, head) pairs fill the SMs
  int c = 1;
  while (c < 8 && 4 * c < windows && static_cast<int64_t>(B) * Hkv * c < 2ll * sm_count()) c *= 2;
  return d == 128
             ? cl::launch_pdl(kv4::compact_kernel<128, true>, c, dim3(c, Hkv, B), dim3(128, 4), 0, st, a)
             : cl::launch_pdl(kv4::compact_kernel<64, true>, c, dim3(c, Hkv, B), dim3(64, 4), 0, st, a);
}
