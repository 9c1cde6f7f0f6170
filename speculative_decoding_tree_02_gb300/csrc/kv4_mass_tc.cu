// kv4_attn_mass for many bf16 rows per KV head: tcgen05 path.
//
//   S [tokens x rows] = K Q^T,  m[t] = sum over rows of 2^(S f_t - l)
// with the tokens as the 128 tensor-memory lanes of an MMA: a thread owns a
// token, turns its codes into the A operand once (tensor memory, 64 columns at
// d = 128), and then sums over the columns of S in registers, the token's scale
// f_t being its own and the rows' -lse (l) a broadcast.  Nothing crosses lanes.
//
// A CTA = 256 tokens (two MMA tiles that share every staged row) of one
// (request, KV head):
//   warps 0..15   consumers, a warpgroup per tile and half of the columns:
//                 exponentials and sums
//   warps 16..19  copy 64 rows at a time into shared memory (cp.async, K-major,
//                 128-byte swizzle)
//   warp 20       the rows' lse and visible lengths
//   warp 21       issues the MMAs
// S has three buffers per tile, so that the MMAs run ahead of the exponentials.
// 8 requests of 1024 rows x 32 heads over 1024..4096 tokens: 193 us (39% of the
// measured matrix rate); 64 rows take a CTA 1000 cycles, of which the 16384
// exponentials are 512 and the issue slots 690.
//
// Every wait is bounded (2 s); a role whose wait expires raises the CTA's abort
// flag, all leave, and the CTA's scores become NaN, with 1 in *err.
#include <algorithm>

#include "kv4_device.cuh"
#include "kv4_mass.cuh"

namespace tv {
namespace kv4 {
namespace {

using namespace tc;

constexpr int kTok = 256;       // tokens of a CTA
constexpr int kRowsC = 64;      // rows of a chunk
constexpr int kSt = 6;          // staged chunks
constexpr int kLag = 3;         // of these on their way
constexpr int kBuf = 3;         // buffers of S per tile
constexpr int kPar = kBuf + 1;  // chunks whose lse and visible lengths are held
constexpr int kConsumers = 16;  // warps
constexpr int kThreadsT = 32 * (kConsumers + 6);
constexpr float kInf = __builtin_huge_valf();

template <int D>
struct MassLay {
  static constexpr uint32_t kHalf = kRowsC * 128;             // 64 rows x 64 dims
  static constexpr uint32_t kStage = (D / 64) * kHalf;
  static constexpr uint32_t kLse = kSt * kStage;              // float [kPar][64], negated
  static constexpr uint32_t kVis = kLse + kPar * 256;         // int [kPar][64]
  static constexpr uint32_t kSpan = kVis + kPar * 256;        // int2 [kPar][2] least and most visible of 32 rows
  static constexpr uint32_t kPart = kSpan + kPar * 16;        // float [2][256]
  static constexpr uint32_t kBars = kPart + 2048;             // full, empty [kSt], pfull [kPar], dfull, dempty [kBuf], done, K
  static constexpr uint32_t kMisc = kBars + 8 * (2 * kSt + kPar + 2 * kBuf + 2);
  // one CTA to an SM: it takes all of the tensor memory
  static constexpr uint32_t kBytes = kMisc + 64 + 1024 > 120 * 1024 ? kMisc + 64 + 1024 : 120 * 1024;
  static constexpr uint32_t tK = 2 * kBuf * kRowsC;           // tensor memory: S [2 tiles][kBuf][64], then K [2 tiles][D / 2]
  static_assert(tK + D <= 512, "tensor memory");
};

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(r));
  return r != 0;
}

template <int D>
__global__ void __launch_bounds__(kThreadsT, 1) mass_tc_kernel(const MassArgs a, const uint32_t parts, const uint32_t magic) {
  using L = MassLay<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ int s_first, s_abort, s_status;
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int r = blockIdx.z, h = blockIdx.y, g = a.Hq / a.Hkv;
  const uint32_t rank = parts > 1 ? cl::rank() : 0;
  const int t0 = static_cast<int>(blockIdx.x / parts) * kTok;
  auto full = [&](int s) { return sb + L::kBars + 8u * s; };
  auto empty = [&](int s) { return sb + L::kBars + 8u * (kSt + s); };
  auto pfull = [&](int s) { return sb + L::kBars + 8u * (2 * kSt + s); };
  auto dfull = [&](int s) { return sb + L::kBars + 8u * (2 * kSt + kPar + s); };
  auto dempty = [&](int s) { return sb + L::kBars + 8u * (2 * kSt + kPar + kBuf + s); };
  const uint32_t done = sb + L::kBars + 8u * (2 * kSt + kPar + 2 * kBuf), kready = done + 8;
  float* part = reinterpret_cast<float*>(sm + L::kPart);
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(sm + L::kMisc);
  volatile int* abort_flag = &s_abort;
  griddep_wait();
  griddep_release();
  const MassSpan sp = mass_span(a, r, &s_first);
  if (blockIdx.x == 0 && h == 0 && tid == 0 && sp.bad && a.err) *a.err = 1;
  if (t0 >= sp.len) return;                       // (all CTAs of the cluster alike)
  if (tid == 0) {
    for (int s = 0; s < kSt; ++s) { mbar_init(full(s), 128); mbar_init(empty(s), 1); }
    for (int s = 0; s < kPar; ++s) mbar_init(pfull(s), 1);
    for (int s = 0; s < kBuf; ++s) { mbar_init(dfull(s), 1); mbar_init(dempty(s), kConsumers); }
    mbar_init(done, 1);
    mbar_init(kready, kConsumers);
    s_abort = 0;
    s_status = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kConsumers + 5) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(sm + L::kMisc)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);

  // this CTA's chunks of rows: first, first + parts, ..
  const int64_t row = static_cast<int64_t>(r) * a.Hkv + h;
  const int rows = sp.count * g, all = (rows + kRowsC - 1) / kRowsC;
  int skip = 0;                                   // chunks whose rows see nothing of these tokens
  if (a.causal && !a.vis_prefix && t0 > sp.old)
    skip = static_cast<int>(min(static_cast<int64_t>(t0 - sp.old) * g, static_cast<int64_t>(rows)) / kRowsC);
  const int first = skip + static_cast<int>((rank + parts - skip % parts) % parts);
  const int chunks = first < all ? (all - first + static_cast<int>(parts) - 1) / static_cast<int>(parts) : 0;

  // consumers: the thread's tile, columns and token
  const int tile = (warp >> 2) & 1, half = (warp >> 3) & 1, t = t0 + (tid & 255);
  float fac = 0.f, sum = 0.f;
  bool ok = false;
  if (warp < kConsumers) {
    // ---- half of the token's key -> operand
    const int page = t < sp.len ? mass_page(a, r, t) : -1;
    if (t < sp.len && page < 0 && a.err) *a.err = 1;
    ok = page >= 0;
    const int slot = t & (a.P - 1);
    const uint8_t* blk = a.cache + (static_cast<int64_t>(max(page, 0)) * a.Hkv + h) * block_bytes(a.P, D);
    uint4 w[D / 64];
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      w[c] = make_uint4(0u, 0u, 0u, 0u);
      if (ok) w[c] = ldg_stream(blk + k_word(a.P, slot, 32 * (c + half * (D / 64))));
    }
    if (ok) fac = bf16_at(reinterpret_cast<const uint16_t*>(blk + k_scale(a.P, D, slot))) * (a.scale * kLog2e);
    const uint32_t to = tmem + L::tK + tile * (D / 2) + half * (D / 4) + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      uint32_t v[16];
      decode8(w[c].x, v, magic);
      decode8(w[c].y, v + 4, magic);
      decode8(w[c].z, v + 8, magic);
      decode8(w[c].w, v + 12, magic);
      tmem_st16(to + 16 * c, v);
    }
    tmem_st_wait();
    tc_fence_before();
    if (lane == 0) mbar_arrive(kready);
  }

  // i / g by a multiplication, exact for 0 <= i < 2^31: with 2^s >= g the factor m = floor(2^(31+s) / g) + 1 < 2^32 makes
  // i m / 2^(31+s) too large by i e / (g 2^(31+s)), 0 < e = m g - 2^(31+s) <= g <= 2^s, that is by less than 1 / g.
  const int shift = 31 + 32 - __clz(g - 1);
  const auto inv_g = static_cast<uint32_t>((1ull << shift) / g + 1);
  auto node_of = [&](int i) { return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(i)) * inv_g >> shift); };
  if (warp >= kConsumers && warp < kConsumers + 4) {
    // ---- copies of the rows
    const int p = tid - 32 * kConsumers;
    auto source = [&](int i) {                    // row i of the request's list: its place in q, -1: none
      if (i >= rows) return static_cast<int64_t>(-1);
      const int j = node_of(i);
      const int64_t src = static_cast<int64_t>(sp.base) + (a.path ? a.path[static_cast<int64_t>(r) * a.path_ld + j] : j);
      return src >= 0 && src < a.total_rows ? src * a.ldq + static_cast<int64_t>(h * g + i - j * g) * D : static_cast<int64_t>(-1);
    };
    // A thread copies the same 16 bytes of rows that lie kStep apart; with rows
    // in order and g dividing kStep these are a constant stride apart in q.
    constexpr int kStep = 128 / (D / 8);
    const int mine = p / (D / 8), x8 = 8 * (p % (D / 8));
    const uint32_t to = (p % (D / 8) >> 3) * L::kHalf + mine * 128 + (((p % (D / 8) & 7) ^ (mine & 7)) << 4);
    const bool even = !a.path && 8 % g == 0 && sp.base >= 0 && static_cast<int64_t>(sp.base) + sp.count <= a.total_rows;
    const int64_t stride = kStep / g * a.ldq;     // (even only)
    const uint16_t* from = static_cast<const uint16_t*>(a.q) + x8;
    if (even) {
      const int i = first * kRowsC + mine, j = node_of(i);
      from += (static_cast<int64_t>(sp.base) + j) * a.ldq + static_cast<int64_t>(h * g + i - j * g) * D;
    }
    for (int c = 0; c < chunks + kLag; ++c) {
      if (c < chunks) {
        const int s = c % kSt;
        if (c >= kSt && !warp_wait(empty(s), (c / kSt - 1) & 1, abort_flag, &s_status, 1)) break;
        const int i0 = (first + c * static_cast<int>(parts)) * kRowsC;
        const uint32_t stage = sb + s * L::kStage + to;
#pragma unroll
        for (int k = 0; k < kRowsC / kStep; ++k) {
          const int64_t at = even ? 0 : source(i0 + mine + kStep * k);
          const uint16_t* src = even ? from + k * stride : from + max(at, static_cast<int64_t>(0));
          const bool some = even ? i0 + mine + kStep * k < rows : at >= 0;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(stage + 128 * kStep * k), "l"(src), "r"(some ? 16 : 0)
                       : "memory");
        }
        if (even) from += static_cast<int64_t>(parts) * (kRowsC / kStep) * stride;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (c >= kLag) {                            // the chunk kLag before has arrived
        asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(full((c - kLag) % kSt));
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (warp == kConsumers + 4) {
    // ---- lse and visible lengths: lane = rows lane and lane + 32 of a chunk
    struct Two {
      float l[2];
      int vis[2];
    };
    auto params = [&](int c) {
      Two x;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = (first + c * static_cast<int>(parts)) * kRowsC + 32 * u + lane;
        x.l[u] = kInf;
        x.vis[u] = 0;
        if (c >= chunks || i >= rows) continue;
        const int j = node_of(i);
        const MassRow m = mass_row(a, sp, r, j);
        if (m.bad && a.err) *a.err = 1;
        if (m.bad) continue;
        x.l[u] = a.lse[m.src * a.Hq + h * g + i - j * g];
        x.vis[u] = m.vis;
      }
      return x;
    };
    Two now = params(0), next = params(1);        // loads take longer than a chunk
    for (int c = 0; c < chunks; ++c) {
      const Two later = params(c + 2);
      // Consumers that have loaded S of chunk c - kBuf are through with the chunk before it, whose place this is.
      // (A barrier may be waited for only by those without whom its next phase cannot end: a parity tells two phases
      // apart. Here that is chunk c's, for which the consumers wait for this warp.)
      if (c >= kBuf && !warp_wait(dempty(c % kBuf), (c / kBuf - 1) & 1, abort_flag, &s_status, 6)) break;
      const int q = c % kPar;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool none = now.l[u] == -kInf;      // (a row that saw nothing weighs nothing)
        if (none) now.vis[u] = 0;
        reinterpret_cast<float*>(sm + L::kLse)[q * kRowsC + 32 * u + lane] = none ? -kInf : -(now.l[u] * kLog2e);
        reinterpret_cast<int*>(sm + L::kVis)[q * kRowsC + 32 * u + lane] = now.vis[u];
        const int lo = __reduce_min_sync(0xffffffffu, now.vis[u]), hi = __reduce_max_sync(0xffffffffu, now.vis[u]);
        if (lane == 0) reinterpret_cast<int2*>(sm + L::kSpan)[2 * q + u] = make_int2(lo, hi);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(pfull(q));
      now = next;
      next = later;
    }
  } else if (warp == kConsumers + 5) {
    // ---- MMAs
    constexpr uint32_t id = idesc_bf16(128, kRowsC, 0);
    const bool keys = warp_wait(kready, 0, abort_flag, &s_status, 7);
    for (int c = 0; c < chunks && keys; ++c) {
      const int s = c % kSt, b = c % kBuf;
      if (c >= kBuf && !warp_wait(dempty(b), (c / kBuf - 1) & 1, abort_flag, &s_status, 2)) break;
      if (!warp_wait(full(s), (c / kSt) & 1, abort_flag, &s_status, 3)) break;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t desc = sdesc(sb + s * L::kStage, 16, 1024);
#pragma unroll
        for (int tile = 0; tile < 2; ++tile)
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)     // descriptors count 16 bytes
            umma_bf16_ts(tmem + (tile * kBuf + b) * kRowsC, tmem + L::tK + tile * (D / 2) + 8 * kk,
                         desc + ((kk >> 2) * L::kHalf + (kk & 3) * 32) / 16, id, kk > 0);
        umma_commit(empty(s));
        umma_commit(dfull(b));
      }
      __syncwarp();
    }
    // nothing is in flight when the CTA frees its tensor memory
    if (elect_one()) umma_commit(done);
    __syncwarp();
    if (!drain(done, 0)) *abort_flag = 1;
  } else {
    // ---- consumers
    const uint32_t from = tmem + tile * (kBuf * kRowsC) + 32 * half + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const int tile0 = t0 + 128 * tile;
    const uint64_t fac2 = pair(fac, fac);
    for (int c = 0; c < chunks; ++c) {
      const int b = c % kBuf, q = c % kPar;
      if (!warp_wait(pfull(q), (c / kPar) & 1, abort_flag, &s_status, 4)) break;
      const int2 v = reinterpret_cast<const int2*>(sm + L::kSpan)[2 * q + half];
      if (!warp_wait(dfull(b), (c / kBuf) & 1, abort_flag, &s_status, 5)) break;
      tc_fence_after();
      uint32_t x[32];
      tmem_ld32(from + b * kRowsC, x);
      tmem_ld_wait();
      tc_fence_before();
      if (lane == 0) mbar_arrive(dempty(b));
      if (v.y <= tile0) continue;                 // none of these rows sees the tile
      const float* nl = reinterpret_cast<const float*>(sm + L::kLse) + q * kRowsC + 32 * half;
      const int* vis = reinterpret_cast<const int*>(sm + L::kVis) + q * kRowsC + 32 * half;
      uint64_t s2[2] = {0ull, 0ull};
      if (v.x >= tile0 + 128) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(nl + i);
#pragma unroll
          for (int j = 0; j < 4; ++j) pin(x[i + j]);
          const uint64_t y0 = fma2(pair(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), fac2, l.x);
          const uint64_t y1 = fma2(pair(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), fac2, l.y);
          float lo, hi;
          split(y0, lo, hi);
          s2[0] = add2(s2[0], pair(ex2(lo), ex2(hi)));
          split(y1, lo, hi);
          s2[1] = add2(s2[1], pair(ex2(lo), ex2(hi)));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(nl + i);
          const int4 see = *reinterpret_cast<const int4*>(vis + i);
#pragma unroll
          for (int j = 0; j < 4; ++j) pin(x[i + j]);
          const uint64_t y0 = fma2(pair(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), fac2, l.x);
          const uint64_t y1 = fma2(pair(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])), fac2, l.y);
          float lo, hi;
          split(y0, lo, hi);
          s2[0] = add2(s2[0], pair(t < see.x ? ex2(lo) : 0.f, t < see.y ? ex2(hi) : 0.f));
          split(y1, lo, hi);
          s2[1] = add2(s2[1], pair(t < see.z ? ex2(lo) : 0.f, t < see.w ? ex2(hi) : 0.f));
        }
      }
      float lo, hi;
      split(add2(s2[0], s2[1]), lo, hi);
      sum += lo + hi;
    }
    part[tid] = ok ? sum : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kConsumers + 5) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(misc[0]), "r"(512) : "memory");
  }
  // ---- sums of the halves and parts, in order (of a CTA that gave up: NaN)
  if (s_abort) {
    if (warp < kConsumers) part[tid] = __uint_as_float(0x7fc00000u);
    if (tid == 0 && a.err) *a.err = 1;
  }
  if (parts > 1) cl::sync();
  else __syncthreads();
  if (rank == 0 && warp < 8) {
    float m = 0.f;
    for (uint32_t c = 0; c < parts; ++c)
      m += parts > 1 ? cl::peek(&part[tid], c) + cl::peek(&part[tid + 256], c) : part[tid] + part[tid + 256];
    if (t < sp.len) a.score_out[row * a.out_ld + t] = mass_before(a, sp, row, t) + m;
  }
  if (parts > 1) cl::sync();                      // no CTA leaves while another may read its shared memory
}

template <int D>
int launch(const MassArgs& a, int B, int parts, cudaStream_t st) {
  if (!smem_limit(mass_tc_kernel<D>, static_cast<int>(MassLay<D>::kBytes))) return TV_ECUDA;
  const dim3 grid(static_cast<unsigned>((a.max_len + kTok - 1) / kTok) * parts, a.Hkv, B);
  return cl::launch_pdl(mass_tc_kernel<D>, parts, grid, dim3(kThreadsT), MassLay<D>::kBytes, st, a,
                        static_cast<uint32_t>(parts), kMagic);
}

}  // namespace

int mass_tc(const MassArgs& a, int B, int d, cudaStream_t st) {
  // a cluster shares a tile's rows where the tiles alone leave SMs idle
  const int64_t tiles = static_cast<int64_t>((a.max_len + kTok - 1) / kTok) * a.Hkv * B;
  const int64_t chunks = (static_cast<int64_t>(a.max_rows) * (a.Hq / a.Hkv) + kRowsC - 1) / kRowsC;
  int parts = 1;
  while (parts < 8 && 4 * parts <= chunks && tiles * parts < sm_count()) parts *= 2;
  return d == 128 ? launch<128>(a, B, parts, st) : launch<64>(a, B, parts, st);
}

}  // namespace kv4
}  // namespace tv
