// kv4_attn_mass: attention weight that cached tokens receive,
//   m[t] = sum over rows i and the query heads of t's KV head of exp(scale q_i.k_t - lse_i),
// the weights being those of an attention whose log-sum-exp is given: no
// maximum, no second pass, and every token is independent of the others.
// Here the kernels for fp32 rows (CUDA cores) and for few bf16 rows (mma.sync), and the entry point.
#include <algorithm>

#include "kv4_device.cuh"
#include "kv4_mass.cuh"

namespace tv {
namespace kv4 {
namespace {

constexpr int kTile = 128;      // tokens of a CTA
constexpr float kInf = __builtin_huge_valf();

// Sums of the parts of a cluster (each part took its share of the rows), in
// the order of their ranks; the first writes.
__device__ __forceinline__ void finish(const MassArgs& a, const MassSpan& sp, int64_t row, int t, bool page_ok, float mine,
                                       float* part, uint32_t rank, uint32_t parts) {
  // `mine` belongs to token t, thread = token
  if (parts > 1) {
    part[threadIdx.x] = mine;
    cl::sync();
    if (rank == 0) {
      mine = 0.f;
      for (uint32_t c = 0; c < parts; ++c) mine += cl::peek(&part[threadIdx.x], c);
    }
    cl::sync();
  }
  if (rank == 0 && t < sp.len) a.score_out[row * a.out_ld + t] = mass_before(a, sp, row, t) + (page_ok ? mine : 0.f);
}

// ------------------------------------------------------------------ fp32 rows
constexpr int kSimtRows = 32;   // rows staged at a time

// Thread = token: its key stays in registers, rows pass through shared memory
// (bf16 MMAs would lose bits of fp32 rows).  60 rows of 4 heads of 64 over 128
// tokens: 14.5 us with the call, which is most of it.
template <int D>
__global__ void __launch_bounds__(kTile) simt_kernel(const MassArgs a, const uint32_t parts) {
  __shared__ __align__(16) float qs[kSimtRows][D];
  __shared__ float s_lse[kSimtRows];
  __shared__ int s_vis[kSimtRows];
  __shared__ float part[kTile];
  __shared__ int s_first;
  griddep_wait();
  griddep_release();
  const int tid = threadIdx.x, r = blockIdx.z, h = blockIdx.y, g = a.Hq / a.Hkv;
  const uint32_t rank = parts > 1 ? cl::rank() : 0;
  const int t0 = static_cast<int>(blockIdx.x / parts) * kTile, t = t0 + tid;
  const MassSpan sp = mass_span(a, r, &s_first);
  if (blockIdx.x == 0 && h == 0 && tid == 0 && sp.bad && a.err) *a.err = 1;
  if (t0 >= sp.len) return;                       // (all CTAs of the cluster alike)
  const int64_t row = static_cast<int64_t>(r) * a.Hkv + h;
  float k[D];
  bool page_ok = false;
  {
    float sc = 0.f;
    const int page = t < sp.len ? mass_page(a, r, t) : -1;
    if (t < sp.len && page < 0 && a.err) *a.err = 1;
    page_ok = page >= 0;
    const uint8_t* blk = a.cache + (static_cast<int64_t>(max(page, 0)) * a.Hkv + h) * block_bytes(a.P, D);
    const int slot = t % a.P;
    if (page_ok) sc = bf16_at(reinterpret_cast<const uint16_t*>(blk + k_scale(a.P, D, slot)));
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (page_ok) w = *reinterpret_cast<const uint4*>(blk + k_word(a.P, slot, 32 * c));
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) k[32 * c + 8 * i + e] = sc * decode(v[i], e);
    }
  }
  const int rows = sp.count * g;
  const float fac = a.scale * kLog2e;
  float sum = 0.f;
  for (int i0 = static_cast<int>(rank) * kSimtRows; i0 < rows; i0 += static_cast<int>(parts) * kSimtRows) {
    __syncthreads();
    if (tid < kSimtRows) {
      int vis = 0;
      float l = kInf;
      if (i0 + tid < rows) {
        const MassRow m = mass_row(a, sp, r, (i0 + tid) / g);
        if (m.bad && a.err) *a.err = 1;
        if (!m.bad) {
          l = a.lse[m.src * a.Hq + h * g + (i0 + tid) % g];
          vis = l == -kInf ? 0 : m.vis;           // (a row that saw nothing weighs nothing)
        }
      }
      s_vis[tid] = vis;
      s_lse[tid] = l * kLog2e;
    }
    for (int u = tid; u < kSimtRows * (D / 4); u += kTile) {
      const int i = u / (D / 4), c = u % (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + i < rows) {
        const MassRow m = mass_row(a, sp, r, (i0 + i) / g);
        if (!m.bad)
          v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + m.src * a.ldq +
                                               static_cast<int64_t>(h * g + (i0 + i) % g) * D + 4 * c);
      }
      *reinterpret_cast<float4*>(&qs[i][4 * c]) = v;
    }
    __syncthreads();
    const int some = min(kSimtRows, rows - i0);
    for (int i = 0; i < some; ++i) {
      if (s_vis[i] <= t0) continue;
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < D / 4; ++c) {
        const float4 v = *reinterpret_cast<const float4*>(&qs[i][4 * c]);
        s[0] = fmaf(v.x, k[4 * c], s[0]);
        s[1] = fmaf(v.y, k[4 * c + 1], s[1]);
        s[2] = fmaf(v.z, k[4 * c + 2], s[2]);
        s[3] = fmaf(v.w, k[4 * c + 3], s[3]);
      }
      const float w = ex2(fmaf((s[0] + s[1]) + (s[2] + s[3]), fac, -s_lse[i]));
      if (t < s_vis[i]) sum += w;
    }
  }
  finish(a, sp, row, t, page_ok, sum, part, rank, parts);
}

// ------------------------------------------------------------------ bf16 rows
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool some) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}

// S = K Q^T with tokens as the rows of the MMA: a warp owns 32 tokens at a
// time, whose codes it turns into operands once and keeps in registers (64 at
// d = 128), and passes over all rows, eight at a time.  The dims are permuted
// alike in both operands so that a lane's share of a token is d / 4 consecutive
// dims, whole words of codes, and its share of a query row is one run of the
// row: staged in fragment order, a block of eight rows is read back in 16-byte
// accesses without conflicts.  The scale of a token and the -lse of a row enter
// in the exponent, exp(scale s_t (n.q) - lse) = 2^(acc f_t - l).
// The query rows of a KV head, kFewRows at most, stay in shared memory and a warp
// walks over tiles of 32 tokens, the next tile's codes on their way
// while it works on one.

// 64 requests over 512..4096 tokens, 8 heads of 128: 4 rows per head 31.1 us (42%
// of the measured copy rate for 66 bytes a token and head and the scores), 4..64
// rows 59.5 us; bound by issue slots (550 instructions per tile, 176 of them the
// codes), then by the rate of mma.sync (16 for eight rows; more
// chains side by side made no difference).
template <int D>
__global__ void __launch_bounds__(kTile, 4) few_kernel(const MassArgs a, const int run, const uint32_t magic) {
  constexpr int kRun = D / 32;                    // words, and 16-byte units of a row, of a lane
  constexpr int kBlock = 8 * D * 2;               // bytes of eight rows
  extern __shared__ __align__(16) uint8_t qs[];
  __shared__ __align__(8) float s_lse[kFewRows];
  __shared__ __align__(8) int s_vis[kFewRows];
  __shared__ int64_t s_at[kFewRows];              // places in q, -1: none
  __shared__ int2 s_span[kFewRows / 8];           // least and most that a block's rows see
  __shared__ int s_first;
  griddep_wait();
  griddep_release();
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int r = blockIdx.z, h = blockIdx.y, g = a.Hq / a.Hkv;
  const MassSpan sp = mass_span(a, r, &s_first);
  if (blockIdx.x == 0 && h == 0 && tid == 0 && sp.bad && a.err) *a.err = 1;
  const int t_lo = static_cast<int>(blockIdx.x) * run, t_hi = min(t_lo + run, sp.len);
  if (t_lo >= t_hi) return;
  const int64_t row = static_cast<int64_t>(r) * a.Hkv + h;
  const int rows = sp.count * g, blocks = (rows + 7) / 8;

  // a warp's tile: codes of tokens t + 8 i (t = the tile's first + lane / 4), and what its own token had
  struct Tile {
    uint32_t w[4][kRun];
    uint16_t sc[4];
    float had;
    int page[2];                                  // of tokens 0..15 and 16..31 of the tile
  };
  const int32_t* table = a.block_table + static_cast<int64_t>(r) * a.table_ld;
  const int ps = 31 - __clz(a.P);
  auto pages = [&](int t0, int (&page)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      page[i] = -1;
      if (t0 + 16 * i < t_hi) page[i] = __ldg(table + ((t0 + 16 * i) >> ps));
    }
  };
  // (a page holds codes in every place, so tokens past the end may be read; their sums go nowhere)
  const int lane_key = k_word(a.P, lane >> 2, (lane & 3) * (D / 4)), lane_sc = k_scale(a.P, D, lane >> 2);
  const uint8_t* heads = a.cache + static_cast<int64_t>(h) * block_bytes(a.P, D);
  const int64_t page_bytes = a.Hkv * block_bytes(a.P, D);
  const bool had = a.score_in && a.decay != 0.f;
  const float* before = a.score_in + row * a.in_ld;
  auto fetch = [&](int t0, Tile& x) {
    if (t0 >= t_hi) return;
#pragma unroll
    for (int m = 0; m < 2 && a.n_pages > 0; ++m) {
      // (a bad page: some page, and the weights are dropped when they are stored)
      const int page = static_cast<unsigned>(x.page[m]) < static_cast<unsigned>(a.n_pages) ? x.page[m] : 0;
      const int slot = (t0 + 16 * m) & (a.P - 1);
      const uint8_t* blk = heads + page * page_bytes;
      const uint8_t* at = blk + lane_key + 16 * slot;
      const uint8_t* sc = blk + lane_sc + 2 * slot;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (D == 128) {
          const uint4 v = ldg_stream(at + 128 * i);
          x.w[2 * m + i][0] = v.x; x.w[2 * m + i][1] = v.y; x.w[2 * m + i][2] = v.z; x.w[2 * m + i][3] = v.w;
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(at + 128 * i));
          x.w[2 * m + i][0] = v.x; x.w[2 * m + i][1] = v.y;
        }
        x.sc[2 * m + i] = __ldg(reinterpret_cast<const uint16_t*>(sc + 16 * i));
      }
    }
    const int t = t0 + (lane >> 2) + 8 * (lane & 3);
    x.had = had && t < min(t_hi, sp.old) ? before[t] : 0.f;
  };
  Tile next = {};
  int t0 = t_lo + 32 * warp;
  pages(t0, next.page);

  // where the rows lie, their lse and what they see; then the rows, in fragment order
  for (int i = tid; i < 8 * blocks; i += kTile) {
    int vis = 0;
    float l = kInf;
    int64_t at = -1;
    if (i < rows) {
      const int j = i / g;
      const MassRow m = mass_row(a, sp, r, j);
      if (m.bad && a.err) *a.err = 1;
      if (!m.bad) {
        at = m.src * a.ldq + static_cast<int64_t>(h * g + i - j * g) * D;
        l = a.lse[m.src * a.Hq + h * g + i - j * g];
        vis = l == -kInf ? 0 : m.vis;             // (a row that saw nothing weighs nothing)
      }
    }
    s_at[i] = at;
    s_vis[i] = vis;
    s_lse[i] = l == -kInf ? kInf : l * kLog2e;
  }
  __syncthreads();
  {
    // a thread copies the same 16 bytes of every 8 (16) rows
    constexpr int kStep = kTile / (D / 8);
    const int i0 = tid / (D / 8), x = tid % (D / 8);
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + 8 * x;
    const uint32_t dst = tc::smem_u32(qs + (i0 / 8) * kBlock + (x % kRun) * 512 + ((i0 % 8) * 4 + x / kRun) * 16);
    for (int i = i0; i < 8 * blocks; i += kStep) {
      const int64_t at = s_at[i];
      cp16(dst + (i - i0) / 8 * kBlock, q + max(at, static_cast<int64_t>(0)), at >= 0);
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  fetch(t0, next);
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  if (tid < blocks) {                             // (blocks <= kFewRows / 8)
    int2 v = make_int2(0x7fffffff, 0);
    for (int i = 8 * tid; i < 8 * tid + 8; ++i) v = make_int2(min(v.x, s_vis[i]), max(v.y, s_vis[i]));
    s_span[tid] = v;
  }
  __syncthreads();

  const float scale2 = a.scale * kLog2e;
  for (; t0 < t_hi; t0 += kTile) {
    const Tile cur = next;
    pages(t0 + kTile, next.page);
    uint32_t ka[2][2 * kRun][4];
    float fac[4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int w = 0; w < kRun; ++w) {
        uint32_t lo[4], hi[4];
        decode8(cur.w[2 * m][w], lo, magic);
        decode8(cur.w[2 * m + 1][w], hi, magic);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          ka[m][2 * w + p][0] = lo[2 * p];
          ka[m][2 * w + p][1] = hi[2 * p];
          ka[m][2 * w + p][2] = lo[2 * p + 1];
          ka[m][2 * w + p][3] = hi[2 * p + 1];
        }
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) fac[i] = __uint_as_float(static_cast<uint32_t>(cur.sc[i]) << 16) * scale2;
    fetch(t0 + kTile, next);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int n = 0; n < blocks; ++n) {
      const int2 span = s_span[n];
      if (span.y <= t0) continue;
      float acc[2][4] = {};
#pragma unroll
      for (int w = 0; w < kRun; ++w) {
        const uint4 v = *reinterpret_cast<const uint4*>(qs + n * kBlock + w * 512 + lane * 16);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          mma16816(acc[m], ka[m][2 * w], v.x, v.y);
          mma16816(acc[m], ka[m][2 * w + 1], v.z, v.w);
        }
      }
      const float2 l = *reinterpret_cast<const float2*>(&s_lse[8 * n + 2 * (lane & 3)]);
      if (span.x >= t0 + 32) {                    // all of them see the whole tile
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sum[i] += ex2(fmaf(acc[i >> 1][2 * (i & 1)], fac[i], -l.x)) + ex2(fmaf(acc[i >> 1][2 * (i & 1) + 1], fac[i], -l.y));
      } else {
        const int2 vis = *reinterpret_cast<const int2*>(&s_vis[8 * n + 2 * (lane & 3)]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + (lane >> 2) + 8 * i;
          if (t < vis.x) sum[i] += ex2(fmaf(acc[i >> 1][2 * (i & 1)], fac[i], -l.x));
          if (t < vis.y) sum[i] += ex2(fmaf(acc[i >> 1][2 * (i & 1) + 1], fac[i], -l.y));
        }
      }
    }
    // a token's sums lie in four lanes, each of which takes one of their four tokens
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
      sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    }
    const int i = lane & 3, t = t0 + (lane >> 2) + 8 * i;
    const float mine = i == 0 ? sum[0] : i == 1 ? sum[1] : i == 2 ? sum[2] : sum[3];
    if (t < t_hi) {
      const int page = i < 2 ? cur.page[0] : cur.page[1];
      const bool ok = page >= 0 && page < a.n_pages;
      if (!ok && a.err) *a.err = 1;
      a.score_out[row * a.out_ld + t] = (had ? a.decay * cur.had : 0.f) + (ok ? mine : 0.f);
    }
  }
}

}  // namespace

int mass_simt(const MassArgs& a, int B, int d, cudaStream_t st) {
  // a cluster shares a tile's rows where the tiles alone leave SMs idle
  const int64_t tiles = static_cast<int64_t>((a.max_len + kTile - 1) / kTile) * a.Hkv * B;
  const int64_t chunks = (static_cast<int64_t>(a.max_rows) * (a.Hq / a.Hkv) + kSimtRows - 1) / kSimtRows;
  int parts = 1;
  while (parts < 8 && 2 * parts <= chunks && tiles * parts < 2ll * sm_count()) parts *= 2;
  const dim3 grid(static_cast<unsigned>((a.max_len + kTile - 1) / kTile) * parts, a.Hkv, B);
  const auto u = static_cast<uint32_t>(parts);
  return d == 128 ? cl::launch_pdl(simt_kernel<128>, parts, grid, dim3(kTile), 0, st, a, u)
                  : cl::launch_pdl(simt_kernel<64>, parts, grid, dim3(kTile), 0, st, a, u);
}
int mass_few(const MassArgs& a, int B, int d, cudaStream_t st) {
  // tokens of a CTA: about four CTAs' worth for each one that is resident, 128 at least
  const int64_t all = static_cast<int64_t>(a.max_len) * a.Hkv * B, rows = static_cast<int64_t>(a.max_rows) * (a.Hq / a.Hkv);
  const int run = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(8, all / (16ll * kTile * sm_count())))) * kTile;
  const dim3 grid(static_cast<unsigned>((a.max_len + run - 1) / run), a.Hkv, B);
  const size_t smem = static_cast<size_t>((rows + 7) / 8) * 16 * d;
  if (smem > 40 << 10 && !(d == 128 ? smem_limit(few_kernel<128>, kFewRows * 256) : smem_limit(few_kernel<64>, kFewRows * 128)))
    return TV_ECUDA;
  return d == 128 ? launch_pdl(few_kernel<128>, grid, dim3(kTile), smem, st, a, run, kMagic)
                  : launch_pdl(few_kernel<64>, grid, dim3(kTile), smem, st, a, run, kMagic);
}

}  // namespace kv4
}  // namespace tv

using namespace tv;

TV_API int kv4_attn_mass(const void* q, int64_t ldq, const float* lse, int dtype, const void* cache, int n_pages,
                         int page_size, const int32_t* block_table, int table_ld, const int32_t* cache_len,
                         const int32_t* row_off, const int32_t* path, int path_ld, const int32_t* vis_prefix,
                         const int32_t* old_len, int causal, int B, int max_rows, int total_rows, int max_len, int Hq,
                         int Hkv, int d, float scale, float decay, const float* score_in, int64_t score_in_ld,
                         float* score_out, int64_t score_out_ld, int32_t* err, tv_stream_t stream) {
  if (dtype != TV_F32 && dtype != TV_BF16) return TV_EINVAL;
  if (B < 0 || max_rows < 0 || total_rows < 0 || max_len < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv) return TV_EINVAL;
  if (n_pages < 0 || table_ld < 0 || page_size <= 0 || path_ld < 0) return TV_EINVAL;
  if (!kv4::page_size_ok(page_size) || (d != 64 && d != 128) || Hq / Hkv > 64) return TV_EUNSUPPORTED;
  if (B > 65535 || Hkv > 65535 || static_cast<int64_t>(table_ld) * page_size > 0x7fffffffll ||
      max_len > 0x7fffffff - 4096 || static_cast<int64_t>(max_rows) * (Hq / Hkv) > 0x7fffffff - 4096)
    return TV_EUNSUPPORTED;
  if (!(scale > 0.f) || scale > 3.402823466e38f || !(decay >= 0.f && decay <= 1.f)) return TV_EINVAL;
  if (score_out_ld < max_len || (score_in && score_in_ld < max_len)) return TV_EINVAL;
  if (score_in && score_in == score_out && score_in_ld != score_out_ld) return TV_EINVAL;
  if (B == 0 || max_len == 0) return TV_OK;
  if (!cache_len || !row_off || !score_out || (causal && !old_len) || (path && path_ld <= 0)) return TV_EINVAL;
  if (table_ld > 0 && !block_table) return TV_EINVAL;
  if (n_pages > 0 && !cache) return TV_EINVAL;
  if (total_rows > 0 && max_rows > 0 && (!q || !lse)) return TV_EINVAL;
  if (ldq < static_cast<int64_t>(Hq) * d || ldq % (dtype == TV_BF16 ? 8 : 4)) return TV_EINVAL;
  if ((q && !aligned(q, 16)) || (cache && !aligned(cache, 16))) return TV_EINVAL;
  if (total_rows == 0) max_rows = 0;      // no row can be read
  const kv4::MassArgs a{q, lse, static_cast<const uint8_t*>(cache), block_table, cache_len, row_off, path, vis_prefix,
                        old_len, score_in, score_out, err, ldq, score_in_ld, score_out_ld, n_pages, page_size, table_ld,
                        path_ld, causal, max_rows, total_rows, max_len, Hq, Hkv, scale, decay};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = static_cast<int64_t>(max_rows) * (Hq / Hkv);
  if (dtype == TV_BF16) return rows <= kv4::kFewRows ? kv4::mass_few(a, B, d, st) : kv4::mass_tc(a, B, d, st);
  return kv4::mass_simt(a, B, d, st);
}
