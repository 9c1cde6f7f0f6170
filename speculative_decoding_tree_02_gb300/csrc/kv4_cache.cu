// Rotation of q/k rows (tv_rope) and the paged 4-bit KV cache: kv4_append
// (rotate, quantise, append) and kv4_gather (cached rows back as values).
// All three move bytes: they are bound by HBM, or by launch latency when a
// step's few rows are all there is.
#include <algorithm>

#include "kv4.cuh"

namespace tv {
namespace kv4 {

// Eight consecutive elements, as loaded and as fp32.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> raw8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.v[i] = ldg_stream(p + 8 / (sizeof(T) / 2) * i);
  return r;
}
__device__ __forceinline__ void widen8(const Raw8<uint16_t>& r, float (&x)[8]) {
  const uint4 v = r.v[0];
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
  x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ void widen8(const Raw8<float>& r, float (&x)[8]) {
  const uint4 a = r.v[0], b = r.v[1];
  x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y); x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
  x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y); x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
}
// fp32 -> bf16, round to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Value of byte i (0..15) of a word, minus 8, by way of the mantissa.
__device__ __forceinline__ float byte_value(uint32_t w, int i) {
  return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540u + i)) - 8388616.f;   // 2^23 + byte - (2^23 + 8)
}

// A row of d elements is d/16 units of 16 elements, in two runs of eight that
// start at i0 and i1: run u of the first and of the second half of the rotated
// part (or of what follows it), so that neighbouring threads touch neighbouring
// 16 bytes.  In halves the two runs are the pairs' first and second elements,
// interleaved each run is four pairs.
struct Unit {
  int i0, i1;
  bool rot;
};
__device__ __forceinline__ Unit unit_of(int u, int d, int rot) {
  Unit r;
  r.rot = 16 * u < rot;
  r.i0 = r.rot ? 8 * u : rot + 8 * (u - (rot >> 4));
  r.i1 = r.i0 + (r.rot ? rot : d - rot) / 2;
  return r;
}
// Rotates a unit in place.  Every product and sum is rounded by itself (no
// fused multiply-add), so the result is the same wherever it is computed.
template <bool kInter>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8]) {
  if constexpr (kInter) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = a[2 * j], y = a[2 * j + 1];
      a[2 * j] = __fsub_rn(__fmul_rn(x, c[j]), __fmul_rn(y, s[j]));
      a[2 * j + 1] = __fadd_rn(__fmul_rn(y, c[j]), __fmul_rn(x, s[j]));
      const float z = b[2 * j], w = b[2 * j + 1];
      b[2 * j] = __fsub_rn(__fmul_rn(z, c[4 + j]), __fmul_rn(w, s[4 + j]));
      b[2 * j + 1] = __fadd_rn(__fmul_rn(w, c[4 + j]), __fmul_rn(z, s[4 + j]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = a[j], y = b[j];
      a[j] = __fsub_rn(__fmul_rn(x, c[j]), __fmul_rn(y, s[j]));
      b[j] = __fadd_rn(__fmul_rn(y, c[j]), __fmul_rn(x, s[j]));
    }
  }
}
// The (cos, sin) of unit u from a table row; rows are reused: cached loads.
template <bool kInter>
__device__ __forceinline__ void table_unit(const float* row, int u, int rot, float (&c)[8], float (&s)[8]) {
  const float* at = row + (kInter ? 4 : 8) * u;
  const int step = kInter ? rot >> 2 : 4, half = rot >> 1;
  const float4 v[4] = {__ldg(reinterpret_cast<const float4*>(at)), __ldg(reinterpret_cast<const float4*>(at + step)),
                       __ldg(reinterpret_cast<const float4*>(at + half)),
                       __ldg(reinterpret_cast<const float4*>(at + half + step))};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    c[4 * i] = v[i].x; c[4 * i + 1] = v[i].y; c[4 * i + 2] = v[i].z; c[4 * i + 3] = v[i].w;
    s[4 * i] = v[2 + i].x; s[4 * i + 1] = v[2 + i].y; s[4 * i + 2] = v[2 + i].z; s[4 * i + 3] = v[2 + i].w;
  }
}

// ------------------------------------------------------------------ rotation
// CTA = one token; thread = (unit of the row, head lane), so a thread reads
// its eight (cos, sin) once for all of its heads.  16411 tokens of 40 heads of
// 128 in bf16: 55 us, 6.2 TB/s (91% of the measured copy rate).
template <typename T, bool kInter>
__global__ void __launch_bounds__(256) rope_kernel(const T* __restrict__ q, int64_t ldq, const T* __restrict__ k,
                                                   int64_t ldk, int Hq, int Hkv, int d,
                                                   const int32_t* __restrict__ pos, const float* __restrict__ table,
                                                   int max_pos, int rot, T* __restrict__ q_out,
                                                   T* __restrict__ k_out, int32_t* err) {
  griddep_wait();
  griddep_release();
  const int64_t t = blockIdx.x;
  const int units = d >> 4;
  const int u = threadIdx.x % units, lane0 = threadIdx.x / units, lanes = blockDim.x / units;
  const int p = pos[t];
  if (rot > 0 && (p < 0 || p >= max_pos)) {
    if (threadIdx.x == 0 && err) *err = 1;
    return;
  }
  const Unit un = unit_of(u, d, rot);
  float c[8], s[8];
  if (un.rot) table_unit<kInter>(table + static_cast<int64_t>(p) * rot, u, rot, c, s);
  for (int h = lane0; h < Hq + Hkv; h += lanes) {
    const T* src = h < Hq ? q + t * ldq + static_cast<int64_t>(h) * d : k + t * ldk + static_cast<int64_t>(h - Hq) * d;
    T* dst = h < Hq ? q_out + (t * Hq + h) * d : k_out + (t * Hkv + h - Hq) * d;
    const Raw8<T> ra = raw8(src + un.i0), rb = raw8(src + un.i1);
    float a[8], b[8];
    widen8(ra, a);
    widen8(rb, b);
    if (un.rot) rotate<kInter>(a, b, c, s);
    store8(dst + un.i0, a);
    store8(dst + un.i1, b);
  }
}

// -------------------------------------------------------------------- append
struct AppendArgs {
  const void* k;
  const void* v;
  int64_t ldk, ldv;
  const int32_t* row_off;
  const int32_t* path;
  const int32_t* pos;
  const float* table;
  const int32_t* block_table;
  const int32_t* cache_len;
  uint8_t* cache;
  int32_t* new_len;
  int32_t* err;
  int total_rows, path_ld, max_new, max_pos, rot, n_pages, P, table_ld, Hkv, heads;
};

// CTA = (16 cache tokens of one V group, `heads` KV heads, request), D
// threads: thread = (token, unit of its row).  A group belongs to one CTA, so
// the nibbles of its tokens in shared V words are merged without atomics: the
// CTA rewrites the group's words whole, keeping the nibbles of tokens that it
// does not append.  The heads of a CTA follow one another with the next head's
// rows on their way: the chain of lengths, tables and positions and the
// (cos, sin) of the token are paid once for them (see heads_per_cta).  8 prompts
// of 512..4096 tokens, 8 heads of 128: 27 us for 95 MB in and out, 3.5 TB/s (52%
// of the measured copy rate); bound by issue slots (66% taken: the maxima, the
// divisions and the packing of 2 x 128 elements a token and head).
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(D, 768 / D) append_kernel(const AppendArgs a) {
  constexpr int kUnits = D / 16;
  __shared__ __align__(16) uint8_t codes[2][16][D];
  __shared__ int s_count;
  __shared__ uint32_t s_live;
  griddep_wait();
  griddep_release();
  const int r = blockIdx.z, h0 = blockIdx.y * a.heads, h1 = min(h0 + a.heads, a.Hkv), tid = threadIdx.x;
  const int len = a.cache_len[r];
  const int base = a.row_off[r];
  int count = min(a.path ? min(a.path_ld, a.max_new) : a.row_off[r + 1] - base, a.max_new);
  if (tid == 0) {
    s_count = count;
    s_live = 0;
  }
  __syncthreads();
  if (a.path) {   // rows up to the first negative entry
    int first = count;
    for (int j = tid; j < count; j += D)
      if (a.path[static_cast<int64_t>(r) * a.path_ld + j] < 0) {
        first = j;
        break;
      }
    if (first < count) atomicMin(&s_count, first);
    __syncthreads();
    count = s_count;
  }
  count = max(count, 0);
  const int64_t cap = static_cast<int64_t>(a.table_ld) * a.P;
  const bool bad = len < 0 || (count > 0 && len + static_cast<int64_t>(count) > cap) ||
                   (!a.path && a.row_off[r + 1] - base > a.max_new);
  if (blockIdx.x == 0 && h0 == 0 && tid == 0) {
    if (a.new_len) a.new_len[r] = len < 0 ? len : len + count;
    if (bad && a.err) *a.err = 1;
  }
  if (len < 0 || count == 0) return;             // (nothing to append: no table entry is needed)
  const int64_t g64 = len / 16 + static_cast<int64_t>(blockIdx.x);   // 16-token group of the request
  if (16 * g64 >= min(len + static_cast<int64_t>(count), cap)) return;   // (beyond the table: reported above)
  const int group = static_cast<int>(g64);
  const int pg = group * 16 / a.P;
  const int page = a.block_table[static_cast<int64_t>(r) * a.table_ld + pg];
  if (page < 0 || page >= a.n_pages) {
    if (tid == 0 && a.err) *a.err = 1;
    return;
  }

  const int tk = tid / kUnits, u = tid % kUnits;
  const int slot = (group * 16 + tk) % a.P;
  const int j = group * 16 + tk - len;           // appended row of the request
  bool live = j >= 0 && j < count;
  int64_t src = 0;
  int p = len + j;
  if (live) {
    src = static_cast<int64_t>(base) + (a.path ? a.path[static_cast<int64_t>(r) * a.path_ld + j] : j);
    live = src >= 0 && src < a.total_rows;
    if (live && a.pos) p = a.pos[src];
    if (live && a.rot > 0) live = p >= 0 && p < a.max_pos;
    if (!live && a.err) *a.err = 1;
  }
  if (live && u == 0) atomicOr(&s_live, 1u << tk);
  const Unit un = unit_of(u, D, a.rot);
  const T* kr = static_cast<const T*>(a.k) + src * a.ldk;
  const T* vr = static_cast<const T*>(a.v) + src * a.ldv;
  float c[8], s[8];
  Raw8<T> next[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int k = 0; k < static_cast<int>(sizeof(T) / 2); ++k) next[i].v[k] = make_uint4(0u, 0u, 0u, 0u);
  auto fetch = [&](int h) {
    if (!live) return;
    next[0] = raw8(kr + static_cast<int64_t>(h) * D + un.i0);
    next[1] = raw8(kr + static_cast<int64_t>(h) * D + un.i1);
    next[2] = raw8(vr + static_cast<int64_t>(h) * D + 8 * u);
    next[3] = raw8(vr + static_cast<int64_t>(h) * D + D / 2 + 8 * u);
  };
  fetch(h0);
  if (live && un.rot) table_unit<kInter>(a.table + static_cast<int64_t>(p) * a.rot, u, a.rot, c, s);
  __syncthreads();
  const uint32_t mask = s_live;
  if (mask == 0) return;
  for (int h = h0; h < h1; ++h) {
    uint8_t* blk = a.cache + (static_cast<int64_t>(page) * a.Hkv + h) * block_bytes(a.P, D);
    uint8_t(*buf)[D] = codes[(h - h0) & 1];
    uint2* dst = reinterpret_cast<uint2*>(blk + v_group(a.P, D, group % (a.P / 16), tid));
    uint2 old = make_uint2(0u, 0u);
    if (mask != 0xffffu) old = *dst;
    float ka[8], kb[8], va[8], vb[8];
    widen8(next[0], ka);
    widen8(next[1], kb);
    widen8(next[2], va);
    widen8(next[3], vb);
    if (h + 1 < h1) fetch(h + 1);
    if (live && un.rot) rotate<kInter>(ka, kb, c, s);
    // row maxima over the units of a token
    float mk = 0.f, mv = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mk = max_abs(mk, ka[i], kb[i]);
      mv = max_abs(mv, va[i], vb[i]);
    }
#pragma unroll
    for (int o = kUnits / 2; o; o >>= 1) {
      mk = max_nan(mk, __shfl_xor_sync(0xffffffffu, mk, o));
      mv = max_nan(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    }
    const float sk = row_scale(mk), sv = row_scale(mv);
    const float ik = row_inverse(sk), iv = row_inverse(sv);
    uint32_t w0 = 0, w1 = 0, cv[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int m = 7; m >= 0; --m) {               // nibble m holds item 2 m (+ 1 - 8 in the upper half)
      const int e = m < 4 ? 2 * m : 2 * m - 7;
      w0 = (w0 << 4) | (encode(ka[e], sk, ik) & 15u);
      w1 = (w1 << 4) | (encode(kb[e], sk, ik) & 15u);
    }
#pragma unroll
    for (int e = 7; e >= 0; --e) {
      cv[e >> 2] = (cv[e >> 2] << 8) | (encode(va[e], sv, iv) & 15u);
      cv[2 + (e >> 2)] = (cv[2 + (e >> 2)] << 8) | (encode(vb[e], sv, iv) & 15u);
    }
    *reinterpret_cast<uint2*>(&buf[tk][8 * u]) = make_uint2(cv[0], cv[1]);
    *reinterpret_cast<uint2*>(&buf[tk][D / 2 + 8 * u]) = make_uint2(cv[2], cv[3]);
    if (live) {
      *reinterpret_cast<uint32_t*>(blk + k_word(a.P, slot, un.i0)) = w0;
      *reinterpret_cast<uint32_t*>(blk + k_word(a.P, slot, un.i1)) = w1;
      if (u == 0) {
        *reinterpret_cast<uint16_t*>(blk + k_scale(a.P, D, slot)) = static_cast<uint16_t>(__float_as_uint(sk) >> 16);
        *reinterpret_cast<uint16_t*>(blk + v_scale(a.P, D, slot)) = static_cast<uint16_t>(__float_as_uint(sv) >> 16);
      }
    }
    __syncthreads();
    // thread = dim: the 16 tokens' nibbles of one dim
    uint32_t w[2] = {0u, 0u}, keep[2] = {0u, 0u};
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const int sh = 4 * nibble_of(t & 7);
      w[t >> 3] |= static_cast<uint32_t>(buf[t][tid]) << sh;
      if (!((mask >> t) & 1u)) keep[t >> 3] |= 15u << sh;
    }
    *dst = make_uint2((w[0] & ~keep[0]) | (old.x & keep[0]), (w[1] & ~keep[1]) | (old.y & keep[1]));
  }
}

// -------------------------------------------------------------------- gather
struct GatherArgs {
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* start;
  const int32_t* out_off;
  void* k_out;
  void* v_out;
  int32_t* err;
  int n_pages, P, table_ld, Hkv, total_rows, max_rows, heads;
};

// CTA = (16 cache tokens, `heads` KV heads, request), D threads: thread =
// (tokens tk and tk + 8, 8 dims) for the rows, so that a warp's store is whole
// rows; V codes pass through shared memory to turn the group's dim-major words
// into rows.  The heads of a CTA follow one another with the next head's codes
// on their way.  64 requests of 512..4096 tokens, 8 heads of 128 to bf16: 118 us,
// 6.4 TB/s (95% of the measured copy rate).
template <typename T, int D>
__global__ void __launch_bounds__(D) gather_kernel(const GatherArgs a) {
  constexpr int kUnits = D / 8;
  __shared__ __align__(16) uint8_t codes[2][16][D];
  griddep_wait();
  griddep_release();
  const int r = blockIdx.z, h0 = blockIdx.y * a.heads, h1 = min(h0 + a.heads, a.Hkv), tid = threadIdx.x;
  const int o0 = a.out_off[r];
  int n = a.out_off[r + 1] - o0;
  const int t0 = a.start ? a.start[r] : 0;
  if (n <= 0) return;
  const int64_t cap = static_cast<int64_t>(a.table_ld) * a.P;
  const bool bad = t0 < 0 || o0 < 0 || static_cast<int64_t>(o0) + n > a.total_rows;
  if (blockIdx.x == 0 && h0 == 0 && tid == 0 && a.err && (bad || n > a.max_rows || t0 + static_cast<int64_t>(n) > cap))
    *a.err = 1;
  if (bad) return;
  n = min(n, a.max_rows);
  const int64_t g64 = t0 / 16 + static_cast<int64_t>(blockIdx.x);
  if (16 * g64 >= min(t0 + static_cast<int64_t>(n), cap)) return;
  const int group = static_cast<int>(g64);
  const int pg = group * 16 / a.P;
  const int page = a.block_table[static_cast<int64_t>(r) * a.table_ld + pg];
  if (page < 0 || page >= a.n_pages) {
    if (tid == 0 && a.err) *a.err = 1;
    return;
  }
  const int tk = tid / kUnits, u = tid % kUnits;
  const int slot = (group * 16) % a.P + tk;
  const int64_t i0 = static_cast<int64_t>(group) * 16 + tk - t0;
  const uint8_t* blk = a.cache + (static_cast<int64_t>(page) * a.Hkv + h0) * block_bytes(a.P, D);
  const int ko = k_word(a.P, slot, 8 * u), vo = v_group(a.P, D, group % (a.P / 16), tid);
  uint32_t kw[2];
  uint2 vw;
  uint16_t ks[2], vs[2];
  auto fetch = [&]() {
    vw = __ldg(reinterpret_cast<const uint2*>(blk + vo));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      kw[t] = __ldg(reinterpret_cast<const uint32_t*>(blk + ko + 128 * t));
      ks[t] = __ldg(reinterpret_cast<const uint16_t*>(blk + k_scale(a.P, D, slot + 8 * t)));
      vs[t] = __ldg(reinterpret_cast<const uint16_t*>(blk + v_scale(a.P, D, slot + 8 * t)));
    }
  };
  fetch();
  for (int h = h0; h < h1; ++h) {
    uint8_t(*buf)[D] = codes[(h - h0) & 1];
    const uint32_t k2[2] = {kw[0], kw[1]};
    const float sk[2] = {bf16_at(&ks[0]), bf16_at(&ks[1])}, sv[2] = {bf16_at(&vs[0]), bf16_at(&vs[1])};
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      buf[t][tid] = static_cast<uint8_t>((vw.x >> (4 * nibble_of(t))) & 15u);
      buf[t + 8][tid] = static_cast<uint8_t>((vw.y >> (4 * nibble_of(t))) & 15u);
    }
    blk += block_bytes(a.P, D);
    if (h + 1 < h1) fetch();
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t i = i0 + 8 * t;
      if (i < 0 || i >= n) continue;
      const int64_t at = ((o0 + i) * a.Hkv + h) * D + 8 * u;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = sk[t] * decode(k2[t], e);
      store8(static_cast<T*>(a.k_out) + at, x);
      const uint2 cv = *reinterpret_cast<const uint2*>(&buf[tk + 8 * t][8 * u]);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = sv[t] * byte_value(e < 4 ? cv.x : cv.y, e & 3);
      store8(static_cast<T*>(a.v_out) + at, x);
    }
  }
}

// KV heads that a CTA of append and gather takes one after another: all of
// them while that leaves enough CTAs for every SM, else fewer.
// One head to a CTA against all eight: the accepted paths of 64 requests in and
// back 12.5 against 15.5 us (the rule: 12.5), prompts of 8 requests 68 against 51
// (51), 64 requests' prefixes back 164 against 121 (121).
int heads_per_cta(int64_t groups, int Hkv) {
  const int64_t want = 8ll * sm_count();
  int heads = Hkv;
  while (heads > 1 && groups * ((Hkv + heads - 1) / heads) < want) heads = (heads + 1) / 2;
  return heads;
}

bool cache_ok(int n_pages, int page_size, int table_ld, int Hkv, int d) {
  return n_pages >= 0 && table_ld >= 0 && Hkv > 0 && page_size > 0 && d > 0 &&
         static_cast<int64_t>(table_ld) * page_size <= 0x7fffffffll;
}

}  // namespace kv4
}  // namespace tv

using namespace tv;

TV_API size_t kv4_cache_size(int n_pages, int page_size, int Hkv, int d) {
  if (n_pages <= 0 || Hkv <= 0 || !kv4::page_size_ok(page_size) || (d != 64 && d != 128)) return 0;
  return static_cast<size_t>(n_pages) * Hkv * kv4::block_bytes(page_size, d);
}

TV_API int tv_rope(const void* q, int64_t ldq, const void* k, int64_t ldk, int dtype, int n, int Hq, int Hkv, int d,
                   const int32_t* pos, const float* table, int max_pos, int rot_dim, int interleaved, void* q_out,
                   void* k_out, int32_t* err, tv_stream_t stream) {
  if (dtype != TV_F32 && dtype != TV_BF16) return TV_EINVAL;
  if (n < 0 || Hq <= 0 || Hkv < 0 || d <= 0 || max_pos < 0 || rot_dim < 0 || rot_dim > d) return TV_EINVAL;
  if (d % 16 || rot_dim % 16 || d > 512) return TV_EUNSUPPORTED;
  if (n == 0) return TV_OK;
  if (!q || !q_out || !pos || (rot_dim > 0 && !table)) return TV_EINVAL;
  if (!k != !k_out) return TV_EINVAL;
  if (!k) Hkv = 0;
  if (k && Hkv == 0) return TV_EINVAL;
  const int vec = dtype == TV_BF16 ? 8 : 4;   // elements of a 16-byte load
  if (ldq < static_cast<int64_t>(Hq) * d || ldq % vec) return TV_EINVAL;
  if (k && (ldk < static_cast<int64_t>(Hkv) * d || ldk % vec)) return TV_EINVAL;
  const void* ptrs[] = {q, k, table, q_out, k_out};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return TV_EINVAL;
  const int units = d / 16, H = Hq + Hkv;
  int lanes = std::max(1, std::min(H, 256 / units));
  const int iters = (H + lanes - 1) / lanes;
  lanes = (H + iters - 1) / iters;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto tag, auto kernel) {
    using T = decltype(tag);
    return launch_pdl(kernel, dim3(n), dim3(units * lanes), 0, st, static_cast<const T*>(q), ldq,
                      static_cast<const T*>(k), ldk, Hq, Hkv, d, pos, table, max_pos, rot_dim, static_cast<T*>(q_out),
                      static_cast<T*>(k_out), err);
  };
  if (dtype == TV_BF16)
    return interleaved ? go(uint16_t{}, kv4::rope_kernel<uint16_t, true>) : go(uint16_t{}, kv4::rope_kernel<uint16_t, false>);
  return interleaved ? go(float{}, kv4::rope_kernel<float, true>) : go(float{}, kv4::rope_kernel<float, false>);
}

TV_API int kv4_append(const void* k, int64_t ldk, const void* v, int64_t ldv, int dtype, int total_rows,
                      const int32_t* row_off, const int32_t* path, int path_ld, int B, int max_new, const int32_t* pos,
                      const float* table, int max_pos, int rot_dim, int interleaved, void* cache, int n_pages,
                      int page_size, const int32_t* block_table, int table_ld, const int32_t* cache_len, int Hkv, int d,
                      int32_t* new_len, int32_t* err, tv_stream_t stream) {
  if (dtype != TV_F32 && dtype != TV_BF16) return TV_EINVAL;
  if (B < 0 || max_new < 0 || total_rows < 0 || max_pos < 0 || rot_dim < 0 || rot_dim > d) return TV_EINVAL;
  if (!kv4::cache_ok(n_pages, page_size, table_ld, Hkv, d)) return TV_EINVAL;
  if (!kv4::page_size_ok(page_size) || (d != 64 && d != 128) || rot_dim % 16) return TV_EUNSUPPORTED;
  if (B > 65535 || Hkv > 65535) return TV_EUNSUPPORTED;
  if (B == 0) return TV_OK;
  if (!row_off || !cache_len || (new_len && new_len == cache_len)) return TV_EINVAL;
  if (path && path_ld <= 0) return TV_EINVAL;
  if (table_ld > 0 && !block_table) return TV_EINVAL;
  if (total_rows > 0 && max_new > 0) {
    if (!k || !v || !cache || !block_table || (rot_dim > 0 && !table)) return TV_EINVAL;
  }
  const int vec = dtype == TV_BF16 ? 8 : 4;
  if (ldk < static_cast<int64_t>(Hkv) * d || ldv < static_cast<int64_t>(Hkv) * d || ldk % vec || ldv % vec)
    return TV_EINVAL;
  const void* ptrs[] = {k, v, table, cache};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return TV_EINVAL;
  kv4::AppendArgs a{k, v, ldk, ldv, row_off, path, pos, table, block_table, cache_len, static_cast<uint8_t*>(cache),
                    new_len, err, total_rows, path_ld, max_new, max_pos, rot_dim, n_pages,
                    page_size, table_ld, Hkv, 1};
  if (total_rows == 0) a.n_pages = 0;     // no row can be read or written
  const int64_t groups = (static_cast<int64_t>(max_new) + 15) / 16 + 1;
  a.heads = kv4::heads_per_cta(std::min(groups * B, static_cast<int64_t>(total_rows) / 16 + B), Hkv);
  const dim3 grid(static_cast<unsigned>(groups), (Hkv + a.heads - 1) / a.heads, B);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto k128, auto k64) {
    return d == 128 ? launch_pdl(k128, grid, dim3(128), 0, st, a) : launch_pdl(k64, grid, dim3(64), 0, st, a);
  };
  if (dtype == TV_BF16)
    return interleaved ? go(kv4::append_kernel<uint16_t, 128, true>, kv4::append_kernel<uint16_t, 64, true>)
                       : go(kv4::append_kernel<uint16_t, 128, false>, kv4::append_kernel<uint16_t, 64, false>);
  return interleaved ? go(kv4::append_kernel<float, 128, true>, kv4::append_kernel<float, 64, true>)
                     : go(kv4::append_kernel<float, 128, false>, kv4::append_kernel<float, 64, false>);
}

TV_API int kv4_gather(const void* cache, int n_pages, int page_size, const int32_t* block_table, int table_ld,
                      const int32_t* start, const int32_t* out_off, int B, int max_rows, int total_rows, int Hkv, int d,
                      int dtype, void* k_out, void* v_out, int32_t* err, tv_stream_t stream) {
  if (dtype != TV_F32 && dtype != TV_BF16) return TV_EINVAL;
  if (B < 0 || max_rows < 0 || total_rows < 0) return TV_EINVAL;
  if (!kv4::cache_ok(n_pages, page_size, table_ld, Hkv, d)) return TV_EINVAL;
  if (!kv4::page_size_ok(page_size) || (d != 64 && d != 128)) return TV_EUNSUPPORTED;
  if (B > 65535 || Hkv > 65535) return TV_EUNSUPPORTED;
  if (B == 0 || max_rows == 0 || total_rows == 0) return TV_OK;
  if (!cache || !block_table || !out_off || !k_out || !v_out) return TV_EINVAL;
  const void* ptrs[] = {cache, k_out, v_out};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return TV_EINVAL;
  kv4::GatherArgs a{static_cast<const uint8_t*>(cache), block_table, start, out_off, k_out, v_out, err, n_pages,
                    page_size, table_ld, Hkv, total_rows, max_rows, 1};
  const int64_t groups = (static_cast<int64_t>(max_rows) + 15) / 16 + (start ? 1 : 0);
  a.heads = kv4::heads_per_cta(std::min(groups * B, static_cast<int64_t>(total_rows) / 16 + B), Hkv);
  const dim3 grid(static_cast<unsigned>(groups), (Hkv + a.heads - 1) / a.heads, B);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == TV_BF16)
    return d == 128 ? launch_pdl(kv4::gather_kernel<uint16_t, 128>, grid, dim3(128), 0, st, a)
                    : launch_pdl(kv4::gather_kernel<uint16_t, 64>, grid, dim3(64), 0, st, a);
  return d == 128 ? launch_pdl(kv4::gather_kernel<float, 128>, grid, dim3(128), 0, st, a)
                  : launch_pdl(kv4::gather_kernel<float, 64>, grid, dim3(64), 0, st, a);
}
