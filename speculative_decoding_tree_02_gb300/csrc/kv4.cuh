// The paged 4-bit KV cache: block layout, code conversions and the parameter
// block of tree_verify_attn_kv4, shared by kv4_cache.cu and the attention paths.
//
// One (page, KV head) block of P tokens, head dimension d, P * (d + 4) bytes:
//   K codes  [d/32][P][16 B]  chunk c of token t: its dims 32c .. 32c+31
//   V codes  [P/16][d][8 B]   dim by dim, the 16 tokens of a group
//   K scales bf16 [P], V scales bf16 [P]
// Eight codes make a 32-bit word: item e (a dim of a key, a token of a value)
// sits in nibble e/2 + 4 * (e % 2), so that (w >> 4i) & 0x000f000f is the pair
// (2i, 2i + 1) in the two halves of a register.  Keys run along the head
// dimension and values along the tokens because those are the contraction
// axes of q.k and of p.v: a thread that owns a key (a tensor-memory lane of K)
// or a dim (a lane of V^T) finds its operand row in whole words.
// A code n + 8 (n in -7..7) stands for s * n; s * n has at most 8 + 3
// significant bits, so it is exact in fp32, and n alone is exact in bf16.
#pragma once

#include "tv_common.cuh"

namespace tv {
namespace kv4 {

constexpr float kScaleMin = 7.888609052210118e-31f;   // 2^-100: keeps 1/s finite

// Scale of a row: max|x| / 7 rounded up to bf16, at least 2^-100; NaN for a
// row with a non-finite entry (amax NaN or infinite), so that the whole row
// reads back as NaN.  The quotient is correctly rounded: 1/7 correctly rounded
// and one remainder step (Markstein 1990).
__device__ __forceinline__ float row_scale(float amax) {
  const float q0 = __fmul_rn(amax, 1.f / 7.f);
  const float a = fmaf(fmaf(-q0, 7.f, amax), 1.f / 7.f, q0);
  const float up = __uint_as_float((__float_as_uint(a) + 0xffffu) & 0xffff0000u);
  return amax <= 3.402823466e38f ? fmaxf(up, kScaleMin) : __uint_as_float(0x7fc00000u);
}
// 1/s correctly rounded, s a row's scale: one Newton step on the hardware's
// approximation.  For each of the 128 significands of a bf16 number the step
// gives the correctly rounded reciprocal from anything within 4 units in the
// last place of it (enumerated), and 2^-100 <= s < 2^126 keeps both normal.
__device__ __forceinline__ float row_inverse(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return fmaf(r, fmaf(-s, r, 1.f), r);
}
// max(m, |x|, |y|); a NaN stays.
__device__ __forceinline__ float max_abs(float m, float x, float y) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(m), "f"(fabsf(x)), "f"(fabsf(y)));
  return d;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(x), "f"(y));
  return d;
}

// Code of x in the low four bits of the result (the others are not zero):
// x / s rounded to the nearest integer, ties to even, plus 8.  The quotient is
// the correctly rounded one (inv = 1/s correctly rounded, one remainder step:
// Markstein 1990): bf16 rows hit exact ties often, and a product with the
// reciprocal alone would break them either way.  |x| <= 7 s, so it needs no
// clamp; adding 1.5 * 2^23 + 8 rounds it to an integer in the low bits.
__device__ __forceinline__ uint32_t encode(float x, float s, float inv) {
  const float q0 = __fmul_rn(x, inv);
  const float q = fmaf(fmaf(-q0, s, x), inv, q0);
  return __float_as_uint(__fadd_rn(q, 12582920.f));
}

__host__ __device__ __forceinline__ constexpr int nibble_of(int e) { return (e >> 1) + 4 * (e & 1); }

// Value n of item e of a code word, by way of the mantissa (2^23 + code).
__device__ __forceinline__ float decode(uint32_t w, int e) {
  return __uint_as_float(((w >> (4 * nibble_of(e))) & 15u) | 0x4b000000u) - 8388616.f;
}

// Byte offsets inside a block.
__host__ __device__ __forceinline__ int k_word(int P, int slot, int dim) {   // word of dims dim & ~7 ..
  return ((dim >> 5) * P + slot) * 16 + ((dim & 31) >> 3) * 4;
}
__host__ __device__ __forceinline__ int v_group(int P, int d, int group, int dim) {   // 16 tokens of one dim
  return P * (d >> 1) + (group * d + dim) * 8;
}
__host__ __device__ __forceinline__ int k_scale(int P, int d, int slot) { return P * d + 2 * slot; }
__host__ __device__ __forceinline__ int v_scale(int P, int d, int slot) { return P * d + 2 * P + 2 * slot; }
__host__ __device__ __forceinline__ int64_t block_bytes(int P, int d) { return static_cast<int64_t>(P) * (d + 4); }

inline bool page_size_ok(int P) { return P == 16 || P == 32 || P == 64 || P == 128; }

struct AttnArgs {
  const void* q;
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* cache_len;
  const void* k_tree;
  const void* v_tree;
  const int32_t* node_off;
  const int32_t* node_cnt;
  const uint64_t* anc;
  const int32_t* vis_prefix;
  void* out;
  float* lse;
  int32_t* err;
  int64_t ldq, ldk, ldv;   // elements between rows of q, k_tree, v_tree
  int n_pages, page_size, table_ld, anc_words;
  int B, max_nodes, total_nodes, Hq, Hkv, d, dtype;
  float scale;
};

// The nodes of request r that exist: first node and count, clipped to the tensors.
struct Span {
  int n0, cnt;
};
__device__ __forceinline__ Span node_span(const AttnArgs& a, int r) {
  Span s;
  s.n0 = max(a.node_off[r], 0);
  int n = min(a.node_off[r + 1], a.total_nodes) - s.n0;
  if (a.node_cnt) n = min(n, a.node_cnt[r]);
  s.cnt = max(0, min(n, a.max_nodes));
  return s;
}
__device__ __forceinline__ int prefix_len(const AttnArgs& a, int r) {
  const int cap = a.table_ld * a.page_size;
  const int raw = a.cache_len[r], len = min(max(raw, 0), cap);
  if (raw != len && a.err) *a.err = 1;
  return len;
}

int attn_simt(const AttnArgs& a, void* ws, cudaStream_t st);            // fp32 rows
int attn_mma(const AttnArgs& a, void* ws, cudaStream_t st);   // bf16, at most 16 rows per KV head
int attn_tc(const AttnArgs& a, void* ws, cudaStream_t st);    // bf16
size_t attn_mma_workspace(int B, int max_nodes, int Hq, int Hkv, int d);
size_t attn_tc_workspace(int B, int max_nodes, int Hq, int Hkv, int d);

}  // namespace kv4
}  // namespace tv
