// Arguments and row lists of kv4_attn_mass, shared by its kernels.
#pragma once

#include "cluster.cuh"
#include "kv4.cuh"

namespace tv {
namespace kv4 {

struct MassArgs {
  const void* q;
  const float* lse;
  const uint8_t* cache;
  const int32_t* block_table;
  const int32_t* cache_len;
  const int32_t* row_off;
  const int32_t* path;
  const int32_t* vis_prefix;
  const int32_t* old_len;
  const float* score_in;
  float* score_out;
  int32_t* err;
  int64_t ldq, in_ld, out_ld;
  int n_pages, P, table_ld, path_ld, causal, max_rows, total_rows, max_len, Hq, Hkv;
  float scale, decay;
};

// What a request brings: its cached tokens, its rows, and whether its arguments are out of bounds.
struct MassSpan {
  int len, old, base, count;
  bool bad;
};
// By all threads of a CTA; `s_first` is a shared word of its own.
__device__ __forceinline__ MassSpan mass_span(const MassArgs& a, int r, int* s_first) {
  MassSpan s;
  const int raw = a.cache_len[r];
  const int64_t cap = min(static_cast<int64_t>(a.table_ld) * a.P, static_cast<int64_t>(a.max_len));
  s.len = static_cast<int>(min(static_cast<int64_t>(max(raw, 0)), cap));
  s.bad = raw != s.len;
  s.old = a.old_len ? max(a.old_len[r], 0) : s.len;
  s.base = a.row_off[r];
  if (a.path) {
    int n = min(a.path_ld, a.max_rows);
    if (threadIdx.x == 0) *s_first = n;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += blockDim.x)
      if (a.path[static_cast<int64_t>(r) * a.path_ld + j] < 0) {
        atomicMin(s_first, j);
        break;
      }
    __syncthreads();
    s.count = *s_first;
    s.bad |= s.count == a.max_rows && a.max_rows < a.path_ld &&
             a.path[static_cast<int64_t>(r) * a.path_ld + a.max_rows] >= 0;
  } else {
    const int n = a.row_off[r + 1] - s.base;
    s.count = max(0, min(n, a.max_rows));
    s.bad |= n > a.max_rows;
  }
  return s;
}
// Row j of the request: its index in q and the cached tokens that it sees (0 for a row outside the tensor).
struct MassRow {
  int64_t src;
  int vis;
  bool bad;
};
__device__ __forceinline__ MassRow mass_row(const MassArgs& a, const MassSpan& s, int r, int j) {
  MassRow m;
  m.src = static_cast<int64_t>(s.base) + (a.path ? a.path[static_cast<int64_t>(r) * a.path_ld + j] : j);
  m.bad = m.src < 0 || m.src >= a.total_rows;
  m.vis = 0;
  if (m.bad) return m;
  m.vis = s.len;
  if (a.causal) m.vis = static_cast<int>(min(static_cast<int64_t>(s.len), static_cast<int64_t>(s.old) + j + 1));
  if (a.vis_prefix) m.vis = min(m.vis, max(a.vis_prefix[m.src], 0));
  return m;
}
// Page of token t of request r, -1 when it has none.
__device__ __forceinline__ int mass_page(const MassArgs& a, int r, int t) {
  const int page = a.block_table[static_cast<int64_t>(r) * a.table_ld + t / a.P];
  return page >= 0 && page < a.n_pages ? page : -1;
}
// What token t has gathered before, decayed.
__device__ __forceinline__ float mass_before(const MassArgs& a, const MassSpan& s, int64_t row, int t) {
  if (!a.score_in || t >= s.old || a.decay == 0.f) return 0.f;
  return a.decay * a.score_in[row * a.in_ld + t];
}

// Query rows per KV head up to which mass_few takes a call; mass_tc pays the set-up
// of 256 tokens (5.6 us) before the rows count.  us for 128, 160, 192 and 224 rows
// of 8 heads of 128, few against tc: 64 requests of 512..4096 tokens 121 146 171
// 209 against 211 231 235 254, 8 of 8192 72 87 99 127 against 77 86 88 97.
constexpr int kFewRows = 192;

int mass_simt(const MassArgs& a, int B, int d, cudaStream_t st);   // fp32 rows
int mass_few(const MassArgs& a, int B, int d, cudaStream_t st);    // bf16, few rows per KV head
int mass_tc(const MassArgs& a, int B, int d, cudaStream_t st);     // bf16, any number

}  // namespace kv4
}  // namespace tv
