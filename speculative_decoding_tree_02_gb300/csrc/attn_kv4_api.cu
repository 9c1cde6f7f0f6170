// tree_verify_attn_kv4 entry point: host validation, workspace, dispatch by type
// (bf16 rows on the tensor cores, fp32 rows on the CUDA cores: their products
// would lose bits in a bf16 MMA).
#include <algorithm>

#include "kv4.cuh"

using namespace tv;

namespace {
bool shape_ok(int B, int max_nodes, int Hq, int Hkv, int d) {
  return B >= 0 && max_nodes >= 0 && Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && (d == 64 || d == 128);
}
// Which bf16 kernel: the warps' own mma.sync up to 16 rows per KV head, the
// tcgen05 tiles above. 64 requests over 512..4096 tokens, 1 over 2048 and 8 over
// 8192 of 8 KV heads of 128, mma.sync against tcgen05: 4 rows 54/15/35 against
// 100/17/50 us, 16 rows 76/18/41 against 103/17/52, 32 rows (with twice the
// accumulators) 152/39/72 against 105/19/53.  max_nodes is the caller's bound:
// the live nodes are known on the device only, and a captured call keeps its
// kernel whatever they are.
bool few_rows(int max_nodes, int Hq, int Hkv) { return static_cast<int64_t>(max_nodes) * (Hq / Hkv) <= 16; }
// The kernels count a request's tokens, the places of its row tile's units (a unit's tiles, and a fixed part) and those of
// a run in 32 bits: tokens with room for a tile beyond the last, 2^38 places in all for at least 2^7 runs.
bool counts_fit(int B, int max_nodes, int Hq, int Hkv, int64_t cap) {
  const int nq = 64 / (Hq / Hkv);
  const int64_t places = (cap / 64 + 24) * Hkv, tiles = static_cast<int64_t>(B) * ((max_nodes + nq - 1) / nq);
  return cap <= 0x7fff0000ll && places <= 0x7fffffffll && tiles * places <= 1ll << 38;
}
}  // namespace

TV_API size_t tree_verify_attn_kv4_workspace_size(int B, int max_nodes, int Hq, int Hkv, int d, int dtype) {
  if (!shape_ok(B, max_nodes, Hq, Hkv, d) || B == 0 || max_nodes == 0 || Hq / Hkv > 64) return 0;
  if (dtype != TV_BF16) return 256;
  // enough for every smaller call too, whichever kernel it takes: a server keeps one workspace for its largest trees
  const int g = Hq / Hkv;
  size_t bytes = few_rows(max_nodes, Hq, Hkv) ? 0 : kv4::attn_tc_workspace(B, max_nodes, Hq, Hkv, d);
  for (const int rows : {8, 16}) {
    const int nodes = std::min(max_nodes, rows / g);
    if (nodes > 0) bytes = std::max(bytes, kv4::attn_mma_workspace(B, nodes, Hq, Hkv, d));
  }
  return bytes;
}

TV_API int tree_verify_attn_kv4(const void* q, int64_t ldq, const void* cache, int n_pages, int page_size,
                                const int32_t* block_table, int table_ld, const int32_t* cache_len, const void* k_tree,
                                int64_t ldk, const void* v_tree, int64_t ldv, const int32_t* node_off,
                                const int32_t* node_cnt, const uint64_t* anc, int anc_words, const int32_t* vis_prefix,
                                int B, int max_nodes, int total_nodes, int Hq, int Hkv, int d, int dtype, float scale,
                                void* out, float* lse, void* ws, size_t ws_bytes, int32_t* err, tv_stream_t stream) {
  if (B < 0 || max_nodes < 0 || total_nodes < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv) return TV_EINVAL;
  if (n_pages < 0 || table_ld < 0 || page_size <= 0) return TV_EINVAL;
  if (dtype != TV_F32 && dtype != TV_BF16) return TV_EINVAL;
  if (d != 64 && d != 128) return TV_EUNSUPPORTED;
  if (!kv4::page_size_ok(page_size) || Hq / Hkv > 64 || max_nodes > TV_MAX_NODES) return TV_EUNSUPPORTED;
  if (static_cast<int64_t>(B) * Hkv > 65535 || Hq > 65535) return TV_EUNSUPPORTED;
  if (!counts_fit(B, max_nodes, Hq, Hkv, static_cast<int64_t>(table_ld) * page_size)) return TV_EUNSUPPORTED;
  if (anc_words < (max_nodes + 63) / 64 || anc_words < 1) return TV_EINVAL;
  if (!(scale > 0.f) || scale > 3.402823466e38f) return TV_EINVAL;
  if (B == 0 || max_nodes == 0 || total_nodes == 0) return TV_OK;
  if (!q || !cache_len || !k_tree || !v_tree || !node_off || !anc || !out) return TV_EINVAL;
  if (table_ld > 0 && !block_table) return TV_EINVAL;
  if (n_pages > 0 && !cache) return TV_EINVAL;
  const int vec = dtype == TV_BF16 ? 8 : 4;
  const int64_t lds[] = {ldq, ldk, ldv};
  const int heads[] = {Hq, Hkv, Hkv};
  for (int i = 0; i < 3; ++i)
    if (lds[i] < static_cast<int64_t>(heads[i]) * d || lds[i] % vec || lds[i] > 0x7fffffffll) return TV_EINVAL;
  const void* ptrs[] = {q, k_tree, v_tree, out, cache};
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return TV_EINVAL;
  if (!ws || ws_bytes < tree_verify_attn_kv4_workspace_size(B, max_nodes, Hq, Hkv, d, dtype) || !aligned(ws, 256))
    return TV_EWORKSPACE;
  const kv4::AttnArgs a{q, static_cast<const uint8_t*>(cache), block_table, cache_len, k_tree, v_tree, node_off,
                        node_cnt, anc, vis_prefix, out, lse, err, ldq, ldk, ldv, n_pages, page_size, table_ld,
                        anc_words, B, max_nodes, total_nodes, Hq, Hkv, d, dtype, scale};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == TV_BF16) return few_rows(max_nodes, Hq, Hkv) ? kv4::attn_mma(a, ws, st) : kv4::attn_tc(a, ws, st);
  return kv4::attn_simt(a, ws, st);
}
