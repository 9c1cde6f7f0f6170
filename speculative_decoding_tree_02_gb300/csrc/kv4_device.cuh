// Device pieces shared by the two tensor-core kernels of tree_verify_attn_kv4.
#pragma once

#include "kv4.cuh"
#include "tc_common.cuh"

namespace tv {
namespace kv4 {

constexpr float kLow = -3.3895314e38f;   // reference of a piece that has seen nothing

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Pairs of fp32 (one instruction for two).
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(x), "f"(y), "f"(z));
  return d;
}

// Codes in bits 0-3 and 16-19 -> bf16 pair of n = code - 8 (128 + code - 136, exact).
// `magic` is kMagic by way of a kernel argument: with both constants known
// the assembler takes two logic instructions, an instruction having room for
// one immediate; the logic pipe is what bounds the dequantisation.
constexpr uint32_t kMagic = 0x43004300u;   // bf16 128, 128
__device__ __forceinline__ uint32_t decode_pair(uint32_t w, uint32_t magic) {
  const uint32_t bias = 0x43084308u;       // bf16 136, 136
  uint32_t x;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "n"(0x000f000f), "r"(magic));   // (w & mask) | magic
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                   *reinterpret_cast<const __nv_bfloat162*>(&bias));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// A code word -> its four pairs (items 2i, 2i + 1).
__device__ __forceinline__ void decode8(uint32_t w, uint32_t* r, uint32_t magic) {
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = decode_pair(w >> (4 * i), magic);
}

// Bounded waits.  A poll is a handful of instructions in a tight loop (the
// warps that wait share the issue slots with those that work); the clock is
// read once in 64 polls.
constexpr long long kWaitClocks = 4000000000ll;   // about 2 s
__device__ __forceinline__ bool poll64(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, 64;\n\t"
      "WAIT%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE%=;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra WAIT%=;\n\t"
      "DONE%=:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int code) {
  if (poll64(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (poll64(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitClocks) break;
  }
  *abort_flag = 1;
  atomicExch(err, code);
  return false;
}
// For work in flight when a kernel ends: until it is done, at most kWaitClocks, whatever became of other waits.
__device__ __forceinline__ bool drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!tc::mbar_try(bar, parity))
    if (clock64() - t0 > kWaitClocks) return false;
  return true;
}
// By a whole warp: true when the phase is over, the same in all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int code) {
  if (__builtin_expect(__all_sync(0xffffffffu, tc::mbar_test(bar, parity)), 1)) return true;
  return __all_sync(0xffffffffu, bounded_wait(bar, parity, abort_flag, err, code));
}

// Per entry (request x row tile of nq nodes) the visible prefix, the first and
// the number of 128-node tree tiles: for calls where these do not follow from
// the lengths alone (nodes with prefixes of their own, larger trees).
constexpr int kTreeTile = 128;
int attn_extents(const AttnArgs& a, int nq, int tiles, int4* out, cudaStream_t st);

// Partial results of units that the end of a run cuts: a run has two slots
// (0: the unit was begun by an earlier run, 1: it begins here), R rows each.
struct Pieces {
  int4* desc;      // [runs] pieces, request, row tile, KV head of a unit that begins in a run and ends in another
  float2* ml;      // [2 runs][R] reference (base-2 units), sum
  float* o;        // [2 runs][R][d] unnormalised
};
inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
size_t pieces_bytes(int runs, int R, int d);
Pieces pieces_at(char* base, int runs, int R);
// `status`: the call's status word, written by the kernel before.
int attn_join(const AttnArgs& a, const Pieces& p, const int* status, int runs, int R, int nq, cudaStream_t st);
// What a call writes to its status word at the start: 0, except when the caller's process plants a failure to test the
// failure path (TV_TEST_ATTN_KV4_STATUS, read on the host).
int initial_status();

}  // namespace kv4
}  // namespace tv
