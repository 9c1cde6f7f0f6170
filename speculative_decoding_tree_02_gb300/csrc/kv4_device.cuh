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

// Bounded waits.  The clock is read only once in many polls: a poll is a few
// cycles, reading a timer in every one delays what is waited for.
constexpr long long kWaitClocks = 4000000000ll;   // about 2 s
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int code) {
  const long long t0 = clock64();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
      if (tc::mbar_try(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitClocks) break;
  }
  *abort_flag = 1;
  atomicExch(err, code);
  return false;
}
// By a whole warp: true when the phase is over, the same in all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int code) {
  bool ok = tc::mbar_try(bar, parity);
  if (!__all_sync(0xffffffffu, ok)) ok = __all_sync(0xffffffffu, ok || wait_slow(bar, parity, abort_flag, err, code));
  return ok;
}

// Per entry (request x row tile of nq nodes) the visible prefix, the first and
// the number of 128-node tree tiles (see attn_kv4_tc.cu): for calls where
// these do not follow from the lengths alone.
int attn_extents(const AttnArgs& a, int nq, int tiles, int4* out, cudaStream_t st);

}  // namespace kv4
}  // namespace tv
