// hca_cache_tc.cuh -- what the tensor-core kernels over the 8-bit cache share:
// the numbers of their fp16 operands and small pieces of PTX.
#pragma once

#include <cuda_bf16.h>

#include <cfloat>
#include <climits>
#include <type_traits>

#include "hca_cache.cuh"
#include "tc_tiles.cuh"

namespace hca {
namespace cache {

using namespace tc;

// The reference exponent of a row is kBias below its largest score so far and is
// raised when that is beaten by 2^kRaiseLog2 (hca_cache_attn_tc.cu).
constexpr float kRaiseLog2 = 11.f, kBias = 2.f;
constexpr int kLeastExp = -15, kMostExp = 7;      // e: 2^-9 .. 448 times 2^e is an fp16 value
constexpr int kLeastUnit = -100, kMostUnit = 127;  // u: 2^u / l is a normal number (l below 2^26)
constexpr int kLeastQExp = -118;                  // exponent of q's factor: so is its reciprocal

// s = 2^exponent * part with part in (0.5, 1], for positive finite s.
__device__ __forceinline__ int split_scale(float s, float &part) {
  const int sub = s < FLT_MIN ? 24 : 0;  // a subnormal one
  const uint32_t u = __float_as_uint(sub ? s * 16777216.f : s), mant = u & 0x7fffffu;
  part = mant ? __uint_as_float(mant | (126u << 23)) : 1.f;
  return (int)(u >> 23) - (mant ? 126 : 127) - sub;
}
// 2^e in both halves, e in [kLeastExp, kMostExp]
__device__ __forceinline__ uint32_t f16x2_exp2(int e) { return (e >= -14 ? (uint32_t)(e + 15) << 10 : 0x400u >> (-14 - e)) * 0x10001u; }
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void st_shared(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void ld_shared(uint32_t addr, uint32_t (&v)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 16 bytes of which the first n come from p and the others are 0
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *p, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
               "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// 4 e4m3 values -> two fp16 pairs
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t &a, uint32_t &b) {
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(w));
}

// A warp's rows of O times f.
template <int D>
static __device__ __noinline__ void scale_o(uint32_t addr, float f) {
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t o[16];
    tmem_ld16(addr + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
    tmem_st16(addr + c, o);
  }
  tmem_wait_st();
}

}  // namespace cache
}  // namespace hca
