// Warp-level primitives of the paged-cache kernels, beside those of
// decode_ptx.cuh.  The CPU emulator (tests/emu) defines the same functions
// on the host, so that the kernels' sources run there unchanged.
#pragma once

#include <cstdint>

#include "decode_ptx.cuh"

namespace cattn {

constexpr unsigned kFullWarp = 0xffffffffu;

// The kernel's dynamic shared memory, 1024-byte aligned, and shared-memory
// addresses as 32-bit numbers (alignment of the number = that of the place).
__device__ __forceinline__ uint8_t* pg_dynamic_smem() {
  extern __shared__ __align__(1024) uint8_t pg_smem_base[];
  return pg_smem_base;
}
__device__ __forceinline__ uint32_t pg_smem_addr(const void* p) { return dec_smem_addr(p); }
// dec_cp_async16, dec_ldsm_x4, _x4_t and _x2 with such an address.
__device__ __forceinline__ void pg_cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void pg_cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void pg_ldsm_x4(uint32_t (&r)[4], uint32_t row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(row)
               : "memory");
}
__device__ __forceinline__ void pg_ldsm_x4_t(uint32_t (&r)[4], uint32_t row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(row)
               : "memory");
}
__device__ __forceinline__ void pg_ldsm_x2(uint32_t (&r)[2], uint32_t row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];\n"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(row)
               : "memory");
}

// The value of lane `src` (0..31) of the warp.
__device__ __forceinline__ int dec_shfl(int v, int src) { return __shfl_sync(kFullWarp, v, src); }
__device__ __forceinline__ float dec_shfl(float v, int src) {
  return __shfl_sync(kFullWarp, v, src);
}
__device__ __forceinline__ long long dec_shfl(long long v, int src) {
  return __shfl_sync(kFullWarp, v, src);
}
__device__ __forceinline__ double dec_shfl(double v, int src) {
  return __shfl_sync(kFullWarp, v, src);
}
// The warp's predicate bits, lane l in bit l.
__device__ __forceinline__ unsigned dec_ballot(bool p) { return __ballot_sync(kFullWarp, p); }
__device__ __forceinline__ int dec_popc(unsigned x) { return __popc(x); }
// Index of the lowest set bit (x != 0).
__device__ __forceinline__ int dec_lowest(unsigned x) { return __ffs(static_cast<int>(x)) - 1; }
__device__ __forceinline__ long long dec_double_bits(double x) { return __double_as_longlong(x); }
__device__ __forceinline__ unsigned dec_float_bits(float x) { return __float_as_uint(x); }
__device__ __forceinline__ float dec_bits_float(unsigned u) { return __uint_as_float(u); }
// 2^x to 2 ulp; results below the smallest normal number are 0.
__device__ __forceinline__ float dec_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// High word of the 128-bit product.
__device__ __forceinline__ unsigned long long dec_mulhi(unsigned long long a,
                                                        unsigned long long b) {
  return __umul64hi(a, b);
}
// Sum over the warp's lanes.
__device__ __forceinline__ int dec_warp_sum(int v) { return __reduce_add_sync(kFullWarp, v); }
__device__ __forceinline__ unsigned dec_warp_min(unsigned v) {
  return __reduce_min_sync(kFullWarp, v);
}
__device__ __forceinline__ unsigned dec_warp_max(unsigned v) {
  return __reduce_max_sync(kFullWarp, v);
}
// atomicAdd on a shared counter.
__device__ __forceinline__ int dec_add_shared(int* p, int v) { return atomicAdd(p, v); }
// Rank of the CTA in its cluster, and the cluster's size.
__device__ __forceinline__ unsigned dec_cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
// Per bf16 half: max(m, |x|), m >= 0 (the bit patterns of magnitudes are in
// their order).
__device__ __forceinline__ uint32_t dec_bf16_absmax(uint32_t m, uint32_t x) {
  return __vmaxu2(m, x & 0x7fff7fffu);
}
// Per bf16 half, the lower and the higher value; a NaN stays.
__device__ __forceinline__ uint32_t dec_bf16_min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t dec_bf16_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// bf16 halves of a word as floats (exact).
__device__ __forceinline__ float dec_bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float dec_bf16_hi(uint32_t w) {
  return __uint_as_float(w & 0xffff0000u);
}

}  // namespace cattn
