// Host definitions of the paged-cache kernels' warp primitives (the functions
// of paged_ptx.cuh), for the CPU emulator: shared-memory addresses, indexed
// shuffles, ballots, the cluster rank, warp sums, bit casts.
#pragma once

#include <atomic>
#include <cstdint>
#include <cstring>
#include <stdexcept>

#include "decode_ptx_emu.h"

struct alignas(16) int4 {
  int x, y, z, w;
};
struct alignas(16) longlong2 {
  long long x, y;
};

namespace cattn {

constexpr unsigned kFullWarp = 0xffffffffu;

// Shared-memory addresses: offsets into the CTA's dynamic shared memory.
inline uint8_t* pg_dynamic_smem() { return emu::t_cta->dsmem; }
inline uint32_t pg_smem_addr(const void* p) {
  return static_cast<uint32_t>(static_cast<const uint8_t*>(p) - emu::t_cta->dsmem);
}
inline void pg_cp_async16(uint32_t dst, const void* src) {
  dec_cp_async16(emu::t_cta->dsmem + dst, src, true);
}
inline void pg_cp_async16(uint32_t dst, const void* src, bool valid) {
  dec_cp_async16(emu::t_cta->dsmem + dst, src, valid);
}
inline void pg_ldsm_x4(uint32_t (&r)[4], uint32_t row) {
  dec_ldsm_x4(r, emu::t_cta->dsmem + row);
}
inline void pg_ldsm_x4_t(uint32_t (&r)[4], uint32_t row) {
  dec_ldsm_x4_t(r, emu::t_cta->dsmem + row);
}
inline void pg_ldsm_x2(uint32_t (&r)[2], uint32_t row) {
  dec_ldsm_x2(r, emu::t_cta->dsmem + row);
}

namespace emu_detail {
template <typename T>
inline T shfl(T v, int src) {
  if (src < 0 || src > 31) throw std::logic_error("shuffle from a lane outside the warp");
  uint64_t mine = 0;
  std::memcpy(&mine, &v, sizeof(T));
  const uint64_t* all = emu::warp_exchange(&mine, 1);
  T r;
  std::memcpy(&r, all + src * emu::kWords, sizeof(T));
  return r;
}
}  // namespace emu_detail

inline int dec_shfl(int v, int src) { return emu_detail::shfl(v, src); }
inline float dec_shfl(float v, int src) { return emu_detail::shfl(v, src); }
inline long long dec_shfl(long long v, int src) { return emu_detail::shfl(v, src); }
inline double dec_shfl(double v, int src) { return emu_detail::shfl(v, src); }
inline unsigned dec_ballot(bool p) {
  const uint64_t mine = p;
  const uint64_t* all = emu::warp_exchange(&mine, 1);
  unsigned r = 0;
  for (int l = 0; l < 32; ++l) r |= (all[l * emu::kWords] ? 1u : 0u) << l;
  return r;
}
inline int dec_popc(unsigned x) { return __builtin_popcount(x); }
inline int dec_lowest(unsigned x) { return __builtin_ctz(x); }
inline unsigned dec_float_bits(float x) {
  unsigned r;
  std::memcpy(&r, &x, 4);
  return r;
}
inline float dec_bits_float(unsigned u) {
  float r;
  std::memcpy(&r, &u, 4);
  return r;
}
inline int dec_warp_sum(int v) {
  const uint64_t mine = static_cast<uint64_t>(static_cast<int64_t>(v));
  const uint64_t* all = emu::warp_exchange(&mine, 1);
  int64_t s = 0;
  for (int l = 0; l < 32; ++l) s += static_cast<int64_t>(all[l * emu::kWords]);
  return static_cast<int>(s);
}
inline unsigned dec_warp_min(unsigned v) {
  const uint64_t mine = v;
  const uint64_t* all = emu::warp_exchange(&mine, 1);
  uint64_t r = all[0];
  for (int l = 1; l < 32; ++l) r = all[l * emu::kWords] < r ? all[l * emu::kWords] : r;
  return static_cast<unsigned>(r);
}
inline unsigned dec_warp_max(unsigned v) { return ~dec_warp_min(~v); }
inline int dec_add_shared(int* p, int v) {
  emu::check_smem(p, 4, 4);
  return std::atomic_ref<int>(*p).fetch_add(v);
}
inline long long dec_double_bits(double x) {
  long long r;
  std::memcpy(&r, &x, 8);
  return r;
}
inline float dec_exp2(float x) {
  const float y = std::exp2(x);
  return y < 0x1p-126f ? 0.f : y;
}
inline unsigned long long dec_mulhi(unsigned long long a, unsigned long long b) {
  return static_cast<unsigned long long>(static_cast<unsigned __int128>(a) * b >> 64);
}
inline unsigned dec_cluster_rank() { return emu::t_cta->rank; }
inline uint32_t dec_bf16_absmax(uint32_t m, uint32_t x) {
  x &= 0x7fff7fffu;
  const uint32_t lo = (m & 0xffffu) > (x & 0xffffu) ? m & 0xffffu : x & 0xffffu;
  const uint32_t hi = (m >> 16) > (x >> 16) ? m >> 16 : x >> 16;
  return lo | hi << 16;
}
inline float dec_bf16_lo(uint32_t w) {
  const uint32_t u = w << 16;
  float f;
  std::memcpy(&f, &u, 4);
  return f;
}
inline float dec_bf16_hi(uint32_t w) {
  const uint32_t u = w & 0xffff0000u;
  float f;
  std::memcpy(&f, &u, 4);
  return f;
}
namespace emu_detail {
template <typename F>
inline uint32_t per_half(uint32_t a, uint32_t b, F f) {
  uint32_t r = 0;
  for (int half = 0; half < 2; ++half) {
    const uint32_t ha = half ? a & 0xffff0000u : a << 16, hb = half ? b & 0xffff0000u : b << 16;
    float x, y;
    std::memcpy(&x, &ha, 4);
    std::memcpy(&y, &hb, 4);
    const uint32_t h = x != x || y != y ? 0x7fffu : (f(x, y) ? ha : hb) >> 16;
    r |= h << (16 * half);
  }
  return r;
}
}  // namespace emu_detail
inline uint32_t dec_bf16_min(uint32_t a, uint32_t b) {
  return emu_detail::per_half(a, b, [](float x, float y) { return x <= y; });
}
inline uint32_t dec_bf16_max(uint32_t a, uint32_t b) {
  return emu_detail::per_half(a, b, [](float x, float y) { return x >= y; });
}

}  // namespace cattn
