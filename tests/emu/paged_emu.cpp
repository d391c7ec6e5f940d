// Runs the paged-cache kernels (the device sources themselves) on the host
// through simt_emu.h, for CPU tests: exactly sized buffers under
// AddressSanitizer and UBSan, so any out-of-bounds or misaligned access of a
// kernel fails the run.
//
//   paged_emu decode|plan|append|select in.bin out.bin
//
// With LATE_WARP=w in the environment, warp w of each CTA goes on late behind
// every CTA barrier.
//
// in.bin is a row of arrays, each an int64 byte count and the bytes; the
// first holds int64 parameters.  out.bin is the outputs, one behind the other.
// The host set-up (grids, strides of packed arrays) follows api.cu.
#define CATTN_HOST_EMULATION 1
#include "simt_emu.h"

#include <cstdio>
#include <cstdlib>
#include <string>

#include "paged_ptx_emu.h"
#include "decode.cuh"
#include "paged_cache.cuh"
#include "paged_decode.cuh"

using namespace cattn;

static std::vector<uint8_t*> g_in;  // exactly sized, never freed before exit
static std::vector<size_t> g_bytes;
static FILE* g_out;

static void read_all(const char* path) {
  FILE* f = std::fopen(path, "rb");
  if (!f) std::exit(3);
  int64_t n;
  while (std::fread(&n, 8, 1, f) == 1) {
    auto* p = static_cast<uint8_t*>(std::malloc(n ? n : 1));
    if (n && std::fread(p, 1, n, f) != static_cast<size_t>(n)) std::exit(3);
    g_in.push_back(p);
    g_bytes.push_back(n);
  }
  std::fclose(f);
}
template <typename T>
static T* in(size_t i) {
  return g_bytes.at(i) ? reinterpret_cast<T*>(g_in.at(i)) : nullptr;
}
// An output buffer filled with a pattern that is no result.
template <typename T>
static T* out(size_t n) {
  auto* p = static_cast<T*>(std::malloc(n ? n * sizeof(T) : 1));
  std::memset(p, 0xa5, n * sizeof(T));
  return p;
}
static void put(const void* p, size_t bytes) {
  if (bytes) std::fwrite(p, 1, bytes, g_out);
}

template <int D, bool UP, bool MULTI>
static void run_decode_as(const PagedParams& p, int grid) {
  if (grid < 0) {
    emu::launch_ex(static_cast<unsigned>(p.B * p.Hkv * p.n_tiles * -grid), kPagedThreads,
                   paged_smem_bytes(D, kItemStages), static_cast<unsigned>(-grid), paged_item_kernel<D, UP, MULTI>,
                   p, -grid);
    return;
  }
  emu::launch_ex(grid, kPagedThreads, paged_smem_bytes(D, kPagedStages), 1, paged_decode_kernel<D, UP, MULTI>,
                 p);
  const int n_y = paged_merge_y(p.R);
  emu::launch_ex(grid * n_y, kMergeThreads, paged_merge_smem_bytes(D), 1, paged_merge_kernel<D>,
                 p, n_y);
}

template <int D>
static void run_decode(const PagedParams& p, int grid) {
  const bool up = p.rows > 8, multi = p.Tq > 1;
  if (up)
    multi ? run_decode_as<D, true, true>(p, grid) : run_decode_as<D, true, false>(p, grid);
  else
    multi ? run_decode_as<D, false, true>(p, grid) : run_decode_as<D, false, false>(p, grid);
}

// params: B H Hkv Tq D n_pages P width n_sel grid layout (grid < 0: -grid CTAs
//         per item); scale as float
// arrays: q, k, v (layout 0: (n_pages, Hkv, P, D), 1: (n_pages, P, Hkv, D)),
//         table, lengths, pages, scale
static void decode() {
  const int64_t* a = in<int64_t>(0);
  PagedParams p{};
  p.B = a[0]; p.H = a[1]; p.Hkv = a[2]; p.Tq = a[3];
  const int D = a[4];
  p.n_pages = a[5]; p.P = a[6]; p.width = a[7]; p.n_sel = a[8];
  const int grid = a[9];
  p.rows = p.H / p.Hkv * p.Tq;
  p.n_tiles = (p.rows + kPagedRows - 1) / kPagedRows;
  p.R = p.rows < kPagedRows ? p.rows : kPagedRows;
  p.q = in<__nv_bfloat16>(1);
  p.k = in<__nv_bfloat16>(2);
  p.v = in<__nv_bfloat16>(3);
  p.table = in<int>(4);
  p.table_sb = p.width;
  p.lengths = in<int>(5);
  p.pages = in<int>(6);
  p.scale_log2 = *in<float>(7) * 1.4426950408889634f;
  p.by_P = PageDivider(p.P);
  p.q_sb = static_cast<long long>(p.H) * p.Tq * D;
  p.q_sh = static_cast<long long>(p.Tq) * D;
  p.q_st = D;
  p.k_sp = static_cast<long long>(p.Hkv) * p.P * D;
  p.k_sh = a[10] ? D : static_cast<long long>(p.P) * D;
  p.k_st = a[10] ? static_cast<long long>(p.Hkv) * D : D;
  p.v_sp = p.k_sp; p.v_sh = p.k_sh; p.v_st = p.k_st;
  p.o_sb = p.q_sb; p.o_sh = p.q_sh; p.o_st = p.q_st;
  const size_t rows = static_cast<size_t>(p.B) * p.H * p.Tq;
  p.o = out<__nv_bfloat16>(rows * D);
  p.lse = out<float>(rows);
  const size_t warps = grid > 0 ? static_cast<size_t>(grid) * kPagedWarps : 0;
  p.cuts = out<PagedCut>(warps);
  p.part_ml = out<float2>(2 * warps * p.R);
  p.part_o = out<float>(2 * warps * p.R * D);
  switch (D) {
    case 16: run_decode<16>(p, grid); break;
    case 32: run_decode<32>(p, grid); break;
    case 64: run_decode<64>(p, grid); break;
    case 128: run_decode<128>(p, grid); break;
    default: std::exit(4);
  }
  put(p.o, rows * D * 2);
  put(p.lse, rows * 4);
}

// params: B width n_pages P n_slots ctas in_place threads prompts
// arrays: asked, lengths, table, ring, state
static void plan() {
  const int64_t* a = in<int64_t>(0);
  PlanParams p{};
  p.B = a[0]; p.width = a[1]; p.n_pages = a[2]; p.P = a[3];
  p.n_slots = a[4];
  const unsigned ctas = a[5];
  p.asked = in<int>(1);
  p.lengths = in<int>(2);
  p.table = in<int>(3);
  p.table_sb = p.width;
  p.ring = in<int>(4);
  p.state = in<long long>(5);
  p.lengths_out = a[6] ? in<int>(2) : out<int>(p.B);
  p.state_out = a[6] ? in<long long>(5) : out<long long>(2);
  p.cu = out<int>(p.B + 1);
  p.slots = out<long long>(p.n_slots);
  p.positions = out<int>(p.n_slots);
  p.status = out<int>(1);
  p.by_P = PageDivider(p.P);
  emu::launch_ex(ctas, a[7], plan_smem_bytes(p.B), ctas,
                 a[8] ? paged_plan_kernel<false> : paged_plan_kernel<true>, p,
                 static_cast<int>(ctas));
  const int64_t per = kSlotsV * kSlotsThreads;
  if (a[8])
    emu::launch_ex(static_cast<unsigned>((p.n_slots + per - 1) / per), kSlotsThreads, 0, 1,
                   paged_slots_kernel, p);
  put(p.lengths_out, 4ull * p.B);
  put(p.state_out, 16);
  put(p.cu, 4ull * (p.B + 1));
  put(p.slots, 8ull * p.n_slots);
  put(p.positions, 4ull * p.n_slots);
  put(p.status, 4);
  put(p.table, 4ull * p.B * p.width);
  put(p.ring, 4ull * p.n_pages);
}

template <int D>
static void run_append(const AppendParams& p, int tile) {
  if (p.bounds) {
    emu::launch_ex(static_cast<unsigned>(2 * ((p.n + tile - 1) / tile)), kBoundsThreads,
                   append_smem_bytes(), 1, cache_append_bounds_kernel<D>, p, tile);
    return;
  }
  const auto blocks =
      static_cast<unsigned>((p.n * p.Hkv * (D / 8) + kAppendThreads - 1) / kAppendThreads);
  emu::launch_ex(blocks, kAppendThreads, 0, 1, cache_append_kernel<D>, p);
}

// params: n Hkv D n_pages P tile; arrays: k_new, v_new (n, Hkv, D), slots, k, v
// (n_pages, P, Hkv, D), bounds
static void append() {
  const int64_t* a = in<int64_t>(0);
  AppendParams p{};
  p.n = a[0]; p.Hkv = a[1];
  const int D = a[2];
  p.P = a[4];
  p.n_rows = a[3] * a[4];
  p.mul = append_mul(p.P);
  p.kn = in<__nv_bfloat16>(1);
  p.vn = in<__nv_bfloat16>(2);
  p.slots = in<long long>(3);
  p.k = in<__nv_bfloat16>(4);
  p.v = in<__nv_bfloat16>(5);
  p.bounds = in<__nv_bfloat16>(6);
  p.kn_st = p.vn_st = static_cast<long long>(p.Hkv) * D;
  p.kn_sh = p.vn_sh = D;
  p.k_sp = p.v_sp = static_cast<long long>(p.P) * p.Hkv * D;
  p.k_sh = p.v_sh = D;
  p.k_st = p.v_st = static_cast<long long>(p.Hkv) * D;
  switch (D) {
    case 16: run_append<16>(p, a[5]); break;
    case 32: run_append<32>(p, a[5]); break;
    case 64: run_append<64>(p, a[5]); break;
    case 128: run_append<128>(p, a[5]); break;
    default: std::exit(4);
  }
  put(p.k, g_bytes[4]);
  put(p.v, g_bytes[5]);
  put(p.bounds, g_bytes[6]);
}

template <int D, bool UP>
static void run_select(const SelectParams& p, bool fused) {
  const auto bh = static_cast<unsigned>(p.B * p.Hkv);
  if (fused) {
    emu::launch_ex(bh * kSelectCtas, kSelectThreads, select_smem_bytes(D), kSelectCtas,
                   page_select_kernel<D, UP>, p);
    return;
  }
  emu::launch_ex(bh * p.n_blocks, kScoreThreads, kScoreWarps * score_ring_bytes(D), 1,
                 page_score_kernel<D, UP>, p);
  emu::launch_ex(bh, kPickThreads, pick_smem_bytes(), 1, page_pick_kernel, p);
}

// params: B H Hkv Tq D n_pages P width n_sel n_first n_last groups (0: the
//         fused kernel)
// arrays: q, bounds, table, lengths
static void select() {
  const int64_t* a = in<int64_t>(0);
  SelectParams p{};
  p.B = a[0]; p.H = a[1]; p.Hkv = a[2]; p.Tq = a[3];
  const int D = a[4];
  p.n_pages = a[5]; p.P = a[6]; p.width = a[7];
  p.n_sel = a[8]; p.n_first = a[9]; p.n_last = a[10];
  p.rows = p.H / p.Hkv * p.Tq;
  p.D = D;
  const bool fused = a[11] == 0;
  p.groups = fused ? 1 : a[11];
  const int per = kScoreWarps * 8 * p.groups;
  p.n_blocks = (p.width + per - 1) / per;
  p.q = in<__nv_bfloat16>(1);
  p.q_sb = static_cast<long long>(p.H) * p.Tq * D;
  p.q_sh = static_cast<long long>(p.Tq) * D;
  p.q_st = D;
  p.bounds = in<__nv_bfloat16>(2);
  p.table = in<int>(3);
  p.table_sb = p.width;
  p.lengths = in<int>(4);
  p.pages = out<int>(static_cast<size_t>(p.B) * p.Hkv * p.n_sel);
  p.exact = out<double>(static_cast<size_t>(p.B) * p.Hkv * p.width);
  p.score = out<float>(static_cast<size_t>(p.B) * p.Hkv * p.width);
  p.largest = out<float>(static_cast<size_t>(p.B) * p.Hkv * (fused ? kSelectCtas * kSelectThreads / 32
                                                                    : p.n_blocks * kScoreWarps));
  const bool up = p.rows > 8;
  switch (D) {
    case 16: up ? run_select<16, true>(p, fused) : run_select<16, false>(p, fused); break;
    case 32: up ? run_select<32, true>(p, fused) : run_select<32, false>(p, fused); break;
    case 64: up ? run_select<64, true>(p, fused) : run_select<64, false>(p, fused); break;
    case 128: up ? run_select<128, true>(p, fused) : run_select<128, false>(p, fused); break;
    default: std::exit(4);
  }
  put(p.pages, 4ull * p.B * p.Hkv * p.n_sel);
}

int main(int argc, char** argv) {
  if (argc != 4) return 2;
  read_all(argv[2]);
  g_out = std::fopen(argv[3], "wb");
  if (!g_out) return 5;
  if (const char* w = std::getenv("LATE_WARP")) emu::g_late_warp = std::atoi(w);
  const std::string op = argv[1];
  if (op == "decode") decode();
  else if (op == "plan") plan();
  else if (op == "append") append();
  else if (op == "select") select();
  else return 2;
  std::fclose(g_out);
  return 0;
}
