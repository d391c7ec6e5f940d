// Kernels that keep a paged key/value cache: the step's plan (pages, slots
// and positions of the new tokens), the append of their keys and values, and
// the selection of pages for the sparse form of decode attention.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "paged_decode.cuh"

namespace cattn {

// -------------------------------------------------------------------- plan
//
// Request b holds `length` tokens in its first ceil(length / P) pages and
// asks for n more (n > 0), for nothing (0), or ends (n < 0).  Free pages lie
// in a ring of n_pages entries between the counters head and tail.  With
//   have = ceil(length / P), need = ceil((length + n) / P) - have,
// and exclusive sums over the requests, new page j of request b is
// ring[head + sum need + j], its token i has position length + i and slot
// table[b][pos / P] P + pos % P, and the pages of the requests that end go to
// ring[tail + sum have ..].  A call that cannot be served as a whole
// changes nothing but its status.
//
// A few kilobytes of whole numbers: bound by latency.  One launch of one
// thread-block cluster: every CTA scans all requests for itself (into shared
// memory), the cluster's barrier separates the last read of the inputs from
// the first write of the outputs (which may be the same arrays), and then the
// CTAs share the tokens and pages.

constexpr int kPlanThreads = 256;
constexpr int kPlanMaxB = 8192;       // requests per call (128 KB of prefix sums)
constexpr int kPlanMaxCtas = 8;       // portable cluster size
constexpr int kPlanStatusInvalid = 1;   // CATTN_ERR_INVALID_ARG
constexpr int kPlanStatusTooLarge = 5;  // CATTN_ERR_TOO_LARGE

struct PlanParams {
  const int* asked;            // (B) new tokens, negative: the request ends
  const int* lengths;          // (B)
  int* table;                  // (B, width), row stride table_sb
  long long table_sb;
  int* ring;                   // (n_pages)
  const long long* state;      // head, tail
  int B, width, n_pages, P;
  long long n_slots;
  int* lengths_out;            // (B)
  long long* state_out;        // head, tail
  int* cu;                     // (B + 1)
  long long* slots;            // (n_slots)
  int* positions;              // (n_slots)
  int* status;                 // (1)
};

__host__ __device__ constexpr int plan_smem_bytes(int B) {
  return 16 * (B + 1) + kPlanThreads / 32 * 32 + 16;
}

__device__ __forceinline__ int pages_of(int n, int P) { return n / P + (n % P != 0); }

// Last index b in [0, n) with cu[b] <= i (cu ascending, cu[0] = 0 <= i).
__device__ __forceinline__ int last_at_most(const int* cu, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (cu[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ long long warp_scan64(long long v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long long u = dec_shfl(v, lane >= d ? lane - d : 0);
    if (lane >= d) v += u;
  }
  return v;
}

// Grid: one cluster of n_ctas <= kPlanMaxCtas CTAs of kPlanThreads threads.
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanParams p, int n_ctas) {
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  constexpr int NW = kPlanThreads / 32;
  uint8_t* smem = dec_dynamic_smem();
  long long* sums = reinterpret_cast<long long*>(smem);  // [NW][3], then the flag
  int* bad = reinterpret_cast<int*>(sums + NW * 4);
  int* len_s = bad + 4;                                   // [B + 1] each
  int* cu_tok = len_s + p.B + 1;
  int* cu_need = cu_tok + p.B + 1;
  int* cu_back = cu_need + p.B + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = n_ctas > 1 ? dec_cluster_rank() : 0u;
  if (tid < 4) bad[tid] = 0;
  __syncthreads();

  // this thread's requests: b0 .. b1 - 1
  const int nb = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = tid * nb < p.B ? tid * nb : p.B, b1 = b0 + nb < p.B ? b0 + nb : p.B;
  const int cap = p.width * p.P;
  long long tok = 0, need = 0, back = 0;
  int fault = 0;  // bit 0: invalid, bit 1: too large
  for (int b = b0; b < b1; ++b) {
    const int len = p.lengths[b], n = p.asked[b];
    if (len < 0) {
      fault |= 1;
    } else if (n > 0) {
      if (len > cap || n > cap - len) {
        fault |= 2;
      } else {
        tok += n;
        need += pages_of(len + n, p.P) - pages_of(len, p.P);
      }
    } else if (n < 0) {
      if (len > cap) fault |= 1; else back += pages_of(len, p.P);
    }
  }
  if (fault & 1) bad[1] = 1;  // (any writer writes the same)
  if (fault & 2) bad[2] = 1;
  const long long it = warp_scan64(tok, lane), in = warp_scan64(need, lane),
                  ib = warp_scan64(back, lane);
  if (lane == 31) {
    sums[warp * 4] = it;
    sums[warp * 4 + 1] = in;
    sums[warp * 4 + 2] = ib;
  }
  __syncthreads();
  long long et = it - tok, en = in - need, eb = ib - back, T = 0, N = 0, R = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) {
      et += sums[w * 4];
      en += sums[w * 4 + 1];
      eb += sums[w * 4 + 2];
    }
    T += sums[w * 4];
    N += sums[w * 4 + 1];
    R += sums[w * 4 + 2];
  }
  const long long head = p.state[0], tail = p.state[1], avail = tail - head;
  int status = 0;
  if (T > p.n_slots || N > avail) status = kPlanStatusTooLarge;
  if (bad[2]) status = kPlanStatusTooLarge;
  if (bad[1] || head < 0 || avail < 0 || avail > p.n_pages || R > p.n_pages - avail)
    status = kPlanStatusInvalid;
  for (int b = b0; b < b1; ++b) {
    const int len = p.lengths[b], n = p.asked[b];
    len_s[b] = status || n >= 0 ? len : -1;  // -1: the request ends
    cu_tok[b] = status ? 0 : static_cast<int>(et);
    cu_need[b] = status ? 0 : static_cast<int>(en);
    cu_back[b] = status ? 0 : static_cast<int>(eb);
    if (!status && n > 0) {
      et += n;
      en += pages_of(len + n, p.P) - pages_of(len, p.P);
    }
    if (!status && n < 0) eb += pages_of(len, p.P);
  }
  if (status) T = N = R = 0;
  if (tid == 0) {
    cu_tok[p.B] = static_cast<int>(T);
    cu_need[p.B] = static_cast<int>(N);
    cu_back[p.B] = static_cast<int>(R);
  }
  __syncthreads();
  if (n_ctas > 1) dec_cluster_sync();  // every CTA has read its inputs

  const int start = static_cast<int>(rank) * kPlanThreads + tid, step = n_ctas * kPlanThreads;
  const int head0 = static_cast<int>(head % p.n_pages >= 0 ? head % p.n_pages : 0);
  const int tail0 = static_cast<int>(tail % p.n_pages >= 0 ? tail % p.n_pages : 0);
  auto at = [&](int base, int k) {  // ring entry of counter base + k, k < n_pages
    const long long i = static_cast<long long>(base) + k;
    return static_cast<int>(i >= p.n_pages ? i - p.n_pages : i);
  };
  for (long long i = start; i < p.n_slots; i += step) {
    long long slot = -1;
    int pos = -1;
    if (i < T) {
      const int b = last_at_most(cu_tok, p.B, static_cast<int>(i));
      const int len = len_s[b], have = pages_of(len, p.P);
      pos = len + (static_cast<int>(i) - cu_tok[b]);
      const int lp = pos / p.P;
      const int page = lp < have ? p.table[b * p.table_sb + lp]
                                 : p.ring[at(head0, cu_need[b] + lp - have)];
      if (page >= 0 && page < p.n_pages) slot = static_cast<long long>(page) * p.P + pos % p.P;
    }
    p.slots[i] = slot;
    p.positions[i] = pos;
  }
  for (int j = start; j < N; j += step) {
    const int b = last_at_most(cu_need, p.B, j);
    p.table[b * p.table_sb + pages_of(len_s[b], p.P) + (j - cu_need[b])] = p.ring[at(head0, j)];
  }
  for (int j = start; j < R; j += step) {
    const int b = last_at_most(cu_back, p.B, j);
    p.ring[at(tail0, j)] = p.table[b * p.table_sb + (j - cu_back[b])];
  }
  for (int b = start; b <= p.B; b += step) {
    p.cu[b] = cu_tok[b];
    if (b < p.B)
      p.lengths_out[b] = len_s[b] < 0 && !status ? 0 : len_s[b] + (cu_tok[b + 1] - cu_tok[b]);
  }
  if (start == 0) {
    p.state_out[0] = head + N;
    p.state_out[1] = tail + R;
    p.status[0] = status;
  }
}

// ------------------------------------------------------------------ append
//
// Row i of the new K and V goes to cache row slots[i] (page slots[i] / P, row
// slots[i] % P); a slot outside the cache is skipped.  With bounds, the lowest
// and highest value of each channel of a page's keys are kept beside it:
//   lo_d = min over the page's keys of k_d,  hi_d = max
// A run of new rows with ascending slots in one page is done by the threads
// of its first row, so nothing is updated twice; a run that starts at the
// page's first row starts its bounds over.  (NaN in, NaN out.)
//
// The bound is memory: each row is read and written once.

struct AppendParams {
  const __nv_bfloat16* kn;  // (n, Hkv, D)
  const __nv_bfloat16* vn;
  long long kn_st, kn_sh, vn_st, vn_sh;
  __nv_bfloat16* k;         // (n_pages, Hkv, P, D)
  __nv_bfloat16* v;
  long long k_sp, k_sh, k_st, v_sp, v_sh, v_st;
  const long long* slots;   // (n)
  __nv_bfloat16* bounds;    // (n_pages, Hkv, 2, D) or null
  long long n;
  int Hkv, P;
  long long n_rows;         // n_pages P
};

constexpr int kAppendThreads = 256;

// min / max of bf16 values that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  return a != a ? a : b != b ? b : fminf(a, b);
}
__device__ __forceinline__ float max_nan(float a, float b) {
  return a != a ? a : b != b ? b : fmaxf(a, b);
}

// Thread: 8 channels of one (row, head).
template <int D, bool BOUNDS>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendParams p) {
  constexpr int PC = D / 8;
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  const long long x = static_cast<long long>(blockIdx.x) * kAppendThreads + threadIdx.x;
  const int pc = static_cast<int>(x % PC);
  const long long unit = x / PC;
  const long long i = unit / p.Hkv;
  const int h = static_cast<int>(unit - i * p.Hkv);
  if (i >= p.n) return;
  const long long slot = p.slots[i];
  if (slot < 0 || slot >= p.n_rows) return;
  const long long page = slot / p.P;
  int off = static_cast<int>(slot - page * p.P);
  if (BOUNDS && off != 0 && i > 0 && p.slots[i - 1] == slot - 1) return;  // inside a run
  const bool fresh = off == 0;
  float lo[8], hi[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    lo[c] = INFINITY;
    hi[c] = -INFINITY;
  }
  const __nv_bfloat16* ks = p.kn + i * p.kn_st + h * p.kn_sh + pc * 8;
  const __nv_bfloat16* vs = p.vn + i * p.vn_st + h * p.vn_sh + pc * 8;
  __nv_bfloat16* kd = p.k + page * p.k_sp + h * p.k_sh + pc * 8;
  __nv_bfloat16* vd = p.v + page * p.v_sp + h * p.v_sh + pc * 8;
  for (long long j = i;; ++j, ++off) {
    const uint4 kw = *reinterpret_cast<const uint4*>(ks + (j - i) * p.kn_st);
    const uint4 vw = *reinterpret_cast<const uint4*>(vs + (j - i) * p.vn_st);
    *reinterpret_cast<uint4*>(kd + off * p.k_st) = kw;
    *reinterpret_cast<uint4*>(vd + off * p.v_st) = vw;
    if (!BOUNDS) return;
    const uint32_t w[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float a = dec_bf16_lo(w[c]), b = dec_bf16_hi(w[c]);
      lo[2 * c] = min_nan(lo[2 * c], a);
      hi[2 * c] = max_nan(hi[2 * c], a);
      lo[2 * c + 1] = min_nan(lo[2 * c + 1], b);
      hi[2 * c + 1] = max_nan(hi[2 * c + 1], b);
    }
    if (off + 1 >= p.P || j + 1 >= p.n || p.slots[j + 1] != slot + (j + 1 - i)) break;
  }
  uint4* bl = reinterpret_cast<uint4*>(p.bounds + ((page * p.Hkv + h) * 2) * D + pc * 8);
  uint4* bh = reinterpret_cast<uint4*>(p.bounds + ((page * p.Hkv + h) * 2 + 1) * D + pc * 8);
  if (!fresh) {
    const uint4 a = *bl, b = *bh;
    const uint32_t wl[4] = {a.x, a.y, a.z, a.w}, wh[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      lo[2 * c] = min_nan(lo[2 * c], dec_bf16_lo(wl[c]));
      lo[2 * c + 1] = min_nan(lo[2 * c + 1], dec_bf16_hi(wl[c]));
      hi[2 * c] = max_nan(hi[2 * c], dec_bf16_lo(wh[c]));
      hi[2 * c + 1] = max_nan(hi[2 * c + 1], dec_bf16_hi(wh[c]));
    }
  }
  // (the values are bf16 values: packing them rounds nothing)
  *bl = uint4{dec_pack_bf16(lo[0], lo[1]), dec_pack_bf16(lo[2], lo[3]),
              dec_pack_bf16(lo[4], lo[5]), dec_pack_bf16(lo[6], lo[7])};
  *bh = uint4{dec_pack_bf16(hi[0], hi[1]), dec_pack_bf16(hi[2], hi[3]),
              dec_pack_bf16(hi[4], hi[5]), dec_pack_bf16(hi[6], hi[7])};
}

// ------------------------------------------------------------------ select
//
// For request b and cache head h, over its G Tq query rows q_r and the bounds
// (lo, hi) of the keys of page i of the request:
//
//   s_i = max_r sum_d max(q_rd, 0) hi_d + min(q_rd, 0) lo_d
//
// an upper bound of every q_r . k in the page.  The n_first first and n_last
// last of the request's pages are always taken, then the highest s_i (the
// lower index where equal) up to n_sel pages; they are listed in ascending
// order, -1 behind the last.  A page that is not held has s = -inf, a NaN
// counts as +inf.
//
// The choice is that of exact sums, so that it does not depend on an order of
// summation.  page_score_kernel sums in fp32: at most 13 roundings lie on the
// way of a term (8 products in a lane, 5 additions between lanes), so with
// V = the largest |bound| of the request's pages and u = 2^-24
//   |s_i - exact| <= 14 u max_r sum_d |q_rd| V = rho.
// The want-th highest of a list moves by at most rho if every entry does, so
// a page more than 2 rho above (below) the want-th highest fp32 score T is
// chosen (is not).  Only if more pages lie within 2 rho of T than there are
// places left for, page_pick_kernel sums those again in 64 bits (a product of
// two bf16 values has 16 bits: a sum of 2 D of them is exact there unless they
// span more than 2^29).
//
// The bound is memory: 4 D bytes per page and cache head, read once.

struct SelectParams {
  const __nv_bfloat16* q;       // (B, H, Tq, D)
  long long q_sb, q_sh, q_st;
  const __nv_bfloat16* bounds;  // (n_pages, Hkv, 2, D)
  const int* table;
  long long table_sb;
  const int* lengths;
  int B, H, Hkv, Tq, D, rows, n_pages, P, width, n_sel, n_first, n_last;
  int n_blocks;                 // ceil(width / score_pages(D))
  int* pages;                   // (B, Hkv, n_sel)
  double* exact;                // [B Hkv][width]
  float* score;                 // [B Hkv][width]
  float* largest;               // [B Hkv][n_blocks][score warps]: |bounds|
};

constexpr int kScoreThreads = 128;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kScoreLoads = 8;     // 16-byte loads of a lane in flight
constexpr int kScoreRows = 4;      // query rows at a time
constexpr int kPickThreads = 512;
constexpr int kPickKeys = 8192;    // scores kept in shared memory

// Pages of a warp and of a CTA: a page's bounds are 4 D bytes, D / 4 lanes.
__host__ __device__ constexpr int score_warp_pages(int D) { return kScoreLoads * 128 / D; }
__host__ __device__ constexpr int score_pages(int D) { return kScoreWarps * score_warp_pages(D); }

__device__ __forceinline__ int select_count(const SelectParams& p, int b) {
  const int len = p.lengths[b];
  const int n = len > 0 ? pages_of(len, p.P) : 0;
  return n < p.width ? n : p.width;
}

__device__ __forceinline__ const __nv_bfloat16* select_row(const SelectParams& p, int b, int h,
                                                           int r) {
  const int gh = r / p.Tq, t = r - gh * p.Tq;
  return p.q + b * p.q_sb + (static_cast<long long>(h) * (p.rows / p.Tq) + gh) * p.q_sh +
         t * p.q_st;
}

// Grid: B * Hkv * n_blocks.  A warp takes score_warp_pages(D) pages, all of
// whose bounds are on their way at once; a lane holds 8 channels of lo or hi
// of one page per load, and of up to four query rows.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const SelectParams p) {
  constexpr int LP = D / 4;                 // lanes per page
  constexpr int PW = score_warp_pages(D);
  constexpr int NV = kScoreLoads * kScoreRows / LP;  // sums that a lane ends up with
  constexpr int KEPT = NV > 0 ? NV : 1;
  static_assert(kScoreLoads * kScoreRows == 32, "one sum per lane at D = 128");
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = static_cast<int>(blockIdx.x) / p.n_blocks;
  const int blk = static_cast<int>(blockIdx.x) - bh * p.n_blocks;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int count = select_count(p, b);
  if (count <= p.n_sel) return;  // every page is taken
  const int first = blk * score_pages(D) + warp * PW;
  if (blk * score_pages(D) >= count) return;
  const int lp = lane % LP;           // the lane's place in its page: lo first
  const bool low = lp < LP / 2;
  const int ch = (lp % (LP / 2)) * 8;
  // the warp's pages, one or more per lane; -1: not held
  uint4 v[kScoreLoads];
  float big = 0.f;
  constexpr int TL = (PW + 31) / 32;
  int pg[TL];
#pragma unroll
  for (int i = 0; i < TL; ++i) {
    const int at = first + 32 * i + lane;
    pg[i] = 32 * i + lane < PW && at < count ? p.table[b * p.table_sb + at] : -1;
    if (pg[i] >= p.n_pages) pg[i] = -1;
  }
#pragma unroll
  for (int j = 0; j < kScoreLoads; ++j) {
    constexpr int PPL = 32 / LP;      // pages per load
    const int i = j * PPL;            // compile-time register, lane within it
    const int page = dec_shfl(pg[i / 32], i % 32 + lane / LP);
    v[j] = page < 0 ? uint4{0, 0, 0, 0}
                    : *reinterpret_cast<const uint4*>(
                          p.bounds + ((static_cast<long long>(page) * p.Hkv + h) * 2 + !low) * D +
                          ch);
  }
#pragma unroll
  for (int j = 0; j < kScoreLoads; ++j) {
    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
    for (int c = 0; c < 4; ++c)
      big = fmaxf(big, fmaxf(fabsf(dec_bf16_lo(w[c])), fabsf(dec_bf16_hi(w[c]))));
  }
  float best[KEPT];
#pragma unroll
  for (int i = 0; i < KEPT; ++i) best[i] = -INFINITY;
  for (int r0 = 0; r0 < p.rows; r0 += kScoreRows) {
    float s[kScoreLoads * kScoreRows];
    // four rows in turn (past the last: the last again)
#pragma unroll
    for (int r = 0; r < kScoreRows; ++r) {
      const uint4 qw = *reinterpret_cast<const uint4*>(
          select_row(p, b, h, r0 + r < p.rows ? r0 + r : p.rows - 1) + ch);
      const uint32_t w[4] = {qw.x, qw.y, qw.z, qw.w};
      float y[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float x = (c & 1) ? dec_bf16_hi(w[c / 2]) : dec_bf16_lo(w[c / 2]);
        y[c] = low ? (x > 0.f ? 0.f : x) : (x < 0.f ? 0.f : x);  // (a NaN stays)
      }
#pragma unroll
      for (int j = 0; j < kScoreLoads; ++j) {
        const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
        float a = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          a = fmaf(y[2 * c], dec_bf16_lo(u[c]), a);
          a = fmaf(y[2 * c + 1], dec_bf16_hi(u[c]), a);
        }
        s[j * kScoreRows + r] = a;
      }
    }
    // sums over the LP lanes of a page: at each step a lane hands half of its
    // values to its partner and takes the other half's, so that lane lp ends
    // with values lp NV .. lp NV + NV - 1
#pragma unroll
    for (int d = LP / 2, n = kScoreLoads * kScoreRows / 2; d > 0; d /= 2, n /= 2) {
      const bool upper = (lane & d) != 0;
#pragma unroll
      for (int i = 0; i < kScoreLoads * kScoreRows / 2; ++i)
        if (i < n) {
          const float keep = upper ? s[i + n] : s[i], give = upper ? s[i] : s[i + n];
          s[i] = keep + __shfl_xor_sync(0xffffffffu, give, d);
        }
    }
    // a sum that is not finite is left to the exact pass: +inf marks it
#pragma unroll
    for (int i = 0; i < KEPT; ++i) best[i] = s[i] - s[i] == 0.f ? fmaxf(best[i], s[i]) : INFINITY;
  }
  // the highest of the four rows: values of one lane, or of 4 / NV lanes
  constexpr int RL = KEPT < kScoreRows ? KEPT : kScoreRows;
  float* out = p.score + static_cast<long long>(bh) * p.width;
#pragma unroll
  for (int i = 0; i < KEPT; i += RL) {
    float m = best[i];
#pragma unroll
    for (int r = 1; r < RL; ++r) m = fmaxf(m, best[i + r]);
#pragma unroll
    for (int d = 1; d < kScoreRows / RL; d *= 2)
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const int value = lp * KEPT + i;  // of the lane's page group
    const int at = (value / kScoreRows) * (32 / LP) + lane / LP;
    // whether the page is held: from the lane that looked it up
    int page = -1;
#pragma unroll
    for (int t = 0; t < TL; ++t) {
      const int x = dec_shfl(pg[t], at % 32);
      if (at / 32 == t) page = x;
    }
    if (value % kScoreRows == 0 && first + at < count) out[first + at] = page < 0 ? -INFINITY : m;
  }
#pragma unroll
  for (int d = 1; d < 32; d *= 2) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
  if (lane == 0)
    p.largest[(static_cast<long long>(bh) * p.n_blocks + blk) * kScoreWarps + warp] = big;
}

// Whole numbers in the order of the scores (both zeros alike).
__device__ __forceinline__ unsigned score_key(float s) {
  const unsigned u = dec_float_bits(s + 0.f);
  return (u >> 31) ? ~u : u | (1u << 31);
}
__device__ __forceinline__ unsigned long long score_key(double s) {
  const unsigned long long u = static_cast<unsigned long long>(dec_double_bits(s + 0.0));
  return (u >> 63) ? ~u : u | (1ull << 63);
}

// Sums of the N values v over the CTA's threads; `sh` has two halves of three
// words per warp, used in turn, so that one barrier is enough.
template <int N>
__device__ __forceinline__ void pick_sums(int (&v)[N], int* sh, int& turn) {
  constexpr int NW = kPickThreads / 32;
  static_assert(N <= 3 && NW <= 32, "sums");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* half = sh + turn * 3 * NW;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = dec_warp_sum(v[i]);
    if (lane == 0) half[i * NW + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dec_warp_sum(lane < NW ? half[i * NW + lane] : 0);
  turn ^= 1;
}
// The highest digit 0 .. 3 that at least `want` keys reach; n: how many reach
// 1, 2 and 3.
__device__ __forceinline__ unsigned pick_digit(const int (&n)[3], int want) {
  return n[2] >= want ? 3u : n[1] >= want ? 2u : n[0] >= want ? 1u : 0u;
}

// Exact score of page i (a warp): the largest row's, in 64 bits; a NaN as +inf.
__device__ __forceinline__ double exact_score(const SelectParams& p, int b, int h, int i) {
  const int lane = threadIdx.x & 31;
  const int page = p.table[b * p.table_sb + i];
  double best = -INFINITY;
  if (page < 0 || page >= p.n_pages) return best;
  const __nv_bfloat16* lo = p.bounds + (static_cast<long long>(page) * p.Hkv + h) * 2 * p.D;
  for (int r = 0; r < p.rows; ++r) {
    const __nv_bfloat16* q = select_row(p, b, h, r);
    double s = 0.0;
    for (int d = lane; d < p.D; d += 32) {
      const float x = __bfloat162float(q[d]);
      const float up = x < 0.f ? 0.f : x, down = x > 0.f ? 0.f : x;
      s += static_cast<double>(up) * static_cast<double>(__bfloat162float(lo[p.D + d]));
      s += static_cast<double>(down) * static_cast<double>(__bfloat162float(lo[d]));
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) s += dec_shfl(s, lane ^ d);
    if (s != s) s = INFINITY;
    best = s > best ? s : best;
  }
  return best;
}

// Grid: B * Hkv CTAs of kPickThreads.
__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelectParams p) {
  constexpr int NW = kPickThreads / 32;
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  unsigned* keys = reinterpret_cast<unsigned*>(dec_dynamic_smem());  // [kPickKeys]
  int* sh = reinterpret_cast<int*>(keys + kPickKeys);                // [2][3][NW]
  float* shf = reinterpret_cast<float*>(sh + 6 * NW);                // [2][NW]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = static_cast<int>(blockIdx.x), b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int count = select_count(p, b);
  int* out = p.pages + static_cast<long long>(bh) * p.n_sel;
  if (count <= p.n_sel) {
    for (int i = tid; i < p.n_sel; i += kPickThreads) out[i] = i < count ? i : -1;
    return;
  }
  const float* score = p.score + static_cast<long long>(bh) * p.width;
  double* exact = p.exact + static_cast<long long>(bh) * p.width;
  const int lo = p.n_first, hi = count - p.n_last;  // candidates: lo <= i < hi
  int want = p.n_sel - p.n_first - p.n_last, turn = 0;

  // rho: the largest |bound| and the largest sum |q| of a row
  float big = 0.f, qsum = 0.f;
  const int n_big = (count + score_pages(p.D) - 1) / score_pages(p.D) * kScoreWarps;
  for (int i = tid; i < n_big; i += kPickThreads)
    big = fmaxf(big, p.largest[static_cast<long long>(bh) * p.n_blocks * kScoreWarps + i]);
  for (int r = warp; r < p.rows; r += NW) {
    const __nv_bfloat16* q = select_row(p, b, h, r);
    float a = 0.f;
    for (int d = lane; d < p.D; d += 32) a += fabsf(__bfloat162float(q[d]));
#pragma unroll
    for (int d = 1; d < 32; d *= 2) a += __shfl_xor_sync(0xffffffffu, a, d);
    qsum = fmaxf(qsum, a);
  }
#pragma unroll
  for (int d = 1; d < 32; d *= 2) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
  if (lane == 0) {
    shf[warp] = big;
    shf[NW + warp] = qsum;
  }
  int odd[1] = {0};  // scores that are not finite, of pages that are held
  for (int i = tid; i < count; i += kPickThreads) {
    const float s = score[i];
    odd[0] += s == INFINITY;
    if (i < kPickKeys) keys[i] = score_key(s);
  }
  pick_sums(odd, sh, turn);  // (a barrier: keys and shf are written)
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    big = fmaxf(big, shf[w]);
    qsum = fmaxf(qsum, shf[NW + w]);
  }
  // 1 percent for the sum's and the product's own roundings; a little for
  // products below the smallest normal number
  const float rho = odd[0] ? INFINITY : 14.14f * 0x1p-24f * (big * qsum) + 1e-42f;
  auto key = [&](int i) { return i < kPickKeys ? keys[i] : score_key(score[i]); };

  // T, the want-th highest score: two bits a round, each the highest digit
  // that at least `want` scores reach
  unsigned T = 0;
  if (want > 0) {
    for (int shift = 30; shift >= 0; shift -= 2) {
      int n[3] = {0, 0, 0};
      for (int i = lo + tid; i < hi; i += kPickThreads) {
        const unsigned k = key(i);
#pragma unroll
        for (int d = 0; d < 3; ++d) n[d] += k >= (T | ((d + 1u) << shift));
      }
      pick_sums(n, sh, turn);
      T |= pick_digit(n, want) << shift;
    }
  }
  const float t = dec_bits_float((T >> 31) ? T & 0x7fffffffu : ~T);
  // sure: above whatever the want-th highest exact score may be; near: may
  // be either (the comparisons with infinities and NaN fall to `near`)
  auto value = [&](int i) {
    const unsigned k = key(i);
    return dec_bits_float((k >> 31) ? k & 0x7fffffffu : ~k);
  };
  const bool none = want == 0;
  auto sure = [&](float s) { return !none && s - rho > t + rho; };
  auto near = [&](float s) { return !none && !(s - rho > t + rho) && !(s + rho < t - rho); };
  int n_of[2] = {0, 0};  // sure, near
  for (int i = lo + tid; i < hi; i += kPickThreads) {
    const float s = value(i);
    n_of[0] += sure(s);
    n_of[1] += near(s);
  }
  pick_sums(n_of, sh, turn);
  want -= n_of[0];
  const bool all_near = n_of[1] <= want;
  unsigned long long E = 0;  // the want-th highest exact score of those near T
  if (!all_near) {
    for (int base = lo; base < hi; base += kPickThreads) {
      const int i = base + warp * 32 + lane;
      unsigned todo = dec_ballot(i < hi && near(value(i < hi ? i : lo)));
      while (todo != 0u) {
        const int at = base + warp * 32 + dec_lowest(todo);
        todo &= todo - 1u;
        const double s = exact_score(p, b, h, at);
        if (lane == 0) exact[at] = s;
      }
    }
    __syncthreads();
    for (int shift = 62; shift >= 0; shift -= 2) {
      int n[3] = {0, 0, 0};
      for (int i = lo + tid; i < hi; i += kPickThreads) {
        if (!near(value(i))) continue;
        const unsigned long long k = score_key(exact[i]);
#pragma unroll
        for (int d = 0; d < 3; ++d) n[d] += k >= (E | ((d + 1ull) << shift));
      }
      pick_sums(n, sh, turn);
      E |= static_cast<unsigned long long>(pick_digit(n, want)) << shift;
    }
    int above[1] = {0};
    for (int i = lo + tid; i < hi; i += kPickThreads)
      above[0] += near(value(i)) && score_key(exact[i]) > E;
    pick_sums(above, sh, turn);
    want -= above[0];  // places for those that equal E
  }

  // listed in order: those chosen, and the first `want` of those equal to E
  int listed = 0, equal = 0;
  for (int base = 0; base < count; base += kPickThreads) {
    const int i = base + tid;
    bool take = i < count && (i < lo || i >= hi), same = false;
    if (i >= lo && i < hi) {
      const float s = value(i);
      take = sure(s);
      if (near(s)) {
        if (all_near) {
          take = true;
        } else {
          const unsigned long long k = score_key(exact[i]);
          take = k > E;
          same = k == E;
        }
      }
    }
    const unsigned below = (1u << lane) - 1u;
    if (!all_near) {
      const unsigned m = dec_ballot(same);
      __syncthreads();
      if (lane == 0) sh[warp] = dec_popc(m);
      __syncthreads();
      int eq = equal + dec_popc(m & below);
      for (int w = 0; w < NW; ++w) {
        if (w < warp) eq += sh[w];
        equal += sh[w];
      }
      take = take || (same && eq < want);
    }
    const unsigned m = dec_ballot(take);
    __syncthreads();
    if (lane == 0) sh[NW + warp] = dec_popc(m);
    __syncthreads();
    int at = listed + dec_popc(m & below);
    for (int w = 0; w < NW; ++w) {
      if (w < warp) at += sh[NW + w];
      listed += sh[NW + w];
    }
    if (take && at < p.n_sel) out[at] = i;
  }
}

__host__ __device__ constexpr int pick_smem_bytes() {
  return kPickKeys * 4 + 8 * (kPickThreads / 32) * 4;
}
// Workspace: the exact scores, the fp32 scores, the largest bounds.
__host__ __device__ constexpr long long select_workspace_bytes(long long bh, int width) {
  const long long blocks = (width + score_pages(128) - 1) / score_pages(128);
  return bh * (width * 12LL + blocks * kScoreWarps * 4);
}

}  // namespace cattn
