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
// The scores are exact to 64 bits, so that the choice does not depend on an
// order of summation (a product of two bf16 values has 16 bits, so a sum of
// 2 D of them is exact unless they span more than 2^29).

struct SelectParams {
  const __nv_bfloat16* q;       // (B, H, Tq, D)
  long long q_sb, q_sh, q_st;
  const __nv_bfloat16* bounds;  // (n_pages, Hkv, 2, D)
  const int* table;
  long long table_sb;
  const int* lengths;
  int B, H, Hkv, Tq, rows, n_pages, P, width, n_sel, n_first, n_last;
  int n_blocks;                 // ceil(width / kScorePages)
  int* pages;                   // (B, Hkv, n_sel)
  double* score;                // [B][Hkv][width]
};

constexpr int kScoreThreads = 128;
constexpr int kScorePages = 32;    // pages per CTA
constexpr int kPickThreads = 256;

__device__ __forceinline__ int select_count(const SelectParams& p, int b) {
  const int len = p.lengths[b];
  const int n = len > 0 ? pages_of(len, p.P) : 0;
  return n < p.width ? n : p.width;
}

// Grid: B * Hkv * n_blocks.  Warp: a page at a time.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const SelectParams p) {
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = static_cast<int>(blockIdx.x) / p.n_blocks;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int count = select_count(p, b);
  if (count <= p.n_sel) return;  // every page is taken
  const int first = (static_cast<int>(blockIdx.x) - bh * p.n_blocks) * kScorePages;
  constexpr int CPL = D / 16;    // channels per lane and bound, 16 lanes
  for (int i = first + warp; i < first + kScorePages && i < count; i += kScoreThreads / 32) {
    const int page = p.table[b * p.table_sb + i];
    double best = -INFINITY;
    if (page >= 0 && page < p.n_pages) {
      // lanes 0-15 take hi, 16-31 lo
      const bool low = lane >= 16;
      const __nv_bfloat16* src =
          p.bounds + ((static_cast<long long>(page) * p.Hkv + h) * 2 + (low ? 0 : 1)) * D +
          (lane & 15) * CPL;
      float v[CPL];
#pragma unroll
      for (int c = 0; c < CPL; ++c) v[c] = __bfloat162float(src[c]);
      for (int r = 0; r < p.rows; ++r) {
        const int gh = r / p.Tq, t = r - gh * p.Tq;
        const __nv_bfloat16* qr = p.q + b * p.q_sb +
                                  (static_cast<long long>(h) * (p.rows / p.Tq) + gh) * p.q_sh +
                                  t * p.q_st + (lane & 15) * CPL;
        double s = 0.0;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          const float x = __bfloat162float(qr[c]);
          const float y = low ? (x > 0.f ? 0.f : x) : (x < 0.f ? 0.f : x);  // (NaN stays)
          s += static_cast<double>(y) * static_cast<double>(v[c]);
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) s += dec_shfl(s, lane ^ d);
        if (s != s) s = INFINITY;
        best = s > best ? s : best;
      }
    }
    if (lane == 0) p.score[static_cast<long long>(bh) * p.width + i] = best;
  }
}

// Whole numbers in the order of the scores (both zeros alike).
__device__ __forceinline__ unsigned long long score_key(double s) {
  const unsigned long long u = static_cast<unsigned long long>(dec_double_bits(s + 0.0));
  return (u >> 63) ? ~u : u | (1ull << 63);
}

// Grid: B * Hkv CTAs.  Radix select, eight bits at a time.
__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelectParams p) {
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  int* sh = reinterpret_cast<int*>(dec_dynamic_smem());
  int* hist = sh;             // [256]
  int* found = sh + 256;      // digit, how many are still wanted
  int* sums = sh + 258;       // [2][warps]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = static_cast<int>(blockIdx.x) / p.Hkv;
  const int count = select_count(p, b);
  int* out = p.pages + static_cast<long long>(blockIdx.x) * p.n_sel;
  if (count <= p.n_sel) {
    for (int i = tid; i < p.n_sel; i += kPickThreads) out[i] = i < count ? i : -1;
    return;
  }
  const double* score = p.score + static_cast<long long>(blockIdx.x) * p.width;
  const int lo = p.n_first, hi = count - p.n_last;  // candidates: lo <= i < hi
  int want = p.n_sel - p.n_first - p.n_last;
  unsigned long long prefix = 0;  // the digits of the want-th highest key so far
  for (int shift = 56; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kPickThreads) {
      const unsigned long long k = score_key(score[i]);
      if (shift == 56 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        dec_add_shared(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int digit = 255, above = 0;
      while (digit > 0 && above + hist[digit] < want) above += hist[digit--];
      found[0] = digit;
      found[1] = want - above;
    }
    __syncthreads();
    prefix |= static_cast<unsigned long long>(found[0]) << shift;
    want = found[1];
    __syncthreads();
  }
  // listed in order: above the key, and the first `want` of those equal to it
  int listed = 0, equal = 0;
  const bool none = p.n_sel == p.n_first + p.n_last;
  for (int base = 0; base < count; base += kPickThreads) {
    const int i = base + tid;
    bool take = i < count && (i < lo || i >= hi), same = false;
    if (!none && i >= lo && i < hi) {
      const unsigned long long k = score_key(score[i]);
      take = k > prefix;
      same = k == prefix;
    }
    const unsigned below = (1u << lane) - 1u;
    const unsigned mt = dec_ballot(same);
    if (lane == 0) sums[warp] = dec_popc(mt);
    __syncthreads();
    int eq = equal + dec_popc(mt & below);
    for (int w = 0; w < kPickThreads / 32; ++w) {
      if (w < warp) eq += sums[w];
      equal += sums[w];
    }
    take = take || (same && eq < want);
    const unsigned ml = dec_ballot(take);
    if (lane == 0) sums[kPickThreads / 32 + warp] = dec_popc(ml);
    __syncthreads();
    int at = listed + dec_popc(ml & below);
    for (int w = 0; w < kPickThreads / 32; ++w) {
      if (w < warp) at += sums[kPickThreads / 32 + w];
      listed += sums[kPickThreads / 32 + w];
    }
    if (take && at < p.n_sel) out[at] = i;
  }
}

__host__ __device__ constexpr int pick_smem_bytes() {
  return (258 + 2 * (kPickThreads / 32)) * 4;
}

}  // namespace cattn
