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
// table[b][pos / P] P + pos % P, and the held pages of the requests that end go
// to ring[tail ..] in order: at sum have + j where all are held.  A call that
// cannot be served as a whole changes nothing but its status.
//
// A few kilobytes of whole numbers: bound by latency.  One thread-block
// cluster: every CTA scans all requests for itself (into shared
// memory), the cluster's barrier separates the last read of the inputs from
// the first write of the outputs (which may be the same arrays), and then the
// CTAs share the tokens and pages.

constexpr int kPlanThreads = 1024;    // at most; 256 for short calls
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
  PageDivider by_P;
};

__host__ __device__ constexpr int plan_smem_bytes(int B) {
  return 16 * (B + 1) + kPlanThreads / 32 * 32 + 16;  // prefix sums, warp totals, faults
}

__device__ __forceinline__ int pages_of(int n, int P) { return n / P + (n % P != 0); }

// Last index b in [lo, hi) with cu[b] <= i (cu ascending, cu[lo] <= i).
__device__ __forceinline__ int last_at_most(const int* cu, int lo, int hi, int i) {
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

// Many tokens (prompts) get a second launch over the whole GPU: the eight SMs of
// a cluster store no more than 0.3 TB/s (145,000 slots: 20.7 us in one launch).
__host__ __device__ constexpr bool plan_prompts(long long n_slots) {
  return n_slots > 2 * kPlanMaxCtas * kPlanThreads;
}
// CTAs of the cluster and their threads: short calls on one small CTA (64
// requests, one token each: 3.1 us); else what the slots, or the pages that
// change hands, can occupy.
__host__ __device__ constexpr int plan_threads(long long n_slots, int B) {
  return n_slots <= 512 && B <= 256 ? 256 : kPlanThreads;
}
__host__ __device__ constexpr int plan_ctas(long long n_slots, int B) {
  const long long pages = n_slots / 16 + 2LL * B, work = plan_prompts(n_slots) ? 0 : n_slots;
  const long long n = ((work > pages ? work : pages) + kPlanThreads - 1) / kPlanThreads;
  return n < 1 ? 1 : n > kPlanMaxCtas ? kPlanMaxCtas : static_cast<int>(n);
}

// Grid: one cluster of n_ctas CTAs.  SLOTS: with the tokens' slots and positions
// (else paged_slots_kernel writes them).
template <bool SLOTS>
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanParams p, int n_ctas) {
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  uint8_t* smem = dec_dynamic_smem();
  long long* sums = reinterpret_cast<long long*>(smem);  // [warps][4]
  int* bad = reinterpret_cast<int*>(sums + kPlanThreads / 32 * 4);
  int* len_s = bad + 4;                                   // [B + 1] each
  int* cu_tok = len_s + p.B + 1;
  int* cu_need = cu_tok + p.B + 1;
  int* cu_back = cu_need + p.B + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nt = static_cast<int>(blockDim.x), nw = nt / 32;
  const unsigned rank = n_ctas > 1 ? dec_cluster_rank() : 0u;
  if (tid < 4) bad[tid] = 0;
  __syncthreads();

  // this thread's requests: b0 .. b1 - 1
  const int nb = (p.B + nt - 1) / nt;
  const int b0 = tid * nb < p.B ? tid * nb : p.B, b1 = b0 + nb < p.B ? b0 + nb : p.B;
  const int cap = p.width * p.P;
  auto pages = [&](int n) {  // n <= 2^30
    const int q = p.by_P(n);
    return q + (n != q * p.P);
  };
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
        need += pages(len + n) - pages(len);
      }
    } else if (n < 0) {
      if (len > cap) fault |= 1; else back += pages(len);
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
  // the warps' totals, scanned by every warp
  long long of[3], all[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const long long v = warp_scan64(lane < nw ? sums[lane * 4 + i] : 0, lane);
    all[i] = dec_shfl(v, 31);
    of[i] = dec_shfl(v, warp > 0 ? warp - 1 : 0);
    if (warp == 0) of[i] = 0;
  }
  long long et = of[0] + it - tok, en = of[1] + in - need, eb = of[2] + ib - back;
  long long T = all[0], N = all[1], R = all[2];
  const long long head = p.state[0], tail = p.state[1], avail = tail - head;
  int status = 0;
  if (T > p.n_slots || N > avail) status = kPlanStatusTooLarge;
  if (bad[2]) status = kPlanStatusTooLarge;
  if (bad[1] || head < 0 || avail < 0 || avail > p.n_pages || R > 0x7fffffffLL)
    status = kPlanStatusInvalid;
  for (int b = b0; b < b1; ++b) {
    const int len = p.lengths[b], n = p.asked[b];
    len_s[b] = status || n >= 0 ? len : ~len;  // below 0: the request ends
    cu_tok[b] = status ? 0 : static_cast<int>(et);
    cu_need[b] = status ? 0 : static_cast<int>(en);
    cu_back[b] = status ? 0 : static_cast<int>(eb);
    if (!status && n > 0) {
      et += n;
      en += pages(len + n) - pages(len);
    }
    if (!status && n < 0) eb += pages(len);
  }
  if (status) T = N = R = 0;
  if (tid == 0) {
    cu_tok[p.B] = static_cast<int>(T);
    cu_need[p.B] = static_cast<int>(N);
    cu_back[p.B] = static_cast<int>(R);
  }
  __syncthreads();
  // Entry j of the rows of the requests that end.
  auto ended = [&](long long j) {
    const int b = last_at_most(cu_back, 0, p.B, static_cast<int>(j));
    return p.table[b * p.table_sb + (j - cu_back[b])];
  };
  auto held = [&](int page) { return page >= 0 && page < p.n_pages; };
  // Where some are not held: f(rank, page, tile) for each held one, a tile of nt
  // entries at a time (every CTA walks all of them); returns their number.
  auto each_held = [&](auto f) {
    long long rank_in = 0;
    for (long long base = 0, tile = 0; base < R; base += nt, ++tile) {
      const int page = base + tid < R ? ended(base + tid) : -1;
      const unsigned m = dec_ballot(held(page));
      __syncthreads();  // the tile before is done with the counts
      if (lane == 0) sums[warp * 4] = dec_popc(m);
      __syncthreads();
      long long at = rank_in + dec_popc(m & ((1u << lane) - 1u));
      for (int w = 0; w < nw; ++w) {
        if (w < warp) at += sums[w * 4];
        rank_in += sums[w * 4];
      }
      if (held(page)) f(at, page, tile);
    }
    return rank_in;
  };
  constexpr int ILP = 4;  // entries in flight per thread
  const int start = static_cast<int>(rank) * nt + tid, step = n_ctas * nt;
  // whether there are any: each CTA looks at its share, of which the first
  // entries stay in registers
  const bool ending = R > 0;  // (alike in every CTA)
  int first[ILP];
  for (long long j0 = start; j0 < R; j0 += ILP * step) {
    int entry[ILP];
#pragma unroll
    for (int u = 0; u < ILP; ++u) entry[u] = j0 + u * step < R ? ended(j0 + u * step) : 0;
#pragma unroll
    for (int u = 0; u < ILP; ++u) {
      if (!held(entry[u])) bad[3] = 1;
      if (j0 == start) first[u] = entry[u];
    }
  }
  if (n_ctas > 1)
    dec_cluster_sync();  // every CTA has read its inputs
  else
    __syncthreads();
  bool holes = false;
  if (ending) {
    const float* flag = reinterpret_cast<const float*>(bad + 3);
    holes = n_ctas > 1
                ? dec_ballot(lane < n_ctas && dec_float_bits(dec_cluster_ld(flag, lane)) != 0u) != 0u
                : bad[3] != 0;
    const long long n_held = holes ? each_held([](long long, int, long long) {}) : R;
    if (n_held > p.n_pages - avail) {  // (every thread of every CTA finds the same)
      status = kPlanStatusInvalid;
      __syncthreads();
      for (int b = b0; b < b1; ++b) {
        if (len_s[b] < 0) len_s[b] = ~len_s[b];
        cu_tok[b] = cu_need[b] = cu_back[b] = 0;
      }
      T = N = R = 0;
      if (tid == 0) cu_tok[p.B] = cu_need[p.B] = cu_back[p.B] = 0;
      holes = false;
      __syncthreads();
    }
  }

  const int head0 = static_cast<int>(head % p.n_pages >= 0 ? head % p.n_pages : 0);
  const int tail0 = static_cast<int>(tail % p.n_pages >= 0 ? tail % p.n_pages : 0);
  auto at = [&](int base, int k) {  // ring entry of counter base + k, k < n_pages
    const long long i = static_cast<long long>(base) + k;
    return static_cast<int>(i >= p.n_pages ? i - p.n_pages : i);
  };
  // a token per thread: its request by a search, its page from the row or, if
  // it is new, from the ring
  for (long long i = start; SLOTS && i < p.n_slots; i += step) {
    long long slot = -1;
    int pos = -1;
    if (i < T) {
      const int b = last_at_most(cu_tok, 0, p.B, static_cast<int>(i));
      const int have = pages(len_s[b]);
      pos = len_s[b] + (static_cast<int>(i) - cu_tok[b]);
      const int lp = p.by_P(pos);
      const int page = lp < have ? p.table[b * p.table_sb + lp]
                                 : p.ring[at(head0, cu_need[b] + lp - have)];
      if (page >= 0 && page < p.n_pages)
        slot = static_cast<long long>(page) * p.P + (pos - lp * p.P);
    }
    p.slots[i] = slot;
    p.positions[i] = pos;
  }
  // new pages into the table, freed ones into the ring, four at a time
  for (long long j0 = start; j0 < N; j0 += ILP * step) {
    int entry[ILP];
#pragma unroll
    for (int u = 0; u < ILP; ++u) {
      const long long j = j0 + u * step;
      entry[u] = j < N ? p.ring[at(head0, static_cast<int>(j))] : -1;
    }
#pragma unroll
    for (int u = 0; u < ILP; ++u) {
      const long long j = j0 + u * step;
      if (j >= N) continue;
      const int b = last_at_most(cu_need, 0, p.B, static_cast<int>(j));
      p.table[b * p.table_sb + pages(len_s[b]) + (j - cu_need[b])] = entry[u];
    }
  }
  if (holes) {
    R = each_held([&](long long j, int page, long long tile) {
      if (tile % n_ctas == rank) p.ring[at(tail0, static_cast<int>(j))] = page;
    });
  } else {
    for (long long j0 = start; j0 < R; j0 += ILP * step) {
#pragma unroll
      for (int u = 0; u < ILP; ++u) {
        const long long j = j0 + u * step;
        if (j < R) p.ring[at(tail0, static_cast<int>(j))] = j0 == start ? first[u] : ended(j);
      }
    }
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
  if (n_ctas > 1 && ending) dec_cluster_sync();  // no CTA leaves while its flag is read
}

// Slots and positions of a planned step's tokens, from what the plan wrote:
// offsets, new lengths and tables.  A warp takes 32 V neighbours, a lane every
// 32nd of them (so that stores coalesce): a search where a lane enters another
// request.  Grid: ceil(n_slots / (V kSlotsThreads)).
constexpr int kSlotsThreads = 256;
constexpr int kSlotsV = 4;
__global__ void __launch_bounds__(kSlotsThreads) paged_slots_kernel(const PlanParams p) {
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long i0 =
      32LL * kSlotsV * (static_cast<long long>(blockIdx.x) * (kSlotsThreads / 32) + warp);
  const int T = p.cu[p.B];
  int page[kSlotsV], pos[kSlotsV], row[kSlotsV];
  int b = 0, end = 0, shift = 0;
#pragma unroll
  for (int u = 0; u < kSlotsV; ++u) {
    page[u] = pos[u] = -1;
    row[u] = 0;
    const long long i = i0 + 32 * u + lane;
    if (i >= T) continue;
    if (u == 0 || i >= end) {
      b = last_at_most(p.cu, b, p.B, static_cast<int>(i));
      end = p.cu[b + 1];
      shift = p.lengths_out[b] - end;  // length before the step - cu[b]
    }
    pos[u] = static_cast<int>(i) + shift;
    const int lp = p.by_P(pos[u]);
    row[u] = pos[u] - lp * p.P;
    page[u] = p.table[b * p.table_sb + lp];
  }
#pragma unroll
  for (int u = 0; u < kSlotsV; ++u) {
    const long long i = i0 + 32 * u + lane;
    if (i >= p.n_slots) continue;
    p.slots[i] = page[u] >= 0 && page[u] < p.n_pages
                     ? static_cast<long long>(page[u]) * p.P + row[u]
                     : -1;
    p.positions[i] = pos[u];
  }
}

// ------------------------------------------------------------------ append
//
// Row i of the new K and V goes to cache row slots[i] (page slots[i] / P, row
// slots[i] % P); a slot outside the cache is skipped.  With bounds, the lowest
// and highest value of each channel of a page's keys are kept beside it:
//   lo_d = min over the page's keys of k_d,  hi_d = max
// A run of neighbouring rows of one page is done by one thread per 8 channels,
// row after row, so nothing is updated twice; the page's first row starts its
// bounds over.  (NaN in, NaN out.)
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
  long long n_rows;         // n_pages P, at most 2^32
  // slot / P as the high word of (2 slot) mul, mul = floor(2^63 / P) + 1: that
  // exceeds slot / P by at most slot / 2^63 < 1 / P (P <= 2^30), too little to
  // reach the next whole number.  (A 64-bit division takes as long as a load; the
  // form without bounds keeps one, by Hkv, where it hardly shows.)
  unsigned long long mul;
  __device__ __forceinline__ long long page(long long slot) const {
    return static_cast<long long>(dec_mulhi(2 * static_cast<unsigned long long>(slot), mul));
  }
};
inline unsigned long long append_mul(int P) { return (1ull << 63) / static_cast<unsigned>(P) + 1; }

constexpr int kAppendThreads = 256;
constexpr int kBoundsThreads = 128;   // of the form with bounds
constexpr int kAppendILP = 8;         // rows of a run in flight per thread
constexpr int kAppendMaxTile = 32;    // tokens per CTA, a lane each

// Tokens per CTA of the form with bounds: about 512 CTAs.
__host__ __device__ constexpr int append_tile(long long n) {
  return n < 1024 ? 1 : n / 512 > kAppendMaxTile ? kAppendMaxTile : static_cast<int>(n / 512);
}

// Without bounds.  Thread: 8 channels of one (row, head).  (16,392 tokens x 8
// heads x 128 from a fused projection: 22.5 us, 0.92 of the copy bandwidth.)
template <int D>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendParams p) {
  constexpr int PC = D / 8;
  dec_grid_dep_wait();
  const long long x = static_cast<long long>(blockIdx.x) * kAppendThreads + threadIdx.x;
  const int pc = static_cast<int>(x % PC);
  const long long unit = x / PC;
  const long long i = unit / p.Hkv;
  const int h = static_cast<int>(unit - i * p.Hkv);
  if (i >= p.n) return;
  const long long slot = p.slots[i];
  if (slot < 0 || slot >= p.n_rows) return;
  const long long page = p.page(slot), off = slot - page * p.P;
  const uint4 k =
      *reinterpret_cast<const uint4*>(p.kn + i * p.kn_st + h * p.kn_sh + pc * 8);
  const uint4 v =
      *reinterpret_cast<const uint4*>(p.vn + i * p.vn_st + h * p.vn_sh + pc * 8);
  *reinterpret_cast<uint4*>(p.k + page * p.k_sp + h * p.k_sh + off * p.k_st + pc * 8) = k;
  *reinterpret_cast<uint4*>(p.v + page * p.v_sp + h * p.v_sh + off * p.v_st + pc * 8) = v;
}

// With bounds.  Grid: two CTAs, one for K and one for V, per `tile` tokens; a
// CTA takes the runs that begin among these, to their ends.  Unit: 8 channels
// of one head of a run; its thread reads kAppendILP rows at a time.
template <int D>
__global__ void __launch_bounds__(kBoundsThreads)
    cache_append_bounds_kernel(const AppendParams p, int tile) {
  constexpr int PC = D / 8;
  dec_grid_dep_wait();
  uint8_t* smem = dec_dynamic_smem();
  long long* run_slot = reinterpret_cast<long long*>(smem);            // [32]
  int* run_at = reinterpret_cast<int*>(run_slot + kAppendMaxTile);     // [32]
  int* run_len = run_at + kAppendMaxTile;                              // [32]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool keys = (blockIdx.x & 1) == 0;
  const long long i0 = static_cast<long long>(blockIdx.x >> 1) * tile;
  auto valid = [&](long long slot) { return slot >= 0 && slot < p.n_rows; };
  // token j goes on with the run of token j - 1: it is in the same page, in the
  // next row (1) or another one (2)
  auto goes_on = [&](long long j) {
    if (j <= 0 || j >= p.n) return 0;
    const long long slot = p.slots[j], before = p.slots[j - 1];
    if (!valid(slot) || !valid(before)) return 0;
    return p.page(slot) != p.page(before) ? 0 : slot == before + 1 ? 1 : 2;
  };
  const bool in = lane < tile && i0 + lane < p.n;
  const long long slot = in ? p.slots[i0 + lane] : -1;
  const int on = in ? goes_on(i0 + lane) : 0;
  const unsigned stops = ~dec_ballot(on != 0);                // no run goes on there
  const unsigned jumps = dec_ballot(on == 2);                 // or not in the next row
  const unsigned leads = dec_ballot(valid(slot) && on == 0);
  const int n_runs = dec_popc(leads);
  if (n_runs == 0) return;
  if (warp == 0) {
    // a run ends before the next stop of the tile, or is followed beyond it
    const unsigned inside = tile < 32 ? (1u << tile) - 1u : ~0u;
    const unsigned behind = lane < 31 ? stops & inside & (~0u << (lane + 1)) : 0u;
    int len = behind != 0u ? dec_lowest(behind) - lane : tile - lane;
    const bool open = ((leads >> lane) & 1u) != 0u && behind == 0u;
    const unsigned until = behind != 0u ? (1u << dec_lowest(behind)) - 1u : ~0u;
    bool jump = lane < 31 && (jumps & inside & until & (~0u << (lane + 1))) != 0u;
    if (dec_ballot(open) != 0u) {
      long long j = i0 + tile;
      for (;; j += 32) {
        const int further = goes_on(j + lane);
        const unsigned end = ~dec_ballot(further != 0), off = dec_ballot(further == 2);
        if (open && (end == 0u ? off : off & ((end & (0u - end)) - 1u)) != 0u) jump = true;
        if (end != 0u) {
          j += dec_lowest(end);
          break;
        }
      }
      if (open) len = static_cast<int>(j - (i0 + lane));
    }
    if ((leads >> lane) & 1u) {
      const int r = dec_popc(leads & ((1u << lane) - 1u));
      run_slot[r] = slot;
      run_at[r] = jump ? lane | 64 : lane;   // 64: the rows are not in order
      run_len[r] = len;
    }
  }
  __syncthreads();
  const int per_run = p.Hkv * PC;
  for (int u = tid; u < n_runs * per_run; u += kBoundsThreads) {
    const int r = u / per_run, hp = u - r * per_run, h = hp / PC, pc = hp - h * PC;
    const long long first = run_slot[r], page = p.page(first), i = i0 + (run_at[r] & 31);
    const int off = static_cast<int>(first - page * p.P);
    const bool jump = (run_at[r] & 64) != 0;
    const int n = run_len[r];
    const long long from_st = keys ? p.kn_st : p.vn_st, to_st = keys ? p.k_st : p.v_st;
    const __nv_bfloat16* from = keys ? p.kn + i * p.kn_st + h * p.kn_sh + pc * 8
                                     : p.vn + i * p.vn_st + h * p.vn_sh + pc * 8;
    __nv_bfloat16* to = keys ? p.k + page * p.k_sp + h * p.k_sh + pc * 8
                             : p.v + page * p.v_sp + h * p.v_sh + pc * 8;
    uint4* bl = reinterpret_cast<uint4*>(p.bounds + ((page * p.Hkv + h) * 2) * D + pc * 8);
    uint4 lo, hi;
    if (keys && off != 0) {  // the page goes on
      lo = *bl;
      hi = bl[D / 8];
    } else if (keys) {
      lo = hi = *reinterpret_cast<const uint4*>(from);
    }
    auto join = [&](const uint4& x) {
      lo.x = dec_bf16_min(lo.x, x.x);
      lo.y = dec_bf16_min(lo.y, x.y);
      lo.z = dec_bf16_min(lo.z, x.z);
      lo.w = dec_bf16_min(lo.w, x.w);
      hi.x = dec_bf16_max(hi.x, x.x);
      hi.y = dec_bf16_max(hi.y, x.y);
      hi.z = dec_bf16_max(hi.z, x.z);
      hi.w = dec_bf16_max(hi.w, x.w);
    };
    if (jump) {  // one after another
      for (int t = 0; t < n; ++t) {
        const uint4 x = *reinterpret_cast<const uint4*>(from + t * from_st);
        const long long row = p.slots[i + t] - page * p.P;
        *reinterpret_cast<uint4*>(to + row * to_st) = x;
        if (keys && row == 0) lo = hi = x;
        if (keys) join(x);
      }
    }
    to += off * to_st;
    for (int t = 0; t < n && !jump; t += kAppendILP) {
      uint4 x[kAppendILP];
#pragma unroll
      for (int j = 0; j < kAppendILP; ++j)  // (past the last: the last again)
        x[j] = *reinterpret_cast<const uint4*>(from + (t + j < n ? t + j : n - 1) * from_st);
#pragma unroll
      for (int j = 0; j < kAppendILP; ++j)
        if (t + j < n) *reinterpret_cast<uint4*>(to + (t + j) * to_st) = x[j];
      if (keys) {
#pragma unroll
        for (int j = 0; j < kAppendILP; ++j) join(x[j]);
      }
    }
    if (keys) {
      *bl = lo;
      bl[D / 8] = hi;
    }
  }
}

__host__ __device__ constexpr int append_smem_bytes() { return kAppendMaxTile * 16; }

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
// The choice is that of sums in 64 bits (exact, see below), so that it does not
// depend on an order of summation.  page_score_kernel sums on the tensor cores (the clipped query
// rows against the pages' bounds, 2 D terms a score): products of two bf16
// values are exact in fp32, and each of the 2 D / 16 steps rounds sums of at
// most S = sum of the terms' magnitudes.  Allowing a step 2^-20 S (the fp32
// rounding is 2^-24; how the hardware aligns its addends is not documented),
// at most 16 of them, and with V = the largest |bound| of the request's pages,
//   |s_i - exact| <= 2^-16 max_r sum_d |q_rd| V = rho.
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
  int groups;                   // groups of 8 pages that a warp takes
  int n_blocks;                 // CTAs per (request, head)
  int* pages;                   // (B, Hkv, n_sel)
  double* exact;                // [B Hkv][width]
  float* score;                 // [B Hkv][width]
  float* largest;               // [B Hkv][n_blocks][score warps]: |bounds|
};

constexpr int kScoreThreads = 128;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kScoreStages = 3;      // groups of 8 pages in flight per warp
constexpr int kPickThreads = 512;
constexpr int kSelectThreads = 256;  // of the fused kernel
constexpr int kSelectCtas = 8;       // its cluster
constexpr int kPickKeys = 8192;      // scores kept in shared memory
constexpr int kPickNear = 256;       // pages near the border that fit its list

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

// Clipped query values: below (low) or above zero, zero instead of the
// others; a NaN stays.
__device__ __forceinline__ uint32_t clip_pair(uint32_t w, bool low) {
  const float a = dec_bf16_lo(w), b = dec_bf16_hi(w);
  const bool drop_a = low ? a > 0.f : a < 0.f, drop_b = low ? b > 0.f : b < 0.f;
  return (drop_a ? 0u : w & 0xffffu) | (drop_b ? 0u : w & 0xffff0000u);
}

__host__ __device__ constexpr int score_ring_bytes(int D) { return kScoreStages * 32 * D; }

// Scores of groups of 8 pages (a warp): groups first, first + step, ... below
// `end`.  Their bounds stream through the warp's ring of kScoreStages slots of
// 32 D bytes with cp.async; lane (g, t4) reads bytes 16 t4 .. + 15 of each
// 64-byte segment of page g's [lo | hi], which are the B fragments of two
// k-steps (the channels of a segment enter the product in the order that this
// gives, on both sides).  The page numbers of four groups are looked up at a
// time, one per lane, ahead of their use.  UP: more than 8 query rows.
// Returns the largest |bound|, infinity where one is NaN.
template <int D, bool UP>
__device__ __forceinline__ float score_groups(const SelectParams& p, int b, int h, int count,
                                              int first, int end, int step, uint8_t* ring) {
  constexpr int SEG = D / 16;         // 64-byte segments of a page's bounds
  constexpr int PCS = D / 4;          // its 16-byte pieces
  constexpr int NR = UP ? 2 : 1;
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  float* out = p.score + (static_cast<long long>(b) * p.Hkv + h) * p.width;
  const __nv_bfloat16* src = p.bounds + static_cast<long long>(h) * 2 * D;
  const long long page_step = static_cast<long long>(p.Hkv) * 2 * D;
  uint32_t big2 = 0u;                 // largest |bound| of the even and odd channels
  if (end > (count + 7) / 8) end = (count + 7) / 8;
  // pages at odd places take the other 64 bytes of each 128: two pages' reads
  // then fall into different banks
  auto at = [](int page, int pc) {
    return page * (4 * D) + (pc ^ (PCS >= 8 ? (page & 1) * 4 : 0)) * 16;
  };
  for (int r0 = 0; r0 < p.rows && first < end; r0 += 8 * NR) {
    const int n = (end - first + step - 1) / step;
    uint32_t qa[SEG][2][2][NR];       // [segment][k-step][half][row g, g + 8]
    // lane l looks up page l % 8 of group l / 8 of four
    auto look_up = [&](int k4) {
      const int i = (first + (4 * k4 + (lane >> 3)) * step) * 8 + (lane & 7);
      const int page = 4 * k4 + (lane >> 3) < n && i < count ? p.table[b * p.table_sb + i] : -1;
      return page < p.n_pages ? page : -1;
    };
    int now = look_up(0), then = look_up(1), have = 0;  // entries of have, have + 1
    uint32_t held = 0u;               // which pages of the groups in the ring are held, 8 bits each
    auto issue = [&](int k) {         // group k of the run into slot k % kScoreStages
      held <<= 8;
      if (k < n) {
        if (k / 4 != have) {
          have = k / 4;
          now = then;
          then = look_up(have + 1);
        }
        held |= (dec_ballot(now >= 0) >> ((k & 3) * 8)) & 0xffu;
        uint8_t* to = ring + (k % kScoreStages) * (32 * D);
#pragma unroll
        for (int u = 0; u < PCS / 4; ++u) {
          const int piece = lane + 32 * u, pg = piece / PCS, pc = piece % PCS;
          const int page = dec_shfl(now, (k & 3) * 8 + pg);
          const bool ok = page >= 0;
          dec_cp_async16(to + at(pg, pc), src + (ok ? page : 0) * page_step + pc * 8, ok);
        }
      }
      dec_cp_async_commit();
    };
#pragma unroll
    for (int k = 0; k < kScoreStages; ++k) issue(k);
#pragma unroll
    for (int s = 0; s < SEG; ++s) {
      const int ch = 32 * s + 8 * t4;
      const bool low = ch < D;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        // (past the last row: the last again)
        const int row = r0 + g + 8 * r < p.rows ? r0 + g + 8 * r : p.rows - 1;
        const uint4 w =
            *reinterpret_cast<const uint4*>(select_row(p, b, h, row) + (low ? ch : ch - D));
        qa[s][0][0][r] = clip_pair(w.x, low);
        qa[s][0][1][r] = clip_pair(w.y, low);
        qa[s][1][0][r] = clip_pair(w.z, low);
        qa[s][1][1][r] = clip_pair(w.w, low);
      }
    }
    for (int k = 0; k < n; ++k) {
      dec_cp_async_wait<kScoreStages - 1>();
      __syncwarp();  // every lane's pieces of the group are in shared memory
      const uint8_t* slot = ring + (k % kScoreStages) * (32 * D);
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < SEG; ++s) {
        const uint4 v = *reinterpret_cast<const uint4*>(slot + at(g, 4 * s + t4));
        dec_mma(c, qa[s][0][0][0], UP ? qa[s][0][0][NR - 1] : 0u, qa[s][0][1][0],
                UP ? qa[s][0][1][NR - 1] : 0u, v.x, v.y);
        dec_mma(c, qa[s][1][0][0], UP ? qa[s][1][0][NR - 1] : 0u, qa[s][1][1][0],
                UP ? qa[s][1][1][NR - 1] : 0u, v.z, v.w);
        if (r0 == 0) {
          big2 = dec_bf16_absmax(big2, v.x);
          big2 = dec_bf16_absmax(big2, v.y);
          big2 = dec_bf16_absmax(big2, v.z);
          big2 = dec_bf16_absmax(big2, v.w);
        }
      }
      const uint32_t there = held >> (8 * (kScoreStages - 1));
      __syncwarp();  // every lane has read the slot: refill it
      issue(k + kScoreStages);
      // the highest row of pages 2 t4 and 2 t4 + 1 of the group; +inf marks a
      // sum that is not finite, which is left to the exact pass
      float m[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m[x] = c[x] - c[x] == 0.f ? c[x] : INFINITY;
        if (UP) m[x] = fmaxf(m[x], c[2 + x] - c[2 + x] == 0.f ? c[2 + x] : INFINITY);
#pragma unroll
        for (int d = 4; d < 32; d *= 2) m[x] = fmaxf(m[x], __shfl_xor_sync(0xffffffffu, m[x], d));
      }
      // lanes 0 .. 7 write: lane l the group's page l, from lane l / 2 (row 0)
      const float even = dec_shfl(m[0], (lane & 7) >> 1), odd = dec_shfl(m[1], (lane & 7) >> 1);
      const int i = (first + k * step) * 8 + lane;
      if (lane < 8 && i < count) {
        float s = ((there >> lane) & 1u) == 0u ? -INFINITY : (lane & 1) ? odd : even;
        if (r0 > 0) s = fmaxf(s, out[i]);  // (this lane wrote it)
        out[i] = s;
      }
    }
    dec_cp_async_wait<0>();
  }
  float big = fmaxf(dec_bf16_lo(big2), dec_bf16_hi(big2));
  // a NaN outranks every number in big2 and may hide the largest
  if ((big2 & 0xffffu) > 0x7f80u || (big2 >> 16) > 0x7f80u) big = INFINITY;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
  return big;
}

// Grid: B * Hkv * n_blocks; a warp takes p.groups groups.  (No early release
// of page_pick_kernel: its CTAs would take registers from the later waves of
// this grid, 5 us of 48 when it was measured at 128 x 1,150 pages.)
template <int D, bool UP>
__global__ void __launch_bounds__(kScoreThreads, 4) page_score_kernel(const SelectParams p) {
  dec_grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bh = static_cast<int>(blockIdx.x) / p.n_blocks;
  const int blk = static_cast<int>(blockIdx.x) - bh * p.n_blocks;
  const int b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int count = select_count(p, b);
  if (count <= p.n_sel) return;  // every page is taken
  const int w = blk * kScoreWarps + warp;
  const float big = score_groups<D, UP>(p, b, h, count, w * p.groups, (w + 1) * p.groups, 1,
                                        dec_dynamic_smem() + warp * score_ring_bytes(D));
  if (lane == 0) p.largest[static_cast<long long>(bh) * p.n_blocks * kScoreWarps + w] = big;
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

// Reductions over the NT threads of a CTA; `sh` has two halves of three words
// per warp, used in turn, so that one barrier each is enough.  (A reduction
// ends with reads of its half: whatever else writes to `sh` needs a barrier
// before it.)
template <int NT>
struct PickReduce {
  static constexpr int NW = NT / 32;
  int* sh;
  int turn;

  template <int N>
  __device__ __forceinline__ void sum(int (&v)[N]) {
    static_assert(N <= 3 && NW <= 32, "words");
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
  __device__ __forceinline__ void min_max(unsigned& lo, unsigned& hi) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned* half = reinterpret_cast<unsigned*>(sh + turn * 3 * NW);
    lo = dec_warp_min(lo);
    hi = dec_warp_max(hi);
    if (lane == 0) {
      half[warp] = lo;
      half[NW + warp] = hi;
    }
    __syncthreads();
    lo = dec_warp_min(lane < NW ? half[lane] : 0xffffffffu);
    hi = dec_warp_max(lane < NW ? half[NW + lane] : 0u);
    turn ^= 1;
  }
};
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

// Keys of no score (they would be NaN): a page that is chosen, and one that is
// not.
constexpr unsigned kKeySure = 0xffffffffu, kKeyOut = 0u;

// The choice for (b, h) from its scores, by the NT threads of a CTA; `largest`:
// n_largest maxima of the |bounds|.
template <int NT>
__device__ __forceinline__ void pick_pages(const SelectParams& p, int b, int h, int count,
                                           const float* largest, int n_largest) {
  constexpr int NW = NT / 32;
  constexpr int KR = 2048 / NT;       // scores that a thread keeps in registers
  unsigned* keys = reinterpret_cast<unsigned*>(dec_dynamic_smem());  // [kPickKeys]
  int* sh = reinterpret_cast<int*>(keys + kPickKeys);                // [2][3][NW]
  float* shf = reinterpret_cast<float*>(sh + 6 * NW);                // [2][NW]
  unsigned long long* sums = reinterpret_cast<unsigned long long*>(shf + 2 * NW);  // [kPickNear]
  int* list = reinterpret_cast<int*>(sums + kPickNear);                            // [kPickNear]
  int* n_list = list + kPickNear;                                                  // its entries
  PickReduce<NT> over{sh, 0};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) *n_list = 0;  // (barriers follow before it is used)
  const long long bh = static_cast<long long>(b) * p.Hkv + h;
  int* out = p.pages + bh * p.n_sel;
  const float* score = p.score + bh * p.width;
  double* exact = p.exact + bh * p.width;
  const int lo = p.n_first, hi = count - p.n_last;  // candidates: lo <= i < hi
  int want = p.n_sel - p.n_first - p.n_last;

  // rho: the largest |bound| and the largest sum |q| of a row
  float big = 0.f, qsum = 0.f;
  unsigned kr[KR], lowest = 0xffffffffu, highest = 0u;
  int odd[1] = {0};  // scores that are not finite, of pages that are held
  auto take_in = [&](int i, float s) {
    const unsigned k = score_key(s);
    odd[0] += s == INFINITY;
    if (i < kPickKeys) keys[i] = k;
    lowest = k < lowest ? k : lowest;
    highest = k > highest ? k : highest;
    return k;
  };
#pragma unroll
  for (int j = 0; j < KR; ++j) {
    const int i = lo + tid + j * NT;
    kr[j] = i < hi ? dec_float_bits(score[i]) : 0u;
  }
  for (int i = tid; i < n_largest; i += NT) big = fmaxf(big, largest[i]);
  for (int r = warp; r < p.rows; r += NW) {
    const __nv_bfloat16* q = select_row(p, b, h, r);
    float a = 0.f;
    for (int d = lane; d < p.D; d += 32) a += fabsf(__bfloat162float(q[d]));
#pragma unroll
    for (int d = 1; d < 32; d *= 2) a += __shfl_xor_sync(0xffffffffu, a, d);
    qsum = fmaxf(qsum, a);
  }
#pragma unroll
  for (int j = 0; j < KR; ++j) {
    const int i = lo + tid + j * NT;
    if (i < hi) kr[j] = take_in(i, dec_bits_float(kr[j]));
  }
  for (int i = lo + tid + KR * NT; i < hi; i += NT) take_in(i, score[i]);
#pragma unroll
  for (int d = 1; d < 32; d *= 2) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
  if (lane == 0) {
    shf[warp] = big;
    shf[NW + warp] = qsum;
  }
  over.sum(odd);  // (a barrier: keys and shf are written)
  over.min_max(lowest, highest);
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    big = fmaxf(big, shf[w]);
    qsum = fmaxf(qsum, shf[NW + w]);
  }
  // 1 percent for the sum's and the product's own roundings; a little for
  // terms below the smallest normal number
  const float rho = odd[0] ? INFINITY : 1.01f * 0x1p-16f * (big * qsum) + 1e-35f;
  auto key = [&](int i) { return i < kPickKeys ? keys[i] : score_key(score[i]); };
  auto each = [&](auto f) {  // f(page, key) of this thread's candidates
#pragma unroll
    for (int j = 0; j < KR; ++j)
      if (lo + tid + j * NT < hi) f(lo + tid + j * NT, kr[j]);
    for (int i = lo + tid + KR * NT; i < hi; i += NT) f(i, key(i));
  };

  // T, the want-th highest score: from the first bit in which the scores
  // differ, two bits a round, each the highest digit that at least `want`
  // scores reach; done when just `want` of them reach it
  unsigned T = 0u;
  if (want > 0) {
    int reach = hi - lo, shift = 30;
    while (shift > 0 && (lowest >> shift) == (highest >> shift)) shift -= 2;
    T = shift + 2 < 32 ? highest >> (shift + 2) << (shift + 2) : 0u;
    for (; shift >= 0 && reach != want; shift -= 2) {
      int n[3] = {0, 0, 0};
      each([&](int, unsigned k) {
#pragma unroll
        for (int d = 0; d < 3; ++d) n[d] += k >= (T | ((d + 1u) << shift));
      });
      over.sum(n);
      const unsigned digit = pick_digit(n, want);
      T |= digit << shift;
      reach = digit == 0u ? reach : n[digit - 1u];
    }
    unsigned least = 0xffffffffu, none = 0u;  // the lowest of those that reach T
    each([&](int, unsigned k) { least = k >= T && k < least ? k : least; });
    over.min_max(least, none);
    T = least;
  }
  // sure: above whatever the want-th highest exact score may be; near: may
  // be either (the comparisons with infinities and NaN fall to `near`)
  auto value = [](unsigned k) { return dec_bits_float((k >> 31) ? k & 0x7fffffffu : ~k); };
  const float t = value(T);
  const bool some = want > 0;
  auto sure = [&](unsigned k) { return some && value(k) - rho > t + rho; };
  auto near = [&](unsigned k) {
    return some && !(value(k) - rho > t + rho) && !(value(k) + rho < t - rho);
  };
  int n_of[2] = {0, 0};  // sure, near
  each([&](int, unsigned k) {
    n_of[0] += sure(k);
    n_of[1] += near(k);
  });
  over.sum(n_of);
  want -= n_of[0];
  const bool all_near = n_of[1] <= want;
  const bool few = !all_near && n_of[1] <= kPickNear && count <= kPickKeys;
  unsigned long long E = 0;  // the want-th highest exact score of those near T
  if (few) {
    // list them, sum them, and rank each among all: the keys of those chosen
    // become the highest, of the others the lowest
    each([&](int i, unsigned k) {
      if (near(k)) list[dec_add_shared(n_list, 1)] = i;  // (in any order)
    });
    __syncthreads();
    for (int j = warp; j < n_of[1]; j += NW) {
      const double s = exact_score(p, b, h, list[j]);
      if (lane == 0) sums[j] = score_key(s);
    }
    __syncthreads();
    for (int j = tid; j < n_of[1]; j += NT) {
      int rank = 0;
      for (int x = 0; x < n_of[1]; ++x)
        rank += sums[x] > sums[j] || (sums[x] == sums[j] && list[x] < list[j]);
      keys[list[j]] = rank < want ? kKeySure : kKeyOut;
    }
    __syncthreads();
  } else if (!all_near) {
    for (int base = lo; base < hi; base += NT) {
      const int i = base + tid;
      unsigned todo = dec_ballot(i < hi && near(key(i < hi ? i : lo)));
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
      each([&](int i, unsigned k32) {
        if (!near(k32)) return;
        const unsigned long long k = score_key(exact[i]);
#pragma unroll
        for (int d = 0; d < 3; ++d) n[d] += k >= (E | ((d + 1ull) << shift));
      });
      over.sum(n);
      E |= static_cast<unsigned long long>(pick_digit(n, want)) << shift;
    }
    int above[1] = {0};
    each([&](int i, unsigned k) { above[0] += near(k) && score_key(exact[i]) > E; });
    over.sum(above);
    want -= above[0];  // places for those that equal E
  }

  // listed in order: those chosen, and the first `want` of those equal to E
  int listed = 0, equal = 0;
  for (int base = 0; base < count; base += NT) {
    const int i = base + tid;
    bool take = i < count && (i < lo || i >= hi), same = false;
    if (i >= lo && i < hi) {
      const unsigned k = key(i);
      if (few && (k == kKeySure || k == kKeyOut)) {
        take = k == kKeySure;
      } else if (!near(k)) {
        take = sure(k);
      } else if (all_near) {
        take = true;
      } else {
        const unsigned long long k64 = score_key(exact[i]);
        take = k64 > E;
        same = k64 == E;
      }
    }
    const unsigned below = (1u << lane) - 1u;
    if (!all_near && !few) {
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

// Every page of (b, h).
__device__ __forceinline__ void pick_all(const SelectParams& p, long long bh, int count) {
  for (int i = threadIdx.x; i < p.n_sel; i += blockDim.x)
    p.pages[bh * p.n_sel + i] = i < count ? i : -1;
}

// Grid: B * Hkv CTAs of kPickThreads.
__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelectParams p) {
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  const int bh = static_cast<int>(blockIdx.x), b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int count = select_count(p, b);
  if (count <= p.n_sel) {
    pick_all(p, bh, count);
    return;
  }
  pick_pages<kPickThreads>(p, b, h, count,
                           p.largest + static_cast<long long>(bh) * p.n_blocks * kScoreWarps,
                           p.n_blocks * kScoreWarps);
}

// Both in one launch: a cluster of kSelectCtas CTAs scores the pages of one
// (request, head), then its first CTA chooses, while other clusters score.
template <int D, bool UP>
__global__ void __launch_bounds__(kSelectThreads, 2) page_select_kernel(const SelectParams p) {
  constexpr int NW = kSelectCtas * kSelectThreads / 32;
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int bh = static_cast<int>(blockIdx.x) / kSelectCtas, b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int rank = static_cast<int>(dec_cluster_rank());
  const int count = select_count(p, b);
  float* largest = p.largest + static_cast<long long>(bh) * NW;
  if (count > p.n_sel) {
    const int w = warp * kSelectCtas + rank;
    const float big = score_groups<D, UP>(p, b, h, count, w, p.width, NW,
                                          dec_dynamic_smem() + warp * score_ring_bytes(D));
    if (lane == 0) largest[w] = big;
  }
  dec_cluster_sync();  // every CTA's scores are written
  if (rank != 0) return;
  if (count <= p.n_sel)
    pick_all(p, bh, count);
  else
    pick_pages<kSelectThreads>(p, b, h, count, largest, NW);
}

__host__ __device__ constexpr int pick_smem_bytes() {
  return kPickKeys * 4 + 8 * (kPickThreads / 32) * 4 + kPickNear * 12 + 16;
}
// Shared memory of the fused kernel: the rings, and then the choice's.
__host__ __device__ constexpr int select_smem_bytes(int D) {
  const int rings = kSelectThreads / 32 * score_ring_bytes(D);
  return rings > pick_smem_bytes() ? rings : pick_smem_bytes();
}

// Whether the fused kernel is taken: for short lists, where it saves a launch
// (device time is the same: 16 heads x 512 pages 11.6 against 11.9 us, x 1,024
// pages 14.2 against 14.1); longer ones are scored faster by a grid of its
// own (64 x 256 pages: 13.9 against 17.9 us, 128 x 1,150: 33.2 against 45.6).
__host__ __device__ constexpr bool select_fused(long long bh, int width) {
  return bh * ((width + 7LL) / 8) <= 2048;
}
// Otherwise: groups of 8 pages per warp, and the CTAs per (request, head) that
// follow.  One group where there are few, so that all are on their way at
// once; up to six, whose query rows then cost little (64 x 512 pages: 17.2 us
// with one, 15.5 with two; 32 x 2,048: 27.4, 22.7 with four; 128 x 1,150:
// 47.0, 33.2 with six).
__host__ __device__ constexpr int score_groups_of(long long bh, int width) {
  const long long n = (bh * ((width + 7LL) / 8) + 2047) / 2048;
  return n < 1 ? 1 : n > 6 ? 6 : static_cast<int>(n);
}
__host__ __device__ constexpr int score_blocks(long long bh, int width) {
  const int pages = kScoreWarps * 8 * score_groups_of(bh, width);
  return (width + pages - 1) / pages;
}
// Workspace: the exact scores, the fp32 scores, the largest bounds.
__host__ __device__ constexpr long long select_workspace_bytes(long long bh, int width) {
  const long long n = select_fused(bh, width) ? kSelectCtas * kSelectThreads / 32
                                              : score_blocks(bh, width) * kScoreWarps;
  return bh * (width * 12LL + n * 4);
}

}  // namespace cattn
