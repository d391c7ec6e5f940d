// Decode attention over a paged key/value cache.
//
// As decode.cuh (the newest Tq positions of a sequence against its cached
// keys and values), for many sequences of different lengths whose keys lie
// in pages of a common pool: request b's position p is row p % P of page
// table[b][p / P].  H query heads read Hkv cache heads, G = H / Hkv query
// heads each.  For the query row at position x = len - Tq + t:
//
//   s_j = scale q . k_j,  o = sum_j exp(s_j) v_j / sum_j exp(s_j),
//   lse = log sum_j exp(s_j)   over the held keys j <= x
//
// (o = 0 and lse = -inf where no key is held).  The sparse form reads the
// keys of K listed pages per (request, cache head) only.
//
// The bound is reading K and V once (4 D bytes per key and cache head for
// 4 D G Tq flops), so the design is about a steady read by every SM however
// the lengths are spread:
//   - the keys of every item (request, cache head, tile of <= 16 query rows)
//     are cut into chunks of paged_chunk(D) keys; all items' chunks in a row
//     form one flat axis that is dealt evenly to the warps of one resident
//     wave, each a contiguous run.  Lengths live on the GPU, so every CTA
//     works out the cuts itself, from one scan of the lengths;
//   - a warp streams its run through a private ring of kPagedStages shared
//     memory slots with cp.async, on across items; per chunk it multiplies
//     q k^T and p v with mma.sync m16n8k16 (query rows as the A operand, at
//     most 16) and keeps the running maximum and sum (online softmax);
//   - an item that ends inside its warp's run is written out directly; a cut
//     item leaves (m, l, o) per warp in the workspace, paged_merge_kernel joins
//     them, in the order of the keys, so results repeat bit for bit.
// p enters the second product as a bf16 pair, hi + lo: a relative error of at
// most 2^-16, little beside the 2^-9 of o's own rounding to bf16.  With at most 8
// rows the pair costs no instruction: hi takes the fragment's rows 0 .. 7, lo its
// rows 8 .. 15, and the two halves of the accumulator are added at the end.  hi
// is p cut off, and lo the rest of p with its last bit set: neither is zero or
// negative where p > 0 (from 2^-110 on, where lo leaves bf16's range), so an
// infinite value of V gives infinity in both products and not 0 inf or inf - inf.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#ifndef CATTN_HOST_EMULATION
#include "paged_ptx.cuh"
#endif

namespace cattn {

constexpr int kPagedWarps = 4;                    // warps per CTA
constexpr int kPagedThreads = 32 * kPagedWarps;
constexpr int kPagedStages = 3;                   // chunks in flight per warp
constexpr int kItemStages = 2;                    // in paged_item_kernel
constexpr int kPagedMaxCtas = 2 * 148;            // resident CTAs of a B200 (2 x 99 KB)
constexpr int kItemSlots = 3 * 148;               // resident CTAs of paged_item_kernel (66 KB)
constexpr int kPagedMaxWarps = kPagedMaxCtas * kPagedWarps;
constexpr int kPagedMinRun = 2;                   // chunks that a warp takes at least
constexpr int kPagedRows = 16;                    // query rows per item
constexpr int kPagedNone = 0x7fffffff;            // position of a key that is not held
constexpr int kMergeThreads = 512;
constexpr float kPagedLag = 8.f;                  // how far scores rise before m_run follows, log2

// Keys per chunk: 4 KB of K and 4 KB of V at D >= 64; at most 32, one lane
// per key.
__host__ __device__ constexpr int paged_chunk(int D) { return D == 128 ? 16 : 32; }
__host__ __device__ constexpr int paged_chunk_bytes(int D) { return paged_chunk(D) * D * 4; }
__host__ __device__ constexpr int paged_ring_bytes(int D, int stages) {
  return kPagedWarps * stages * paged_chunk_bytes(D);
}
// Dynamic shared memory: the rings, the key positions of their slots, the
// scan's prefix sums and warp totals.
__host__ __device__ constexpr int paged_smem_bytes(int D, int stages) {
  return paged_ring_bytes(D, stages) + kPagedWarps * stages * 32 * 4 + (kPagedThreads + 8) * 4;
}

// Where a cut item begins (n_parts = 0: none does in this warp), and where its
// parts are: slot 1 of this warp; slot 0 of the n_same warps behind it in its
// CTA; of the first warp of the n_mid CTAs behind that, whose shares lie in the
// item as a whole; and of the first warps of one more CTA.
struct PagedCut {
  int b, ht, n_parts, where;  // where = 4 n_mid + n_same

  // The slot of part i of an item that begins in warp gw.
  __host__ __device__ long long slot(int gw, int i) const {
    const int n_same = where & 3, n_mid = where >> 2, cta = gw / kPagedWarps;
    if (i == 0) return 2LL * gw + 1;
    if (i <= n_same) return 2LL * (gw + i);
    i -= n_same;
    if (i <= n_mid) return 2LL * kPagedWarps * (cta + i);
    return 2LL * (kPagedWarps * (cta + n_mid + 1) + i - n_mid - 1);
  }
};
static_assert(kPagedWarps == 4, "PagedCut packs a warp's place in two bits");

// Workspace: PagedCut[kPagedMaxWarps], then (m, l) and o of two slots per
// warp with R = min(16, G Tq) rows each.
__host__ __device__ constexpr long long paged_ml_offset() {
  return static_cast<long long>(kPagedMaxWarps) * static_cast<long long>(sizeof(PagedCut));
}
__host__ __device__ constexpr long long paged_o_offset(int R) {
  return paged_ml_offset() + 2LL * kPagedMaxWarps * R * 8;
}
__host__ __device__ constexpr long long paged_workspace_bytes(int R, int D) {
  return paged_o_offset(R) + 2LL * kPagedMaxWarps * R * D * 4;
}

// n / P for 0 <= n < 2^31 as (n mul) >> shift: with shift = 31 + L, 2^L >= P,
// and mul = floor(2^shift / P) + 1 <= 2^32, n mul / 2^shift exceeds n / P by at
// most n / 2^shift < 1 / P, too little to reach the next whole number.
struct PageDivider {
  unsigned long long mul;
  int shift;
  __host__ __device__ explicit PageDivider(int P = 1) {
    int L = 0;
    while ((1LL << L) < P) ++L;
    shift = 31 + L;
    mul = (1ull << shift) / static_cast<unsigned>(P) + 1;
  }
  __host__ __device__ int operator()(int n) const {
    return static_cast<int>((static_cast<unsigned long long>(n) * mul) >> shift);
  }
};

struct PagedParams {
  const __nv_bfloat16* q;  // (B, H, Tq, D)
  const __nv_bfloat16* k;  // (n_pages, Hkv, P, D)
  const __nv_bfloat16* v;
  long long q_sb, q_sh, q_st, k_sp, k_sh, k_st, v_sp, v_sh, v_st;
  __nv_bfloat16* o;        // (B, H, Tq, D)
  long long o_sb, o_sh, o_st;
  float* lse;              // (B, H, Tq) contiguous, natural log
  const int* table;        // (B, width), row stride table_sb
  long long table_sb;
  const int* lengths;      // (B)
  const int* pages;        // (B, Hkv, n_sel) logical pages, or null: all
  int B, H, Hkv, Tq, rows; // rows = G Tq
  int n_tiles;             // ceil(rows / 16)
  int n_pages, P, width, n_sel;
  int R;                   // rows of a partial slot, min(16, rows)
  float scale_log2;        // scale * log2(e)
  PageDivider by_P;
  PagedCut* cuts;
  float2* part_ml;         // [2 warps][R]
  float* part_o;           // [2 warps][R][D]
};

// Keys of request b that its items enumerate (sparse: of the listed pages),
// and the chunks they take; an item without keys has one, empty, chunk.
__device__ __forceinline__ int paged_length(const PagedParams& p, int b) {
  const int len = p.lengths[b];
  return len > 0 ? len : 0;
}
__device__ __forceinline__ int paged_keys(const PagedParams& p, int len) {
  if (p.pages != nullptr)  // (a list holds at most 2^30 keys)
    return len >= p.n_sel * p.P ? p.n_sel * p.P : p.by_P(len + p.P - 1) * p.P;
  const int cap = p.width * p.P;
  return len < cap ? len : cap;
}
template <int D>
__device__ __forceinline__ int paged_chunks(const PagedParams& p, int len) {
  const int n = (paged_keys(p, len) + paged_chunk(D) - 1) / paged_chunk(D);
  return n > 0 ? n : 1;
}

// What an item costs its warp beside its chunks, in chunks: its query rows,
// lengths and table row are trips to memory that nothing hides.  On the flat
// axis every item begins with that many empty places (c < 0).  (64 requests of
// 10 to 12,453 keys x 8 heads of 128: 108 us without, 88 with 2; of 64: 70 and
// 55 with 4; twice as many change nothing or cost 5 percent at D <= 32.)
__host__ __device__ constexpr int paged_item_cost(int D) { return D == 128 ? 2 : 4; }

// A place on the flat axis: chunk c of the n of item (b, ht).
struct PagedPlace {
  int b, ht, c, n, len;
};

// A key: where its rows of K and V begin (bytes from head 0 of the pool; -1: it
// is not held), and its position.
struct PagedKey {
  long long k, v;
  int pos;
};

// On to the next chunk; `units` are the places from x to the end of the run.
template <int D>
__device__ __forceinline__ void paged_next(const PagedParams& p, int HT, PagedPlace& x,
                                           int& units) {
  --units;
  if (++x.c < x.n) return;
  x.c = 0;
  units -= paged_item_cost(D);
  if (++x.ht < HT) return;
  x.ht = 0;
  if (++x.b >= p.B) return;  // behind the last item
  x.len = paged_length(p, x.b);
  x.n = paged_chunks<D>(p, x.len);
}

// Natural log-sum-exp from a base-2 reference and the sum relative to it, which
// lies 2 kPagedLag below the largest score at the most: brought there, so that the
// two parts do not cancel.
__device__ __forceinline__ float paged_lse(float m, float l) {
  constexpr float up = 1 << static_cast<int>(2 * kPagedLag);
  return l == 0.f ? -INFINITY : (m - 2.f * kPagedLag + log2f(l * up)) * 0.69314718055994531f;
}

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int warp_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int u = dec_shfl(v, lane >= d ? lane - d : 0);
    if (lane >= d) v += u;
  }
  return v;
}

// Flat place x: request b holds the places HT * before(b) up to
// HT * before(b + 1), before = the chunks and costs of one head of the requests
// in front.  pre[t] is before(t * nb).  (The lengths are read again here; the
// clamps keep every index in range should a caller change them meanwhile.)
template <int D>
__device__ __forceinline__ PagedPlace paged_locate(const PagedParams& p, int HT, int nb,
                                                   const int* pre, long long x, int lane) {
  const int y = static_cast<int>(x / HT);
  int t = -1;  // pre[0] = 0 <= y: at least 0 in the end
#pragma unroll
  for (int i = 0; i < kPagedThreads / 32; ++i) t += dec_popc(dec_ballot(pre[32 * i + lane] <= y));
  int run = pre[t];
  for (int b0 = t * nb; b0 < (t + 1) * nb; b0 += 32) {
    const int b = b0 + lane;
    const bool in = lane < (t + 1) * nb - b0 && b < p.B;
    const int len = in ? paged_length(p, b) : 0;
    const int n = in ? paged_chunks<D>(p, len) + paged_item_cost(D) : 0;
    const int incl = warp_scan(n, lane);
    const unsigned hit = dec_ballot(run + incl > y);
    if (hit != 0u) {
      const int src = dec_lowest(hit);
      PagedPlace r;
      r.b = b0 + src;
      r.n = dec_shfl(n, src);
      r.len = dec_shfl(len, src);
      const int before = run + dec_shfl(incl, src) - r.n;
      const long long rem = x - static_cast<long long>(before) * HT;
      r.ht = static_cast<int>(rem / r.n);
      r.c = static_cast<int>(rem - static_cast<long long>(r.ht) * r.n) - paged_item_cost(D);
      r.n -= paged_item_cost(D);
      if (r.ht >= HT) r.ht = HT - 1;
      return r;
    }
    run += dec_shfl(incl, 31);
  }
  return PagedPlace{p.B, 0, 0, 1, 0};
}

// One warp's work on chunks: its ring of shared memory slots and the running
// state of the item it is in.  UP: rows 8 .. 15 of the tile are used.  MULTI:
// several new positions (Tq > 1), so that rows may see different keys.
//
// A warp waits for memory most of the time, but it has few companions (8 to 12
// on an SM, for the rings' sake), so the length of its instruction stream
// counts: the swizzled addresses of a slot differ from one per-lane offset by an
// exclusive or with constants, and the running reference m_run, which the
// weights 2^(s - m_run) are relative to, is set 2^16 above the largest score and
// only moves when a score comes within 2^8 of it.  (Weights stay below 2^-8, so
// the sums over values near the largest bf16 have room for 2^8 such weights, and
// neither the quad's exchange of maxima nor the rescaling of o is on the usual
// path.)
template <int D, bool UP, bool MULTI, int STAGES>
struct PagedWarp {
  static constexpr int CK = paged_chunk(D);  // keys per chunk
  static constexpr int PC = D / 8;           // 16-byte pieces per row
  static constexpr int NS = CK / 8;          // score n-tiles per chunk
  static constexpr int KS = D / 16;          // k-steps of q k^T
  static constexpr int NO = D / 8;           // output n-tiles
  static constexpr int TILE = CK * D * 2;    // bytes of K (of V) per chunk
  static constexpr int CB = 2 * TILE;
  static constexpr int NR = UP ? 2 : 1;      // fragment rows of a lane: g, g + 8
  static constexpr int RU = 32 / PC;         // rows that a 16-byte copy per lane covers
  static_assert(TILE / 16 % 32 == 0 && CK % 16 == 0 && CK <= 32 && 32 % PC == 0, "chunk");
  static_assert(TILE % 256 == 0, "offsets inside 256 bytes may be changed by exclusive or");

  const PagedParams& p;
  int lane, g, t4;             // lane, fragment row, column pair
  bool same;                   // K and V have one layout
  uint8_t* ring;
  uint32_t ring_at;            // its shared-memory address
  uint32_t at_copy, at_k, at_v;  // the lane's offsets in a tile: copies, ldmatrix of K, of V
  int* slot_pos;               // positions of the slots' keys
  uint32_t qa[KS][4];          // query rows as mma A fragments
  float o[NO][4];              // running state of rows g (and g + 8)
  float m_run[NR], l_run[NR];  // (l is the lane's part)
  int row_pos[NR];             // the rows' positions

  __device__ __forceinline__ PagedWarp(const PagedParams& params, uint8_t* smem, int warp,
                                       int lane_)
      : p(params), lane(lane_), g(lane_ >> 2), t4(lane_ & 3),
        same(params.k_sp == params.v_sp && params.k_st == params.v_st) {
    ring = smem + warp * (STAGES * CB);
    ring_at = pg_smem_addr(ring);
    slot_pos = reinterpret_cast<int*>(smem + paged_ring_bytes(D, STAGES)) + warp * STAGES * 32;
    const int l7 = lane & 7, mi = lane >> 3;
    at_copy = dec_swz<D>(lane / PC, lane % PC);
    at_k = dec_swz<D>(l7, PC >= 4 ? mi : mi & 1);
    at_v = dec_swz<D>((mi & 1) * 8 + l7, mi >> 1);
    clear();
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      m_run[r] = -INFINITY;
      l_run[r] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < NO; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  }

  // The lane's key of chunk x.  (The list and the table are read as far as they
  // go, whatever the length: its own load need not have arrived.)
  __device__ __forceinline__ PagedKey look_up(const PagedPlace& x) const {
    const int vk = x.c * CK + lane;
    const int li = p.by_P(vk);
    const int row = vk - li * p.P;
    int lp = -1, page = -1;
    if (lane < CK && x.b < p.B) {
      lp = li;
      if (p.pages != nullptr)
        lp = li < p.n_sel ? p.pages[(static_cast<long long>(x.b) * p.Hkv + x.ht / p.n_tiles) *
                                        p.n_sel + li]
                          : -1;
      if (lp >= 0 && lp < p.width) page = p.table[x.b * p.table_sb + lp];
    }
    PagedKey key{-1, -1, kPagedNone};
    if (page >= 0 && page < p.n_pages && lp * p.P + row < x.len &&
        (p.pages == nullptr || vk < paged_keys(p, x.len))) {
      key.k = (page * p.k_sp + row * p.k_st) * 2;
      key.v = same ? key.k : (page * p.v_sp + row * p.v_st) * 2;
      key.pos = lp * p.P + row;
    }
    return key;
  }

  // A chunk of item (b, ht) into ring slot `slot`; rows of keys that are not
  // held are zero-filled (and masked in chunk()).  A lane copies the same
  // 16 bytes of every RU-th row.
  __device__ __forceinline__ void issue(int ht, const PagedKey& key, int slot) {
    const uint32_t to = ring_at + slot * CB + at_copy;
    const int h = ht / p.n_tiles;
    const char* kb = reinterpret_cast<const char*>(p.k + h * p.k_sh) + lane % PC * 16;
    const char* vb = reinterpret_cast<const char*>(p.v + h * p.v_sh) + lane % PC * 16;
    slot_pos[slot * 32 + lane] = key.pos;
    const bool full = dec_ballot(lane < CK && key.k < 0) == 0u;
#pragma unroll
    for (int u = 0; u < TILE / 16 / 32; ++u) {
      // row lane / PC + RU u: 512 u bytes on, its swizzle changed by constants
      constexpr int RPL = PC >= 8 ? 1 : 8 / PC, MASK = (PC >= 8 ? 8 : PC) - 1;
      const uint32_t at = (to ^ ((RU * u / RPL & MASK) * 16)) + 512 * u;
      const int row = lane / PC + RU * u;
      const long long ko = dec_shfl(key.k, row), vo = same ? ko : dec_shfl(key.v, row);
      if (full) {
        pg_cp_async16(at, kb + ko);
        pg_cp_async16(at + TILE, vb + vo);
      } else {
        pg_cp_async16(at, kb + (ko < 0 ? 0 : ko), ko >= 0);
        pg_cp_async16(at + TILE, vb + (ko < 0 ? 0 : vo), ko >= 0);
      }
    }
  }

  // Query row `gr` of cache head h: its head and new position.
  __device__ __forceinline__ long long row_head(int h, int gr, int* t) const {
    const int gh = MULTI ? gr / p.Tq : gr;
    *t = gr - gh * p.Tq;
    return static_cast<long long>(h) * (p.H / p.Hkv) + gh;
  }

  // A new item: its query rows (zero past the last) and an empty state.
  __device__ __forceinline__ void begin(const PagedPlace& x) {
    clear();
    const int h = x.ht / p.n_tiles, r0 = (x.ht - h * p.n_tiles) * kPagedRows;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int gr = r0 + g + 8 * r;
      const bool ok = r < NR && gr < p.rows && x.b < p.B;
      int t = 0;
      const long long hq = ok ? row_head(h, gr, &t) : 0;
      const __nv_bfloat16* qr = p.q + (ok ? x.b : 0) * p.q_sb + hq * p.q_sh + t * p.q_st;
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) {
        qa[kk][r] = ok ? *reinterpret_cast<const uint32_t*>(qr + 16 * kk + 2 * t4) : 0u;
        qa[kk][2 + r] = ok ? *reinterpret_cast<const uint32_t*>(qr + 16 * kk + 8 + 2 * t4) : 0u;
      }
      if (r < NR) row_pos[r] = x.len - p.Tq + t;
    }
  }

  // The chunk in ring slot `slot` of a request of length len.
  __device__ __forceinline__ void chunk(int slot, int len) {
    const float sl2 = p.scale_log2;
    const uint32_t sk = ring_at + slot * CB + at_k, sv = ring_at + slot * CB + TILE + at_v;
    const int* pos = slot_pos + slot * 32;
    const int pos0 = len - p.Tq;  // position of query t = 0
    const int my_pos = lane < CK ? pos[lane] : -1;

    // s = q k^T: lane's c0, c1 are row g, keys 8 nt + 2 t4, + 1; c2, c3 row g + 8.
    // Two sums of every other k-step each, so that the products' chain is short.
    float sc[NS][4];
#pragma unroll
    for (int nt = 0; nt < NS; ++nt) {
      float s2[4] = {0.f, 0.f, 0.f, 0.f};
      sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
      if constexpr (PC >= 4) {
#pragma unroll
        for (int x = 0; x < PC / 4; ++x) {
          uint32_t r[4];
          pg_ldsm_x4(r, (sk ^ (64 * x)) + nt * (8 * PC * 16));
          dec_mma(sc[nt], qa[2 * x][0], qa[2 * x][1], qa[2 * x][2], qa[2 * x][3], r[0], r[1]);
          dec_mma(s2, qa[2 * x + 1][0], qa[2 * x + 1][1], qa[2 * x + 1][2], qa[2 * x + 1][3],
                  r[2], r[3]);
        }
#pragma unroll
        for (int c = 0; c < 2 * NR; ++c) sc[nt][c] += s2[c];
      } else {  // D = 16: one k-step
        uint32_t r[2];
        pg_ldsm_x2(r, sk + nt * (8 * PC * 16));
        dec_mma(sc[nt], qa[0][0], qa[0][1], qa[0][2], qa[0][3], r[0], r[1]);
      }
    }
    // keys that are not held, and keys behind a row's position
    const bool masked = dec_ballot(MULTI ? my_pos > pos0 : my_pos == kPagedNone) != 0u;
    if (masked) {
#pragma unroll
      for (int nt = 0; nt < NS; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int kp = pos[nt * 8 + 2 * t4 + c];
#pragma unroll
          for (int r = 0; r < NR; ++r)
            if (MULTI ? kp > row_pos[r] : kp == kPagedNone) sc[nt][2 * r + c] = -INFINITY;
        }
    }

    // online softmax of the rows over this chunk (m_run: see the class)
    float mx[NR];
    bool moves = false;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      mx[r] = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NS; ++nt)
        mx[r] = fmaxf(mx[r], fmaxf(sc[nt][2 * r], sc[nt][2 * r + 1]));
      moves = moves || mx[r] * sl2 > m_run[r] - kPagedLag;
    }
    if (dec_ballot(moves) != 0u) {
      float alpha[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        const float m_new = fmaxf(m_run[r], fmaf(mx[r], sl2, 2.f * kPagedLag));
        alpha[r] = dec_exp2(m_run[r] - (m_new == -INFINITY ? 0.f : m_new));  // 0 from -inf
        m_run[r] = m_new;
        l_run[r] *= alpha[r];
      }
#pragma unroll
      for (int j = 0; j < NO; ++j) {
        o[j][0] *= alpha[0];
        o[j][1] *= alpha[0];
        o[j][2] *= alpha[NR - 1];  // without UP: the lo half of row g
        o[j][3] *= alpha[NR - 1];
      }
    }
    uint32_t hi[NS][NR], lo[NS][NR];  // the weights as bf16 pairs, hi + lo (see the top)
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float mu = m_run[r] == -INFINITY ? 0.f : m_run[r];  // no visible key yet
#pragma unroll
      for (int nt = 0; nt < NS; ++nt) {
        const float p0 = dec_exp2(fmaf(sc[nt][2 * r], sl2, -mu));
        const float p1 = dec_exp2(fmaf(sc[nt][2 * r + 1], sl2, -mu));
        l_run[r] += p0 + p1;
        if (MULTI) {
          sc[nt][2 * r] = p0;
          sc[nt][2 * r + 1] = p1;
        }
        const unsigned u0 = dec_float_bits(p0), u1 = dec_float_bits(p1);
        hi[nt][r] = u0 >> 16 | (u1 & 0xffff0000u);
        lo[nt][r] =
            dec_pack_bf16(dec_bits_float(u0 | 1u) - dec_bits_float(u0 & 0xffff0000u),
                          dec_bits_float(u1 | 1u) - dec_bits_float(u1 & 0xffff0000u));
      }
    }
    // A key that some rows see and others do not: its value must not touch
    // those others, not even as 0 * NaN.  Its products are done one by one,
    // and its row of V is cleared for the matrix product below.
    if (MULTI && masked) {
      uint8_t* v = ring + slot * CB + TILE;
      for (int key = 0; key < CK; ++key) {
        const int kp = pos[key];
        if (kp <= pos0 || kp == kPagedNone) continue;
        const int nt = key >> 3, src = (lane & ~3) | ((key & 7) >> 1);
        float w[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float x = 0.f;
#pragma unroll
          for (int n = 0; n < NS; ++n)
            if (n == nt) x = (key & 1) ? sc[n][2 * r + 1] : sc[n][2 * r];
          w[r] = dec_shfl(x, src);
        }
#pragma unroll
        for (int j = 0; j < NO; ++j) {
          const uint32_t vv = *reinterpret_cast<const uint32_t*>(v + dec_swz<D>(key, j) + 4 * t4);
#pragma unroll
          for (int r = 0; r < NR; ++r)
            if (kp <= row_pos[r]) {
              o[j][2 * r] = fmaf(w[r], dec_bf16_lo(vv), o[j][2 * r]);
              o[j][2 * r + 1] = fmaf(w[r], dec_bf16_hi(vv), o[j][2 * r + 1]);
            }
        }
        __syncwarp();  // every lane has read the row
        if (lane < PC) *reinterpret_cast<uint4*>(v + dec_swz<D>(key, lane)) = uint4{0, 0, 0, 0};
      }
      __syncwarp();  // the cleared rows are visible
    }

    // o += p v over the chunk's 16-key steps; one transposed x4 covers 16
    // keys x 16 columns (two output n-tiles)
#pragma unroll
    for (int kk = 0; kk < CK / 16; ++kk) {
#pragma unroll
      for (int jj = 0; jj < D / 16; ++jj) {
        uint32_t r[4];
        pg_ldsm_x4_t(r, (sv ^ (32 * jj)) + kk * (16 * PC * 16));
        const uint32_t b1 = UP ? hi[2 * kk][NR - 1] : lo[2 * kk][0];
        const uint32_t b3 = UP ? hi[2 * kk + 1][NR - 1] : lo[2 * kk + 1][0];
        dec_mma(o[2 * jj], hi[2 * kk][0], b1, hi[2 * kk + 1][0], b3, r[0], r[1]);
        dec_mma(o[2 * jj + 1], hi[2 * kk][0], b1, hi[2 * kk + 1][0], b3, r[2], r[3]);
        if constexpr (UP) {
          dec_mma(o[2 * jj], lo[2 * kk][0], lo[2 * kk][1], lo[2 * kk + 1][0], lo[2 * kk + 1][1],
                  r[0], r[1]);
          dec_mma(o[2 * jj + 1], lo[2 * kk][0], lo[2 * kk][1], lo[2 * kk + 1][0],
                  lo[2 * kk + 1][1], r[2], r[3]);
        }
      }
    }
  }

  // Column pair c of row r of n-tile j.
  __device__ __forceinline__ float out(int j, int r, int c) const {
    return UP ? o[j][2 * r + c] : o[j][c] + o[j][2 + c];
  }

  // Row r's sum over the quad that shares it.
  __device__ __forceinline__ float row_sum(int r) const {
    float l = l_run[r];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    return l + __shfl_xor_sync(0xffffffffu, l, 2);
  }

  // The item x, done: its rows' o and lse.
  __device__ __forceinline__ void finish(const PagedPlace& x) {
    const int h = x.ht / p.n_tiles, r0 = (x.ht - h * p.n_tiles) * kPagedRows;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float l = row_sum(r);
      const int gr = r0 + g + 8 * r;
      if (gr >= p.rows || x.b >= p.B) continue;
      int t;
      const long long hq = row_head(h, gr, &t);
      __nv_bfloat16* ob = p.o + x.b * p.o_sb + hq * p.o_sh + t * p.o_st;
      const float inv = l == 0.f ? 0.f : 1.f / l;  // no key: zeros
#pragma unroll
      for (int j = 0; j < NO; ++j)
        *reinterpret_cast<uint32_t*>(ob + 8 * j + 2 * t4) =
            dec_pack_bf16(out(j, r, 0) * inv, out(j, r, 1) * inv);
      if (t4 == 0)
        p.lse[(x.b * static_cast<long long>(p.H) + hq) * p.Tq + t] = paged_lse(m_run[r], l);
    }
  }

  // The state as rows [r] of ml (m, l) and of ov (o, `pitch` floats apart), R of
  // them.
  __device__ __forceinline__ void store(float2* ml, float* ov, int R, int pitch) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const float l = row_sum(r);
      const int row = g + 8 * r;
      if (row >= R) continue;
      if (t4 == 0) ml[row] = float2{m_run[r], l};
#pragma unroll
      for (int j = 0; j < NO; ++j)
        *reinterpret_cast<float2*>(ov + row * pitch + 8 * j + 2 * t4) =
            float2{out(j, r, 0), out(j, r, 1)};
    }
  }
};

// Shared memory of a CTA's merge, over the rings: (m, l) and o of each warp,
// then the CTA's own.  Rows of o are 8 floats longer than D, so that the eight
// rows of a fragment fall into different banks.
template <int D>
struct PagedMerge {
  static constexpr int PITCH = D + 8;
  static_assert((kPagedWarps + 1) * kPagedRows * (PITCH + 2) * 4 <=
                    paged_ring_bytes(D, kItemStages), "merge area");
  float2 *ml, *cta_ml;
  float *ov, *cta_ov;
  __device__ __forceinline__ explicit PagedMerge(uint8_t* smem) {
    ml = reinterpret_cast<float2*>(smem);
    cta_ml = ml + kPagedWarps * kPagedRows;
    ov = reinterpret_cast<float*>(cta_ml + kPagedRows);
    cta_ov = ov + kPagedWarps * kPagedRows * PITCH;
  }
  // Row r's column d over n parts (m, l, o): M, L and the sum.  A part without
  // keys has l = 0; l = NaN goes on whatever its m.
  template <int N>
  static __device__ __forceinline__ float sum(const float2 (&part)[N], const float (&o)[N],
                                              float& M, float& L) {
    M = part[0].x;
#pragma unroll
    for (int i = 1; i < N; ++i) M = fmaxf(M, part[i].x);
    const float mu = M == -INFINITY ? 0.f : M;
    float acc = 0.f;
    L = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float f =
          part[i].x == -INFINITY ? (part[i].y == 0.f ? 0.f : 1.f) : dec_exp2(part[i].x - mu);
      L = fmaf(f, part[i].y, L);
      acc = fmaf(f, o[i], acc);
    }
    return acc;
  }
  // Over the CTA's warps.
  __device__ __forceinline__ float warps(int r, int d, float& M, float& L) const {
    float2 part[kPagedWarps];
    float o[kPagedWarps];
#pragma unroll
    for (int w = 0; w < kPagedWarps; ++w) {
      part[w] = ml[w * kPagedRows + r];
      o[w] = ov[(w * kPagedRows + r) * PITCH + d];
    }
    return sum(part, o, M, L);
  }
  // Over the cluster's CTAs.
  __device__ __forceinline__ float ctas(int n, int r, int d, float& M, float& L) const {
    float2 part[8];
    float o[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      part[c] = float2{-INFINITY, 0.f};
      o[c] = 0.f;
      if (c < n) {
        part[c].x = dec_cluster_ld(&cta_ml[r].x, c);
        part[c].y = dec_cluster_ld(&cta_ml[r].y, c);
        o[c] = dec_cluster_ld(cta_ov + r * PITCH + d, c);
      }
    }
    return sum(part, o, M, L);
  }
};

// One more part (m, l) for a running (M, L): the factors of the two.  A part
// without keys has l = 0; l = NaN goes on whatever its m.
__device__ __forceinline__ void paged_join(float m, float l, float& M, float& L, float& fa,
                                           float& fb) {
  const float m_new = fmaxf(M, m), mu = m_new == -INFINITY ? 0.f : m_new;
  fa = exp2f(M - mu);
  fb = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2f(m - mu);
  M = m_new;
  L = fmaf(L, fa, fb * l);
}

// o and lse of row r (of tile r0), column d of item x.
__device__ __forceinline__ void paged_write(const PagedParams& p, const PagedPlace& x, int h,
                                            int gr, int d, float M, float L, float acc) {
  const int gh = gr / p.Tq, t = gr - gh * p.Tq;
  const long long hq = static_cast<long long>(h) * (p.rows / p.Tq) + gh;
  p.o[x.b * p.o_sb + hq * p.o_sh + t * p.o_st + d] =
      __float2bfloat16_rn(L == 0.f ? 0.f : acc / L);
  if (d == 0) p.lse[(x.b * static_cast<long long>(p.H) + hq) * p.Tq + t] = paged_lse(M, L);
}

// One item per thread-block cluster: for calls whose longest item is short, or
// whose items are few.  The warps of its CTAs take turns at its chunks; their
// results are joined in shared memory, the CTAs' in distributed shared memory.
// Nothing to scan, no workspace, one launch.  Grid: items * ctas in clusters of
// ctas.
template <int D, bool UP, bool MULTI>
__global__ void __launch_bounds__(kPagedThreads, UP && D == 128 ? 2 : 3)
    paged_item_kernel(const PagedParams p, int ctas) {
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  uint8_t* smem = pg_dynamic_smem();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int HT = p.Hkv * p.n_tiles, item = static_cast<int>(blockIdx.x) / ctas;
  const int rank = static_cast<int>(blockIdx.x) - item * ctas;
  PagedPlace x;
  x.b = item / HT;
  x.ht = item - x.b * HT;
  x.len = paged_length(p, x.b);
  x.n = paged_chunks<D>(p, x.len);
  x.c = rank * kPagedWarps + warp;
  const int step = ctas * kPagedWarps, h = x.ht / p.n_tiles;
  const int left = x.n > x.c ? (x.n - x.c + step - 1) / step : 0;
  PagedWarp<D, UP, MULTI, kItemStages> k(p, smem, warp, lane);
  // the first chunks' keys are looked up together, then one ahead
  PagedKey key[kItemStages], next{-1, -1, kPagedNone};
  auto look_up = [&](int i) {
    PagedPlace y = x;
    y.c = x.c + i * step;
    return k.look_up(y);
  };
#pragma unroll
  for (int i = 0; i < kItemStages; ++i) key[i] = look_up(i);
#pragma unroll
  for (int i = 0; i < kItemStages; ++i) {
    if (i < left) k.issue(x.ht, key[i], i);
    dec_cp_async_commit();
  }
  if (kItemStages < left) next = look_up(kItemStages);
  k.begin(x);
  int slot = 0;
  for (int i = 0; i < left; ++i) {
    dec_cp_async_wait<kItemStages - 1>();
    __syncwarp();  // every lane's pieces of the chunk are in shared memory
    k.chunk(slot, x.len);
    __syncwarp();  // every lane has read the slot: refill it
    if (i + kItemStages < left) {
      k.issue(x.ht, next, slot);
      if (i + kItemStages + 1 < left) next = look_up(i + kItemStages + 1);
    }
    dec_cp_async_commit();
    slot = slot + 1 == kItemStages ? 0 : slot + 1;
  }
  dec_cp_async_wait<0>();
  const PagedMerge<D> a(smem);
  __syncthreads();  // every warp is done with its ring
  k.store(a.ml + warp * kPagedRows, a.ov + warp * kPagedRows * a.PITCH, p.R, a.PITCH);
  __syncthreads();
  const int r0 = (x.ht - h * p.n_tiles) * kPagedRows;
  const int rows = p.rows - r0 < kPagedRows ? p.rows - r0 : kPagedRows;
  for (int i = tid; i < rows * D; i += kPagedThreads) {
    const int r = i / D, d = i - r * D;
    float M, L;
    const float acc = a.warps(r, d, M, L);
    if (ctas == 1) {
      paged_write(p, x, h, r0 + r, d, M, L, acc);
    } else {
      a.cta_ov[r * a.PITCH + d] = acc;
      if (d == 0) a.cta_ml[r] = float2{M, L};
    }
  }
  if (ctas == 1) return;
  dec_cluster_sync();  // every CTA's part is in its shared memory
  for (int i = rank * kPagedThreads + tid; i < rows * D; i += ctas * kPagedThreads) {
    const int r = i / D, d = i - r * D;
    float M, L;
    const float acc = a.ctas(ctas, r, d, M, L);
    paged_write(p, x, h, r0 + r, d, M, L, acc);
  }
  dec_cluster_sync();  // no CTA leaves while its shared memory is read
}

// Grid: up to kPagedMaxCtas CTAs of kPagedThreads.
//
// A CTA takes an even share of the flat axis.  If all of it lies in one item
// the warps take turns at its chunks and join their results in shared
// memory; otherwise each takes a quarter of the share.  Where the table has
// room for long requests: 726 MB of K and V (64 x 8 heads x 2,770 keys of 128)
// in 127 us with the merge, 2.9 GB in 458 us (6.3 TB/s).
template <int D, bool UP, bool MULTI>
__global__ void __launch_bounds__(kPagedThreads, 2) paged_decode_kernel(const PagedParams p) {
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  uint8_t* smem = pg_dynamic_smem();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* pre = reinterpret_cast<int*>(smem + paged_ring_bytes(D, kPagedStages)) +
             kPagedWarps * kPagedStages * 32;
  int* totals = pre + kPagedThreads;
  const int HT = p.Hkv * p.n_tiles;

  // prefix sums of the requests' chunks, nb requests per thread
  const int nb = (p.B + kPagedThreads - 1) / kPagedThreads;
  int mine = 0;
  for (int i = 0; i < nb; ++i) {
    const int b = tid * nb + i;
    if (b < p.B) mine += paged_chunks<D>(p, paged_length(p, b)) + paged_item_cost(D);
  }
  const int incl = warp_scan(mine, lane);
  if (lane == 31) totals[warp] = incl;
  __syncthreads();
  int before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kPagedWarps; ++w) {
    if (w < warp) before += totals[w];
    total += totals[w];
  }
  pre[tid] = before;
  __syncthreads();

  // this CTA's share [S, E) of the flat axis
  const long long W = static_cast<long long>(total) * HT;
  long long nc = (W + kPagedMinRun * kPagedWarps - 1) / (kPagedMinRun * kPagedWarps);
  if (nc > gridDim.x) nc = gridDim.x;
  const int cta = static_cast<int>(blockIdx.x), gw = cta * kPagedWarps + warp;
  if (cta >= nc) {
    if (lane == 0) p.cuts[gw] = PagedCut{0, 0, 0, 0};
    return;
  }
  const long long S = cta * W / nc, E = (cta + 1) * W / nc;
  const int share = static_cast<int>(E - S);
  PagedPlace use = paged_locate<D>(p, HT, nb, pre, S, lane);
  const bool together = use.c + share <= use.n;  // one item's
  // its first place that is a chunk, and how many of them
  PagedPlace first = use;
  if (first.c < 0) first.c = 0;
  const int chunks = use.c + share - first.c;
  // this warp's places: `units` of them up to flat place e (together: turns)
  long long e = E;
  int units = share;
  if (together) {
    use.c = first.c + warp;
    units = chunks > warp ? (chunks - warp + kPagedWarps - 1) / kPagedWarps : 0;
  } else {
    const long long s = S + static_cast<long long>(warp) * share / kPagedWarps;
    e = S + static_cast<long long>(warp + 1) * share / kPagedWarps;
    units = static_cast<int>(e - s);
    if (units > 0) use = paged_locate<D>(p, HT, nb, pre, s, lane);
    if (use.c < 0) {
      units += use.c;
      use.c = 0;
    }
  }
  // the cut of an item that begins in this warp and ends with flat place x
  auto cut_to = [&](const PagedPlace& item, long long x) {
    if (x >= W) x = W - 1;
    const long long c = ((x + 1) * nc - 1) / W, cs = c * W / nc, ce = (c + 1) * W / nc;
    // the last warp that holds some of it; only the first if all of c's share is the item's
    const int w = static_cast<int>(((x - cs + 1) * kPagedWarps - 1) / (ce - cs));
    const int last = c > cta && x == ce - 1 ? 0 : w;
    const int n_same = together ? 0 : c > cta ? kPagedWarps - 1 - warp : w - warp;
    const int n_mid = c > cta ? static_cast<int>(c) - cta - 1 : 0;
    return PagedCut{item.b, item.ht, 1 + n_same + n_mid + (c > cta ? last + 1 : 0),
                    4 * n_mid + n_same};
  };

  PagedWarp<D, UP, MULTI, kPagedStages> k(p, smem, warp, lane);
  const bool none = units <= 0;
  PagedPlace get = use;
  int ahead = units;  // the places from `get` on
  PagedKey key[kPagedStages], next{-1, -1, kPagedNone};
  int hts[kPagedStages], next_ht = 0;
  auto on = [&](PagedPlace& x, int& left) {
    if (together) {
      x.c += kPagedWarps;
      --left;
    } else {
      paged_next<D>(p, HT, x, left);
    }
  };
  auto look_up = [&](PagedKey& to, int& ht) {  // the next chunk's keys, and on to the one behind
    if (ahead <= 0) return false;
    to = k.look_up(get);
    ht = get.ht;
    on(get, ahead);
    return true;
  };
  // the first chunks' keys are looked up together, then one ahead; one commit
  // group per ring slot, empty when the run is shorter
  bool there[kPagedStages];
#pragma unroll
  for (int i = 0; i < kPagedStages; ++i) there[i] = look_up(key[i], hts[i]);
#pragma unroll
  for (int i = 0; i < kPagedStages; ++i) {
    if (there[i]) k.issue(hts[i], key[i], i);
    dec_cp_async_commit();
  }
  bool more = look_up(next, next_ht);

  bool begins = use.c == 0;  // the current item's first chunk is this warp's
  bool fresh = true;
  PagedCut cut{0, 0, 0, 0};
  int slot = 0;
  while (units > 0) {
    if (fresh) {
      fresh = false;
      k.begin(use);
    }
    dec_cp_async_wait<kPagedStages - 1>();
    __syncwarp();  // every lane's pieces of the chunk are in shared memory
    k.chunk(slot, use.len);
    __syncwarp();  // every lane has read the slot: refill it
    if (more) {
      k.issue(next_ht, next, slot);
      more = look_up(next, next_ht);
    }
    dec_cp_async_commit();
    slot = slot + 1 == kPagedStages ? 0 : slot + 1;
    const PagedPlace done = use;
    const long long at = e - units;  // its flat place
    on(use, units);
    if (together) continue;
    const bool ends = done.c + 1 == done.n;
    if (ends || units <= 0) {
      if (ends && begins) {
        k.finish(done);
      } else {
        const long long part = (2LL * gw + begins) * p.R;
        k.store(p.part_ml + part, p.part_o + part * D, p.R, D);
      }
      if (begins && !ends)  // cut here: the warps that hold its other chunks
        cut = cut_to(done, at + (done.n - 1 - done.c));
      begins = true;
      fresh = true;
    }
  }
  dec_cp_async_wait<0>();

  if (together && chunks > 0) {
    const bool whole = first.c == 0 && chunks == first.n;
    const PagedMerge<D> a(smem);
    __syncthreads();  // every warp is done with its ring
    k.store(a.ml + warp * kPagedRows, a.ov + warp * kPagedRows * a.PITCH, p.R, a.PITCH);
    __syncthreads();
    const int h = first.ht / p.n_tiles, r0 = (first.ht - h * p.n_tiles) * kPagedRows;
    const int rows = p.rows - r0 < kPagedRows ? p.rows - r0 : kPagedRows;
    const long long part = (2LL * cta * kPagedWarps + (first.c == 0)) * p.R;
    for (int i = tid; i < rows * D && first.b < p.B; i += kPagedThreads) {
      const int r = i / D, d = i - r * D;
      float M, L;
      const float acc = a.warps(r, d, M, L);
      if (whole) {
        paged_write(p, first, h, r0 + r, d, M, L, acc);
      } else {
        p.part_o[(part + r) * D + d] = acc;
        if (d == 0) p.part_ml[part + r] = float2{M, L};
      }
    }
    if (warp == 0 && first.c == 0 && !whole)
      cut = cut_to(first, E - chunks + first.n - 1);
  }
  // nothing in slot 0 of a warp without chunks
  if (!together && none)
    if (lane < p.R) p.part_ml[2LL * gw * p.R + lane] = float2{-INFINITY, 0.f};
  if (lane == 0) p.cuts[gw] = cut;
}

// CTAs per item of paged_item_kernel, or 0 for paged_decode_kernel, from the
// items and the chunks that the table (the list) has room for; the lengths are
// not known here.  As many CTAs as are resident at once (128 items of 2,048
// listed keys of 128: 37.9, 31.6 and 42.8 us with 2, 3 and 4); then the item
// kernel where no warp has more than 12 chunks (those: 38.6 us for the other
// kernel; 16 x 12 heads x 1,024 keys of 64: 14.1, 20.8; 4 x 8 x 2,048 of 128:
// 12.6, 17.2), the other one for longer items, whose lengths may differ more
// (32 x 8 x 100 to 1,000 keys of 128: 24.4, 22.4; 2 x 16 x 8,192: 33.1, 32.2).
__host__ __device__ constexpr int paged_item_ctas(long long items, long long chunks) {
  long long ctas = kItemSlots / items, most = (chunks + kPagedWarps - 1) / kPagedWarps;
  if (ctas > 8) ctas = 8;
  if (ctas > most) ctas = most;
  if (ctas < 1) ctas = 1;
  return items * ctas <= 2 * kItemSlots && chunks <= 12 * kPagedWarps * ctas
             ? static_cast<int>(ctas) : 0;
}

// Joins the parts of the cut items:  M = max m_i,
//   o = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
// Grid: (CTAs of paged_decode_kernel) * n_y; CTA (c, y) takes rows y, y + n_y,
// ... of the items that begin in CTA c's warps.  A team of warps takes a row
// of an item, each four parts at a time.  Latency is all that counts here, and
// part of it is the fetch of the code itself: the kernel is kept small, and
// its registers few, so that it is resident before the last CTA ends.
template <int D>
__global__ void __launch_bounds__(kMergeThreads, 2) paged_merge_kernel(const PagedParams p, int n_y) {
  constexpr int NW = kMergeThreads / 32;
  constexpr int VEC = D >= 128 ? 4 : D >= 64 ? 2 : 1;  // columns of a lane
  constexpr int ILP = 4;                               // parts in flight
  dec_grid_dep_wait();
  dec_grid_dep_launch();
  float* sh = reinterpret_cast<float*>(dec_dynamic_smem());  // [NW][2 + D]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = static_cast<int>(blockIdx.x) / n_y, y = static_cast<int>(blockIdx.x) - cta * n_y;
  // lanes 0 .. 3 read the cuts of the CTA's warps
  PagedCut mine = lane < kPagedWarps ? p.cuts[cta * kPagedWarps + lane] : PagedCut{0, 0, 0, 0};
  const unsigned begun = dec_ballot(mine.n_parts > 0);
  if (begun == 0u) return;
  const int per_y = (p.R - y + n_y - 1) / n_y;  // rows of an item for this CTA
  const int units = dec_popc(begun) * per_y;
  int team = NW;                                // warps per (item, row)
  while (team > 1 && team * units > NW) team /= 2;
  const int k = warp & (team - 1);
  const bool has = lane * VEC < D;
#pragma unroll 1
  for (int base = 0; base < units; base += NW / team) {
    const int unit = base + warp / team, nth = unit / per_y, row = y + (unit - nth * per_y) * n_y;
    unsigned left = begun;
    for (int i = 0; i < nth; ++i) left &= left - 1u;
    const int w = left != 0u ? dec_lowest(left) : 0, gw = cta * kPagedWarps + w;
    PagedCut c;
    c.b = dec_shfl(mine.b, w);
    c.ht = dec_shfl(mine.ht, w);
    c.n_parts = dec_shfl(mine.n_parts, w);
    c.where = dec_shfl(mine.where, w);
    const int h = c.ht / p.n_tiles, gr = (c.ht - h * p.n_tiles) * kPagedRows + row;
    const bool in = unit < units && gr < p.rows;
    float M = -INFINITY, L = 0.f, acc[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) acc[v] = 0.f;
#pragma unroll 1
    for (int i = k; in && i < c.n_parts; i += ILP * team) {
      float2 ml[ILP];
      float x[ILP][VEC];
#pragma unroll
      for (int u = 0; u < ILP; ++u) {
        const bool there = i + u * team < c.n_parts;
        const long long at = c.slot(gw, there ? i + u * team : 0) * p.R + row;
        ml[u] = p.part_ml[at];
        if (!there) ml[u] = float2{-INFINITY, 0.f};
#pragma unroll
        for (int v = 0; v < VEC; ++v) x[u][v] = has ? p.part_o[at * D + lane * VEC + v] : 0.f;
      }
      float m = M;
#pragma unroll
      for (int u = 0; u < ILP; ++u) m = fmaxf(m, ml[u].x);
      const float mu = m == -INFINITY ? 0.f : m, fa = dec_exp2(M - mu);
      M = m;
      L *= fa;
#pragma unroll
      for (int v = 0; v < VEC; ++v) acc[v] *= fa;
#pragma unroll
      for (int u = 0; u < ILP; ++u) {
        const bool empty = ml[u].y == 0.f;  // (its o may not have been written; a NaN goes on)
        const float f = empty ? 0.f : ml[u].x == -INFINITY ? 1.f : dec_exp2(ml[u].x - mu);
        L = fmaf(f, ml[u].y, L);
#pragma unroll
        for (int v = 0; v < VEC; ++v) acc[v] = fmaf(f, empty ? 0.f : x[u][v], acc[v]);
      }
    }
    if (team > 1) {
      if (in && k > 0) {
        float* to = sh + warp * (2 + D);
        to[0] = M;
        to[1] = L;
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          if (has) to[2 + lane * VEC + v] = acc[v];
      }
      __syncthreads();
#pragma unroll 1
      for (int j = 1; in && k == 0 && j < team; ++j) {
        const float* from = sh + (warp + j) * (2 + D);
        float fa, fb;
        paged_join(from[0], from[1], M, L, fa, fb);
#pragma unroll
        for (int v = 0; v < VEC; ++v)
          acc[v] = fmaf(acc[v], fa, has ? fb * from[2 + lane * VEC + v] : 0.f);
      }
    }
    if (in && k == 0) {
      const int gh = gr / p.Tq, t = gr - gh * p.Tq;
      const long long hq = static_cast<long long>(h) * (p.H / p.Hkv) + gh;
      __nv_bfloat16* ob = p.o + c.b * p.o_sb + hq * p.o_sh + t * p.o_st;
      const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        if (has) ob[lane * VEC + v] = __float2bfloat16_rn(acc[v] * inv);
      if (lane == 0)
        p.lse[(c.b * static_cast<long long>(p.H) + hq) * p.Tq + t] = paged_lse(M, L);
    }
    if (team > 1) __syncthreads();
  }
}

__host__ __device__ constexpr int paged_merge_smem_bytes(int D) {
  return kMergeThreads / 32 * (2 + D) * 4;
}
// CTAs of the merge per CTA of the decode: four rows of an item each.
__host__ __device__ constexpr int paged_merge_y(int R) { return (R + 3) / 4; }

}  // namespace cattn
