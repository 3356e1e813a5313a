// The paged KV cache: bookkeeping of pages (reserving, forking, giving back, compacting) and the copies of rows that go
// with it (writing new rows, accepting drafted ones, pages copied on write or moved).
//
// The bookkeeping is integer work on a few KB and bound by latency: one CTA, or one per sequence or block of columns,
// and no value that depends on the order of atomics (counts only; which page goes where follows from prefix sums).  The
// copies are bound by memory: 16 bytes a thread, eight loads in flight, nothing staged.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "qevict.h"
#include "sm_count.h"

namespace qv {
namespace {

constexpr int PG_BATCH = 1024;   // sequences of a cache: a thread each where one CTA plans for all
constexpr int PG_PATH = 256;     // accepted rows of a sequence
constexpr int PG_HEADER = 64;    // int32 in front of the arrays

struct PagesDev {
  uint16_t *k, *v;
  int64_t sk[4], sv[4];          // layer, page, token, head
  int layers, pages, page, lg, h_kv, batch, max_pages, words;   // lg: log2 page; words: of the free bits, a multiple of 4
  int *status, *n_free, *moves, *n_copies;
  unsigned long long *drawn;     // units of a copy given out
  int *length, *held, *table, *refs;
  uint32_t *bits;
  int *tickets;                  // [batch + 1] CTAs that have read what the last one changes; 0 between calls
  int4 *copies;                  // [batch] of a reserve: page, its copy, rows to copy
  int *from, *to, *goes;         // [pages] of a compaction: r-th page that moves, its new place; new place of each
};

// (Programmatic launches: a kernel's setup overlaps the end of the one before.  Nothing is read before the wait, and the
// next kernel is let in only behind it.)
__device__ __forceinline__ void pages_begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Tokens of a sequence, whatever stands in the arrays: within the pages that it holds.
__device__ __forceinline__ int held_of(const PagesDev &P, int b) { return min(max(P.held[b], 0), P.max_pages); }
__device__ __forceinline__ int length_of(const PagesDev &P, int b, int held) { return min(max(P.length[b], 0), held << P.lg); }
__device__ __forceinline__ bool is_page(const PagesDev &P, int p) { return (unsigned)p < (unsigned)P.pages; }
__device__ __forceinline__ int *row_of(const PagesDev &P, int b) { return P.table + (int64_t)b * P.max_pages; }

// One table entry of page p less.  True: it was the last, and the page is free now.
__device__ __forceinline__ bool give_back(const PagesDev &P, int p) {
  if (atomicSub(&P.refs[p], 1) != 1) return false;
  atomicOr(&P.bits[p >> 5], 1u << (p & 31));
  return true;
}

// Exclusive sums of x and y over a CTA of 32 warps, and their totals, the same for every thread.  Two barriers.
struct Sums {
  int x, y, all_x, all_y;
};
__device__ __forceinline__ Sums scan_1024(int x, int y, int2 *warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sx = x, sy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ux = __shfl_up_sync(0xffffffffu, sx, o), uy = __shfl_up_sync(0xffffffffu, sy, o);
    if (lane >= o) sx += ux, sy += uy;
  }
  __syncthreads();   // what stood in warps has been read
  if (lane == 31) warps[warp] = make_int2(sx, sy);
  __syncthreads();
  const int2 w = warps[lane];
  Sums S;
  S.x = __reduce_add_sync(0xffffffffu, lane < warp ? w.x : 0) + sx - x;
  S.y = __reduce_add_sync(0xffffffffu, lane < warp ? w.y : 0) + sy - y;
  S.all_x = __reduce_add_sync(0xffffffffu, w.x);
  S.all_y = __reduce_add_sync(0xffffffffu, w.y);
  return S;
}

// ----------------------------------------------------------------------------- start

__global__ void pages_clear_kernel(PagesDev P) {
  pages_begin();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < PG_HEADER) P.status[i] = 0;
  if (i <= P.batch) P.tickets[i] = 0;
  if (i < P.pages) {
    P.refs[i] = 0;
    P.goes[i] = -1;   // here: the place in the tables where the page was first seen
  }
}

__global__ void pages_adopt_kernel(PagesDev P, const int *table, const int *length) {
  __shared__ int first_none;
  pages_begin();
  const int b = blockIdx.x;
  const int *src = table ? table + (int64_t)b * P.max_pages : nullptr;
  if (threadIdx.x == 0) first_none = P.max_pages;
  __syncthreads();
  if (table)
    for (int c = threadIdx.x; c < P.max_pages; c += blockDim.x)
      if (!is_page(P, src[c])) {
        atomicMin(&first_none, c);
        break;   // this thread's later ones lie behind it
      }
  __syncthreads();
  const int held = table ? first_none : 0;
  int *dst = row_of(P, b);
  for (int c = threadIdx.x; c < P.max_pages; c += blockDim.x) {
    const int p = table ? src[c] : -1;
    dst[c] = c < held ? p : -1;
    if (c < held) {
      atomicAdd(&P.refs[p], 1);
      const int seen = atomicCAS(&P.goes[p], -1, c);
      if (seen != -1 && seen != c) atomicOr(P.status, QV_ERR_STATE);
    } else if (c == held && p != -1) {
      atomicOr(P.status, QV_ERR_BOUNDS);
    }
  }
  if (threadIdx.x == 0) {
    const int n = length ? length[b] : 0, fit = min(max(n, 0), held << P.lg);
    if (n != fit) atomicOr(P.status, QV_ERR_BOUNDS);
    P.length[b] = fit;
    P.held[b] = held;
  }
}

__global__ void pages_free_bits_kernel(PagesDev P) {
  pages_begin();
  const int w = blockIdx.x * blockDim.x + threadIdx.x;
  uint32_t x = 0;
  for (int i = 0; i < 32 && w * 32 + i < P.pages; ++i)
    if (P.refs[w * 32 + i] == 0) x |= 1u << i;
  if (w < P.words) P.bits[w] = x;
  const int n = __reduce_add_sync(0xffffffffu, __popc(x));
  if ((threadIdx.x & 31) == 0 && n) atomicAdd(P.n_free, n);
}

// ----------------------------------------------------------------------------- rows

// A part (of PART_PIECES pieces of 16 bytes) of the first `rows` rows of page a, copied to page z by a CTA of 256 threads.
// DENSE: rows follow one another, so that one address and eight offsets do.
constexpr int PART_PIECES = 2048;
template <bool DENSE>
__device__ __forceinline__ void copy_part(uint16_t *pool, const int64_t (&st)[4], int layer, int a, int z, int rows, int h_kv,
                                          int part) {
  const int n = rows * h_kv * 16, x = part * PART_PIECES + threadIdx.x;
  const uint16_t *src = pool + layer * st[0] + a * st[1];
  uint16_t *dst = pool + layer * st[0] + z * st[1];
  auto place = [&](auto *page, int i) {   // of piece x + 256 i: (row, head, 16th of the channels)
    if (DENSE) return page + (int64_t)x * 8 + i * (256 * 8);
    const uint32_t y = x + i * 256, h = y >> 4, r = h / (uint32_t)h_kv;
    return page + r * st[2] + (h - r * h_kv) * st[3] + (y & 15) * 8;
  };
  uint4 w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (x + i * 256 < n) w[i] = *reinterpret_cast<const uint4 *>(place(src, i));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (x + i * 256 < n) *reinterpret_cast<uint4 *>(place(dst, i)) = w[i];
}

// n copies drawn by the CTAs: a unit is a part of one copy's page in one layer, keys or values.  (In fixed turns CTAs
// far from the memory at hand end last: 64 samples of 4 prompts 84 us, drawn 70.  A unit a CTA does as well, but a grid for the
// most copies possible costs a step without any 1 us a thousand CTAs.)
template <bool DENSE, typename Copy>
__device__ __forceinline__ void copy_all(const PagesDev &P, int n, const Copy &copy) {
  __shared__ unsigned long long next[2];
  const int parts = (P.page * P.h_kv * 16 + PART_PIECES - 1) / PART_PIECES, per = parts * 2 * P.layers;
  const unsigned long long units = (unsigned long long)n * per;
  int turn = 0;
  for (unsigned long long u = blockIdx.x; u < units; turn ^= 1) {
    if (threadIdx.x == 0) next[turn] = gridDim.x + atomicAdd(P.drawn, 1ull);
    const int r = (int)(u / per), y = (int)(u - (unsigned long long)r * per), l2 = y / parts, part = y - l2 * parts;
    const int4 c = copy(r);
    if (l2 & 1)
      copy_part<DENSE>(P.v, P.sv, l2 >> 1, c.x, c.y, c.z, P.h_kv, part);
    else
      copy_part<DENSE>(P.k, P.sk, l2 >> 1, c.x, c.y, c.z, P.h_kv, part);
    __syncthreads();
    u = next[turn];
  }
}

struct RowsDev {
  const uint16_t *k, *v;
  int64_t sk[4], sv[4];          // layer, sequence, token, head
  int layer, layers, n;
  const int *d_n;
};

// New rows: a CTA takes 4 pieces a thread of one (layer, sequence), keys and values, so eight loads are in flight.  Bound by
// memory: 4099 + 3075 rows of 8 heads in 8 layers 71 us (6.6 TB/s; with addresses kept over the loads, 90 registers, 81).
constexpr int APPEND_THREADS = 256, APPEND_PIECES = 4;
__global__ void __launch_bounds__(APPEND_THREADS, 4) pages_append_kernel(const __grid_constant__ PagesDev P,
                                                                        const __grid_constant__ RowsDev R) {
  pages_begin();
  const int b = blockIdx.y, held = held_of(P, b), len = length_of(P, b, held);
  int n = R.n;
  if (R.d_n) {
    const int want = R.d_n[b];
    n = min(max(want, 0), R.n);
    if (want != n && threadIdx.x == 0 && blockIdx.x == 0) atomicOr(P.status, QV_ERR_BOUNDS);
  }
  const int *row = row_of(P, b);
  const uint32_t per_row = (uint32_t)P.h_kv * 16, all = (uint32_t)n * per_row;
  const uint32_t x0 = blockIdx.x * (APPEND_THREADS * APPEND_PIECES) + threadIdx.x;
  if (x0 >= all) return;
  for (int l = blockIdx.z; l < R.layers; l += gridDim.z) {
    uint4 wk[APPEND_PIECES], wv[APPEND_PIECES];
    int to[APPEND_PIECES];   // page << 7 | row; -1: nowhere
#pragma unroll
    for (int i = 0; i < APPEND_PIECES; ++i) {
      const uint32_t x = x0 + i * APPEND_THREADS;
      to[i] = -1;
      if (x >= all) continue;
      const uint32_t t = x / per_row, y = x - t * per_row, h = y >> 4, c = (y & 15) * 8;
      wk[i] = *reinterpret_cast<const uint4 *>(R.k + l * R.sk[0] + b * R.sk[1] + t * R.sk[2] + h * R.sk[3] + c);
      wv[i] = *reinterpret_cast<const uint4 *>(R.v + l * R.sv[0] + b * R.sv[1] + t * R.sv[2] + h * R.sv[3] + c);
      const int64_t pos = (int64_t)len + t;
      const int pg = pos < (int64_t)held << P.lg ? row[pos >> P.lg] : -1;
      if (is_page(P, pg) && P.refs[pg] == 1)
        to[i] = pg << 7 | ((int)pos & (P.page - 1));
      else if (y == 0)
        atomicOr(P.status, QV_ERR_BOUNDS);
    }
    uint16_t *k = P.k + (R.layer + l) * P.sk[0], *v = P.v + (R.layer + l) * P.sv[0];
#pragma unroll
    for (int i = 0; i < APPEND_PIECES; ++i) {
      if (to[i] < 0) continue;
      const uint32_t y = (x0 + i * APPEND_THREADS) % per_row, h = y >> 4, c = (y & 15) * 8;
      const int pg = to[i] >> 7, off = to[i] & 127;
      *reinterpret_cast<uint4 *>(k + pg * P.sk[1] + off * P.sk[2] + h * P.sk[3] + c) = wk[i];
      *reinterpret_cast<uint4 *>(v + pg * P.sv[1] + off * P.sv[2] + h * P.sv[3] + c) = wv[i];
    }
  }
}

// Accepted rows move down their sequence.  A thread owns 16 bytes of every row of one (layer, K or V, head) and moves them in
// ascending order, eight rows at a time, all loads before the stores: row path[j] >= j, so a row is read before anything
// lands on it, and no other thread touches these bytes.  The sequence's last CTA to have read its length counts the rows in.
// Bound by the chain from lengths over path and table to the rows (4 sequences in 32 layers 3 us), then by memory in
// pieces of a row: 256 sequences in 8 layers 14 us, 4.2 TB/s (17 with places worked out by every thread; 16 with keys and
// values by one thread, sixteen loads in flight).  The counts of the pages written to are looked up while the first rows
// are on their way.
__global__ void __launch_bounds__(256) pages_accept_kernel(const __grid_constant__ PagesDev P, const int *d_count,
                                                          const int *d_path, int max_path) {
  __shared__ int64_t s_from[2][PG_PATH], s_to[2][PG_PATH];   // places of the rows that move, keys and values
  __shared__ int s_moved[8], last;
  pages_begin();
  const int b = blockIdx.y, j = threadIdx.x, held = held_of(P, b), len = length_of(P, b, held), count = d_count[b];
  const int *row = row_of(P, b);
  const int64_t room = (int64_t)held << P.lg;
  int at = -1, before = -1;
  if (d_path && j < max_path) {
    const int *path = d_path + (int64_t)b * max_path;
    at = path[j];
    if (j) before = path[j - 1];
  }
  const bool fits = count >= 0 && (!d_path || count <= max_path) && (int64_t)len + count <= room;
  bool ok = fits, moves = false;
  int src = -1, dst = -1;
  if (fits && d_path && j < count) {
    ok = at > before && at >= 0 && (int64_t)len + at < room;
    src = ok ? row[(len + at) >> P.lg] : -1;
    dst = row[(len + j) >> P.lg];
    ok = ok && is_page(P, src) && is_page(P, dst);
    moves = ok && at != j;
    if (ok) ok = P.refs[dst] == 1;   // rows of shared pages are never written
  } else if (fits && !d_path && count > 0) {   // (no row: the last page may stay another's too)
    for (int c = (len >> P.lg) + j; (int64_t)c << P.lg < (int64_t)len + count; c += blockDim.x)
      if (!is_page(P, row[c]) || P.refs[row[c]] != 1) ok = false;
  }
  auto settle = [&]() {   // whether the sequence's rows may move, and what follows for its length
    ok = __syncthreads_and(ok);
    if (threadIdx.x == 0) {
      last = gridDim.x == 1;
      if (!last) {
        __threadfence();
        last = atomicAdd(&P.tickets[b], 1) == (int)gridDim.x - 1;
        if (last) P.tickets[b] = 0;
      }
      if (last && !ok) atomicOr(P.status, QV_ERR_BOUNDS);
      if (last && ok) P.length[b] = len + count;
    }
    return ok;
  };
  const uint32_t here = __ballot_sync(0xffffffffu, moves);
  if ((j & 31) == 0) s_moved[j >> 5] = __popc(here);
  __syncthreads();
  int n = 0, mine = __popc(here & ((1u << (j & 31)) - 1));   // rows that move, and those in front of this one
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < j >> 5) mine += s_moved[w];
    n += s_moved[w];
  }
  if (n == 0) {
    settle();
    return;
  }
  if (moves) {
    const int a = (len + at) & (P.page - 1), z = (len + j) & (P.page - 1);
    s_from[0][mine] = src * P.sk[1] + a * P.sk[2], s_from[1][mine] = src * P.sv[1] + a * P.sv[2];
    s_to[0][mine] = dst * P.sk[1] + z * P.sk[2], s_to[1][mine] = dst * P.sv[1] + z * P.sv[2];
  }
  __syncthreads();
  const uint32_t all = 2u * P.layers * P.h_kv * 16;
  bool settled = false;
  for (uint32_t x0 = blockIdx.x * 256; x0 < all; x0 += gridDim.x * 256) {
    const uint32_t x = min(x0 + threadIdx.x, all - 1), h = x >> 4, l2 = h / (uint32_t)P.h_kv, is_v = l2 & 1;
    const bool in = x0 + threadIdx.x < all;
    uint16_t *pool = is_v ? P.v : P.k;
    pool += (l2 >> 1) * (is_v ? P.sv[0] : P.sk[0]) + (h - l2 * P.h_kv) * (is_v ? P.sv[3] : P.sk[3]) + (x & 15) * 8;
    for (int i0 = 0; i0 < n; i0 += 8) {
      uint4 w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (in && i0 + i < n) w[i] = *reinterpret_cast<const uint4 *>(pool + s_from[is_v][i0 + i]);
      if (!settled && !settle()) return;
      settled = true;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (in && i0 + i < n) *reinterpret_cast<uint4 *>(pool + s_to[is_v][i0 + i]) = w[i];
    }
  }
}

// ----------------------------------------------------------------------------- pages

// Who needs which pages, a thread a sequence; then the free bits are walked from the lowest page on, a word a thread, and
// the r-th free page goes to whom the running sum of needs says, a thread a page: it finds word and sequence by their sums.
// Nothing is written before the pages are known to suffice.  Held pages behind a sequence's tokens that the rows reach and that
// stand in other sequences too (a loaded table, a length written back) are given back first: each thread looks at the first
// OWN pages from its sequence's last token on, the CTA at the others (16 sequences that hold 8 pages in advance 4 us, 1100
// pages 11.5).  Bound by latency: lengths, table, counts in a chain of
// loads, then a few barriers for every 32768 pages: 2.5 us with the copying kernel where nothing is needed, 5 for 16
// sequences of 33K tokens that grow.  (A thread that hands out all pages of its 128 bits took 30 us for 64 samples of 4 prompts.)
constexpr int OWN = 3;   // a step of a few rows reaches no more
__global__ void __launch_bounds__(1024, 1) pages_reserve_kernel(const __grid_constant__ PagesDev P, const int *d_new, int n_new) {
  __shared__ int s_tail[PG_BATCH], s_start[PG_BATCH], s_len[PG_BATCH], s_held[PG_BATCH], s_copy[PG_BATCH], s_rank[1024];
  __shared__ uint32_t s_word[1024];
  __shared__ int2 s_warp[32];
  pages_begin();
  const int t = threadIdx.x;
  uint32_t word = t < P.words ? P.bits[t] : 0u;
  const int n_free = *P.n_free;
  int len = 0, held = 0, keep = 0, want = 0, tail = -1, refs = 0;   // keep: held pages that it goes on with
  int lo = 0, hi = 0;   // those that the CTA looks at
  bool bad = false;
  if (t < P.batch) {
    held = keep = held_of(P, t);
    len = length_of(P, t, held);
    const int64_t n = d_new ? d_new[t] : n_new, up = (len + n + P.page - 1) >> P.lg;
    bad = n < 0 || up > P.max_pages;
    if (!bad && n > 0) {
      want = (int)up;
      const int *row = row_of(P, t), c0 = len >> P.lg, reach = min(want, held);
      const bool part = len & (P.page - 1);   // page c0 holds tokens
      int entry[OWN], holders[OWN];
#pragma unroll
      for (int i = 0; i < OWN; ++i) entry[i] = c0 + i < reach ? row[c0 + i] : -1;
#pragma unroll
      for (int i = 0; i < OWN; ++i) holders[i] = is_page(P, entry[i]) ? P.refs[entry[i]] : 0;
      if (part) tail = entry[0], refs = holders[0], bad = !is_page(P, tail);
#pragma unroll
      for (int i = OWN - 1; i >= 0; --i)
        if (holders[i] > 1 && (i > 0 || !part)) keep = c0 + i;
      if (keep == held) lo = c0 + OWN, hi = reach;
    }
    s_len[t] = len, s_held[t] = keep;
  }
  s_tail[t] = tail;
  if (t == 0) *P.n_copies = 0, *P.drawn = 0;
  bool rare = __syncthreads_or(bad || lo < hi || keep < held);   // one barrier for a step without any of them
  if (__builtin_expect(rare, false) && __syncthreads_or(bad)) {
    if (t == 0) atomicOr(P.status, QV_ERR_BOUNDS);
    return;
  }
  auto owner = [&](int r) {   // the last sequence that starts at r or before: it has some
    int a = 0, z = P.batch - 1;
    while (a < z) {
      const int mid = (a + z + 1) >> 1;
      if (s_start[mid] <= r)
        a = mid;
      else
        z = mid - 1;
    }
    return a;
  };
  if (__builtin_expect(rare, false) && __syncthreads_or(lo < hi)) {
    const Sums at = scan_1024(max(hi - lo, 0), 0, s_warp);
    if (t < P.batch) s_start[t] = at.x, s_copy[t] = lo;
    __syncthreads();
    for (int r = t; r < at.all_x; r += 4 * 1024) {
      int b[4], c[4], p[4], n[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = -1;
        if (r + i * 1024 >= at.all_x) continue;
        b[i] = owner(r + i * 1024), c[i] = s_copy[b[i]] + r + i * 1024 - s_start[b[i]];
        p[i] = row_of(P, b[i])[c[i]];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] = is_page(P, p[i]) ? P.refs[p[i]] : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n[i] > 1) atomicMin(&s_held[b[i]], c[i]);
    }
    __syncthreads();
    if (t < P.batch) keep = s_held[t];
  }
  if (__builtin_expect(rare, false)) rare = __syncthreads_or(keep < held);   // some give pages back
  const int add = max(want - keep, 0);
  bool copy = false;
  // Shared pages: how many that reserve now hold each, and is this the first of them.  A look at every other sequence costs
  // 8 of them 0.6 us less than counts in memory, 256 the same, 1024 30 us more.
  if (P.batch <= 256) {
    int same = 0, before = 0;
    if (refs > 1) {
#pragma unroll 8
      for (int j = 0; j < P.batch; ++j)
        if (s_tail[j] == tail) {
          ++same;
          before += j < t;
        }
      copy = same < refs || before > 0;
    }
  } else if (__syncthreads_or(refs > 1)) {
    if (refs > 1) P.goes[tail] = P.batch, P.to[tail] = 0;   // (scratch of a compaction)
    __syncthreads();
    if (refs > 1) {
      atomicMin(&P.goes[tail], t);
      atomicAdd(&P.to[tail], 1);
    }
    __syncthreads();
    if (refs > 1) copy = __ldcg(&P.to[tail]) < refs || __ldcg(&P.goes[tail]) < t;
  }
  const Sums need = scan_1024(add + copy, copy, s_warp);
  const int total = need.all_x;
  if (total > n_free) {
    if (t == 0) atomicOr(P.status, QV_ERR_SLOT);
    return;
  }
  if (total == 0) return;
  if (t < P.batch) s_start[t] = need.x, s_copy[t] = copy ? need.y : -1;
  if (t == 0) {
    *P.n_copies = need.all_y;
    *P.n_free = n_free - total;
  }
  if (__builtin_expect(rare, false)) {
    __syncthreads();   // the count is written
    int free = 0;
    if (keep < held) {
      int *row = row_of(P, t);
      for (int c = keep; c < held; ++c) {
        const int p = row[c];
        row[c] = -1;
        if (is_page(P, p)) free += give_back(P, p);
      }
    }
    if (free) atomicAdd(P.n_free, free);
    __syncthreads();
    word = t < P.words ? __ldcg(&P.bits[t]) : 0u;   // (not the line that this SM has read before)
  }
  auto assign = [&](int r, int id) {
    const int b = owner(r), k = r - s_start[b], l = s_len[b];
    int *row = row_of(P, b);
    if (s_copy[b] >= 0 && k == 0) {
      P.copies[s_copy[b]] = make_int4(s_tail[b], id, l & (P.page - 1), 0);
      row[l >> P.lg] = id;
    } else {
      row[s_held[b] + k - (s_copy[b] >= 0)] = id;
    }
    P.refs[id] = 1;
  };
  int found = 0;
  for (int base = 0; base < P.words && found < total; base += 1024) {
    const int w = base + t;
    if (base) word = w < P.words ? __ldcg(&P.bits[w]) : 0u;
    const int here = __popc(word);
    const Sums at = scan_1024(here, 0, s_warp);   // (its barriers also part this round's lists from the last one's readers)
    s_rank[t] = at.x, s_word[t] = word;
    const int take = min(here, total - found - at.x);
    if (take > 0) {
      uint32_t left = take == here ? 0u : word;
      if (left)
        for (int i = 0; i < take; ++i) left &= left - 1;
      P.bits[w] = left;
    }
    __syncthreads();
    for (int r = t; r < min(at.all_x, total - found); r += 1024) {
      int lo = 0, hi = 1023;   // the last word whose free pages start at r or before: it has some
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_rank[mid] <= r)
          lo = mid;
        else
          hi = mid - 1;
      }
      uint32_t x = s_word[lo];
      for (int i = r - s_rank[lo]; i > 0; --i) x &= x - 1;
      const int id = (base + lo) * 32 + __ffs(x) - 1;
      if (is_page(P, id)) assign(found + r, id);
    }
    found += at.all_x;
  }
  if (__builtin_expect(!rare, true)) {
    if (copy) atomicSub(&P.refs[tail], 1);
  } else if (copy && give_back(P, tail)) {   // its other holders gave the page back in this call (all words are written)
    atomicAdd(P.n_free, 1);
  }
  if (add) P.held[t] = keep + add;
  if (t == 0 && found < total) {   // the count and the bits disagree: not every copy has a page
    *P.n_copies = 0;
    atomicOr(P.status, QV_ERR_STATE);
  }
}

// The rows of the pages that a reserve copied.  Bound by memory: 60 copies of 4 pages in 16 layers, 24 MB read and 356 written,
// 62 us.
template <bool DENSE>
__global__ void __launch_bounds__(256) pages_tail_kernel(const __grid_constant__ PagesDev P) {
  pages_begin();
  copy_all<DENSE>(P, *P.n_copies, [&](int r) { return P.copies[r]; });
}

// Tables rearranged.  A CTA takes the same places of all sequences, up to 8192 entries: it reads them all before it writes
// any, and since a page stands at one place of the tables, it counts every entry that a page gains before the ones it loses.
// Lengths change once all CTAs have read them: by the last of them.  Bound by its chain of loads and atomics: 8 beams 2.5 us,
// 64 samples of 9 pages 3, 1024 sequences of 32 pages 10.
constexpr int SELECT_CELLS = 8;   // entries of a thread
__global__ void __launch_bounds__(1024) pages_select_kernel(const __grid_constant__ PagesDev P, const int *d_src, int cols) {
  __shared__ int s_old[1024 * SELECT_CELLS];
  __shared__ int s_src[PG_BATCH], s_held[PG_BATCH], s_new[PG_BATCH], s_len[PG_BATCH];   // 48 KB in all
  pages_begin();
  const int t = threadIdx.x, c0 = blockIdx.x * cols, n = min(cols, P.max_pages - c0), cells = P.batch * n;
  int cell[SELECT_CELLS];
#pragma unroll
  for (int k = 0; k < SELECT_CELLS; ++k) {   // all entries, while it is worked out which of them count
    const int i = t + 1024 * k;
    if (i < cells) cell[k] = row_of(P, i / n)[c0 + i % n];
  }
  int src = t, held = 0, len = 0;
  if (t < P.batch) {
    src = d_src[t];
    if (src < -1 || src >= P.batch) {
      if (blockIdx.x == 0) atomicOr(P.status, QV_ERR_BOUNDS);
      src = t;
    }
    held = held_of(P, t), len = length_of(P, t, held);
    s_held[t] = held, s_len[t] = len, s_src[t] = src;
  }
#pragma unroll
  for (int k = 0; k < SELECT_CELLS; ++k)
    if (t + 1024 * k < cells) s_old[t + 1024 * k] = cell[k];
  __syncthreads();
  int n_held = held, n_len = len;
  if (src != t) {
    n_len = src < 0 ? 0 : s_len[src];
    n_held = (n_len + P.page - 1) >> P.lg;
  }
  if (t < P.batch) s_new[t] = n_held;
  if (__syncthreads_or(src != t && c0 < max(held, n_held))) {
#pragma unroll
    for (int k = 0; k < SELECT_CELLS; ++k) {
      const int i = t + 1024 * k;
      if (i >= cells) break;
      const int b = i / n, c = i - b * n, from = s_src[b];
      if (from == b) continue;
      const int p = c0 + c < s_new[b] ? s_old[from * n + c] : -1;
      if (is_page(P, p)) atomicAdd(&P.refs[p], 1);
      if (p != cell[k]) row_of(P, b)[c0 + c] = p;
    }
    __syncthreads();
    int free = 0;
#pragma unroll
    for (int k = 0; k < SELECT_CELLS; ++k) {
      const int i = t + 1024 * k;
      if (i >= cells) break;
      const int b = i / n, c = i - b * n;
      if (s_src[b] != b && c0 + c < s_held[b] && is_page(P, cell[k])) free += give_back(P, cell[k]);
    }
    free = __reduce_add_sync(0xffffffffu, free);
    if (free && (t & 31) == 0) atomicAdd(P.n_free, free);
  }
  if (gridDim.x > 1) {
    bool last = false;
    if (t == 0) {
      __threadfence();
      last = atomicAdd(&P.tickets[P.batch], 1) == (int)gridDim.x - 1;
      if (last) P.tickets[P.batch] = 0;
    }
    if (!__syncthreads_or(last)) return;
  }
  if (t < P.batch && src != t) {   // every thread of every CTA has read lengths
    P.length[t] = n_len;
    P.held[t] = n_held;
  }
}

// A CTA a sequence.  Bound by latency: 1.4 us where nothing is given back.
__global__ void __launch_bounds__(256) pages_trim_kernel(const __grid_constant__ PagesDev P, const int *d_length) {
  __shared__ int given;
  pages_begin();
  const int b = blockIdx.x, want = d_length[b], held = held_of(P, b), len = min(length_of(P, b, held), want);
  if (want < 0) return;
  if (threadIdx.x == 0) given = 0;
  __syncthreads();   // also: held and length have been read
  const int keep = (len + P.page - 1) >> P.lg;
  int *row = row_of(P, b), free = 0;
  for (int c = keep + threadIdx.x; c < held; c += blockDim.x) {
    const int p = row[c];
    row[c] = -1;
    if (is_page(P, p)) free += give_back(P, p);
  }
  if (free) atomicAdd(&given, free);
  __syncthreads();
  if (threadIdx.x == 0) {
    P.length[b] = len;
    P.held[b] = min(held, keep);
    if (given) atomicAdd(P.n_free, given);
  }
}

// Which pages move where: the r-th used page from n on to the r-th free one below n, n pages being in use.  Bound by latency: a
// round of barriers for every 32768 pages, 2.5 us with the copying kernel where nothing moves, 20 for a pool of a million pages.
__global__ void __launch_bounds__(1024) pages_plan_kernel(const __grid_constant__ PagesDev P) {
  __shared__ int2 s_warp[32];
  pages_begin();
  const int t = threadIdx.x, n = P.pages - *P.n_free;
  auto below = [](int edge, int w) {   // bits of word w whose page is below edge
    const int k = edge - w * 32;
    return k >= 32 ? ~0u : k <= 0 ? 0u : (1u << k) - 1u;
  };
  int from = 0, to = 0;
  for (int base = 0; base < P.words; base += 1024) {
    const int w = base + t;
    const uint32_t x = w < P.words ? P.bits[w] : 0u;
    const uint32_t hole = x & below(n, w), used = ~x & below(P.pages, w) & ~below(n, w);
    const Sums at = scan_1024(__popc(hole), __popc(used), s_warp);
    int rh = to + at.x, ru = from + at.y;
    for (uint32_t y = hole; y; y &= y - 1) P.to[rh++] = w * 32 + __ffs(y) - 1;
    for (uint32_t y = used; y; y &= y - 1) P.from[ru++] = w * 32 + __ffs(y) - 1;
    to += at.all_x, from += at.all_y;
  }
  const bool fits = from == to;   // else the count of free pages and their bits disagree: nothing moves
  if (t == 0) {
    *P.moves = fits ? from : 0;
    *P.drawn = 0;
    if (!fits) atomicOr(P.status, QV_ERR_STATE);
  }
  if (!fits || !from) return;
  __syncthreads();
  for (int r = t; r < from; r += 1024) {
    const int a = P.from[r], z = P.to[r];
    P.refs[z] = P.refs[a];
    P.refs[a] = 0;
    P.goes[a] = z;
  }
  for (int w = t; w < P.words; w += 1024) P.bits[w] = below(P.pages, w) & ~below(n, w);
}

// The moves themselves, and the tables.  Bound by memory: 700 pages of 64 tokens and 8 heads in 8 layers, 174 of which move, 107
// us (6.8 TB/s).
template <bool DENSE>
__global__ void __launch_bounds__(256) pages_move_kernel(const __grid_constant__ PagesDev P) {
  pages_begin();
  const int moves = *P.moves, n = P.pages - *P.n_free;
  if (!moves) return;
  copy_all<DENSE>(P, moves, [&](int r) { return make_int4(P.from[r], P.to[r], P.page, 0); });
  const int cells = P.batch * P.max_pages;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < cells; i += (int64_t)gridDim.x * 256) {
    const int p = P.table[i];
    if (p >= n && is_page(P, p)) P.table[i] = P.goes[p];
  }
}

// ----------------------------------------------------------------------------- host

bool dims_ok(const int64_t *st, const int64_t *size, int dims, bool zero) {
  for (int i = 0; i < dims; ++i)
    if (size[i] > 1 && (st[i] % 8 || st[i] >= (1ll << 40) || st[i] > (1ll << 48) / (size[i] - 1) || st[i] < (zero ? 0 : 8)))
      return false;
  return true;
}

// No two elements in one place: each dimension steps over all that the smaller steps reach.
bool apart(const int64_t *st, const int64_t *size_in, int dims) {
  int64_t size[4], reach = D;
  for (int i = 0; i < dims; ++i) size[i] = size_in[i];
  for (int n = 0; n < dims; ++n) {
    int best = -1;
    for (int i = 0; i < dims; ++i)
      if (size[i] > 1 && (best < 0 || st[i] < st[best])) best = i;
    if (best < 0) break;
    if (st[best] < reach) return false;
    reach += st[best] * (size[best] - 1);
    size[best] = 1;
  }
  return true;
}

struct PagesPlan {
  qevict_pages_layout lay;
  int64_t tickets, copies, from, to, goes;
  int words;
  bool dense;
};

qevict_status pages_plan(const qevict_pages_desc *d, PagesPlan *p) {
  if (!d || d->layers < 1 || d->layers > 32767 || d->pages < 1 || d->pages > (1 << 24) ||
      (d->page != 16 && d->page != 32 && d->page != 64 && d->page != 128) || d->h_kv < 1 || d->h_kv > 4096 || d->d_head != D ||
      d->batch < 1 || d->batch > PG_BATCH || d->max_pages < 1 || d->max_pages > (1 << 30) / d->page ||
      (int64_t)d->batch * d->max_pages > (1 << 30) || d->reserved0)
    return QEVICT_EINVAL;
  const int64_t size[4] = {d->layers, d->pages, d->page, d->h_kv};
  if (!dims_ok(d->k, size, 4, false) || !dims_ok(d->v, size, 4, false) || !apart(d->k, size, 4) || !apart(d->v, size, 4))
    return QEVICT_EINVAL;
  int64_t off = PG_HEADER;
  auto take = [&](int64_t n) {
    const int64_t o = off;
    off += (n + 63) & ~int64_t(63);   // 256 bytes
    return o;
  };
  p->words = (d->pages + 127) / 128 * 4;
  p->lay.status = 0;
  p->lay.n_free = 1;
  p->lay.length = take(d->batch);
  p->lay.held = take(d->batch);
  p->lay.table = take((int64_t)d->batch * d->max_pages);
  p->lay.refs = take(d->pages);
  p->lay.free_bits = take(p->words);
  p->tickets = take(d->batch + 1);
  p->copies = take((int64_t)d->batch * 4);
  p->from = take(d->pages);
  p->to = take(d->pages);
  p->goes = take(d->pages);
  p->lay.ints = off;
  auto rows_follow = [&](const int64_t *st) {
    return (d->h_kv == 1 || st[3] == D) && st[2] == (int64_t)d->h_kv * D;
  };
  p->dense = rows_follow(d->k) && rows_follow(d->v);
  return QEVICT_OK;
}

qevict_status pages_args(const qevict_pages_desc *d, bool pool, void *k, void *v, void *d_state, PagesPlan *p, PagesDev *P) {
  const qevict_status st = pages_plan(d, p);
  if (st != QEVICT_OK) return st;
  if (!d_state || ((uintptr_t)d_state & 255) || (pool && (!k || !v || (((uintptr_t)k | (uintptr_t)v) & 15))))
    return QEVICT_EINVAL;
  int *s = static_cast<int *>(d_state);
  *P = PagesDev();
  P->k = static_cast<uint16_t *>(k), P->v = static_cast<uint16_t *>(v);
  for (int i = 0; i < 4; ++i) P->sk[i] = d->k[i], P->sv[i] = d->v[i];
  P->layers = d->layers, P->pages = d->pages, P->page = d->page, P->h_kv = d->h_kv, P->batch = d->batch;
  P->max_pages = d->max_pages, P->words = p->words;
  P->lg = d->page == 16 ? 4 : d->page == 32 ? 5 : d->page == 64 ? 6 : 7;
  P->status = s, P->n_free = s + 1, P->moves = s + 2, P->n_copies = s + 3;
  P->drawn = reinterpret_cast<unsigned long long *>(s + 4);
  P->length = s + p->lay.length, P->held = s + p->lay.held, P->table = s + p->lay.table, P->refs = s + p->lay.refs;
  P->bits = reinterpret_cast<uint32_t *>(s + p->lay.free_bits);
  P->tickets = s + p->tickets, P->copies = reinterpret_cast<int4 *>(s + p->copies);
  P->from = s + p->from, P->to = s + p->to, P->goes = s + p->goes;
  return QEVICT_OK;
}

template <typename... Params, typename... Args>
bool launch(void (*kern)(Params...), dim3 grid, int threads, qevict_stream_t stream, const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

unsigned ceil_div(int64_t x, int64_t y) { return (unsigned)((x + y - 1) / y); }
// At most `most` pages to copy: no more CTAs than fit on the SMs at once, three on each.
dim3 copy_grid(const PagesDev &P, int64_t most) {
  const int64_t parts = ceil_div((int64_t)P.page * P.h_kv * 16, PART_PIECES);
  return dim3((unsigned)std::min<int64_t>(most * parts * 2 * P.layers, qv::sm_count() * 3));
}
bool word_ok(const void *p, bool needed) { return !((uintptr_t)p & 3) && (p || !needed); }

}  // namespace
}  // namespace qv

extern "C" {

qevict_status qevict_pages_get_layout(const qevict_pages_desc *desc, qevict_pages_layout *layout) {
  qv::PagesPlan p;
  if (!layout) return QEVICT_EINVAL;
  const qevict_status st = qv::pages_plan(desc, &p);
  if (st == QEVICT_OK) *layout = p.lay;
  return st;
}

qevict_status qevict_pages_load(const qevict_pages_desc *desc, void *d_state, const int32_t *d_table, const int32_t *d_length,
                                qevict_stream_t stream) {
  qv::PagesPlan p;
  qv::PagesDev P;
  const qevict_status st = qv::pages_args(desc, false, nullptr, nullptr, d_state, &p, &P);
  if (st != QEVICT_OK) return st;
  if (!qv::word_ok(d_table, false) || !qv::word_ok(d_length, false) || !d_table != !d_length) return QEVICT_EINVAL;
  const int64_t n = std::max<int64_t>(std::max(P.pages, P.batch + 1), qv::PG_HEADER);
  const bool ok = qv::launch(qv::pages_clear_kernel, dim3(qv::ceil_div(n, 256)), 256, stream, P) &&
                  qv::launch(qv::pages_adopt_kernel, dim3(P.batch), 256, stream, P, (const int *)d_table, (const int *)d_length) &&
                  qv::launch(qv::pages_free_bits_kernel, dim3(qv::ceil_div(P.words, 256)), 256, stream, P);
  return ok ? QEVICT_OK : QEVICT_ECUDA;
}

qevict_status qevict_pages_reserve(const qevict_pages_desc *desc, void *k, void *v, void *d_state, const int32_t *d_new,
                                   int32_t n_new, qevict_stream_t stream) {
  qv::PagesPlan p;
  qv::PagesDev P;
  const qevict_status st = qv::pages_args(desc, true, k, v, d_state, &p, &P);
  if (st != QEVICT_OK) return st;
  if (!qv::word_ok(d_new, false) || (!d_new && n_new < 0)) return QEVICT_EINVAL;
  const auto tail = p.dense ? qv::pages_tail_kernel<true> : qv::pages_tail_kernel<false>;
  const bool ok = qv::launch(qv::pages_reserve_kernel, dim3(1), 1024, stream, P, (const int *)d_new, (int)n_new) &&
                  qv::launch(tail, qv::copy_grid(P, P.batch), 256, stream, P);
  return ok ? QEVICT_OK : QEVICT_ECUDA;
}

qevict_status qevict_pages_append(const qevict_pages_desc *desc, const qevict_pages_rows *rows, void *k, void *v,
                                  void *d_state, const void *k_new, const void *v_new, const int32_t *d_n,
                                  qevict_stream_t stream) {
  qv::PagesPlan p;
  qv::PagesDev P;
  const qevict_status st = qv::pages_args(desc, true, k, v, d_state, &p, &P);
  if (st != QEVICT_OK) return st;
  if (!rows || rows->layer < 0 || rows->layers < 1 || rows->layer > P.layers - rows->layers || rows->n < 1 || rows->reserved0 ||
      rows->n > (1 << 30) / (P.h_kv * 16) || !k_new || !v_new || (((uintptr_t)k_new | (uintptr_t)v_new) & 15) ||
      !qv::word_ok(d_n, false))
    return QEVICT_EINVAL;
  const int64_t size[4] = {rows->layers, P.batch, rows->n, P.h_kv};
  if (!qv::dims_ok(rows->k, size, 4, true) || !qv::dims_ok(rows->v, size, 4, true)) return QEVICT_EINVAL;
  qv::RowsDev R = {};
  R.k = static_cast<const uint16_t *>(k_new), R.v = static_cast<const uint16_t *>(v_new);
  for (int i = 0; i < 4; ++i) R.sk[i] = rows->k[i], R.sv[i] = rows->v[i];
  R.layer = rows->layer, R.layers = rows->layers, R.n = rows->n, R.d_n = d_n;
  const dim3 grid(qv::ceil_div((int64_t)R.n * P.h_kv * 16, qv::APPEND_THREADS * qv::APPEND_PIECES), P.batch, R.layers);
  return qv::launch(qv::pages_append_kernel, grid, qv::APPEND_THREADS, stream, P, R) ? QEVICT_OK : QEVICT_ECUDA;
}

qevict_status qevict_pages_accept(const qevict_pages_desc *desc, void *k, void *v, void *d_state, const int32_t *d_count,
                                  const int32_t *d_path, int32_t max_path, qevict_stream_t stream) {
  qv::PagesPlan p;
  qv::PagesDev P;
  const qevict_status st = qv::pages_args(desc, true, k, v, d_state, &p, &P);
  if (st != QEVICT_OK) return st;
  if (!qv::word_ok(d_count, true) || !qv::word_ok(d_path, false) ||
      (d_path ? max_path < 1 || max_path > qv::PG_PATH : max_path != 0))
    return QEVICT_EINVAL;
  // CTAs for every 256 columns of 16 bytes, or four on each SM over all sequences: the table and path are looked
  // up once a CTA
  const unsigned cols = qv::ceil_div((int64_t)P.layers * 2 * P.h_kv * 16, 256);
  const dim3 grid(d_path ? std::min(cols, std::max(1u, 4u * qv::sm_count() / P.batch)) : 1, P.batch);
  return qv::launch(qv::pages_accept_kernel, grid, 256, stream, P, (const int *)d_count, (const int *)d_path, (int)max_path)
             ? QEVICT_OK : QEVICT_ECUDA;
}

qevict_status qevict_pages_select(const qevict_pages_desc *desc, void *d_state, const int32_t *d_src, qevict_stream_t stream) {
  qv::PagesPlan p;
  qv::PagesDev P;
  const qevict_status st = qv::pages_args(desc, false, nullptr, nullptr, d_state, &p, &P);
  if (st != QEVICT_OK) return st;
  if (!qv::word_ok(d_src, true)) return QEVICT_EINVAL;
  const int cols = std::min(P.max_pages, 1024 * qv::SELECT_CELLS / P.batch);
  return qv::launch(qv::pages_select_kernel, dim3(qv::ceil_div(P.max_pages, cols)), 1024, stream, P, (const int *)d_src,
                    (int)cols) ? QEVICT_OK : QEVICT_ECUDA;
}

qevict_status qevict_pages_trim(const qevict_pages_desc *desc, void *d_state, const int32_t *d_length, qevict_stream_t stream) {
  qv::PagesPlan p;
  qv::PagesDev P;
  const qevict_status st = qv::pages_args(desc, false, nullptr, nullptr, d_state, &p, &P);
  if (st != QEVICT_OK) return st;
  if (!qv::word_ok(d_length, true)) return QEVICT_EINVAL;
  return qv::launch(qv::pages_trim_kernel, dim3(P.batch), 256, stream, P, (const int *)d_length) ? QEVICT_OK : QEVICT_ECUDA;
}

qevict_status qevict_pages_compact(const qevict_pages_desc *desc, void *k, void *v, void *d_state, qevict_stream_t stream) {
  qv::PagesPlan p;
  qv::PagesDev P;
  const qevict_status st = qv::pages_args(desc, true, k, v, d_state, &p, &P);
  if (st != QEVICT_OK) return st;
  const auto move = p.dense ? qv::pages_move_kernel<true> : qv::pages_move_kernel<false>;
  const bool ok = qv::launch(qv::pages_plan_kernel, dim3(1), 1024, stream, P) &&
                  qv::launch(move, qv::copy_grid(P, P.pages / 2 + 1), 256, stream, P);
  return ok ? QEVICT_OK : QEVICT_ECUDA;
}

}  // extern "C"
