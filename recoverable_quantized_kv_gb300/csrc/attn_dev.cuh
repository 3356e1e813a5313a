// Attention over a dense KV cache on the 5th-generation tensor cores: parameters shared by the kernel's
// translation units and the host side, and the kernel itself.
//
// Online softmax in base 2 over key tiles of 128: with x_j the (capped, biased) logit times log2 e,
//   m' = max(m, max x),  l' = l 2^(m - m') + sum 2^(x - m'),  O' = O 2^(m - m') + 2^(x - m') V,
// out = O / l, lse = (m + log2 l) ln 2.
#pragma once

#include <type_traits>

#include "smem_optin.h"
#include "tc_dev.cuh"

namespace qv {

constexpr int AT_TILE = 128;                          // rows of a query tile, keys of a key tile
constexpr int AT_STAGES = 5;                          // key / value tiles in flight
constexpr int AT_TILE_BYTES = AT_TILE * D * 2;        // 32 KB: two 128-byte-swizzled halves of 64 channels
constexpr int AT_HALF_BYTES = AT_TILE_BYTES / 2;
constexpr int AT_SOFT = 16;                           // softmax warps: four for each quarter of the columns
constexpr int AT_W_LOAD = AT_SOFT, AT_W_MMA = AT_SOFT + 1, AT_W_PLAN = AT_SOFT + 2;   // TMA, MMA, work items
constexpr int AT_THREADS = (AT_SOFT + 3) * 32;        // five warps on an SM sub-partition: 96 registers a thread
constexpr int AT_COLS = AT_TILE / 4;                  // columns of S, and channels of O, per softmax thread
constexpr int AT_ITEMS = 4;                           // work items described ahead
constexpr int AT_OFF_KV = 2 * AT_TILE_BYTES;
constexpr int AT_OFF_X = AT_OFF_KV + AT_STAGES * AT_TILE_BYTES;    // [4 quarters][128] fp32 exchange
constexpr int AT_OFF_BAR = AT_OFF_X + 4 * AT_TILE * 4;
constexpr int AT_NBAR = 2 * AT_STAGES + 4 + 6 + 2 * AT_ITEMS + 2;   // (one unused: 16-byte steps)
constexpr int AT_OFF_MISC = AT_OFF_BAR + AT_NBAR * 8;              // tmem address, flags
constexpr int AT_OFF_ITEM = AT_OFF_MISC + 16;                     // work item ring
constexpr int AT_SMEM = AT_OFF_ITEM + AT_ITEMS * 64;
static_assert(AT_SMEM <= 232448, "one CTA per SM");
// tanh(u) / u in powers of u^2 up to |u| = 0.6
constexpr double TANH_0 = 0.9999999403953552, TANH_1 = -0.33332324028015137, TANH_2 = 0.13310357928276062,
                 TANH_3 = -0.052109625190496445, TANH_4 = 0.01548669021576643;
constexpr float AT_BIG = 8388608.f;                   // 2^23: fp32 numbers beyond are whole
constexpr int AT_PADDING = 0x7fffffff;                // end of the visible keys of a row that is none (others: up to 2^30)
constexpr int AT_BAR_ALL = 1, AT_BAR_ROWS = 2;        // named barriers (of the four warps that share rows: 2 .. 5)

struct AttnArgs {
  CUtensorMap tq, tk, tv;      // queries and own keys of each sequence
  CUtensorMap tqp, tkp, tvp;   // queries of all sequences stacked, shared prefix
  const void *k, *v, *q, *kp, *vp;
  void *out;
  float *lse;
  // Own keys, [part][row]: output [128], and (m, l) with maximum m (log2 domain) and sum l of 2^(x - m), 0 where the row sees
  // no key.  One number m + log2 l would lose l behind a maximum of 10^6.
  float *part_o;
  float2 *part_l;
  float *pre_o;                // the same of the prefix
  float2 *pre_l;
  int *status, *drawn;         // status word; units given out (whole units)
  const float *slopes;
  const int *q_len, *kv_len, *prefix_len;
  const int2 *runs;            // [batch][s_kv]: first and past-the-last position of every position's document
  int64_t sq[3], sk[3], sv[3], so[3], skp[2], svp[2];
  int batch, s_q, s_kv, h_q, h_kv, G, causal;
  int mul_q, mul_k, mul_v;     // batch coordinate of the tensor maps: 0 for a batch stride of 0
  int tpt, n_pr;               // own keys: tokens per row tile, pairs of row tiles
  int pre, nb, n_prp;          // prefix: keys, sequences per row tile, pairs of row tiles
  int part_rows, pre_rows;     // rows of a part
  int wide_out;                // rows of out start on 32 bytes
  int stream, min_tiles;       // the key tiles of all units as one stream, cut into equal shares of at least min_tiles
  float scale_log2;            // logit scale * log2 e
  float cap_u, cap_s;          // softcap: scale / cap, cap / scale
  float cap_q[5], cap_r[3];    // tanh(u) / u in powers of the product's square, u = product * cap_u: to 0.6, to 0.25
  float cap_near, cap_mid;     // the |u| up to which they serve: 0.25 and 0.6, or below 0 (never)
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// A unit of work is one KV head's pair of row tiles against the keys it sees; the units of a pair of row tiles (a
// group) differ in the KV head only and have the same key tiles.  Group gi = pair * batch + sequence.
struct AttnGroup {
  int b, tile0;
  int kl, ql, pfx;             // keys, queries, prefix mask of the sequence
  int clean_lo, clean_hi;      // keys that every row sees
  int key_lo, key_hi;          // keys that some row sees
  int tiles;                   // key tiles from key_lo on
};

// Visible keys [x, y) of position p.  Both ends grow with p.
__device__ __forceinline__ int2 attn_interval(const AttnArgs &P, int b, int p, int kl, int pfx) {
  int lo = 0, hi = P.causal ? min(max(p + 1, pfx), kl) : kl;
  if (P.runs) {
    if (p < 0) return make_int2(0, 0);
    const int2 r = P.runs[(size_t)b * P.s_kv + p];
    lo = r.x;
    hi = min(hi, r.y);
  }
  return make_int2(lo, max(hi, lo));
}

__device__ __forceinline__ AttnGroup attn_group(const AttnArgs &P, int gi) {
  AttnGroup A;
  const int pr = P.n_pr == 1 ? 0 : gi / P.batch;
  A.b = gi - pr * P.batch;
  A.tile0 = 2 * pr;
  A.kl = P.kv_len ? clampi(P.kv_len[A.b], 0, P.s_kv) : P.s_kv;
  A.ql = P.q_len ? clampi(P.q_len[A.b], 0, P.s_q) : P.s_q;
  A.pfx = P.prefix_len ? clampi(P.prefix_len[A.b], 0, A.kl) : 0;
  const int i0 = A.tile0 * P.tpt, i1 = min(A.ql, i0 + 2 * P.tpt);
  A.clean_lo = A.clean_hi = A.key_lo = A.key_hi = A.tiles = 0;
  if (i0 < i1) {
    const int p0 = A.kl - A.ql + i0;
    const int2 a = attn_interval(P, A.b, p0, A.kl, A.pfx), z = attn_interval(P, A.b, p0 + (i1 - 1 - i0), A.kl, A.pfx);
    A.key_lo = a.x;
    A.key_hi = z.y;
    A.clean_lo = z.x;
    A.clean_hi = a.y;
    A.tiles = (A.key_hi - A.key_lo + AT_TILE - 1) / AT_TILE;   // (a document's units share its tiles)
  }
  return A;
}

// Places that a unit of t key tiles takes in the stream: its tiles, and behind them the cost of beginning and ending
// a unit in tiles, so that a CTA with many short units gets fewer tiles.
constexpr int AT_UNIT_COST = 4;
__device__ __forceinline__ int attn_places(int t) { return t ? t + AT_UNIT_COST : 0; }
// Share of the stream that each of `ctas` CTAs takes.
__device__ __forceinline__ int attn_share(int total, int ctas, int min_tiles) {
  return max((total + ctas - 1) / ctas, min_tiles);
}

// A work item: a unit, or the part of it that falls into a CTA's share.  pair: slot 0 and 1 hold two row tiles and
// both see every key tile.  Otherwise one row tile in both slots, slot s taking every second key tile.
struct AttnItem {
  int kind;                    // bit 0 prefix, bit 1 pair, bit 2 written as a part; -1: no more items
  int b, g, tile0, kl, ql, pfx;
  int n, t_hi;                 // key tiles t_hi - 1, t_hi - 2, ... (n of them), tile t from key k0 + 128 t on
  int k0;
  int clean_lo, clean_hi, key_hi;   // counted from k0
  int part;
  int pad[2];
  __device__ __forceinline__ bool prefix() const { return kind & 1; }
  __device__ __forceinline__ bool pair() const { return kind & 2; }
  __device__ __forceinline__ bool parts() const { return kind & 4; }
};
static_assert(sizeof(AttnItem) == 64, "item ring");

// What row r of a slot's tile is, in every item: token r / G of the tile and query head r % G of the group.
struct AttnRow {
  int tok, hr, bl, ip;         // in a prefix item the token is query ip of the tile's sequence bl
};
__device__ __forceinline__ AttnRow attn_row_of(const AttnArgs &P, int r) {
  AttnRow R;
  R.tok = r / P.G;
  R.hr = r - R.tok * P.G;
  R.bl = R.tok / P.s_q;
  R.ip = R.tok - R.bl * P.s_q;
  return R;
}
// Sequence b, query i and head h of the row; its row of a part.  False: the row is padding.
template <bool STREAM>
__device__ __forceinline__ bool attn_row(const AttnArgs &P, const AttnItem &I, int slot, const AttnRow &R, int &b, int &i,
                                         int &h, int &prow) {
  const int second = !STREAM || I.pair() ? slot : 0;
  h = I.g * P.G + R.hr;
  if (STREAM && I.prefix()) {
    const int bt = second * P.nb + R.bl;
    b = I.tile0 * P.nb + bt;
    i = R.ip;
    prow = (bt * P.s_q + i) * P.G + R.hr;
    return R.bl < P.nb && b < P.batch;
  }
  b = I.b;
  const int il = second * P.tpt + R.tok;
  i = I.tile0 * P.tpt + il;
  prow = il * P.G + R.hr;
  return R.tok < P.tpt && i < I.ql;
}

// Position of query i of sequence b behind the prefix.
__device__ __forceinline__ int attn_prefix_pos(const AttnArgs &P, int b, int i) {
  return P.pre + ((P.kv_len ? clampi(P.kv_len[b], 0, P.s_kv) : P.s_kv) - P.s_q + i);
}

// Until the kernel before, which may still run, has ended and its writes are visible.
__device__ __forceinline__ void attn_wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Bounded wait on an mbarrier phase.  The limit is about 4 s (8e9 SM cycles), longer than the 200 ms of the other
// kernels' waits, since a slot that recomputes rows on the CUDA cores (attn_exact_rows) holds the others up.  The
// SM's own clock is read, and only now and then: a first read of the global timer costs more than a tile's wait.
__device__ __forceinline__ bool attn_wait(uint64_t *bar, uint32_t parity, int *status) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 255u) == 255u && clock64() - t0 > 8000000000ll) {
      atomicOr(status, QV_ERR_TIMEOUT);
      return false;
    }
  }
}

// The same by a whole warp, one answer for all its lanes.
__device__ __forceinline__ bool attn_wait_warp(uint64_t *bar, uint32_t parity, int *status) {
  return __all_sync(0xffffffffu, attn_wait(bar, parity, status));
}

// ----------------------------------------------------------------------------- tensor memory and products

__device__ __forceinline__ void tma_load_4d_at(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                               uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}
// The eight products (16 deep each) of one 128 x 128 x 128 tile, issued by one elected lane of a converged warp:
// descriptors stay in uniform registers, where a lane-0 branch needs a vector-to-uniform move for every operand of
// every instruction (about 80 cycles per product, more than the 64 that the tensor pipe takes).
// S = Q K^T: both operands in shared memory, 64-channel halves 16 KB apart (descriptor units of 16 bytes).
__device__ __forceinline__ void tc_mma_tile_ss(uint32_t tmem, uint64_t da, uint64_t db, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred e, f, t;\n .reg .b64 a, b;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 f, 0, 0;\n setp.eq.b32 t, 0, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n"
      " add.s64 a, %1, 2;\n add.s64 b, %2, 2;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.s64 a, %1, 4;\n add.s64 b, %2, 4;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.s64 a, %1, 6;\n add.s64 b, %2, 6;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.s64 a, %1, 1024;\n add.s64 b, %2, 1024;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.s64 a, %1, 1026;\n add.s64 b, %2, 1026;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.s64 a, %1, 1028;\n add.s64 b, %2, 1028;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.s64 a, %1, 1030;\n add.s64 b, %2, 1030;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n}" ::"r"(tmem),
      "l"(da), "l"(db), "r"(idesc)
      : "memory");
}
// O (+)= P V: P in tensor memory (8 columns per 16 keys, 32 keys at the start of each 32 columns), 16 keys of V 2048 bytes
// apart
__device__ __forceinline__ void tc_mma_tile_ts(uint32_t tmem, uint32_t ta, uint64_t db, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred e, f, t;\n .reg .b64 b;\n .reg .b32 a;\n elect.sync _|e, 0xffffffff;\n"
      " setp.ne.b32 f, %4, 0;\n setp.eq.b32 t, 0, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n"
      " add.s32 a, %1, 8;\n add.s64 b, %2, 128;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
      " add.s32 a, %1, 32;\n add.s64 b, %2, 256;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
      " add.s32 a, %1, 40;\n add.s64 b, %2, 384;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
      " add.s32 a, %1, 64;\n add.s64 b, %2, 512;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
      " add.s32 a, %1, 72;\n add.s64 b, %2, 640;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
      " add.s32 a, %1, 96;\n add.s64 b, %2, 768;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
      " add.s32 a, %1, 104;\n add.s64 b, %2, 896;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n}" ::"r"(tmem),
      "r"(ta), "l"(db), "r"(idesc), "r"(accumulate)
      : "memory");
}
// tcgen05.commit by the same elected lane
__device__ __forceinline__ void tc_commit_elect(uint64_t *bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar))
      : "memory");
}
// shared-memory descriptor of a value tile: [128 keys][64 channels] halves, channels contiguous (the N side of
// P V is the contiguous one), 128-byte swizzle; 64-channel blocks 16 KB apart, 8-key groups 1024 B apart
__device__ __forceinline__ uint64_t umma_desc_v(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(AT_HALF_BYTES >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

#define QV_R16(r, o)                                                                                               \
  "r"((r)[(o) + 0]), "r"((r)[(o) + 1]), "r"((r)[(o) + 2]), "r"((r)[(o) + 3]), "r"((r)[(o) + 4]), "r"((r)[(o) + 5]), \
      "r"((r)[(o) + 6]), "r"((r)[(o) + 7]), "r"((r)[(o) + 8]), "r"((r)[(o) + 9]), "r"((r)[(o) + 10]),               \
      "r"((r)[(o) + 11]), "r"((r)[(o) + 12]), "r"((r)[(o) + 13]), "r"((r)[(o) + 14]), "r"((r)[(o) + 15])
#define QV_W16(r, o)                                                                                                  \
  "=r"((r)[(o) + 0]), "=r"((r)[(o) + 1]), "=r"((r)[(o) + 2]), "=r"((r)[(o) + 3]), "=r"((r)[(o) + 4]),                 \
      "=r"((r)[(o) + 5]), "=r"((r)[(o) + 6]), "=r"((r)[(o) + 7]), "=r"((r)[(o) + 8]), "=r"((r)[(o) + 9]),             \
      "=r"((r)[(o) + 10]), "=r"((r)[(o) + 11]), "=r"((r)[(o) + 12]), "=r"((r)[(o) + 13]), "=r"((r)[(o) + 14]),        \
      "=r"((r)[(o) + 15])

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : QV_W16(r, 0)
      : "r"(addr));
}
// 32 columns of this thread's lane; the caller waits (tmem_wait_ld) before it uses them
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : QV_W16(r, 0), QV_W16(r, 16)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::QV_R16(
          r, 0),
      "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_global_v8(void *p, const uint32_t *r) {   // 32 bytes, 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ float lg2_approx(float x) {   // absolute error 2^-22 around 1, relative 2^-22 elsewhere
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float min_nan(float x, float y) {   // NaN if one is
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(x), "f"(y));
  return d;
}

// Packed fp32 pairs as 64-bit values: what stays the same over a loop is packed once
__device__ __forceinline__ uint64_t pack_f2(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ void unpack_f2(float &x, float &y, uint64_t v) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float rcp_approx(float x) {   // relative error about 2^-23
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool FP16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (FP16) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
  }
  return pack_bf16(lo, hi);
}
template <bool FP16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if (FP16) return __half22float2(*reinterpret_cast<__half2 *>(&v));
  return make_float2(bf16_lo(v), bf16_hi(v));
}

// 64 bytes of every lane's row (at element `at` of out; rows: the lanes that have one).  Lanes trade 32 bytes with their
// neighbour, so that each store of the warp writes 64 bytes of 16 rows, 32 of them a lane where the rows allow (`wide`);
// rows stored by their own lanes touch 32 lines an instruction.
__device__ __forceinline__ void attn_store_rows(uint16_t *out, int64_t at, uint32_t rows, int lane, bool wide,
                                                uint32_t (&w)[16]) {
  const bool odd = lane & 1;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t x = __shfl_xor_sync(0xffffffffu, odd ? w[c] : w[c + 8], 1);
    if (odd)
      w[c] = x;
    else
      w[c + 8] = x;
  }
  const int64_t mate = __shfl_xor_sync(0xffffffffu, at, 1);
#pragma unroll
  for (int r = 0; r < 2; ++r) {   // the pair's rows
    if (!(rows >> ((lane & 30) + r) & 1)) continue;
    uint16_t *dst = out + (odd == (r == 1) ? at : mate) + (odd ? 16 : 0);
    if (wide) {
      st_global_v8(dst, w + 8 * r);
    } else {
      reinterpret_cast<uint4 *>(dst)[0] = make_uint4(w[8 * r], w[8 * r + 1], w[8 * r + 2], w[8 * r + 3]);
      reinterpret_cast<uint4 *>(dst)[1] = make_uint4(w[8 * r + 4], w[8 * r + 5], w[8 * r + 6], w[8 * r + 7]);
    }
  }
}

// ----------------------------------------------------------------------------- rows with values that are not finite

// The keys of tile t that not every row of the item sees: their values that are not finite become 0 in shared memory,
// thread `who` of 512 taking a quarter of a key's channels.  If some row sees such a key, *flag = mark.
template <bool FP16>
__device__ __forceinline__ void attn_clean_values(const AttnItem &I, int t, uint8_t *v, int who, volatile int *flag, int mark) {
  const int k = who >> 2, key = t * AT_TILE + k;
  if (key >= I.clean_lo && key < I.clean_hi) return;
  constexpr uint32_t E = FP16 ? 0x7C00u : 0x7F80u, E2 = E | (E << 16);   // all exponent bits set: infinity or NaN
  uint32_t *p = reinterpret_cast<uint32_t *>(v + (who >> 1 & 1) * AT_HALF_BYTES + k * 128 + (who & 1) * 64);
  // ~w & E2 has an empty half exactly where the half is not finite; taking 1 from both halves then sets its top bit
  uint32_t hit = 0;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint4 x = lds128(p + ((c + k) & 3) * 4);   // neighbours start in other banks
    hit |= ((~x.x & E2) - 0x00010001u) | ((~x.y & E2) - 0x00010001u) | ((~x.z & E2) - 0x00010001u) |
           ((~x.w & E2) - 0x00010001u);
  }
  if (hit & 0x80008000u) {
    if (key < I.key_hi) *flag = mark;   // key 0 is the first that some row sees
#pragma unroll 1
    for (int c = 0; c < 16; ++c) {
      const uint32_t w = p[c];
      const bool lo = (w & E) == E, hi = (w & (E << 16)) == (E << 16);
      if (lo | hi) p[c] = (lo ? 0u : w & 0xFFFFu) | (hi ? 0u : w & 0xFFFF0000u);
    }
    fence_proxy_async();   // the product reads shared memory through the async proxy
  }
}

// The rows of one warp of a slot recomputed on the CUDA cores, every visible key of the item's own tiles in turn and no
// masked value touched.  Reached when a value that some row of the item sees and another does not is an infinity or NaN
// (the tensor-core product then ran with that value as 0), and when the maximum of one of the rows is beyond AT_BIG.  Writes
// O (unnormalised), m, l of row r through `emit`, the warp's lanes holding four channels each.
template <bool FP16, bool STREAM, typename Emit>
__device__ __forceinline__ void attn_exact_rows(const AttnArgs &P, const AttnItem &I, int slot, int warp, int lane, bool cap,
                                                const Emit &emit) {
  const uint16_t *kb, *vb;
  int64_t kst, vst;
  if (I.prefix()) {
    kb = static_cast<const uint16_t *>(P.kp) + I.g * P.skp[1];
    vb = static_cast<const uint16_t *>(P.vp) + I.g * P.svp[1];
    kst = P.skp[0], vst = P.svp[0];
  } else {
    kb = static_cast<const uint16_t *>(P.k) + I.b * P.sk[0] + I.g * P.sk[2];
    vb = static_cast<const uint16_t *>(P.v) + I.b * P.sv[0] + I.g * P.sv[2];
    kst = P.sk[1], vst = P.sv[1];
  }
  for (int rr = 0; rr < 32; ++rr) {
    int b, i, h, prow;
    if (!attn_row<STREAM>(P, I, slot, attn_row_of(P, warp * 32 + rr), b, i, h, prow)) continue;
    const uint16_t *q = static_cast<const uint16_t *>(P.q) + b * P.sq[0] + i * P.sq[1] + h * P.sq[2];
    int p, lo, hi;
    if (I.prefix()) {
      p = attn_prefix_pos(P, b, i);
      lo = 0, hi = clampi(p + 1, 0, P.pre);
    } else {
      p = I.kl - I.ql + i;
      const int2 v = attn_interval(P, b, p, I.kl, I.pfx);
      lo = v.x, hi = v.y;
    }
    const float slope = P.slopes ? P.slopes[h] * 1.4426950408889634f : 0.f;
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < I.n; ++j) {
      const int k0 = I.k0 + (I.t_hi - 1 - j) * AT_TILE;
      for (int c0 = k0; c0 < k0 + AT_TILE; c0 += 32) {
        if (c0 + 32 <= lo || c0 >= hi) continue;
        const int key = c0 + lane;
        const bool seen = key >= lo && key < hi;
        float x = -INFINITY;
        if (seen) {
          const uint32_t *kr = reinterpret_cast<const uint32_t *>(kb + (int64_t)key * kst);
          const uint32_t *qr = reinterpret_cast<const uint32_t *>(q);
          float s = 0.f;
          for (int d = 0; d < D / 2; ++d) {
            const float2 a = unpack2<FP16>(kr[d]), c = unpack2<FP16>(qr[d]);
            s = fmaf(a.x, c.x, s);
            s = fmaf(a.y, c.y, s);
          }
          x = (cap ? P.cap_s * tanhf(s * P.cap_u) : s) * P.scale_log2;
          x -= slope * fabsf((float)(p - key));
        }
        float mx = x;
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
        const float f = ex2(m - mu), pr = seen ? ex2(x - mu) : 0.f;
        m = mn;
        l = l * f;
        for (int c = 0; c < 4; ++c) acc[c] *= f;
        float ps = pr;
        for (int o = 16; o; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
        l += ps;
        for (int k = max(0, lo - c0); k < min(32, hi - c0); ++k) {   // visible keys only
          const float pk = __shfl_sync(0xffffffffu, pr, k);
          const uint2 w = *reinterpret_cast<const uint2 *>(vb + (int64_t)(c0 + k) * vst + lane * 4);
          const float2 a = unpack2<FP16>(w.x), c = unpack2<FP16>(w.y);
          acc[0] = fmaf(pk, a.x, acc[0]);
          acc[1] = fmaf(pk, a.y, acc[1]);
          acc[2] = fmaf(pk, c.x, acc[2]);
          acc[3] = fmaf(pk, c.y, acc[3]);
        }
      }
    }
    emit(b, i, h, prow, acc, m, l);
  }
}

// ----------------------------------------------------------------------------- the kernel

// One persistent CTA per SM: sixteen softmax warps, a thread owning one row and a quarter of the columns of the 128-row
// tile at hand; a TMA warp; an MMA warp; a warp that lays out the work items ahead of the others.  Rows of a tile are
// (token, query head of the group), so the group's heads share every key tile.  Tensor memory: S of slot s at columns
// 128 s, overwritten in place by the probabilities (each quarter of the keys over its own quarter of S), O of slot s at
// 256 + 128 s.  The probabilities are rounded to the input type, which the product takes as its A operand; the row sums
// take them unrounded.  The softmax warps and the tensor pipe alternate between the slots: while all warps turn slot 0's
// S into P, the pipe runs slot 1's products.  (With eight warps a slot, a half row a thread, a 32K prompt of 32 heads
// takes 5.45 ms instead of 5.16.)
// What bounds it: prompts by a step's chain of S load, row maximum, exponentials and P store, which takes the softmax
// warps about 1450 cycles where the tensor pipe needs 1180 (32K prompt of 32 heads: 5.16 ms, 1.70 PFLOP/s; 4.25 ms with
// the softmax left out); single tokens by memory (16 of 32 heads against caches of 33K keys: 211 us, 6.7 TB/s).
// Key tiles are taken from the last to the first, so a causal row meets its diagonal, and a distance bias its largest
// logits, first.  The running max moves only when a row's max has grown by more than 2^8 (then the warps rescale their
// rows of O in tensor memory): until then p reaches at most 2^8 of its scale, which fp32 sums and 16-bit probabilities hold
// as well.
// Every wait is bounded; the TMEM columns are released on every path.
// STREAM = false: whole units, always as pairs (of a last odd row tile the second is empty).  CAP: 0 none, 1 up to 64, 2 wider
// (instances of their own: its code in the others costs capped prompts 2%).
template <bool FP16, int CAP, bool BIAS, bool STREAM>
__global__ void __launch_bounds__(AT_THREADS, 1) attn_kernel(const __grid_constant__ AttnArgs P) {
  extern __shared__ __align__(1024) uint8_t sm[];   // swizzle atoms: 1024-aligned
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + AT_OFF_BAR);
  uint64_t *full = bars, *empty = full + AT_STAGES, *qfull = empty + AT_STAGES, *qempty = qfull + 2;
  uint64_t *sfull = qempty + 2, *pfull = sfull + 2, *ofull = pfull + 2, *ifull = ofull + 2, *iempty = ifull + AT_ITEMS;
  uint64_t *loaded = iempty + AT_ITEMS;
  uint32_t *misc = reinterpret_cast<uint32_t *>(sm + AT_OFF_MISC);
  uint32_t *tmem_slot = misc;
  volatile int *bad_item = reinterpret_cast<int *>(misc + 2);   // [item parity]: 1 + the item with values to recompute
  AttnItem *items = reinterpret_cast<AttnItem *>(sm + AT_OFF_ITEM);
  float *xch = reinterpret_cast<float *>(sm + AT_OFF_X);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int *status = P.status;
  if (smem_u32(sm) & 1023) {   // cannot be swizzled: nothing runs
    attn_wait_previous();
    if (threadIdx.x == 0) atomicOr(status, QV_ERR_STATE);
    return;
  }

  if (warp == AT_W_MMA) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (threadIdx.x < AT_NBAR) {
    const uint64_t *p = &bars[threadIdx.x];
    const int n = p < pfull ? 1 : p < ofull ? AT_SOFT :
                  p < ifull ? 2 : p < iempty ? 1 : p < loaded ? AT_SOFT + 2 : 1;
    mbar_init(&bars[threadIdx.x], n);
    fence_mbar_init();
    if (threadIdx.x < 2) bad_item[threadIdx.x] = 0;
  }
  // The launch may overlap the previous kernel's end: nothing is read from device memory before this wait, and the next
  // kernel is let in only after it, so whatever starts early still finds the kernel two launches back complete.
  attn_wait_previous();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  AttnGroup plan_a;        // the plan warp's lane: its group of the first 32, worked out while the others set up
  int plan_places = 0;     // and the places of all groups
  if (warp == AT_W_PLAN && STREAM) {
    const int groups = P.n_pr * P.batch;
#pragma unroll 1
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const AttnGroup A = attn_group(P, min(g0 + lane, groups - 1));
      if (g0 == 0) plan_a = A;
      plan_places += __reduce_add_sync(0xffffffffu, g0 + lane < groups ? attn_places(A.tiles) : 0) * P.h_kv;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Next work item of a role: waits for its description, copies what the role keeps and hands the ring place back.
  uint32_t seq = 0;
  auto next_item = [&](AttnItem &I) {
    const uint32_t e = seq % AT_ITEMS;
    bool ok = attn_wait_warp(&ifull[e], (seq / AT_ITEMS) & 1, status);
    I.kind = -1;
    if (ok) {
      I = items[e];
      __syncwarp();
      if (lane == 0) mbar_arrive(&iempty[e]);
      ++seq;
    }
    return ok;
  };

  if (warp == AT_W_PLAN) {
    // ---- work items, in order.  Every lane works everything out, lane 0 writes.
    bool ok = true;
    auto put = [&](const AttnItem &I) {
      const uint32_t e = seq % AT_ITEMS;
      if (!ok || !(ok = attn_wait_warp(&iempty[e], ((seq / AT_ITEMS) & 1) ^ 1, status))) return;
      if (lane == 0) {
        items[e] = I;
        mbar_arrive(&ifull[e]);
      }
      ++seq;
    };
    auto own_item = [&](const AttnGroup &A, int g) {
      AttnItem I;
      I.kind = !STREAM || A.tile0 * P.tpt + P.tpt < A.ql ? 2 : 0;
      I.b = A.b, I.g = g, I.tile0 = A.tile0, I.kl = A.kl, I.ql = A.ql, I.pfx = A.pfx;
      I.n = A.tiles;
      I.t_hi = A.tiles;
      I.k0 = A.key_lo;
      I.clean_lo = A.clean_lo - I.k0, I.clean_hi = A.clean_hi - I.k0, I.key_hi = A.key_hi - I.k0;
      I.part = 0;
      return I;
    };
    const int groups = P.n_pr * P.batch;
    if (!STREAM) {
      // Whole units, the longest (last rows of causal prompts) first, each to the CTA that is ready next: lengths and
      // documents make units differ, and a fixed turn leaves some CTAs twice the mean (a padded batch of prefix-mask
      // prompts 54 us, drawn 31).  A CTA's first unit is its own number; it draws the next when its TMA warp has asked
      // for the last one's tiles, two or three tiles before it needs it.  Every CTA draws once past the end, so the draw
      // that takes the count to the number of units is the last, and starts it again for the next call.
      const int units = groups * P.h_kv;
      int u = blockIdx.x;
      uint32_t drawn = 0;
      while (u < units) {
        const int x = u / P.h_kv, pr = x / P.batch;
        const AttnGroup A = attn_group(P, (P.n_pr - 1 - pr) * P.batch + (x - pr * P.batch));
        if (A.tile0 * P.tpt < A.ql) {   // the padding of a shorter sequence has no rows to write
          put(own_item(A, u - x * P.h_kv));
          if (ok) ok = attn_wait_warp(loaded, drawn++ & 1, status);
        }
        int n = 0;
        if (lane == 0) {
          n = atomicAdd(P.drawn, 1);
          if (n == units - 1) *P.drawn = 0;
        }
        u = gridDim.x + __shfl_sync(0xffffffffu, n, 0);
      }
    } else {
      // The key tiles of all units, prefix first, as one stream; CTA c takes tiles [c share, (c + 1) share).  A unit cut
      // by a share's end is written as parts, numbered CTA + unit: the numbers of a unit's parts are consecutive, and
      // none is used twice, since both terms only grow along the stream.
      const int tp = P.pre ? (P.pre + AT_TILE - 1) / AT_TILE : 0, wp = attn_places(tp);
      const int all_p = P.pre ? P.n_prp * P.h_kv * wp : 0;
      const int64_t total = (int64_t)all_p + plan_places;
      const int share = attn_share((int)total, gridDim.x, P.min_tiles);
      const int begin = (int)min((int64_t)blockIdx.x * share, total), end = (int)min((int64_t)begin + share, total);
      int pos = begin;
      while (ok && pos < min(end, all_p)) {
        const int u = pos / wp, o = pos - u * wp, pr = u / P.h_kv;
        if (o < tp) {
          AttnItem I;
          I.tile0 = 2 * pr;
          I.kind = 1 | 4 | ((I.tile0 + 1) * P.nb < P.batch ? 2 : 0);
          I.b = 0, I.g = u - pr * P.h_kv, I.kl = P.pre, I.ql = P.s_q, I.pfx = 0;
          I.n = min(tp - o, end - pos);
          I.t_hi = tp - o;
          I.k0 = I.clean_lo = 0;
          I.key_hi = P.pre;
          // a sequence with fewer own keys than queries has rows that sit inside the prefix
          I.clean_hi = max(0, P.pre - max(0, P.s_q - 1 - (P.kv_len ? 0 : P.s_kv)));
          I.part = blockIdx.x + u;
          put(I);
        }
        pos = (u + 1) * wp;
      }
      int done = all_p;   // stream position of the groups at hand
#pragma unroll 1
      for (int g0 = 0; ok && pos < end && g0 < groups; g0 += 32) {
        const AttnGroup A = g0 == 0 ? plan_a : attn_group(P, min(g0 + lane, groups - 1));
        const int t = g0 + lane < groups ? A.tiles : 0;
        const int here = __reduce_add_sync(0xffffffffu, attn_places(t)) * P.h_kv;
        if (done + here <= pos) {
          done += here;
          continue;
        }
#pragma unroll 1
        for (int q = 0; ok && pos < end && q < 32; ++q) {
          const int tq = __shfl_sync(0xffffffffu, t, q), wq = attn_places(tq);
          if (done + wq * P.h_kv <= pos) {
            done += wq * P.h_kv;
            continue;
          }
          AttnGroup B;
          B.b = __shfl_sync(0xffffffffu, A.b, q), B.tile0 = __shfl_sync(0xffffffffu, A.tile0, q);
          B.kl = __shfl_sync(0xffffffffu, A.kl, q), B.ql = __shfl_sync(0xffffffffu, A.ql, q);
          B.pfx = __shfl_sync(0xffffffffu, A.pfx, q);
          B.clean_lo = __shfl_sync(0xffffffffu, A.clean_lo, q), B.clean_hi = __shfl_sync(0xffffffffu, A.clean_hi, q);
          B.key_lo = __shfl_sync(0xffffffffu, A.key_lo, q), B.key_hi = __shfl_sync(0xffffffffu, A.key_hi, q);
          B.tiles = tq;
          while (ok && pos < min(end, done + wq * P.h_kv)) {
            const int g = (pos - done) / wq, u0 = done + g * wq, o = pos - u0;
            if (o < tq) {
              AttnItem I = own_item(B, g);
              I.n = min(tq - o, end - pos);
              I.t_hi -= o;
              I.part = blockIdx.x + (g0 + q) * P.h_kv + g;
              if (P.pre || u0 < begin || u0 + tq > begin + share) I.kind |= 4;   // not all in this share
              put(I);
            }
            pos = u0 + wq;
          }
          done += wq * P.h_kv;
        }
      }
    }
    AttnItem I = {};
    I.kind = -1;
    put(I);
    if (blockIdx.x == 0)   // lengths out of range are clamped everywhere; here they are reported
      for (int b = lane; b < P.batch; b += 32)
        if ((P.kv_len && (P.kv_len[b] < 0 || P.kv_len[b] > P.s_kv)) || (P.q_len && (P.q_len[b] < 0 || P.q_len[b] > P.s_q)))
          atomicOr(status, QV_ERR_BOUNDS);
  } else if (warp == AT_W_LOAD) {
    // ---- TMA loads
    const uint32_t qbytes = (uint32_t)(P.G * P.tpt) * 256u, qpbytes = (uint32_t)(P.G * P.s_q * P.nb) * 256u;
    uint32_t c = 0, qn = 0;
    bool ok = true;
    AttnItem I;
    while (ok && next_item(I) && I.kind >= 0) {
      if (I.n > 0 && lane == 0) {
        const bool prefix = STREAM && I.prefix(), pair = !STREAM || I.pair();
        const CUtensorMap *mq = prefix ? &P.tqp : &P.tq, *mk = prefix ? &P.tkp : &P.tk, *mv = prefix ? &P.tvp : &P.tv;
        auto load = [&](const CUtensorMap *map, int j, int bb) {
          const uint32_t st = c % AT_STAGES;
          if (!ok || !(ok = attn_wait(&empty[st], ((c / AT_STAGES) & 1) ^ 1, status))) return;
          const uint32_t dst = smem_u32(sm) + AT_OFF_KV + st * AT_TILE_BYTES;
          const int t = I.t_hi - 1 - j;
          mbar_arrive_expect_tx(&full[st], AT_TILE_BYTES);
          tma_load_4d_at(dst, map, 0, I.g, I.k0 + t * AT_TILE, bb, &full[st]);
          tma_load_4d_at(dst + AT_HALF_BYTES, map, 64, I.g, I.k0 + t * AT_TILE, bb, &full[st]);
          ++c;
        };
        for (int s = 0; ok && s < (pair ? 2 : 1); ++s) {
          const uint32_t qb = qn & 1, dst = smem_u32(sm) + qb * AT_TILE_BYTES;
          if (!(ok = attn_wait(&qempty[qb], ((qn >> 1) & 1) ^ 1, status))) break;
          mbar_arrive_expect_tx(&qfull[qb], prefix ? qpbytes : qbytes);
          const int tok = prefix ? 0 : (I.tile0 + s) * P.tpt, bb = prefix ? (I.tile0 + s) * P.nb : I.b * P.mul_q;
          tma_load_4d_at(dst, mq, 0, I.g * P.G, tok, bb, &qfull[qb]);
          tma_load_4d_at(dst + AT_HALF_BYTES, mq, 64, I.g * P.G, tok, bb, &qfull[qb]);
          ++qn;
        }
        const int bk = I.b * P.mul_k, bv = I.b * P.mul_v;
        // in the order of their last use: K0 V0 K1 V1 .. for a pair; K0 K1 V0 K2 V1 K3 .. otherwise
        load(mk, 0, bk);
        if (!pair && I.n > 1) load(mk, 1, bk);
        for (int j = 0; ok && j < I.n; ++j) {
          load(mv, j, bv);
          const int jk = j + (pair ? 1 : 2);
          if (jk < I.n) load(mk, jk, bk);
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0);
      if (!STREAM && lane == 0) mbar_arrive(loaded);
    }
    if (lane == 0) {   // copies still in flight land before the CTA leaves
      for (uint32_t i = c > AT_STAGES ? c - AT_STAGES : 0; i < c; ++i)
        attn_wait(&full[i % AT_STAGES], (i / AT_STAGES) & 1, status);
      for (uint32_t i = qn > 2 ? qn - 2 : 0; i < qn; ++i) attn_wait(&qfull[i & 1], (i >> 1) & 1, status);
    }
    __syncwarp();
  } else if (warp == AT_W_MMA) {
    // ---- MMA issue, the whole warp in step, slot after slot: P V and the next S of slot 0, then of slot 1.  (A warp per
    // slot lets the products of both slots interleave, so each finishes as late as both, and the slots fall into step
    // instead of alternating: 6.99 ms against 5.6 for a 32K prompt of 32 heads.)  A slot's S(i + 1) overwrites P(i) after
    // P V(i): the tensor pipe runs in the order of issue.  The warp meets the ring's tiles in order, so a phase parity is
    // enough.
    constexpr uint32_t ab = FP16 ? 0u : 1u;
    constexpr uint32_t ID_S = (1u << 4) | (ab << 7) | (ab << 10) | ((uint32_t)(AT_TILE >> 3) << 17) |
                              ((uint32_t)(AT_TILE >> 4) << 24);
    constexpr uint32_t ID_O = ID_S | (1u << 16);   // B (values) with its N side contiguous
    const uint64_t dq0 = umma_desc(smem_u32(sm)), dk0 = umma_desc(smem_u32(sm) + AT_OFF_KV),
                   dv0 = umma_desc_v(smem_u32(sm) + AT_OFF_KV);
    uint32_t base = 0, qn = 0, pc0 = 0, pc1 = 0;
    bool ok = true;
    AttnItem I;
    auto issue_s = [&](int s, uint32_t kpos, uint32_t qb, bool last) {
      const uint32_t st = kpos % AT_STAGES;
      ok = attn_wait_warp(&full[st], (kpos / AT_STAGES) & 1, status);
      tc_fence_after();
      tc_mma_tile_ss(tmem + 128 * s, dq0 + qb * (AT_TILE_BYTES >> 4), dk0 + st * (AT_TILE_BYTES >> 4), ID_S);
      tc_commit_elect(&sfull[s]);
      if (last) tc_commit_elect(&empty[st]);
    };
    auto issue_pv = [&](int s, uint32_t vpos, uint32_t pph, bool first, bool final, bool last) {
      const uint32_t st = vpos % AT_STAGES;
      attn_wait(&full[st], (vpos / AT_STAGES) & 1, status);
      ok = attn_wait_warp(&pfull[s], pph, status);
      tc_fence_after();
      tc_mma_tile_ts(tmem + 256 + 128 * s, tmem + 128 * s, dv0 + st * (AT_TILE_BYTES >> 4), ID_O, !first);
      if (last) tc_commit_elect(&empty[st]);
      if (final) {
        tc_commit_elect(&ofull[s]);
        if (lane == 0) mbar_arrive(&ofull[s]);   // orders what the slots wrote (bad_item) before the reader
        __syncwarp();
      }
    };
    while (ok && next_item(I) && I.kind >= 0) {
      const int n = I.n;
      if (n == 0) continue;
      const bool pair = !STREAM || I.pair();
      const uint32_t q0 = qn & 1, q1 = pair ? (qn + 1) & 1 : q0;
      ok = attn_wait_warp(&qfull[q0], (qn >> 1) & 1, status);
      if (pair) ok = ok && attn_wait_warp(&qfull[q1], ((qn + 1) >> 1) & 1, status);
      qn += pair ? 2 : 1;
      if (ok && pair) {
        issue_s(0, base, q0, false);
        if (ok) issue_s(1, base, q1, true);
        for (int i = 0; ok && i < n; ++i) {
          const bool end = i == n - 1;
          if (end) {   // every S of the item has been issued
            tc_commit_elect(&qempty[q0]);
            tc_commit_elect(&qempty[q1]);
          }
          issue_pv(0, base + 1, pc0++ & 1, i == 0, end, false);
          if (ok && !end) issue_s(0, base + 2, q0, false);
          if (ok) issue_pv(1, base + 1, pc1++ & 1, i == 0, end, true);
          if (ok && !end) issue_s(1, base + 2, q1, true);
          base += 2;
        }
      } else if (ok) {
        const int n0 = (n + 1) >> 1, n1 = n >> 1;
        auto kpos = [&](int j) { return base + (j < 2 ? j : 2 * j - 1); };
        auto vpos = [&](int j) { return base + (j + min(n, j + 2)); };
        issue_s(0, base, q0, true);
        if (ok && n1) issue_s(1, base + 1, q0, true);
        for (int i = 0; ok && i < n0; ++i) {
          if (i == n0 - 1) tc_commit_elect(&qempty[q0]);
          issue_pv(0, vpos(2 * i), pc0++ & 1, i == 0, i == n0 - 1, true);
          if (ok && i + 1 < n0) issue_s(0, kpos(2 * i + 2), q0, true);
          if (ok && i < n1) {
            issue_pv(1, vpos(2 * i + 1), pc1++ & 1, i == 0, i == n1 - 1, true);
            if (ok && i + 1 < n1) issue_s(1, kpos(2 * i + 3), q0, true);
          }
        }
        base += 2 * n;
      }
    }
    // every product issued above has completed before the CTA leaves: the softmax warps wait for ofull
  } else {
    // ---- softmax: thread = one row of a tile, one quarter of its columns, slot after slot
    const int quarter = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16) + AT_COLS * quarter;   // S, P and O (+ 256) of slot 0
    float *x_own = xch + quarter * AT_TILE + row;
    const int row_bar = AT_BAR_ROWS + wq;   // the four warps that share these rows
    const AttnRow R = attn_row_of(P, row);
    uint32_t sc0 = 0, sc1 = 0, oc0 = 0, oc1 = 0, base = 0;
    bool ok = true;   // after a wait that ran out the loops go on without waiting, so all warps meet at every barrier
    for (;;) {
      AttnItem I;
      const bool got = next_item(I);
      // all softmax warps go on together or stop together: none is left alone at a barrier
      int stop;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.or.aligned.pred q, %2, %3, p;\n"
          " selp.s32 %0, 1, 0, q;\n}"
          : "=r"(stop)
          : "r"((int)(!got || I.kind < 0)), "r"(AT_BAR_ALL), "r"(AT_SOFT * 32)
          : "memory");
      if (stop) break;
      const bool prefix = STREAM && I.prefix(), pair = !STREAM || I.pair(), parts = STREAM && I.parts();
      // what a thread keeps of its row in each slot (in a single row tile both are the same row)
      struct Slot {
        float m, l;
        int lo, hi, pos;   // pos: an integer, as positions past 2^24 are not all fp32 numbers
        bool any;
      } S0, S1;
      float slope = 0.f;
      auto setup = [&](int slot, Slot &S) {
        int b, i, h, prow;
        const bool valid = attn_row<STREAM>(P, I, slot, R, b, i, h, prow);
        S.any = __any_sync(0xffffffffu, valid);
        S.lo = 0, S.hi = AT_PADDING;   // padding rows take no masks: nothing reads what they compute
        S.m = -AT_BIG, S.l = 0.f, S.pos = 0;
        if (valid) {
          if (prefix) {
            const int p = attn_prefix_pos(P, b, i);
            S.hi = clampi(p + 1, 0, P.pre);
            if (BIAS) S.pos = p;
          } else {
            const int p = I.kl - I.ql + i;
            if (I.clean_lo > 0) {
              const int2 v = attn_interval(P, b, p, I.kl, I.pfx);
              S.lo = v.x - I.k0, S.hi = v.y - I.k0;   // counted from k0, as the tiles are
            } else {   // one document: the rows' first key is k0, their last the item's or their own
              S.hi = P.causal ? min(max(p + 1, I.pfx) - I.k0, I.key_hi) : I.key_hi;
              if (S.hi < 0 || (P.runs && p < 0)) S.hi = 0;
            }
            if (BIAS) S.pos = p - I.k0;
          }
          if (BIAS) slope = P.slopes[h] * 1.4426950408889634f;
        }
      };
      setup(0, S0);
      if (pair)
        setup(1, S1);
      else
        S1 = S0;
      // x = value * scale2: the products themselves, or with BIAS the finished logit
      const float scale2 = BIAS ? 1.f : P.scale_log2;
      const uint64_t scale22 = pack_f2(scale2, scale2);
      // tiles that every row sees whole
      const int clean_lo = (I.clean_lo + AT_TILE - 1) / AT_TILE, clean_hi = I.clean_hi / AT_TILE;
      // Capped products: y with y scale = cap tanh(v scale / cap), tanh(u) = u Q(u^2) with Q fitted at Chebyshev nodes, its
      // coefficients scaled to take v: of degree 2 where no |u| of the warp's rows exceeds 0.25, of degree 4 up to 0.6 (errors
      // 1e-7 and 7e-8 of tanh in fp32).  Beyond, 1 - 2 / (1 + 2^(2 log2e u)) with one reciprocal for two, 1 / a = b / (a b),
      // where 2^60 bounds the exponentials so that the product stays finite.  A 4K prompt of 32 heads takes 99 us without a
      // cap, 137 with one that no logit reaches a quarter of, 153, 175 and 192 with logits two, four and twelve times as
      // large: bound by the FMA pipe's share of each step.
      // Which form a row takes depends on what it sees alone: in a partly masked tile each row goes by its visible keys; in the
      // others, whose keys every row sees, the warp's rows agree, padding rows (whose queries may be anything) having no say.
      auto capped = [&](auto masks, float *v, uint32_t see, bool valid) {
        constexpr bool mixed = decltype(masks)::value;
        auto largest = [&]() {   // |u| of the row's columns; a NaN is passed over, and propagates in every form
          float x0 = 0.f, x1 = 0.f;
#pragma unroll
          for (int c = 0; c < AT_COLS; c += 4) {
            x0 = max3(x0, fabsf(v[c]), fabsf(v[c + 1]));
            x1 = max3(x1, fabsf(v[c + 2]), fabsf(v[c + 3]));
          }
          return valid ? fmaxf(x0, x1) * P.cap_u : 0.f;
        };
        float most = largest();
        if (mixed && see != ~0u && !(most <= P.cap_near)) {   // without the hidden keys
#pragma unroll
          for (int c = 0; c < AT_COLS; ++c)
            if (!(see & (1u << c))) v[c] = 0.f;
          most = largest();
        }
        auto agreed = [&](bool x) { return mixed ? x : (bool)__all_sync(0xffffffffu, x); };
        if (agreed(most <= P.cap_near)) {
          const uint64_t q0 = pack_f2(P.cap_r[0], P.cap_r[0]), q1 = pack_f2(P.cap_r[1], P.cap_r[1]),
                         q2 = pack_f2(P.cap_r[2], P.cap_r[2]);
#pragma unroll
          for (int c = 0; c < AT_COLS; c += 2) {
            const uint64_t v2 = pack_f2(v[c], v[c + 1]), z = mul_f2(v2, v2);
            unpack_f2(v[c], v[c + 1], mul_f2(v2, fma_f2(z, fma_f2(z, q2, q1), q0)));
          }
        } else if (!mixed && agreed(most <= P.cap_mid)) {   // (rows that differ take turns: two forms are enough there)
          const uint64_t q0 = pack_f2(P.cap_q[0], P.cap_q[0]), q1 = pack_f2(P.cap_q[1], P.cap_q[1]),
                         q2 = pack_f2(P.cap_q[2], P.cap_q[2]), q3 = pack_f2(P.cap_q[3], P.cap_q[3]),
                         q4 = pack_f2(P.cap_q[4], P.cap_q[4]);
#pragma unroll
          for (int c = 0; c < AT_COLS; c += 2) {
            const uint64_t v2 = pack_f2(v[c], v[c + 1]), z = mul_f2(v2, v2);
            const uint64_t q = fma_f2(z, fma_f2(z, fma_f2(z, fma_f2(z, q4, q3), q2), q1), q0);
            unpack_f2(v[c], v[c + 1], mul_f2(v2, q));
          }
        } else {
          const float in = P.cap_u * 2.8853900817779268f;   // 2 log2 e
          auto pair_of = [&](float &x, float &y) {   // (hidden keys are 0 here, so no NaN of theirs reaches a neighbour)
            const float a = 1.f + ex2(min_nan(x * in, 60.f)), b = 1.f + ex2(min_nan(y * in, 60.f));
            const float r = rcp_approx(a * b) * (-2.f * P.cap_s);
            x = fmaf(b, r, P.cap_s);
            y = fmaf(a, r, P.cap_s);
          };
          if (CAP == 2) {
            // The difference from cap_s is off by about 2^-22 of the cap, which small logits of a wide cap would feel: up to
            // 0.6 the polynomial of u itself.
            auto near = [&](float x, float far) {
              const float u = x * P.cap_u, z = u * u;
              float y = fmaf(z, (float)TANH_4, (float)TANH_3);
              y = fmaf(z, y, (float)TANH_2);
              y = fmaf(z, y, (float)TANH_1);
              y = fmaf(z, y, (float)TANH_0);
              return fabsf(u) <= 0.6f ? u * y * P.cap_s : far;
            };
#pragma unroll
            for (int c = 0; c < AT_COLS; c += 2) {
              float x = v[c], y = v[c + 1];
              pair_of(x, y);
              v[c] = near(v[c], x);
              v[c + 1] = near(v[c + 1], y);
            }
          } else {
#pragma unroll
            for (int c = 0; c < AT_COLS; c += 2) pair_of(v[c], v[c + 1]);
          }
        }
      };
      // fp16 holds 2^-24 to 2^15 of a power of two: the reference m is the maximum less 7, so that a row's largest probability
      // lies between 2^7 and 2^15, and what is lost below 2^-25 is below 2^-32 of it.  (bf16 has fp32's exponents.)
      constexpr float LIFT = FP16 ? 7.f : 0.f, RISE = 8.f + LIFT, DROP = FP16 ? 0.0078125f : 1.f;   // DROP = 2^-LIFT
      // The exponents are taken from unrounded logits, the maximum is rounded: beyond 2^24 the row's largest may come out as
      // 2^-30 or 2^30, or further.  Running maxima start at -AT_BIG, so that logits far below weigh nothing, and the warp's rows are
      // recomputed from rounded logits when one has ended above AT_BIG, or sees keys and holds a sum l of 0.  (Rounding the
      // logits as they come costs a prompt 6%.)  The four warps that share the rows hold the same maxima and sums.
      auto far_out = [&](const Slot &S, float l) {
        const bool sees = max(S.lo, (I.t_hi - I.n) * AT_TILE) < min(S.hi, I.t_hi * AT_TILE);
        return (bool)__any_sync(0xffffffffu, S.hi != AT_PADDING && ((S.m > AT_BIG && S.m < INFINITY) || (l == 0.f && sees)));
      };
      // One slot's S of key tile j (from the last) into probabilities; first: the slot's first tile
      auto step_of = [&](auto masks, const int slot, Slot &S, uint32_t &sc, int j, bool first) {
        // Some row does not see some key of the tile: a body of its own, since its branches in the common one cost a
        // prompt of 8192 tokens 5%.
        constexpr bool mixed = decltype(masks)::value;
        const int t = I.t_hi - 1 - j;
        const uint32_t ts = lane_base + 128 * slot;
        // Values of a partly masked tile are looked over before P V may run, once for both slots of a pair.  This S, and so
        // every tile of the ring before its keys, has come: the stage's phase cannot be mistaken for the one before.
        auto look = [&]() {
          const uint32_t vpos = base + (pair ? 2 * j + 1 : j + min(I.n, j + 2)), st = vpos % AT_STAGES;
          if (ok) ok = attn_wait(&full[st], (vpos / AT_STAGES) & 1, status);
          attn_clean_values<FP16>(I, t, sm + AT_OFF_KV + st * AT_TILE_BYTES, threadIdx.x, &bad_item[seq & 1], seq);
        };
        if (ok) ok = attn_wait(&sfull[slot], sc & 1, status);
        ++sc;
        __syncwarp();
        tc_fence_after();
        if (S.any) {
          uint32_t raw[AT_COLS];
          float *v = reinterpret_cast<float *>(raw);
          tmem_ld32(ts, raw);
          tmem_wait_ld();
          const int c0 = t * AT_TILE + quarter * AT_COLS;
          uint32_t see = ~0u;
          bool none = false, part = false;   // of the warp's rows and columns none is visible, not all are
          if (mixed) {   // the row sees keys [lo, hi)
            const int a = clampi(S.lo - c0, 0, 32), z = clampi(S.hi - c0, 0, 32);
            see = (z == 32 ? ~0u : (1u << z) - 1u) & (a == 32 ? 0u : ~0u << a);
            none = __all_sync(0xffffffffu, see == 0u);
            part = !__all_sync(0xffffffffu, see == ~0u);
          }
          float base2 = 0.f;       // of every logit of the row in this tile
          float x0 = -INFINITY, x1;
          if (!none) {
            if (CAP) capped(masks, v, see, S.hi != AT_PADDING);
            if (BIAS) {
              const float sl = P.scale_log2, d0 = (float)(S.pos - c0);
              if ((P.causal && !P.prefix_len) || __all_sync(0xffffffffu, d0 >= (float)(AT_COLS - 1))) {
                // no key behind the row's position is seen: -slope |p - j| = -slope (p - c0) + slope (j - c0)
                const uint64_t sl2 = pack_f2(sl, sl), hop = pack_f2(2.f * slope, 2.f * slope);
                uint64_t b2 = pack_f2(0.f, slope);
#pragma unroll
                for (int c = 0; c < AT_COLS; c += 2) {
                  unpack_f2(v[c], v[c + 1], fma_f2(pack_f2(v[c], v[c + 1]), sl2, b2));
                  b2 = add_f2(b2, hop);
                }
                base2 = -slope * d0;
              } else {
#pragma unroll
                for (int c = 0; c < AT_COLS; ++c) v[c] = fmaf(-slope, fabsf(d0 - (float)c), v[c] * sl);
              }
            }
            if (part) {
#pragma unroll
              for (int c = 0; c < AT_COLS; ++c)
                if (!(see & (1u << c))) v[c] = -INFINITY;
            }
            x0 = v[0], x1 = v[1];
#pragma unroll
            for (int c = 2; c < AT_COLS - 2; c += 4) {
              x0 = max3(x0, v[c], v[c + 1]);
              x1 = max3(x1, v[c + 2], v[c + 3]);
            }
            x0 = fmaxf(max3(x0, v[AT_COLS - 2], v[AT_COLS - 1]), x1);
          }
          const float mx = fmaf(x0, scale2, base2);
          const bool grow = mx > S.m + RISE;   // also the first max
          int any;   // one barrier of the four warps: whether a row has grown in one of them
          asm volatile(
              "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.or.aligned.pred q, %2, 128, p;\n"
              " selp.s32 %0, 1, 0, q;\n}"
              : "=r"(any)
              : "r"((int)grow), "r"(row_bar)
              : "memory");
          if (any) {
            *x_own = mx;
            asm volatile("bar.sync %0, 128;" ::"r"(row_bar) : "memory");
            const float all = fmaxf(fmaxf(xch[row], xch[AT_TILE + row]), fmaxf(xch[2 * AT_TILE + row], xch[3 * AT_TILE + row]));
            float f = 1.f;
            if (all > S.m + RISE) {
              f = ex2(S.m - (all - LIFT));
              S.m = all - LIFT;
            }
            S.l *= f;
            if (!first) {
#pragma unroll 1
              for (int q = 0; q < 2; ++q) {
                uint32_t o[16];
                tmem_ld16(ts + 256 + 16 * q, o);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
                tmem_st16(ts + 256 + 16 * q, o);
              }
            }
          }
          const uint64_t mu2 = pack_f2(base2 - S.m, base2 - S.m);
          uint64_t sa = 0, sb = 0;
          uint32_t pk[16];
          if (none) {
#pragma unroll
            for (int c = 0; c < 16; ++c) pk[c] = 0;
            tmem_st16(ts, pk);
          } else {
#pragma unroll
            for (int c = 0; c < AT_COLS; c += 4) {
              float e0, e1, e2, e3;
              unpack_f2(e0, e1, fma_f2(pack_f2(v[c], v[c + 1]), scale22, mu2));
              unpack_f2(e2, e3, fma_f2(pack_f2(v[c + 2], v[c + 3]), scale22, mu2));
              e0 = ex2(e0), e1 = ex2(e1), e2 = ex2(e2), e3 = ex2(e3);
              sa = add_f2(sa, pack_f2(e0, e1));
              sb = add_f2(sb, pack_f2(e2, e3));
              pk[c / 2] = pack2<FP16>(e0, e1);
              pk[c / 2 + 1] = pack2<FP16>(e2, e3);
            }
            tmem_st16(ts, pk);   // over this quarter of S
            unpack_f2(x0, x1, add_f2(sa, sb));
            S.l += x0 + x1;
          }
          tmem_wait_st();
        }
        if (mixed && (slot == 0 || !pair)) look();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[slot]);
      };
      auto step = [&](const int slot, Slot &S, uint32_t &sc, int j, bool first) {
        const int t = I.t_hi - 1 - j;
        if (__builtin_expect(t < clean_lo || t >= clean_hi, 0))
          step_of(std::true_type(), slot, S, sc, j, first);
        else
          step_of(std::false_type(), slot, S, sc, j, first);
      };
      if (pair) {
        for (int j = 0; j < I.n; ++j) {
          const int t = I.t_hi - 1 - j;
          if (__builtin_expect(t < clean_lo || t >= clean_hi, 0)) {
#pragma unroll 1
            for (int s = 0; s < 2; ++s) {   // one copy of the code: it is run once or twice a unit
              Slot S = s ? S1 : S0;
              uint32_t sc = s ? sc1 : sc0;
              step_of(std::true_type(), s, S, sc, j, j == 0);
              if (s)
                S1 = S, sc1 = sc;
              else
                S0 = S, sc0 = sc;
            }
          } else {
            step_of(std::false_type(), 0, S0, sc0, j, j == 0);
            step_of(std::false_type(), 1, S1, sc1, j, j == 0);
          }
        }
      } else if (STREAM) {
        for (int j = 0; j < I.n; j += 2) {
          step(0, S0, sc0, j, j == 0);
          if (j + 1 < I.n) step(1, S1, sc1, j + 1, j == 0);
        }
      }
      // ---- the item's rows are done: the sums over the quarters, and the outputs
      if (!STREAM) {
        // Whole units: two quarters of the warps finish each slot, half of its columns a thread, so that what a row costs
        // is paid once.  The sums change hands while the last products run.
        const int slot = quarter >> 1, side = quarter & 1;
        float l = 0.f;
        bool bad = false;
        if (I.n > 0) {
          auto row_sum = [&](float x) {
            asm volatile("bar.sync %0, 128;" ::"r"(row_bar) : "memory");   // what stood in xch has been read
            *x_own = x;
            asm volatile("bar.sync %0, 128;" ::"r"(row_bar) : "memory");
            return (xch[row] + xch[AT_TILE + row]) + (xch[2 * AT_TILE + row] + xch[3 * AT_TILE + row]);
          };
          const float l0 = row_sum(S0.l), l1 = row_sum(S1.l);
          l = slot ? l1 : l0;
          if (ok) ok = attn_wait(&ofull[slot], oc0 & 1, status);
          ++oc0;
          __syncwarp();
          tc_fence_after();
          bad = bad_item[seq & 1] == (int)seq || far_out(slot ? S1 : S0, l);
        }
        const uint32_t to = tmem + ((uint32_t)(wq * 32) << 16) + 256 + 128 * slot + 64 * side;
        const bool any_row = slot ? S1.any : S0.any;
        int b, i, h, prow;
        const bool valid = attn_row<false>(P, I, slot, R, b, i, h, prow);
        if (any_row && !bad) {
          const float inv = l == 0.f ? 0.f : rcp_approx(l);   // an empty row is 0
          if (valid && side == 0 && P.lse)
            P.lse[((int64_t)b * P.s_q + i) * P.h_q + h] =
                l == 0.f ? -INFINITY : ((slot ? S1.m : S0.m) + LIFT + lg2_approx(l * DROP)) * 0.69314718055994531f;
          const int64_t at = b * P.so[0] + i * P.so[1] + h * P.so[2] + 64 * side;
          const uint32_t rows = __ballot_sync(0xffffffffu, valid);
#pragma unroll 1
          for (int part = 0; part < 2; ++part) {
            uint32_t o[32];
            const float *of = reinterpret_cast<const float *>(o);
            if (I.n > 0) {
              tmem_ld32(to + 32 * part, o);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = 0;
            }
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) w[c] = pack2<FP16>(of[2 * c] * inv, of[2 * c + 1] * inv);
            attn_store_rows(static_cast<uint16_t *>(P.out) + 32 * part, at, rows, lane, P.wide_out, w);
            __syncwarp();
          }
        } else if (any_row && side == 0) {
          attn_exact_rows<FP16, false>(P, I, slot, wq, lane, CAP,
                                       [&](int rb, int ri, int rh, int, const float (&acc)[4], float rm, float rl) {
            const float f = rl == 0.f ? 0.f : 1.f / rl;
            if (lane == 0 && P.lse)
              P.lse[((int64_t)rb * P.s_q + ri) * P.h_q + rh] = rl == 0.f ? -INFINITY : (rm + log2f(rl)) * 0.69314718055994531f;
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.out) + rb * P.so[0] + ri * P.so[1] + rh * P.so[2] + 4 * lane) =
                rl == 0.f ? make_uint2(0, 0) : make_uint2(pack2<FP16>(acc[0] * f, acc[1] * f), pack2<FP16>(acc[2] * f, acc[3] * f));
          });
        }
        base += 2 * I.n;
        continue;
      }
      const bool join = STREAM && !pair && I.n > 1;   // a single row tile: slot 1 holds the same rows' other key tiles
      const int slots = I.n == 0 ? 0 : pair || join ? 2 : 1;
      auto whole_row = [&](const int slot, Slot &S, uint32_t &oc) {
        if (ok) ok = attn_wait(&ofull[slot], oc & 1, status);
        ++oc;
        asm volatile("bar.sync %0, 128;" ::"r"(row_bar) : "memory");   // what stood in xch has been read
        *x_own = S.l;
        asm volatile("bar.sync %0, 128;" ::"r"(row_bar) : "memory");
        S.l = (xch[row] + xch[AT_TILE + row]) + (xch[2 * AT_TILE + row] + xch[3 * AT_TILE + row]);
      };
      if (slots > 0) whole_row(0, S0, oc0);
      if (slots > 1) whole_row(1, S1, oc1);
      __syncwarp();
      tc_fence_after();
      const bool bad_values = I.n > 0 && bad_item[seq & 1] == (int)seq;
      float *part_o = prefix ? P.pre_o : P.part_o;
      float2 *part_l = prefix ? P.pre_l : P.part_l;
      const int64_t part_row = (int64_t)I.part * (prefix ? P.pre_rows : P.part_rows);
#pragma unroll 1
      for (int slot = 0; slot < (pair ? 2 : 1); ++slot) {
        const float m0 = slot ? S1.m : S0.m, l0 = slot ? S1.l : S0.l, m1 = join ? S1.m : -AT_BIG, l1 = join ? S1.l : 0.f;
        const bool any_row = slot ? S1.any : S0.any;
        const uint32_t to = lane_base + 256 + 128 * slot;
        int b, i, h, prow;
        const bool valid = attn_row<STREAM>(P, I, slot, R, b, i, h, prow);
        if (!any_row) continue;
        const float mu = fmaxf(m0, m1);
        const float w0 = join ? ex2(m0 - mu) : 1.f, w1 = join ? ex2(m1 - mu) : 0.f;
        const float lt = join ? l0 * w0 + l1 * w1 : l0;
        const float inv = lt == 0.f ? 0.f : rcp_approx(lt);   // an empty row is 0
        Slot Sm = slot ? S1 : S0;
        Sm.m = mu;
        if (!bad_values && !(I.n > 0 && far_out(Sm, lt))) {
          if (valid && quarter == 0) {
            if (parts)
              part_l[part_row + prow] = make_float2(mu, lt);
            else if (P.lse)
              P.lse[((int64_t)b * P.s_q + i) * P.h_q + h] =
                  lt == 0.f ? -INFINITY : (mu + LIFT + lg2_approx(lt * DROP)) * 0.69314718055994531f;
          }
          const bool have0 = I.n > 0;
          const float f0 = w0 * inv, f1 = w1 * inv;
          // 16 channels of the row, scaled, as fp32
          auto take = [&](int q, uint32_t (&o)[16]) {
            float *of = reinterpret_cast<float *>(o);
            __syncwarp();
            if (have0) {
              tmem_ld16(to + 16 * q, o);
              if (join) {
                uint32_t o1[16];
                tmem_ld16(to + 128 + 16 * q, o1);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; ++c) of[c] = of[c] * f0 + __uint_as_float(o1[c]) * f1;
              } else {
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; ++c) of[c] = of[c] * f0;
              }
            }
            else {
#pragma unroll
              for (int c = 0; c < 16; ++c) of[c] = 0.f;
            }
          };
          if (parts) {
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
              uint32_t o[16];
              take(q, o);
              float *dst = part_o + (part_row + prow) * D + AT_COLS * quarter + 16 * q;
              if (valid && lt != 0.f) {
                st_global_v8(dst, o);
                st_global_v8(dst + 8, o + 8);
              }
            }
          } else {
            uint32_t w[16];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t o[16];
              take(q, o);
              const float *of = reinterpret_cast<const float *>(o);
#pragma unroll
              for (int c = 0; c < 8; ++c) w[8 * q + c] = pack2<FP16>(of[2 * c], of[2 * c + 1]);
            }
            attn_store_rows(static_cast<uint16_t *>(P.out), b * P.so[0] + i * P.so[1] + h * P.so[2] + AT_COLS * quarter,
                            __ballot_sync(0xffffffffu, valid), lane, P.wide_out, w);
          }
        } else if (quarter == 0) {
          attn_exact_rows<FP16, true>(P, I, slot, wq, lane, CAP,
                                [&](int rb, int ri, int rh, int rp, const float (&acc)[4], float rm, float rl) {
            const float ri_l = rl == 0.f ? 0.f : 1.f / rl;
            const float o0 = rl == 0.f ? 0.f : acc[0] * ri_l, o1 = rl == 0.f ? 0.f : acc[1] * ri_l;
            const float o2 = rl == 0.f ? 0.f : acc[2] * ri_l, o3 = rl == 0.f ? 0.f : acc[3] * ri_l;
            if (parts) {
              if (lane == 0) part_l[part_row + rp] = make_float2(rm, rl);
              *reinterpret_cast<float4 *>(part_o + (part_row + rp) * D + 4 * lane) = make_float4(o0, o1, o2, o3);
            } else {
              if (lane == 0 && P.lse)
                P.lse[((int64_t)rb * P.s_q + ri) * P.h_q + rh] =
                    rl == 0.f ? -INFINITY : (rm + log2f(rl)) * 0.69314718055994531f;
              *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.out) + rb * P.so[0] + ri * P.so[1] + rh * P.so[2] +
                                         4 * lane) = make_uint2(pack2<FP16>(o0, o1), pack2<FP16>(o2, o3));
            }
          });
        }
      }
      base += 2 * I.n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == AT_W_MMA) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// (Programmatic launch: the kernel's setup overlaps the end of the one before.)
template <typename Kernel>
cudaError_t launch_attn_kernel(Kernel kern, const AttnArgs &P, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(AT_THREADS);
  cfg.dynamicSmemBytes = AT_SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, P);
}

template <bool FP16, int CAP, bool BIAS>
cudaError_t launch_attn_variant(const AttnArgs &P, int grid, cudaStream_t s) {
  static SmemOptIn units, stream;
  cudaError_t e = P.stream ? stream.ensure(attn_kernel<FP16, CAP, BIAS, true>, AT_SMEM)
                           : units.ensure(attn_kernel<FP16, CAP, BIAS, false>, AT_SMEM);
  if (e != cudaSuccess) return e;
  return P.stream ? launch_attn_kernel(attn_kernel<FP16, CAP, BIAS, true>, P, grid, s)
                  : launch_attn_kernel(attn_kernel<FP16, CAP, BIAS, false>, P, grid, s);
}

}  // namespace qv
