// Attention over a dense KV cache and of a batch behind a shared prefix: argument checks, split rules,
// workspace layout, the document scan and the merge of split results.  The attention kernel itself is in
// attn_dev.cuh.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn_dev.cuh"
#include "qevict.h"

namespace qv {
cudaError_t launch_attn_bf16(const AttnArgs &P, int grid, bool bias, cudaStream_t s);
cudaError_t launch_attn_fp16(const AttnArgs &P, int grid, bool bias, cudaStream_t s);
cudaError_t launch_attn_bf16_cap(const AttnArgs &P, int grid, bool bias, cudaStream_t s);
cudaError_t launch_attn_fp16_cap(const AttnArgs &P, int grid, bool bias, cudaStream_t s);
cudaError_t launch_attn_bf16_wide(const AttnArgs &P, int grid, bool bias, cudaStream_t s);
cudaError_t launch_attn_fp16_wide(const AttnArgs &P, int grid, bool bias, cudaStream_t s);

// First and past-the-last position of every position's run of equal ids.  One CTA per sequence; thread i takes the i-th of
// 1024 consecutive pieces, finds the first and last run start in it, and scans over the warp and then over the warps carry
// the last start before and the first start after each piece.  Bound by latency: reads 4 bytes and writes 8 a position.
constexpr int RUN_THREADS = 1024;
__global__ void __launch_bounds__(RUN_THREADS) doc_runs_kernel(const int *ids, int s_kv, int2 *runs) {
  __shared__ int w_last[32], w_first[32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the attention kernel waits for this one to end
  const int *id = ids + (size_t)blockIdx.x * s_kv;
  int2 *out = runs + (size_t)blockIdx.x * s_kv;
  const int piece = (s_kv + RUN_THREADS - 1) / RUN_THREADS, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int lo = min((int64_t)s_kv, (int64_t)t * piece), hi = min(s_kv, lo + piece);
  auto starts = [&](int p) { return p == 0 || id[p] != id[p - 1]; };
  int f = s_kv, l = -1;
  for (int p = lo; p < hi; ++p)
    if (starts(p)) {
      if (f == s_kv) f = p;
      l = p;
    }
  auto scan = [&](int &a, int &b) {   // inclusive over the lanes: maximum from the left, minimum from the right
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_down_sync(0xffffffffu, b, o);
      if (lane >= o) a = max(a, x);
      if (lane + o < 32) b = min(b, y);
    }
  };
  int wl = l, wf = f;
  scan(wl, wf);
  if (lane == 31) w_last[warp] = wl;
  if (lane == 0) w_first[warp] = wf;
  __syncthreads();
  if (warp == 0) {
    int a = w_last[lane], b = w_first[lane];
    scan(a, b);
    w_last[lane] = a;
    w_first[lane] = b;
  }
  __syncthreads();
  // last start before this thread's piece, first start behind it
  int before = __shfl_up_sync(0xffffffffu, wl, 1), after = __shfl_down_sync(0xffffffffu, wf, 1);
  if (lane == 0) before = -1;
  if (lane == 31) after = s_kv;
  if (warp > 0) before = max(before, w_last[warp - 1]);
  if (warp < 31) after = min(after, w_first[warp + 1]);
  int begin = max(before, 0), end = 0;   // of the run at hand
  for (int p = lo; p < hi; ++p) {
    if (p == lo || starts(p)) {
      if (starts(p)) begin = p;
      end = p + 1;
      while (end < hi && !starts(end)) ++end;
      if (end == hi) end = after;
    }
    out[p] = make_int2(begin, end);
  }
}

// WARPS warps per row (sequence, query, head): out = sum_s w_s out_s / sum_s w_s over the parts of the row's units, with
// w_s = l_s 2^(m_s - max m); 520 bytes per part and row, read once, eight loads of a warp at a time.  Which parts a row has
// is worked out as the attention kernel did, before that kernel is waited for.  Four warps a row where rows are few: latency.
// A thread without work waits too: what follows in the stream is ordered behind this kernel, and through it behind that one.
template <bool FP16, int WARPS>
__global__ void __launch_bounds__(128) attn_combine_kernel(const __grid_constant__ AttnArgs P, int ctas) {
  const int lane = threadIdx.x & 31, warp = WARPS == 1 ? 0 : threadIdx.x >> 5;
  const uint32_t row = WARPS == 1 ? blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;   // fewer than 2^31
  const uint32_t x = row / (uint32_t)P.h_q;
  const int h = (int)(row - x * P.h_q), b = (int)(x / (uint32_t)P.s_q), i = (int)(x - (uint32_t)b * P.s_q);
  if (b >= P.batch) return attn_wait_previous();
  const int g = h / P.G, hr = h - g * P.G, pr = i / (2 * P.tpt), gi = pr * P.batch + b;
  const AttnGroup A = attn_group(P, gi);
  if (i >= A.ql) return attn_wait_previous();
  const int tp = P.pre ? (P.pre + AT_TILE - 1) / AT_TILE : 0, wp = attn_places(tp);
  const int all_p = P.pre ? P.n_prp * P.h_kv * wp : 0;
  int all = 0, before = 0;   // places of all groups, and of those before this one
#pragma unroll 2
  for (int j = lane; j < P.n_pr * P.batch; j += 32) {
    const AttnGroup B = attn_group(P, j);
    const int w = attn_places(B.tiles);
    all += w;
    if (j < gi) before += w;
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  const int share = attn_share(all_p + all * P.h_kv, ctas, P.min_tiles);
  const int t = A.tiles, u0 = all_p + before * P.h_kv + g * attn_places(t);
  // own parts: the CTAs whose shares hold tiles u0 .. u0 + t - 1
  const int c_own = u0 / share, n_own = t ? (u0 + t - 1) / share - c_own + 1 : 0;
  if (!P.pre && n_own == 1) return attn_wait_previous();   // the unit was not cut: the row is written
  const int64_t own_row = (int64_t)(c_own + gi * P.h_kv + g) * P.part_rows + (int64_t)(i - pr * 2 * P.tpt) * P.G + hr;
  int n_pre = 0;
  int64_t pre_row = 0;
  if (P.pre) {
    const int prp = b / (2 * P.nb), u = prp * P.h_kv + g, c0 = u * wp / share;
    n_pre = (u * wp + tp - 1) / share - c0 + 1;
    pre_row = (int64_t)(c0 + u) * P.pre_rows + (int64_t)((b - prp * 2 * P.nb) * P.s_q + i) * P.G + hr;
  }
  const int n = n_pre + n_own;
  attn_wait_previous();
  auto sum_of = [&](int s) {   // (m, l)
    return s < n_pre ? P.pre_l[pre_row + (int64_t)s * P.pre_rows] : P.part_l[own_row + (int64_t)(s - n_pre) * P.part_rows];
  };
  float mx = -INFINITY;
  for (int s = lane; s < n; s += 32) {
    const float2 ml = sum_of(s);
    if (ml.y != 0.f) mx = fmaxf(mx, ml.x);
  }
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float mu = mx == -INFINITY ? 0.f : mx;
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < n; s0 += 8 * WARPS) {   // every warp knows the weights of these parts, and reads its eight
    // -1: no such part, or one without keys for the row, which wrote no output.  A weight that underflows to 0 counts: what
    // is infinite or NaN in a visible value stays so.
    float w = -1.f;
    if (lane < 8 * WARPS && s0 + lane < n) {
      const float2 ml = sum_of(s0 + lane);
      if (ml.y != 0.f) {
        w = ml.y * ex2(ml.x - mu);
        l += w;
      }
    }
    float4 o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int s = s0 + WARPS * k + warp;
      const float *src = s < n_pre ? P.pre_o + (pre_row + (int64_t)s * P.pre_rows) * D
                                   : P.part_o + (own_row + (int64_t)(s - n_pre) * P.part_rows) * D;
      if (s < n) o[k] = *reinterpret_cast<const float4 *>(src + 4 * lane);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float ws = __shfl_sync(0xffffffffu, w, WARPS * k + warp);
      if (!(ws < 0.f)) {   // a NaN weight goes on
        acc.x = fmaf(ws, o[k].x, acc.x);
        acc.y = fmaf(ws, o[k].y, acc.y);
        acc.z = fmaf(ws, o[k].z, acc.z);
        acc.w = fmaf(ws, o[k].w, acc.w);
      }
    }
  }
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (WARPS > 1) {
    __shared__ float4 sums[WARPS][32];
    sums[warp][lane] = acc;
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int k = 1; k < WARPS; ++k) {
      const float4 o = sums[k][lane];
      acc.x += o.x;
      acc.y += o.y;
      acc.z += o.z;
      acc.w += o.w;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.out) + b * P.so[0] + i * P.so[1] + h * P.so[2] + 4 * lane) =
      make_uint2(pack2<FP16>(acc.x * inv, acc.y * inv), pack2<FP16>(acc.z * inv, acc.w * inv));
  if (lane == 0 && P.lse) P.lse[row] = l == 0.f ? -INFINITY : (mu + log2f(l)) * 0.69314718055994531f;
}

namespace {

int64_t align256(int64_t x) { return (x + 255) & ~int64_t(255); }

int sm_count() {   // of the current device
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64) {
    if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0) {
      known[dev].store(n, std::memory_order_relaxed);
      return n;
    }
  }
  cudaGetLastError();
  return 152;
}

// [tokens][heads][128] tensors of `batch` sequences as a 4-D tensor map; a box is 64 channels x `bh` heads x
// `bt` tokens x `bb` sequences, 128-byte swizzled.  batch: 1 when the batch stride is 0.
bool dense_map(CUtensorMap *map, bool fp16, const void *base, int64_t heads, int64_t tokens, int64_t batch, int64_t st_h,
               int64_t st_t, int64_t st_b, int bh, int bt, int bb) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)batch};
  // a dimension of one element has no step: any valid one will do
  const cuuint64_t strides[3] = {(cuuint64_t)(heads > 1 ? st_h : D) * 2, (cuuint64_t)(tokens > 1 ? st_t : D) * 2,
                                 (cuuint64_t)(batch > 1 ? st_b : D) * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)bh, (cuuint32_t)bt, (cuuint32_t)bb};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct AttnPlan {
  int G, tpt, n_pr, stream, grid;
  int pre, nb, n_prp;
  int part_rows, pre_rows;
  int64_t rows, off_runs, off_l, off_o, off_pl, off_po, bytes;
};

// Key tiles that a CTA takes at least: a token of 8 heads against 16K keys takes 12 us with 2, 13.6 with 1, 13.2 with 6;
// against 1K keys 10, 9.6 and 13 us.
constexpr int MIN_TILES = 2;
// Row tiles against up to this many key tiles are not cut where there are half as many of them as SMs: 16 tokens of 32 heads
// against 1K keys take 16 us whole, 19 as parts; 64 of different lengths up to 1K 42 and 48 us.
constexpr int WHOLE_TILES = 8;

// Caps from here on take the instances that keep small logits exact beside large ones: the others' error of 2^-22 of the cap
// is 2^-16 of a weight at 64.
constexpr float WIDE_CAP = 64.f;

bool stride_ok(int64_t st, int64_t size, bool zero) {
  if (size <= 1) return true;
  return st % 8 == 0 && st < (1ll << 38) && st <= (1ll << 48) / (size - 1) && (st > 0 || (zero && st == 0));
}

float logit_scale(const qevict_attn_desc *d) { return d->scale > 0.f ? d->scale : 1.f / std::sqrt((float)D); }

qevict_status attn_plan(const qevict_attn_desc *d, int s_prefix, AttnPlan *p) {
  if (!d || d->dtype < 0 || d->dtype > 1 || d->batch < 1 || d->s_q < 1 || d->s_kv < 1 || d->h_kv < 1 || d->h_q < d->h_kv ||
      d->h_q % d->h_kv || d->h_q / d->h_kv > AT_TILE || d->d_head != D || d->causal < 0 || d->causal > 1 ||
      !(d->scale >= 0.f) || !std::isfinite(d->scale) || !(d->softcap >= 0.f) || !std::isfinite(d->softcap))
    return QEVICT_EINVAL;
  if (d->softcap > 0.f) {   // scale / cap to its eighth power, and cap / scale, stay finite in fp32
    const double cap = (double)d->softcap / logit_scale(d);
    if (cap < 0x1p-14 || cap > 0x1p100) return QEVICT_EINVAL;
  }
  if (d->s_q > (1 << 30) || d->s_kv > (1 << 30) || s_prefix < 0 || s_prefix > (1 << 30)) return QEVICT_EINVAL;
  for (int n = 0; n < 3; ++n) {
    const int64_t *st = n == 0 ? d->q : n == 1 ? d->k : d->v;
    if (!stride_ok(st[0], d->batch, true) || !stride_ok(st[1], n ? d->s_kv : d->s_q, false) ||
        !stride_ok(st[2], n ? d->h_kv : d->h_q, false))
      return QEVICT_EINVAL;
  }
  if (!stride_ok(d->o[0], d->batch, false) || !stride_ok(d->o[1], d->s_q, false) || !stride_ok(d->o[2], d->h_q, false))
    return QEVICT_EINVAL;
  *p = AttnPlan();
  p->G = d->h_q / d->h_kv;
  p->tpt = AT_TILE / p->G;
  const int64_t sms = sm_count();
  const int64_t n_qt = (d->s_q + p->tpt - 1) / p->tpt, n_pr = (n_qt + 1) / 2, groups = n_pr * d->batch;
  if (groups > (1 << 24) || groups * d->h_kv > (1 << 24)) return QEVICT_EINVAL;   // each factor first: no product wraps
  const int64_t units = groups * d->h_kv, tiles = (d->s_kv + AT_TILE - 1) / AT_TILE;
  p->rows = (int64_t)d->batch * d->s_q * d->h_q;   // at most 256 a unit
  int64_t total = units * (tiles + AT_UNIT_COST);   // places of the stream, at most
  p->n_pr = (int)n_pr;
  if (s_prefix) {
    if (!d->causal || (int64_t)d->s_q * p->G > AT_TILE) return QEVICT_EINVAL;
    p->pre = s_prefix;
    p->nb = std::min(p->tpt / d->s_q, 256);
    const int64_t n_qtp = (d->batch + p->nb - 1) / p->nb;
    p->n_prp = (int)((n_qtp + 1) / 2);
    total += (int64_t)p->n_prp * d->h_kv * ((s_prefix + AT_TILE - 1) / AT_TILE + AT_UNIT_COST);
  }
  // One stream of key tiles cut into equal shares, or whole units in turn.  The stream evens out caches of different
  // lengths and fills the SMs when there are few units, at the price of parts that are merged afterwards.  Units of one
  // row tile have few rows to merge.  Pairs have 256, which costs as much as about 16 key tiles: prompts of 512 and 1024
  // tokens of 32 heads take 29 and 43 us as a stream, 12.5 and 19 as units; the last 256 tokens of 32K, which would fill
  // 32 of the SMs as units, 113 us as a stream.
  p->stream = s_prefix || (tiles > MIN_TILES && (n_qt == 1 ? tiles > WHOLE_TILES || 2 * units < sms
                                                           : tiles * (sms - std::min(units, sms)) >= 16 * sms));
  if ((total > (1 << 30) || p->rows > (1ll << 30)) && p->stream) {
    if (s_prefix) return QEVICT_EINVAL;
    p->stream = 0;
  }
  p->grid = (int)std::min(sms, p->stream ? (total + MIN_TILES - 1) / MIN_TILES : units);
  int64_t off = 256;
  auto take = [&](int64_t n) {
    const int64_t o = off;
    off += align256(n);
    return o;
  };
  if (!s_prefix) p->off_runs = take((int64_t)d->batch * d->s_kv * 8);
  if (p->stream) {
    p->part_rows = std::min(d->s_q, 2 * p->tpt) * p->G;
    const int64_t parts = p->grid + units;
    p->off_l = take(parts * p->part_rows * 8);
    p->off_o = take(parts * p->part_rows * D * 4);
  }
  if (s_prefix) {
    p->pre_rows = std::min(d->batch, 2 * p->nb) * d->s_q * p->G;
    const int64_t parts = p->grid + (int64_t)p->n_prp * d->h_kv;
    p->off_pl = take(parts * p->pre_rows * 8);
    p->off_po = take(parts * p->pre_rows * D * 4);
  }
  p->bytes = off;
  return QEVICT_OK;
}

bool o_disjoint(const qevict_attn_desc *d) {
  int64_t size[3] = {d->batch, d->s_q, d->h_q}, reach = D;
  for (int n = 0; n < 3; ++n) {
    int best = -1;
    for (int i = 0; i < 3; ++i)
      if (size[i] > 1 && (best < 0 || d->o[i] < d->o[best])) best = i;
    if (best < 0) break;
    if (d->o[best] < reach) return false;
    reach += d->o[best] * (size[best] - 1);
    size[best] = 1;
  }
  return true;
}

qevict_status attn_launch(const qevict_attn_desc *d, const AttnPlan &pl, const qevict_attn_mask *mask,
                          const qevict_prefix_attn_desc *pd, const void *q, const void *kp, const void *vp, const void *k,
                          const void *v, void *out, float *lse, void *d_work, size_t bytes, cudaStream_t s) {
  if (!q || !k || !v || !out || !d_work || (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)out) & 15) ||
      ((uintptr_t)lse & 3) || ((uintptr_t)d_work & 255) || !o_disjoint(d))
    return QEVICT_EINVAL;
  qevict_attn_mask none = {};
  const qevict_attn_mask &m = mask ? *mask : none;
  if (((uintptr_t)m.slopes | (uintptr_t)m.q_len | (uintptr_t)m.kv_len | (uintptr_t)m.prefix_len | (uintptr_t)m.doc_ids) & 3)
    return QEVICT_EINVAL;
  if (m.prefix_len && !d->causal) return QEVICT_EINVAL;
  if ((int64_t)bytes < pl.bytes) return QEVICT_ENOMEM;
  uint8_t *w = static_cast<uint8_t *>(d_work);
  AttnArgs A = {};
  A.q = q, A.k = k, A.v = v, A.kp = kp, A.vp = vp;
  A.out = out;
  A.lse = lse;
  A.status = reinterpret_cast<int *>(w);
  A.drawn = A.status + 32;
  A.slopes = m.slopes, A.q_len = m.q_len, A.kv_len = m.kv_len, A.prefix_len = m.prefix_len;
  for (int i = 0; i < 3; ++i) A.sq[i] = d->q[i], A.sk[i] = d->k[i], A.sv[i] = d->v[i], A.so[i] = d->o[i];
  A.batch = d->batch, A.s_q = d->s_q, A.s_kv = d->s_kv, A.h_q = d->h_q, A.h_kv = d->h_kv, A.G = pl.G, A.causal = d->causal;
  A.mul_q = d->batch > 1 && d->q[0] ? 1 : 0;
  A.mul_k = d->batch > 1 && d->k[0] ? 1 : 0;
  A.mul_v = d->batch > 1 && d->v[0] ? 1 : 0;
  A.wide_out = ((uintptr_t)out & 31) == 0 && (d->batch == 1 || d->o[0] % 16 == 0) && (d->s_q == 1 || d->o[1] % 16 == 0) &&
               (d->h_q == 1 || d->o[2] % 16 == 0);
  A.tpt = pl.tpt, A.n_pr = pl.n_pr;
  A.pre = pl.pre, A.nb = std::max(1, pl.nb), A.n_prp = pl.n_prp;
  A.part_rows = pl.part_rows, A.pre_rows = pl.pre_rows;
  A.stream = pl.stream, A.min_tiles = MIN_TILES;
  const float scale = logit_scale(d), log2e = 1.4426950408889634f;
  A.scale_log2 = scale * log2e;
  if (d->softcap > 0.f) {
    A.cap_u = scale / d->softcap;
    A.cap_s = d->softcap / scale;
    const double q[5] = {TANH_0, TANH_1, TANH_2, TANH_3, TANH_4};
    const double r[3] = {0.9999995827674866, -0.3332192897796631, 0.12841935455799103};
    const double u = A.cap_u;
    for (int i = 0; i < 5; ++i) A.cap_q[i] = (float)(q[i] * std::pow(u, 2 * i));
    for (int i = 0; i < 3; ++i) A.cap_r[i] = (float)(r[i] * std::pow(u, 2 * i));
    // where the last coefficients are normal numbers: 0.128 u^4 and 0.0155 u^8 above 2^-126 (and so the squares of products up
    // to the cap below 2^128)
    A.cap_near = A.cap_s <= 0x1p30f ? 0.25f : -1.f;
    A.cap_mid = A.cap_s <= 0x1p15f ? 0.6f : -1.f;
  }
  const bool fp16 = d->dtype == QEVICT_FP16;
  const int qb = A.mul_q ? d->batch : 1, kb = A.mul_k ? d->batch : 1, vb = A.mul_v ? d->batch : 1;
  bool ok = dense_map(&A.tq, fp16, q, d->h_q, d->s_q, qb, d->q[2], d->q[1], d->q[0], pl.G, pl.tpt, 1) &&
            dense_map(&A.tk, fp16, k, d->h_kv, d->s_kv, kb, d->k[2], d->k[1], d->k[0], 1, AT_TILE, 1) &&
            dense_map(&A.tv, fp16, v, d->h_kv, d->s_kv, vb, d->v[2], d->v[1], d->v[0], 1, AT_TILE, 1);
  if (pd) {
    A.skp[0] = pd->k_prefix[0], A.skp[1] = pd->k_prefix[1], A.svp[0] = pd->v_prefix[0], A.svp[1] = pd->v_prefix[1];
    ok = ok && dense_map(&A.tqp, fp16, q, d->h_q, d->s_q, d->batch, d->q[2], d->q[1], d->q[0], pl.G, d->s_q, pl.nb) &&
         dense_map(&A.tkp, fp16, kp, d->h_kv, pl.pre, 1, pd->k_prefix[1], pd->k_prefix[0], 0, 1, AT_TILE, 1) &&
         dense_map(&A.tvp, fp16, vp, d->h_kv, pl.pre, 1, pd->v_prefix[1], pd->v_prefix[0], 0, 1, AT_TILE, 1);
  }
  if (!ok) return QEVICT_EINVAL;
  if (m.doc_ids) {
    A.runs = reinterpret_cast<int2 *>(w + pl.off_runs);
    doc_runs_kernel<<<d->batch, RUN_THREADS, 0, s>>>(m.doc_ids, d->s_kv, const_cast<int2 *>(A.runs));
    if (cudaGetLastError() != cudaSuccess) return QEVICT_ECUDA;
  }
  if (pl.stream) {
    A.part_l = reinterpret_cast<float2 *>(w + pl.off_l);
    A.part_o = reinterpret_cast<float *>(w + pl.off_o);
    A.pre_l = reinterpret_cast<float2 *>(w + pl.off_pl);
    A.pre_o = reinterpret_cast<float *>(w + pl.off_po);
  }
  const auto launch = d->softcap > WIDE_CAP ? (fp16 ? launch_attn_fp16_wide : launch_attn_bf16_wide)
                      : d->softcap > 0.f    ? (fp16 ? launch_attn_fp16_cap : launch_attn_bf16_cap)
                                            : (fp16 ? launch_attn_fp16 : launch_attn_bf16);
  if (launch(A, pl.grid, m.slopes != nullptr, s) != cudaSuccess) return QEVICT_ECUDA;
  if (pl.stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const bool few = pl.rows <= 1024;
    cfg.gridDim = dim3((unsigned)(few ? pl.rows : (pl.rows + 3) / 4));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const auto combine = few ? (fp16 ? attn_combine_kernel<true, 4> : attn_combine_kernel<false, 4>)
                             : (fp16 ? attn_combine_kernel<true, 1> : attn_combine_kernel<false, 1>);
    if (cudaLaunchKernelEx(&cfg, combine, A, pl.grid) != cudaSuccess) return QEVICT_ECUDA;
  }
  return QEVICT_OK;
}

}  // namespace
}  // namespace qv

extern "C" {

qevict_status qevict_attn_bytes(const qevict_attn_desc *desc, size_t *bytes) {
  qv::AttnPlan p;
  if (!bytes) return QEVICT_EINVAL;
  const qevict_status st = qv::attn_plan(desc, 0, &p);
  if (st == QEVICT_OK) *bytes = (size_t)p.bytes;
  return st;
}

qevict_status qevict_attn(const qevict_attn_desc *desc, const qevict_attn_mask *mask, const void *q, const void *k,
                          const void *v, void *out, float *lse, void *d_work, size_t bytes, qevict_stream_t stream) {
  qv::AttnPlan p;
  const qevict_status st = qv::attn_plan(desc, 0, &p);
  if (st != QEVICT_OK) return st;
  return qv::attn_launch(desc, p, mask, nullptr, q, nullptr, nullptr, k, v, out, lse, d_work, bytes,
                         reinterpret_cast<cudaStream_t>(stream));
}

static qevict_status prefix_plan(const qevict_prefix_attn_desc *d, qv::AttnPlan *p) {
  if (!d || d->s_prefix < 1) return QEVICT_EINVAL;
  if (!qv::stride_ok(d->k_prefix[0], d->s_prefix, false) || !qv::stride_ok(d->v_prefix[0], d->s_prefix, false) ||
      !qv::stride_ok(d->k_prefix[1], d->attn.h_kv, false) || !qv::stride_ok(d->v_prefix[1], d->attn.h_kv, false))
    return QEVICT_EINVAL;
  if (d->attn.batch > 1 && d->attn.q[0] == 0) return QEVICT_EINVAL;
  return qv::attn_plan(&d->attn, d->s_prefix, p);
}

qevict_status qevict_prefix_attn_bytes(const qevict_prefix_attn_desc *desc, size_t *bytes) {
  qv::AttnPlan p;
  if (!bytes) return QEVICT_EINVAL;
  const qevict_status st = prefix_plan(desc, &p);
  if (st == QEVICT_OK) *bytes = (size_t)p.bytes;
  return st;
}

qevict_status qevict_prefix_attn(const qevict_prefix_attn_desc *desc, const float *slopes, const int32_t *kv_len,
                                 const void *q, const void *k_prefix, const void *v_prefix, const void *k,
                                 const void *v, void *out, float *lse, void *d_work, size_t bytes,
                                 qevict_stream_t stream) {
  qv::AttnPlan p;
  const qevict_status st = prefix_plan(desc, &p);
  if (st != QEVICT_OK) return st;
  if (!k_prefix || !v_prefix || (((uintptr_t)k_prefix | (uintptr_t)v_prefix) & 15)) return QEVICT_EINVAL;
  qevict_attn_mask m = {};
  m.slopes = slopes;
  m.kv_len = kv_len;
  return qv::attn_launch(&desc->attn, p, &m, desc, q, k_prefix, v_prefix, k, v, out, lse, d_work, bytes,
                         reinterpret_cast<cudaStream_t>(stream));
}

qevict_status qevict_ops_status(void *d_status, int32_t *host_word, qevict_stream_t stream) {
  if (!d_status || ((uintptr_t)d_status & 3)) return QEVICT_EINVAL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int word = 0;
  if (cudaMemcpyAsync(&word, d_status, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return QEVICT_ECUDA;
  // cleared only where it was set: a bit that another stream's call sets after a clean read stays for the next one
  if (word && (cudaMemsetAsync(d_status, 0, sizeof(int), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess))
    return QEVICT_ECUDA;
  if (host_word) *host_word = word;
  return word ? QEVICT_EDEVICE : QEVICT_OK;
}

}  // extern "C"
