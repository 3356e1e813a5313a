// Rotary positions: the (cos, sin) table and its application to queries and keys.
//
// Position p turns channel pair i by the angle p * theta_i.  A pair (x1, x2) becomes
//   y1 = f (x1 c - x2 s),  y2 = f (x2 c + x1 s),   c = cos(p theta_i), s = sin(p theta_i),
// and the inverse (also the gradient with respect to x, the transpose of a rotation) has s negated.
// The half layout pairs channels (i, i + rot/2), the interleaved one (2i, 2i + 1); channels from
// rot on pass unchanged.  The table is the one qevict_set_rope_table takes for rot = 128.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "qevict.h"

namespace qv {

// ----------------------------------------------------------------------------- table

constexpr int MAX_PAIRS = 256;

// theta_i / (2 pi) as a 64-bit fraction of a turn, one per pair
struct TableArgs {
  uint64_t turn[MAX_PAIRS];
  int pairs;
  int64_t first, rows;
  float2 *out;
};

// One thread per (row, pair).  The angle in turns is p * turn[i] mod 2^64: whole turns fall away in
// the integer product, exactly, so a position of 2^31 still has an angle to 2^-33 turns, and no
// fp64 is needed (whose rate bounds this kernel at ten times its write time).  The eighth of a turn
// around the nearest quadrant goes to fp32 in two parts, hi and lo, and the Taylor polynomials of
// sine and cosine on [-pi/4, pi/4] (first terms left out: x^11/11! < 2e-9, x^12/12! < 2e-10) take
// hi with a first-order correction for lo.
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ TableArgs A) {
  const int64_t n = A.rows * A.pairs;
  for (int64_t idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; idx < n; idx += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = idx / A.pairs;
    const int i = (int)(idx - row * A.pairs);
    const uint64_t ph = (uint64_t)(A.first + row) * A.turn[i];
    const uint64_t sh = ph + (1ull << 61);            // nearest quadrant: add an eighth of a turn
    const int quad = (int)(sh >> 62);
    const int64_t r = (int64_t)((sh & ((1ull << 62) - 1)) - (1ull << 61));   // in [-1/8, 1/8) turn, times 2^64
    const float rh = (float)(int)(r >> 38), rl = (float)(uint32_t)((uint64_t)(r & ((1ll << 38) - 1)) >> 6);
    // turns -> radians: 2 pi = C + C2; units of rh are 2^-26 turns, of rl 2^-58
    constexpr float C = 6.28318548202514648437f, C2 = -1.74845553146e-07f;
    const float ah = rh * 1.490116119384765625e-8f, al0 = rl * 3.4694469519536141888e-18f;
    const float p = ah * C;
    const float e = fmaf(ah, C, -p) + fmaf(ah, C2, al0 * C);
    const float x = p + e, d = e - (x - p);
    const float z = x * x;
    float sn = fmaf(z, 2.75573192e-6f, -1.98412698e-4f);
    sn = fmaf(z, sn, 8.33333333e-3f);
    sn = fmaf(z, sn, -1.66666667e-1f);
    sn = fmaf(x * z, sn, x);
    float cs = fmaf(z, -2.75573192e-7f, 2.48015873e-5f);
    cs = fmaf(z, cs, -1.38888889e-3f);
    cs = fmaf(z, cs, 4.16666667e-2f);
    cs = fmaf(z, cs, -0.5f);
    cs = fmaf(z, cs, 1.0f);
    const float s0 = fmaf(d, cs, sn), c0 = fmaf(-d, sn, cs);
    float c = (quad & 1) ? s0 : c0, s = (quad & 1) ? c0 : s0;
    if (quad == 1 || quad == 2) c = -c;
    if (quad >= 2) s = -s;
    A.out[idx] = make_float2(c, s);
  }
}

// ----------------------------------------------------------------------------- application

struct RopeArgs {
  const void *q, *k;
  void *qo, *ko;
  const float2 *table;
  const int32_t *pos;
  int32_t *status;
  int64_t rows, pos0;
  int64_t qi[3], qo_[3], ki[3], ko_[3];   // strides in elements: batch, token, head
  int64_t tokens;                         // batch * seq
  int seq, h_q, heads;                    // heads: queries and keys together
  int half;                               // rotated pairs
  int units, pair_units;                  // vectors of work per head, those of them that rotate
  int lanes;                              // heads in flight per token
  float f, fs;                            // magnitude factor; fs = -f for the inverse
};

template <typename T>
__device__ __forceinline__ float to_f(T x) {
  return (float)x;
}
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
  T v[VEC];
};

// A thread owns one unit (VEC pairs of the half layout, VEC / 2 pairs of the interleaved one, or VEC
// channels that pass) of one token and walks over `lanes`-strided heads with the unit's cosines and
// sines in registers, so the table row is read once per unit and token however many heads there are.
// VEC fills 16 bytes where sizes, strides and alignment allow, else 1.  Rounded once, at the store.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(256) rope_apply_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int NP = INTER ? (VEC > 1 ? VEC / 2 : 1) : VEC;   // pairs of a rotating unit
  const int per_tok = A.units * A.lanes;
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t tok = id / per_tok;
  if (tok >= A.tokens) return;
  const int rest = (int)(id - tok * per_tok), u = rest % A.units, lane = rest / A.units;
  const int64_t b = tok / A.seq, t = tok - b * A.seq;
  const int64_t pos = A.pos ? (int64_t)A.pos[tok] : A.pos0 + t;
  if (pos < 0 || pos >= A.rows) {   // no such table row: the token's heads are not written
    if (rest == 0) atomicOr(A.status, QV_ERR_BOUNDS);
    return;
  }
  const bool rotates = u < A.pair_units;
  float c[NP], s[NP];
  if (rotates) {
    const float2 *row = A.table + pos * A.half + (int64_t)u * NP;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      float2 cs;
      if (NP % 2 == 0) {   // 16-byte loads of two pairs
        const float4 w = *reinterpret_cast<const float4 *>(row + (j & ~1));
        cs = (j & 1) ? make_float2(w.z, w.w) : make_float2(w.x, w.y);
      } else {
        cs = row[j];
      }
      c[j] = cs.x * A.f;
      s[j] = cs.y * A.fs;
    }
  }
  // channels of the unit: half layout ch and ch + half; interleaved ch .. ; passing ch ..
  const int ch = rotates ? (INTER ? u * NP * 2 : u * NP) : 2 * A.half + (u - A.pair_units) * VEC;
  for (int h = lane; h < A.heads; h += A.lanes) {
    const bool is_q = h < A.h_q;
    const int hh = is_q ? h : h - A.h_q;
    const int64_t *si = is_q ? A.qi : A.ki, *so = is_q ? A.qo_ : A.ko_;
    const T *src = reinterpret_cast<const T *>(is_q ? A.q : A.k) + b * si[0] + t * si[1] + hh * si[2] + ch;
    T *dst = reinterpret_cast<T *>(is_q ? A.qo : A.ko) + b * so[0] + t * so[1] + hh * so[2] + ch;
    if (!rotates) {
      if (src != dst) *reinterpret_cast<Pack<T, VEC> *>(dst) = *reinterpret_cast<const Pack<T, VEC> *>(src);
    } else if (INTER) {
      constexpr int N = VEC > 1 ? VEC : 2;
      T x[N];
      if (VEC > 1) {
        *reinterpret_cast<Pack<T, VEC> *>(x) = *reinterpret_cast<const Pack<T, VEC> *>(src);
      } else {
        x[0] = src[0];
        x[1] = src[1];
      }
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const float x1 = to_f(x[2 * j]), x2 = to_f(x[2 * j + 1]);
        x[2 * j] = from_f<T>(fmaf(x1, c[j], -x2 * s[j]));
        x[2 * j + 1] = from_f<T>(fmaf(x2, c[j], x1 * s[j]));
      }
      if (VEC > 1) {
        *reinterpret_cast<Pack<T, VEC> *>(dst) = *reinterpret_cast<const Pack<T, VEC> *>(x);
      } else {
        dst[0] = x[0];
        dst[1] = x[1];
      }
    } else {
      Pack<T, VEC> x = *reinterpret_cast<const Pack<T, VEC> *>(src);
      Pack<T, VEC> y = *reinterpret_cast<const Pack<T, VEC> *>(src + A.half);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float x1 = to_f(x.v[j]), x2 = to_f(y.v[j]);
        x.v[j] = from_f<T>(fmaf(x1, c[j], -x2 * s[j]));
        y.v[j] = from_f<T>(fmaf(x2, c[j], x1 * s[j]));
      }
      *reinterpret_cast<Pack<T, VEC> *>(dst) = x;
      *reinterpret_cast<Pack<T, VEC> *>(dst + A.half) = y;
    }
  }
}

namespace {

template <typename T, bool INTER>
void launch_apply(const RopeArgs &A, int vec, int64_t blocks, int threads, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  if (vec > 1)
    rope_apply_kernel<T, V, INTER><<<(unsigned)blocks, threads, 0, s>>>(A);
  else
    rope_apply_kernel<T, 1, INTER><<<(unsigned)blocks, threads, 0, s>>>(A);
}

// The strides of a written tensor put no two elements in one place: by ascending stride, every
// dimension steps over all that the smaller ones reach.
bool no_overlap(const int64_t *st, int64_t batch, int64_t seq, int64_t heads, int64_t d) {
  int64_t size[3] = {batch, seq, heads}, stride[3] = {st[0], st[1], st[2]};
  int64_t reach = d;   // elements from the first to past the last
  for (int n = 0; n < 3; ++n) {
    int best = -1;
    for (int i = 0; i < 3; ++i)
      if (size[i] > 1 && (best < 0 || stride[i] < stride[best])) best = i;
    if (best < 0) break;
    if (stride[best] < reach) return false;
    reach += stride[best] * (size[best] - 1);
    size[best] = 1;
  }
  return true;
}

int64_t extent(const int64_t *st, int64_t batch, int64_t seq, int64_t heads, int64_t d) {
  return st[0] * (batch - 1) + st[1] * (seq - 1) + st[2] * (heads - 1) + d;
}

}  // namespace
}  // namespace qv

extern "C" {

qevict_status qevict_rope_angles(const qevict_rope_config *cfg, double *theta) {
  if (!cfg || !theta) return QEVICT_EINVAL;
  const int rot = cfg->rot_dim;
  if (rot < 2 || rot > 2 * qv::MAX_PAIRS || rot % 2 || cfg->scaling < 0 || cfg->scaling > 3) return QEVICT_EINVAL;
  if (!(cfg->base > 0) || !std::isfinite(cfg->base)) return QEVICT_EINVAL;
  double base = cfg->base;
  if (cfg->scaling != QEVICT_ROPE_NONE && (!(cfg->factor > 0) || !std::isfinite(cfg->factor))) return QEVICT_EINVAL;
  if (cfg->scaling == QEVICT_ROPE_NTK) {
    if (rot < 4) return QEVICT_EINVAL;
    base *= std::pow(cfg->factor, (double)rot / (rot - 2));
  }
  if (cfg->scaling == QEVICT_ROPE_PARTS &&
      (!(cfg->orig_len > 0) || !std::isfinite(cfg->orig_len) || !(cfg->low >= 0) || !(cfg->high > cfg->low) ||
       !std::isfinite(cfg->high)))
    return QEVICT_EINVAL;
  const double two_pi = 6.283185307179586476925286766559;
  for (int i = 0; i < rot / 2; ++i) {
    double th = std::pow(base, -2.0 * i / rot);
    if (cfg->scaling == QEVICT_ROPE_LINEAR) th /= cfg->factor;
    if (cfg->scaling == QEVICT_ROPE_PARTS) {
      double keep = (cfg->orig_len * th / two_pi - cfg->low) / (cfg->high - cfg->low);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      th = keep * th + (1.0 - keep) * (th / cfg->factor);
    }
    if (!std::isfinite(th)) return QEVICT_EINVAL;
    theta[i] = th;
  }
  return QEVICT_OK;
}

qevict_status qevict_rope_table(const qevict_rope_config *cfg, int64_t first, int64_t rows, float *d_table,
                                qevict_stream_t stream) {
  double theta[qv::MAX_PAIRS];
  qevict_status st = qevict_rope_angles(cfg, theta);
  if (st != QEVICT_OK) return st;
  if (!d_table || ((uintptr_t)d_table & 7) || first < 0 || rows < 1 || first > (1ll << 31) || rows > (1ll << 31) ||
      first + rows > (1ll << 31))
    return QEVICT_EINVAL;
  qv::TableArgs A;
  A.pairs = cfg->rot_dim / 2;
  A.first = first;
  A.rows = rows;
  A.out = reinterpret_cast<float2 *>(d_table);
  const double two_pi = 6.283185307179586476925286766559;
  for (int i = 0; i < A.pairs; ++i) {
    const double turns = std::fmod(theta[i] / two_pi, 1.0);   // whole turns per position change nothing
    // split so that the product below 2^64 stays exact in a double
    const double hi = std::floor(std::ldexp(turns, 32)), lo = std::ldexp(turns, 32) - hi;
    A.turn[i] = ((uint64_t)hi << 32) + (uint64_t)std::floor(std::ldexp(lo, 32));
  }
  const int64_t blocks = (rows * A.pairs + 255) / 256;
  qv::rope_table_kernel<<<(unsigned)(blocks < 152 * 32 ? blocks : 152 * 32), 256, 0,
                          reinterpret_cast<cudaStream_t>(stream)>>>(A);
  return cudaGetLastError() == cudaSuccess ? QEVICT_OK : QEVICT_ECUDA;
}

qevict_status qevict_rope_apply(const qevict_rope_desc *d, const float *d_table, const int32_t *d_positions,
                                const void *q_in, void *q_out, const void *k_in, void *k_out, int32_t *d_status,
                                qevict_stream_t stream) {
  using namespace qv;
  if (!d || !d_table || !d_status || ((uintptr_t)d_table & 15) || ((uintptr_t)d_positions & 3) ||
      ((uintptr_t)d_status & 3))
    return QEVICT_EINVAL;
  if (d->dtype < 0 || d->dtype > 2 || d->batch < 1 || d->seq < 1 || d->h_q < 0 || d->h_k < 0 || d->h_q + (int64_t)d->h_k < 1 ||
      d->d_head < 2 || d->d_head > 1024 || d->rot_dim < 2 || d->rot_dim > d->d_head || d->rot_dim % 2 ||
      d->rot_dim > 2 * MAX_PAIRS || d->interleaved < 0 || d->interleaved > 1 || d->inverse < 0 || d->inverse > 1 ||
      d->h_q > (1 << 20) || d->h_k > (1 << 20) || !std::isfinite(d->factor) || d->table_rows < 1 || d->pos0 < 0)
    return QEVICT_EINVAL;
  if (!d_positions && (d->pos0 > d->table_rows || d->seq > d->table_rows - d->pos0)) return QEVICT_EINVAL;
  if ((d->h_q > 0) != (q_in != nullptr && q_out != nullptr) || (d->h_k > 0) != (k_in != nullptr && k_out != nullptr))
    return QEVICT_EINVAL;
  const int size = d->dtype == QEVICT_FP32 ? 4 : 2, V = 16 / size;
  int64_t align = 0;   // of every pointer in bytes and stride in elements
  for (int n = 0; n < 2; ++n) {
    const int heads = n ? d->h_k : d->h_q;
    if (!heads) continue;
    const int64_t *si = n ? d->k_in : d->q_in, *so = n ? d->k_out : d->q_out;
    const void *in = n ? k_in : q_in;
    void *out = n ? k_out : q_out;
    if (((uintptr_t)in | (uintptr_t)out) % size) return QEVICT_EINVAL;
    bool same = in == out;
    const int64_t dim[3] = {d->batch, d->seq, heads};
    for (int i = 0; i < 3; ++i) {
      if (si[i] < 0 || so[i] < 0 || si[i] > (1ll << 40) || so[i] > (1ll << 40)) return QEVICT_EINVAL;
      if (dim[i] > 1) {
        align |= (si[i] | so[i]) % V;
        same = same && si[i] == so[i];
      }
    }
    align |= ((uintptr_t)in | (uintptr_t)out) & 15;
    if (!no_overlap(so, d->batch, d->seq, heads, d->d_head)) return QEVICT_EINVAL;
    // in place, or apart: a partial overlap would read what another thread has written
    const char *i0 = static_cast<const char *>(in), *o0 = static_cast<const char *>(out);
    const char *i1 = i0 + extent(si, d->batch, d->seq, heads, d->d_head) * size;
    const char *o1 = o0 + extent(so, d->batch, d->seq, heads, d->d_head) * size;
    if (!same && i0 < o1 && o0 < i1) return QEVICT_EINVAL;
  }
  RopeArgs A = {};
  A.q = q_in, A.k = k_in, A.qo = q_out, A.ko = k_out;
  A.table = reinterpret_cast<const float2 *>(d_table);
  A.pos = d_positions;
  A.status = d_status;
  A.rows = d->table_rows;
  A.pos0 = d->pos0;
  for (int i = 0; i < 3; ++i) A.qi[i] = d->q_in[i], A.qo_[i] = d->q_out[i], A.ki[i] = d->k_in[i], A.ko_[i] = d->k_out[i];
  A.seq = d->seq;
  A.tokens = (int64_t)d->batch * d->seq;
  A.h_q = d->h_q;
  A.heads = d->h_q + d->h_k;
  A.half = d->rot_dim / 2;
  A.f = d->factor;
  A.fs = d->inverse ? -d->factor : d->factor;
  const int pass = d->d_head - d->rot_dim;
  const int np = d->interleaved ? V / 2 : V;   // pairs of a full vector
  // full vectors need every start on 16 bytes, table rows (8 bytes a pair) included
  const bool vec = align == 0 && A.half % np == 0 && pass % V == 0 && (A.half % 2 == 0 || np == 1);
  A.pair_units = vec ? A.half / np : A.half;
  A.units = A.pair_units + (vec ? pass / V : pass);
  // heads in flight: all of them for few tokens (latency), else about three heads a thread, which
  // reads each table row a third as often
  const int64_t all = A.tokens * A.units * A.heads;
  A.lanes = all <= 152 * 2048 ? A.heads : (A.heads + 2) / 3;
  const int64_t n = A.tokens * A.units * A.lanes;
  const int64_t blocks = (n + 255) / 256;
  if (blocks > 0x7fffffffll) return QEVICT_EINVAL;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
#define QV_ROPE(T) (d->interleaved ? launch_apply<T, true>(A, vec ? V : 1, blocks, 256, s) : launch_apply<T, false>(A, vec ? V : 1, blocks, 256, s))
  if (d->dtype == QEVICT_BF16)
    QV_ROPE(__nv_bfloat16);
  else if (d->dtype == QEVICT_FP16)
    QV_ROPE(__half);
  else
    QV_ROPE(float);
#undef QV_ROPE
  return cudaGetLastError() == cudaSuccess ? QEVICT_OK : QEVICT_ECUDA;
}

}  // extern "C"
