// Rotary positions: the (cos, sin) table and its application to queries and keys.
//
// Position p turns channel pair i by the angle p * theta_i.  A pair (x1, x2) becomes
//   y1 = f (x1 c - x2 s),  y2 = f (x2 c + x1 s),   c = cos(p theta_i), s = sin(p theta_i),
// and the inverse (also the gradient with respect to x, the transpose of a rotation) has s negated.
// The half layout pairs channels (i, i + rot/2), the interleaved one (2i, 2i + 1); channels from
// rot on pass unchanged.  The table is the one qevict_set_rope_table takes for rot = 128.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstdint>

#include "common.cuh"
#include "qevict.h"

namespace qv {

// ----------------------------------------------------------------------------- table

constexpr int MAX_PAIRS = 256;

// theta_i / (2 pi) as a 64-bit fraction of a turn, one per pair
struct TableArgs {
  uint64_t turn[MAX_PAIRS];
  int pairs, step;             // rows between a thread's entries
  int64_t first, rows;
  float2 *out;
};

// cos and sin of the angle ph * 2^-64 turns.  The eighth of a turn around the nearest quadrant goes to fp32 in two parts
// and from turns to radians with the product's error kept, x + d; the Taylor polynomials of sine and cosine on
// [-pi/4, pi/4] (first terms left out: x^11/11! < 2e-9, x^12/12! < 2e-10) take x, with a first-order correction for d.
__device__ __forceinline__ float2 cos_sin_turns(uint64_t ph) {
  const uint64_t sh = ph + (1ull << 61);            // nearest quadrant: add an eighth of a turn
  const int quad = (int)(sh >> 62);
  const int64_t r = (int64_t)((sh & ((1ull << 62) - 1)) - (1ull << 61));   // in [-1/8, 1/8) turn, times 2^64
  const float rh = (float)(int)(r >> 38), rl = (float)(uint32_t)((uint64_t)(r & ((1ll << 38) - 1)) >> 6);
  // 2 pi = C + C2; units of rh are 2^-26 turns, of rl 2^-58
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
  return make_float2(c, s);
}

// A thread owns N neighbouring pairs (N = 2: 16-byte stores) and walks down the rows.  The angle in turns is
// p * turn[i] mod 2^64: whole turns fall away in the integer product, exactly, so a position of 2^31 still has an angle to
// 2^-33 turns, and no fp64 is needed (whose rate would bound this kernel at ten times its write time); a step down adds
// step * turn[i].  Bound by its arithmetic, 52 instructions for 8 bytes: 131200 rows of 64 pairs take 16.5 us, 71% of the
// issue slots; writing them alone would take 9.9.
template <int N>
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ TableArgs A) {
  const int groups = A.pairs / N;
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  const uint32_t row0 = id / groups, i = (id - row0 * groups) * N;
  if (row0 >= (uint32_t)A.step) return;
  uint64_t ph[N], inc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    ph[j] = (uint64_t)(A.first + row0) * A.turn[i + j];
    inc[j] = (uint64_t)A.step * A.turn[i + j];
  }
  float2 *out = A.out + (int64_t)row0 * A.pairs + i;
  const int64_t hop = (int64_t)A.step * A.pairs;
  for (int64_t row = row0; row < A.rows; row += A.step, out += hop) {
    float2 cs[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      cs[j] = cos_sin_turns(ph[j]);
      ph[j] += inc[j];
    }
    if (N == 2)
      *reinterpret_cast<float4 *>(out) = make_float4(cs[0].x, cs[0].y, cs[N - 1].x, cs[N - 1].y);
    else
      *out = cs[0];
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
  int seq, h_q, h_k;
  int groups_q;                           // of the groups of neighbouring heads, those of queries
  int half;                               // rotated pairs
  int pair_units;                         // of a head's vectors of work (blockDim.x), those that rotate
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

// Who holds the two channels of a pair: one thread, from two places of the half layout (any size and alignment), one
// thread in the interleaved layout, or two lanes of a warp, each with 16 bytes of the half layout, that swap them.  The
// last keeps every load and store of a warp on whole heads.
enum : int { ROPE_TWO_PLACES = 0, ROPE_INTERLEAVED = 1, ROPE_SWAP = 2 };

// Two neighbouring channels as fp32 and back, rounded once
template <typename T>
__device__ __forceinline__ float2 two(const T *p) {
  return make_float2(to_f(p[0]), to_f(p[1]));
}
template <>
__device__ __forceinline__ float2 two(const __nv_bfloat16 *p) {
  const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <>
__device__ __forceinline__ float2 two(const __half *p) {
  return __half22float2(*reinterpret_cast<const __half2 *>(p));
}
__device__ __forceinline__ void put_two(float *p, float a, float b) { p[0] = a, p[1] = b; }
__device__ __forceinline__ void put_two(__nv_bfloat16 *p, float a, float b) { *reinterpret_cast<uint32_t *>(p) = pack_bf16(a, b); }
__device__ __forceinline__ void put_two(__half *p, float a, float b) { *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(a, b); }

// A thread owns one unit of one token (VEC channels; with ROPE_TWO_PLACES VEC pairs) in HPT heads, blockDim.y apart,
// with the unit's cosines and sines in registers, so the table row is read once per unit for all of them; the heads'
// loads are issued before the position is looked at.  Block: (units, heads side by side); grid: (tokens, groups of
// HPT * blockDim.y neighbouring heads, queries' before keys').  VEC fills 16 bytes where sizes, strides and
// alignment allow, else 1.  Rounded once, at the store.  Memory bound.
template <typename T, int VEC, int MODE, int HPT>
__global__ void __launch_bounds__(VEC > 1 ? 256 : 1024) rope_apply_kernel(const __grid_constant__ RopeArgs A) {
  constexpr int NP = MODE == ROPE_INTERLEAVED ? (VEC > 1 ? VEC / 2 : 1) : VEC;   // pairs of a rotating unit
  constexpr int NV = MODE == ROPE_INTERLEAVED && VEC == 1 ? 2 : VEC;             // elements loaded at one place
  const int64_t tok = blockIdx.x;   // fewer than 2^31
  const uint32_t b = blockIdx.x / (uint32_t)A.seq, t = blockIdx.x - b * (uint32_t)A.seq;
  const int64_t pos = A.pos ? (int64_t)A.pos[tok] : A.pos0 + t;
  const int u = threadIdx.x;
  const bool rotates = u < A.pair_units;
  const int hu = A.pair_units / 2;                         // ROPE_SWAP: units of first channels
  const bool second = MODE == ROPE_SWAP && u >= hu;
  // first channel of the unit
  const int ch = MODE == ROPE_SWAP ? u * VEC
                 : rotates         ? u * NP * (MODE == ROPE_INTERLEAVED ? 2 : 1)
                                   : 2 * A.half + (u - A.pair_units) * VEC;
  const int group = blockIdx.y;
  const bool is_q = group < A.groups_q;
  const int h0 = (is_q ? group : group - A.groups_q) * blockDim.y * HPT + threadIdx.y, heads = is_q ? A.h_q : A.h_k;
  const int64_t s0 = is_q ? A.qi[0] : A.ki[0], s1 = is_q ? A.qi[1] : A.ki[1], s2 = is_q ? A.qi[2] : A.ki[2];
  const T *src = static_cast<const T *>(is_q ? A.q : A.k) + b * s0 + t * s1 + h0 * s2 + ch;
  const int64_t shop = s2 * blockDim.y;
  using V = Pack<T, NV>;
  V x[HPT], y[MODE == ROPE_TWO_PLACES ? HPT : 1];
#pragma unroll
  for (int k = 0; k < HPT; ++k, src += shop) {
    if (h0 + k * (int)blockDim.y < heads) {
      if (NV == VEC) {
        x[k] = *reinterpret_cast<const V *>(src);
      } else {   // one pair (or passing channel) at any alignment
        x[k].v[0] = src[0];
        if (rotates) x[k].v[NV - 1] = src[1];
      }
      if (MODE == ROPE_TWO_PLACES && rotates) y[k] = *reinterpret_cast<const V *>(src + A.half);
    }
  }
  if (pos < 0 || pos >= A.rows) {   // no such table row: the token's heads are not written
    if (u == 0 && threadIdx.y == 0) atomicOr(A.status, QV_ERR_BOUNDS);
    return;
  }
  float c[NP], s[NP];
  if (rotates) {
    const float2 *row = A.table + pos * A.half + (int64_t)(second ? u - hu : u) * NP;
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
      s[j] = cs.y * (MODE == ROPE_SWAP && !second ? -A.fs : A.fs);   // swapped: y = own c +- other s
    }
  }
  const int64_t d0 = is_q ? A.qo_[0] : A.ko_[0], d1 = is_q ? A.qo_[1] : A.ko_[1], d2 = is_q ? A.qo_[2] : A.ko_[2];
  T *dst = static_cast<T *>(is_q ? A.qo : A.ko) + b * d0 + t * d1 + h0 * d2 + ch;
  const int64_t dhop = d2 * blockDim.y;
#pragma unroll
  for (int k = 0; k < HPT; ++k, dst += dhop) {
    if (h0 + k * (int)blockDim.y >= heads) break;
    if (MODE == ROPE_SWAP) {   // the head's lanes are together here
      const int lane = (threadIdx.x + blockDim.x * threadIdx.y) & 31;
      const int n = blockDim.x;   // lanes of a head: a power of two up to 32
      const uint32_t mates = (n == 32 ? ~0u : (1u << n) - 1u) << (lane & ~(n - 1));
      const int from = rotates ? (second ? lane - hu : lane + hu) : lane;
      uint4 w = *reinterpret_cast<uint4 *>(&x[k]);
      w.x = __shfl_sync(mates, w.x, from);
      w.y = __shfl_sync(mates, w.y, from);
      w.z = __shfl_sync(mates, w.z, from);
      w.w = __shfl_sync(mates, w.w, from);
      if (rotates) {
        const V o = *reinterpret_cast<V *>(&w);
#pragma unroll
        for (int j = 0; j + 1 < VEC; j += 2) {
          const float2 a = two(x[k].v + j), q = two(o.v + j);
          put_two(x[k].v + j, fmaf(a.x, c[j], q.x * s[j]), fmaf(a.y, c[j + 1], q.y * s[j + 1]));
        }
      }
      *reinterpret_cast<V *>(dst) = x[k];   // passing channels in place: what stands there
    } else if (!rotates) {
      if (NV == VEC)
        *reinterpret_cast<V *>(dst) = x[k];
      else
        dst[0] = x[k].v[0];
    } else if (MODE == ROPE_INTERLEAVED) {
      if (NV == VEC) {
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          const float2 a = two(x[k].v + 2 * j);
          put_two(x[k].v + 2 * j, fmaf(a.x, c[j], -a.y * s[j]), fmaf(a.y, c[j], a.x * s[j]));
        }
        *reinterpret_cast<V *>(dst) = x[k];
      } else {
        const float x1 = to_f(x[k].v[0]), x2 = to_f(x[k].v[NV - 1]);
        dst[0] = from_f<T>(fmaf(x1, c[0], -x2 * s[0]));
        dst[1] = from_f<T>(fmaf(x2, c[0], x1 * s[0]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float x1 = to_f(x[k].v[j]), x2 = to_f(y[k].v[j]);
        x[k].v[j] = from_f<T>(fmaf(x1, c[j], -x2 * s[j]));
        y[k].v[j] = from_f<T>(fmaf(x2, c[j], x1 * s[j]));
      }
      *reinterpret_cast<V *>(dst) = x[k];
      *reinterpret_cast<V *>(dst + A.half) = y[k];
    }
  }
}

// Rotations whose pairs do not fall on whole vectors (37 pairs of a head, say) where heads still start on 16 bytes: a block
// takes up to hc heads of one token through shared memory, in and out 16 bytes a thread, and turns them there pair by pair,
// a lane's cosine and sine serving all the heads of its warp.  8192 tokens of 32 + 8 bf16 heads, 37 pairs: half layout 40 us
// (167 by single loads and stores), interleaved 40 (51); fp32 65 (167) and 66 (55), so interleaved fp32, whose pairs are
// 8 bytes each, is left to single loads.  24.7 and 49.4 at the rate of a copy.
template <typename T>
__global__ void __launch_bounds__(128) rope_staged_kernel(const __grid_constant__ RopeArgs A, int d, int hc, bool inter) {
  extern __shared__ uint4 staged[];
  constexpr int V = 16 / (int)sizeof(T);
  const int64_t tok = blockIdx.x;
  const uint32_t b = blockIdx.x / (uint32_t)A.seq, t = blockIdx.x - b * (uint32_t)A.seq;
  const int64_t pos = A.pos ? (int64_t)A.pos[tok] : A.pos0 + t;
  if (pos < 0 || pos >= A.rows) {   // no such table row: the token's heads are not written
    if (threadIdx.x == 0) atomicOr(A.status, QV_ERR_BOUNDS);
    return;
  }
  const int group = blockIdx.y;
  const bool is_q = group < A.groups_q;
  const int h0 = (is_q ? group : group - A.groups_q) * hc, n = min(hc, (is_q ? A.h_q : A.h_k) - h0);
  const int64_t s2 = is_q ? A.qi[2] : A.ki[2], d2 = is_q ? A.qo_[2] : A.ko_[2];
  const T *src = static_cast<const T *>(is_q ? A.q : A.k) + b * (is_q ? A.qi[0] : A.ki[0]) + t * (is_q ? A.qi[1] : A.ki[1]) +
                 h0 * s2;
  T *dst = static_cast<T *>(is_q ? A.qo : A.ko) + b * (is_q ? A.qo_[0] : A.ko_[0]) + t * (is_q ? A.qo_[1] : A.ko_[1]) + h0 * d2;
  const int nu = d / V, h_first = threadIdx.x / nu, u_first = threadIdx.x - h_first * nu;
  const int dh = blockDim.x / nu, du = blockDim.x - dh * nu;   // a block's step in heads and vectors
  for (int h = h_first, u = u_first; h < n;) {
    staged[h * nu + u] = *reinterpret_cast<const uint4 *>(src + h * s2 + u * V);
    h += dh, u += du;
    if (u >= nu) u -= nu, ++h;
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = lane; i < A.half; i += 32) {
    const float2 cs = A.table[pos * A.half + i];
    const float c = cs.x * A.f, s = cs.y * A.fs;
    T *p = reinterpret_cast<T *>(staged) + warp * d + (inter ? 2 * i : i);
    const int other = inter ? 1 : A.half;
    for (int h = warp; h < n; h += 4, p += 4 * d) {
      const float x1 = to_f(p[0]), x2 = to_f(p[other]);
      p[0] = from_f<T>(fmaf(x1, c, -x2 * s));
      p[other] = from_f<T>(fmaf(x2, c, x1 * s));
    }
  }
  __syncthreads();
  for (int h = h_first, u = u_first; h < n;) {
    *reinterpret_cast<uint4 *>(dst + h * d2 + u * V) = staged[h * nu + u];
    h += dh, u += du;
    if (u >= nu) u -= nu, ++h;
  }
}

namespace {

template <typename T>
bool launch_staged(RopeArgs &A, bool inter, int d_head, cudaStream_t s) {
  const int bytes = d_head * (int)sizeof(T);
  int hc = std::min(std::max(1, 8192 / bytes), std::max(A.h_q, A.h_k));
  while (hc > 4 && A.tokens * ((A.h_q + A.h_k + hc - 1) / hc) < 304) hc = (hc + 1) / 2;   // few tokens: two blocks an SM
  A.groups_q = (A.h_q + hc - 1) / hc;
  const int64_t gy = A.groups_q + (A.h_k + hc - 1) / hc;
  if (gy > 65535) return false;
  rope_staged_kernel<T><<<dim3((unsigned)A.tokens, (unsigned)gy), 128, hc * bytes, s>>>(A, d_head, hc, inter);
  return true;
}

// Block and grid for `units` vectors a head: a warp a block, four neighbouring heads a thread, so that a warp has 2 KB of
// one place in flight, unless there are so few tokens that one head a thread does not fill the GPU.  A 32K prompt of
// 32 + 8 heads takes 111 us (6.2 TB/s, 91% of a plain copy); two heads a thread 167, eight 110, five warps a block 113.
template <typename T, int VEC, int MODE>
bool launch_apply(RopeArgs &A, int units, cudaStream_t s) {
  const bool one = MODE == ROPE_TWO_PLACES || A.tokens * units * (A.h_q + A.h_k) <= 152 * 2048;
  const int ny = std::max(1, 32 / units), per = ny * (one ? 1 : 4);
  A.groups_q = (A.h_q + per - 1) / per;
  const int64_t gx = A.tokens, gy = A.groups_q + (A.h_k + per - 1) / per;
  if (gy > 65535) return false;
  const dim3 grid((unsigned)gx, (unsigned)gy), block(units, ny);
  if (one)
    rope_apply_kernel<T, VEC, MODE, 1><<<grid, block, 0, s>>>(A);
  else
    rope_apply_kernel<T, VEC, MODE, MODE == ROPE_TWO_PLACES ? 1 : 4><<<grid, block, 0, s>>>(A);
  return true;
}
template <typename T>
bool launch_apply_type(RopeArgs &A, bool vec, bool wide, bool inter, int d_head, cudaStream_t s) {
  constexpr int V = 16 / (int)sizeof(T);
  if (!vec && wide && (!inter || sizeof(T) == 2)) return launch_staged<T>(A, inter, d_head, s);
  const int pass = d_head - 2 * A.half;
  if (inter) {
    A.pair_units = vec ? 2 * A.half / V : A.half;
    return vec ? launch_apply<T, V, ROPE_INTERLEAVED>(A, d_head / V, s)
               : launch_apply<T, 1, ROPE_INTERLEAVED>(A, A.half + pass, s);
  }
  if (vec && 32 % (d_head / V) == 0 && d_head % V == 0) {   // a head's lanes in one warp
    A.pair_units = 2 * A.half / V;
    return launch_apply<T, V, ROPE_SWAP>(A, d_head / V, s);
  }
  A.pair_units = vec ? A.half / V : A.half;
  return vec ? launch_apply<T, V, ROPE_TWO_PLACES>(A, A.half / V + pass / V, s)
             : launch_apply<T, 1, ROPE_TWO_PLACES>(A, A.half + pass, s);
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
  // theta / (2 pi) in two doubles, off by about 2^-104 of it: up to theta = 2^40 the 64-bit fraction is off by one at most
  const double inv = 0.15915494309189535, inv_low = -9.839338337591243e-18;   // 1 / (2 pi) = inv + inv_low
  for (int i = 0; i < A.pairs; ++i) {
    const double hi = theta[i] * inv, lo = std::fma(theta[i], inv, -hi) + theta[i] * inv_low;
    // whole turns per position change nothing and fall away exactly; lo may be negative, its low bit is dropped
    const uint64_t low = (uint64_t)std::llround(std::ldexp(lo - std::rint(lo), 63));
    A.turn[i] = (uint64_t)std::ldexp(hi - std::floor(hi), 64) + (low << 1);
  }
  const bool two = A.pairs % 2 == 0 && ((uintptr_t)d_table & 15) == 0;
  const int groups = two ? A.pairs / 2 : A.pairs;
  // rows side by side: all of a short table's, else as many as fill the GPU's 152 x 2048 threads
  const int64_t fill = (152 * 2048 + groups - 1) / groups;
  A.step = (int)(rows < fill ? rows : fill);
  const unsigned blocks = (unsigned)(((int64_t)A.step * groups + 255) / 256);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (two)
    qv::rope_table_kernel<2><<<blocks, 256, 0, s>>>(A);
  else
    qv::rope_table_kernel<1><<<blocks, 256, 0, s>>>(A);
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
      d->h_q > (1 << 20) || d->h_k > (1 << 20) || (int64_t)d->batch * d->seq > 0x7fffffffll || !std::isfinite(d->factor) ||
      d->table_rows < 1 || d->pos0 < 0)
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
        if (std::max(si[i], so[i]) > (1ll << 48) / (dim[i] - 1)) return QEVICT_EINVAL;
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
  // queries and keys may lie between one another, but what is written of one may not be the other
  if (d->h_q && d->h_k && (q_out == k_out || q_out == k_in || k_out == q_in)) return QEVICT_EINVAL;
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
  A.h_k = d->h_k;
  A.half = d->rot_dim / 2;
  A.f = d->factor;
  A.fs = d->inverse ? -d->factor : d->factor;
  const int pass = d->d_head - d->rot_dim;
  const int np = d->interleaved ? V / 2 : V;   // pairs of a full vector
  // full vectors need every start on 16 bytes, table rows (8 bytes a pair) included
  const bool vec = align == 0 && A.half % np == 0 && pass % V == 0 && (A.half % 2 == 0 || np == 1);
  const bool wide = align == 0 && d->d_head % V == 0;   // heads, at least, are whole vectors
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool ok = d->dtype == QEVICT_BF16   ? launch_apply_type<__nv_bfloat16>(A, vec, wide, d->interleaved, d->d_head, s)
                  : d->dtype == QEVICT_FP16 ? launch_apply_type<__half>(A, vec, wide, d->interleaved, d->d_head, s)
                                            : launch_apply_type<float>(A, vec, wide, d->interleaved, d->d_head, s);
  if (!ok) return QEVICT_EINVAL;
  return cudaGetLastError() == cudaSuccess ? QEVICT_OK : QEVICT_ECUDA;
}

}  // extern "C"
