// Norm of the queries and keys of each head with the position rotation in
// the same pass (Video DeltaNet, Section 5: the Softmax branch's fused
// QK-norm + RoPE), optionally appending K and V to a paged cache, and its
// gradient.  B200 (sm_100a).
//
//   x^ = x / sqrt(mean(x^2) + eps),  z = w x^,  y = R(phi) z
//   g = R(phi)^T dy,  dw = sum g x^,  dx = (g w - x^ mean(g w x^)) / sqrt(mean(x^2) + eps)
//
// R turns the pairs (p, p + rot / 2), or (2 p, 2 p + 1) when interleaved, of
// the first rot channels by phi_p = position[axis_p] * frequency_p.
//
// Bound by memory: one read and one write per value against ~15 fp32
// operations.  D / 8 lanes hold one row (a token's head), 8 channels (16 B
// of bf16) each, so the norm is a few shuffles and nothing is staged in shared
// memory.  A warp takes consecutive rows of one token: the token's angles,
// with the weights multiplied in, stay in registers over all its rows.  The
// arithmetic is paired (f32x2) and paired channels are exchanged as loaded
// (bf16 pairs): with 157 instructions for two rows instead of 113 the
// kernel was bound by issue.
//
// Measured, bf16, 60480 tokens of 48 + 48 heads of 128, three axes: 542 to 562 us
// with 80 registers and 6 blocks an SM (2.97 GB, 81 to 84% of a plain copy's rate;
// 778 us with 157 instructions).  The gradient, 20160 such tokens: 302 us with 128
// registers and 4 blocks an SM (1.49 GB, 75%).  Both then wait for memory
// with the warps that their registers allow.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "vda.h"

namespace vda {
namespace qk {

constexpr int kThreads = 128;
constexpr int kBatch = 4;   // rows in flight per lane group

// 8 consecutive channels as loaded
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  }
  __device__ __forceinline__ void get(float2 (&x)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void set(const float2 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ptx::pack_bf16(x[i].x, x[i].y);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ Raw8 from(int lane) const {   // what another lane holds
    Raw8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.w[i] = __shfl_sync(0xffffffffu, w[i], lane);
    return o;
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float2 (&x)[4]) const {
    x[0] = make_float2(a.x, a.y); x[1] = make_float2(a.z, a.w);
    x[2] = make_float2(b.x, b.y); x[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ void set(const float2 (&x)[4]) {
    a = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    b = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ Raw8 from(int lane) const {
    Raw8 o;
    o.a.x = __shfl_sync(0xffffffffu, a.x, lane); o.a.y = __shfl_sync(0xffffffffu, a.y, lane);
    o.a.z = __shfl_sync(0xffffffffu, a.z, lane); o.a.w = __shfl_sync(0xffffffffu, a.w, lane);
    o.b.x = __shfl_sync(0xffffffffu, b.x, lane); o.b.y = __shfl_sync(0xffffffffu, b.y, lane);
    o.b.z = __shfl_sync(0xffffffffu, b.z, lane); o.b.w = __shfl_sync(0xffffffffu, b.w, lane);
    return o;
  }
};

template <typename T>
struct Rows {   // one tensor of rows: channel 0 of (token, head) at p + token * ts + head * hs
  T* p;
  int64_t ts, hs;
  __device__ __forceinline__ T* at(int64_t token, int head) const { return p + token * ts + head * hs; }
};

struct Turn {
  const int* pos;          // [N, axes]
  const double* freq;      // [rot / 2] radians per position
  const int* axis;         // [rot / 2]
  int axes, rot;
};

// Where a lane's 8 channels [c0, c0 + 8) stand in the rotation.
struct Place {
  int lane;        // lane that holds the paired channels
  int pc0;         // the first of them
  int p0;          // first pair
  bool turned;     // the channels are rotated
  bool second;     // they come second in their pairs
};
template <bool INTER>
__device__ __forceinline__ Place place_of(int lane, int c0, int rot) {
  const int half = rot >> 1;
  Place p;
  p.turned = c0 < rot;
  p.second = !INTER && p.turned && c0 >= half;
  const int d = INTER || !p.turned ? 0 : (p.second ? -half : half);
  p.lane = lane + d / 8;
  p.pc0 = c0 + d;
  p.p0 = INTER ? c0 >> 1 : (p.second ? c0 - half : c0);
  return p;
}

// cos and sin of one pair's angle.  It is held in turns as a 64-bit binary
// fraction: the frequency is brought to one, and its product with the integer
// position wraps without rounding, so a far position keeps its angle where a
// 32-bit product of radians loses it.  1 / (2 pi) comes in two parts and the
// product's rounding error is kept, as the whole turns of a frequency above one
// radian would take the digits behind them: the step is off by at most 2^-64
// turns (|frequency| <= 2^40; with one part it was 2^-49 turns at 100 radians).
// The phase is then rounded to the 24 bits of a float, 2^-25 turns with what is
// cut before; fp32 functions of it are off by 2^-23, and more bits of their
// argument would not show in a result of 24.
__device__ __forceinline__ void pair_angle(const Turn& t, int64_t token, int pair, float& c, float& s) {
  c = 1.f;
  s = 0.f;
  const int ax = __ldg(t.axis + pair);
  if (ax < 0 || ax >= t.axes) return;
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;   // 1 / (2 pi)
  const double f = __ldg(t.freq + pair), turns = f * kHi;
  double rest = fma(f, kLo, fma(f, kHi, -turns));   // what the product lost
  rest -= rint(rest);
  constexpr double kTurn = 18446744073709551616.0;
  const unsigned long long step = (unsigned long long)__double2ll_rn((turns - rint(turns)) * kTurn) +
                                  (unsigned long long)__double2ll_rn(rest * kTurn);
  const long long pos = __ldg(t.pos + token * t.axes + ax);
  const int frac = (int)(((unsigned long long)pos * step + 0x80000000ull) >> 32);   // signed: half a turn either way
  sincospif((float)frac * 4.656612873077392578125e-10f, &s, &c);
}

// cos and sin of this lane's 8 channels, the sin with the sign that it takes
// in y_i = z_i cos_i + z_paired sin_i.  The two lanes of a pair of channels
// share its angles: each computes four of the eight.
template <bool INTER>
__device__ __forceinline__ void lane_angles(const Turn& t, int64_t token, const Place& pl, float2 (&cs)[4], float2 (&sn)[4]) {
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (pl.turned) {
#pragma unroll
    for (int i = 0; i < 4; ++i) pair_angle(t, token, pl.p0 + i + (!INTER && pl.second ? 4 : 0), c[i], s[i]);
  }
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[i] = make_float2(c[i], c[i]);
      sn[i] = make_float2(-s[i], s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float oc = __shfl_sync(0xffffffffu, c[i], pl.lane), os = __shfl_sync(0xffffffffu, s[i], pl.lane);
      if (pl.second) {
        c[i + 4] = c[i]; s[i + 4] = s[i];
        c[i] = oc; s[i] = os;
      } else {
        c[i + 4] = oc; s[i + 4] = os;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[i] = make_float2(c[2 * i], c[2 * i + 1]);
      sn[i] = pl.second ? make_float2(s[2 * i], s[2 * i + 1]) : make_float2(-s[2 * i], -s[2 * i + 1]);
    }
  }
}

// the values that the channels are paired with, as fp32
template <bool INTER, typename T>
__device__ __forceinline__ void paired(const Raw8<T>& r, const float2 (&x)[4], int lane, float2 (&xp)[4]) {
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) xp[i] = make_float2(x[i].y, x[i].x);
  } else {
    r.from(lane).get(xp);
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
// sum over the row of the squares, then 1 / sqrt(mean + eps)
template <int D>
__device__ __forceinline__ float row_inv(const float2 (&x)[4], float eps) {
  float2 a = __fmul2_rn(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) a = __ffma2_rn(x[i], x[i], a);
  return rsqrtf(row_sum<D / 8>(a.x + a.y) * (1.f / D) + eps);
}

__device__ __forceinline__ float2 weight2(const float* w, int c) {
  return w ? make_float2(__ldg(w + c), __ldg(w + c + 1)) : make_float2(1.f, 1.f);
}

template <typename T>
struct FwdArgs {
  Rows<const T> q, k, v;
  Rows<T> qo, ko;          // ko.p may be null (K goes to the cache alone)
  T *kc, *vc;              // paged cache [pages, Hk, page, D], or null
  const int64_t* slots;    // [N] place in the cache (page * page_size + offset); outside it: not stored
  const float *wq, *wk;
  Turn turn;
  int64_t slot_end;        // pages * page_size
  int N, Hq, Hk, page, rows, rpw, segs;   // rows of a token; rows of a warp; warps of a token
  float eps;
};

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 6)
k_qk_norm_rope(const __grid_constant__ FwdArgs<T> a) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const int64_t wid = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  ptx::grid_wait_prerequisites();
  ptx::grid_launch_dependents();
  const int64_t token = wid / a.segs;
  if (token >= a.N) return;
  const int r0 = (int)(wid - token * a.segs) * a.rpw, r1 = min(a.rows, r0 + a.rpw);
  const int g = lane / LPR, c0 = (lane % LPR) * 8;
  const Place pl = place_of<INTER>(lane, c0, a.turn.rot);
  // the first rows are on their way while the angles are computed
  Raw8<T> raw[kBatch];
  auto load = [&](const T* src, int64_t hs, int hb, int h1) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int h = hb + u * GPW + g;
      if (h < h1) raw[u].load(src + h * hs);
    }
  };
  if (r0 < a.Hq) load(a.q.at(token, 0) + c0, a.q.hs, r0, min(r1, a.Hq));
  float2 cs[4], sn[4];
  lane_angles<INTER>(a.turn, token, pl, cs, sn);
  int64_t slot = a.slots ? __ldg(a.slots + token) : -1;
  if (slot >= a.slot_end) slot = -1;
  // element offset of (page, head 0, offset) in the cache
  const int64_t cbase = slot < 0 ? 0 : ((slot / a.page) * a.Hk * a.page + slot % a.page) * D;

  // rows [h0, h1) of q or of k
  auto heads = [&](bool isq, int h0, int h1) {
    const float* w = isq ? a.wq : a.wk;
    // weight times cos, the paired channel's weight times sin: once a token instead
    // of once a row, for one more rounding of 2^-24
    float2 wc[4], ws[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 wi = weight2(w, c0 + 2 * i), wp = weight2(w, pl.pc0 + 2 * i);
      wc[i] = __fmul2_rn(wi, cs[i]);
      ws[i] = __fmul2_rn(INTER ? make_float2(wp.y, wp.x) : wp, sn[i]);
    }
    const int64_t hs = isq ? a.q.hs : a.k.hs;
    const T* src = (isq ? a.q.at(token, 0) : a.k.at(token, 0)) + c0;
    const bool plain = isq || a.ko.p;   // the result goes to q_out or k_out ...
    const bool cached = !isq && slot >= 0;   // ... and to the cache
    const int64_t os = isq ? a.qo.hs : a.ko.hs, ks = (int64_t)a.page * D;
    T* dst = (isq ? a.qo.at(token, 0) : a.ko.at(token, 0)) + c0;
    T* kc = a.kc + cbase + c0;
    for (int hb = h0; hb < h1; hb += GPW * kBatch) {
      if (!isq || hb != h0) load(src, hs, hb, h1);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (hb + u * GPW >= h1) break;   // the same for the whole warp
        const int h = hb + u * GPW + g;
        float2 x[4], xp[4];
        raw[u].get(x);
        paired<INTER>(raw[u], x, pl.lane, xp);
        const float inv = row_inv<D>(x, a.eps);
        const float2 inv2 = make_float2(inv, inv);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = __ffma2_rn(__fmul2_rn(x[i], inv2), wc[i], __fmul2_rn(__fmul2_rn(xp[i], inv2), ws[i]));
        if (h >= h1) continue;
        raw[u].set(x);
        if (plain) raw[u].store(dst + h * os);
        if (cached) raw[u].store(kc + h * ks);
      }
    }
  };
  if (r0 < a.Hq) heads(true, r0, min(r1, a.Hq));
  if (r1 > a.Hq && r0 < a.Hq + a.Hk) heads(false, max(r0 - a.Hq, 0), min(r1 - a.Hq, a.Hk));
  const int hk = a.Hq + a.Hk;
  if (slot >= 0)   // V goes along as it is
    for (int h = max(r0 - hk, 0) + g; h < r1 - hk; h += GPW) {
      Raw8<T> raw;
      raw.load(a.v.at(token, h) + c0);
      raw.store(a.vc + cbase + (int64_t)h * a.page * D + c0);
    }
}

// Rows of one tensor, q or k, of the gradient.
template <typename T>
struct BwdSide {
  Rows<const T> x, dy;
  Rows<T> dx;
  const float* w;
  int H, rpw, segs;        // heads; heads of a warp; warps of a token
  int blocks;
};
template <typename T>
struct BwdArgs {
  BwdSide<T> side[2];      // q, then k: the first side[0].blocks blocks are q's
  Turn turn;
  float* part;             // [blocks][D] weight gradients of each block, or null: not wanted
  int N;
  float eps;
};

// Persistent: a block takes q's rows or k's; its warps walk the (token, heads)
// units with the blocks' stride and keep their share of the weight gradient
// in registers; each block leaves one partial sum, and k_qk_weight_grad adds
// the blocks' partials in a fixed order (no atomics: the same inputs give the
// same bits).
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 4)
k_qk_norm_rope_bwd(const __grid_constant__ BwdArgs<T> a) {
  constexpr int LPR = D / 8, GPW = 32 / LPR, NW = kThreads / 32;
  constexpr int NB = 3;   // rows in flight per lane group (two tensors each)
  __shared__ float red[NW][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ptx::grid_wait_prerequisites();
  ptx::grid_launch_dependents();
  const bool isq = (int)blockIdx.x < a.side[0].blocks;
  const BwdSide<T>& sd = isq ? a.side[0] : a.side[1];
  const int g = lane / LPR, c0 = (lane % LPR) * 8;
  const Place pl = place_of<INTER>(lane, c0, a.turn.rot);
  float2 w[4], acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = weight2(sd.w, c0 + 2 * i);
    acc[i] = make_float2(0.f, 0.f);
  }
  const int64_t units = (int64_t)a.N * sd.segs;
  const int64_t first = (int64_t)(isq ? blockIdx.x : blockIdx.x - a.side[0].blocks) * NW + warp;
  for (int64_t wid = first; wid < units; wid += (int64_t)sd.blocks * NW) {
    const int64_t token = wid / sd.segs;
    const int h0 = (int)(wid - token * sd.segs) * sd.rpw, h1 = min(sd.H, h0 + sd.rpw);
    const T* px = sd.x.at(token, 0) + c0;
    const T* py = sd.dy.at(token, 0) + c0;
    T* pd = sd.dx.at(token, 0) + c0;
    Raw8<T> rx[NB], rd[NB];
    auto load = [&](int hb) {
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        const int h = hb + u * GPW + g;
        if (h < h1) {
          rx[u].load(px + h * sd.x.hs);
          rd[u].load(py + h * sd.dy.hs);
        }
      }
    };
    load(h0);   // on their way while the angles are computed
    float2 cs[4], sn[4];
    lane_angles<INTER>(a.turn, token, pl, cs, sn);
#pragma unroll
    for (int i = 0; i < 4; ++i) sn[i] = make_float2(-sn[i].x, -sn[i].y);   // the transposed rotation
    for (int hb = h0; hb < h1; hb += GPW * NB) {
      if (hb != h0) load(hb);
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        if (hb + u * GPW >= h1) break;
        const int h = hb + u * GPW + g;
        const bool live = h < h1;
        float2 x[4], d[4], dp[4];
        rx[u].get(x);
        rd[u].get(d);
        paired<INTER>(rd[u], d, pl.lane, dp);
        const float inv = row_inv<D>(x, a.eps);
        const float2 inv2 = make_float2(inv, inv);
        float2 dot = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 gi = __ffma2_rn(d[i], cs[i], __fmul2_rn(dp[i], sn[i]));
          x[i] = __fmul2_rn(x[i], inv2);
          if (live) acc[i] = __ffma2_rn(gi, x[i], acc[i]);
          d[i] = __fmul2_rn(gi, w[i]);
          dot = __ffma2_rn(d[i], x[i], dot);
        }
        const float along = -row_sum<LPR>(dot.x + dot.y) * (1.f / D);
        if (!live) continue;
        const float2 along2 = make_float2(along, along);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = __fmul2_rn(inv2, __ffma2_rn(x[i], along2, d[i]));
        rd[u].set(d);
        rd[u].store(pd + h * sd.dx.hs);
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int off = 16; off >= LPR; off >>= 1) {
      acc[i].x += __shfl_xor_sync(0xffffffffu, acc[i].x, off);
      acc[i].y += __shfl_xor_sync(0xffffffffu, acc[i].y, off);
    }
    if (g == 0) {
      red[warp][c0 + 2 * i] = acc[i].x;
      red[warp][c0 + 2 * i + 1] = acc[i].y;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) s += red[k][e];
    a.part[(size_t)blockIdx.x * D + e] = s;
  }
}

// dw[c] = sum over a tensor's blocks of part[block][c]; a CTA adds 16 columns,
// 64 blocks at a time
__global__ void __launch_bounds__(1024)
k_qk_weight_grad(const float* part, int blocks_q, int blocks_k, int D, float* dwq, float* dwk) {
  __shared__ float red[16][65];
  ptx::grid_wait_prerequisites();
  ptx::grid_launch_dependents();
  const int per = D / 16;   // CTAs of one tensor
  const bool isq = (int)blockIdx.x < per;
  float* dst = isq ? dwq : dwk;
  if (!dst) return;
  const int col0 = ((int)blockIdx.x - (isq ? 0 : per)) * 16;
  const int b0 = isq ? 0 : blocks_q, nb = isq ? blocks_q : blocks_k;
  const int cx = threadIdx.x & 15, by = threadIdx.x >> 4;
  float s = 0.f;
#pragma unroll 4
  for (int b = by; b < nb; b += 64) s += part[(size_t)(b0 + b) * D + col0 + cx];
  red[cx][by] = s;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < 16) {
    s = red[warp][lane] + red[warp][lane + 32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) dst[col0 + warp] = s;
  }
}

// ------------------------------------------------------------------- host
constexpr int kBwdBlocksPerSm = 4;
constexpr int kBwdMaxBlocks = 1024;

// Rows of a token per warp: as many as leave the GPU's warps (24 an SM) all
// at work, so that the angles are computed as rarely as that allows.
inline int rows_per_warp(int64_t N, int rows, int d, int sms) {
  const int gpw = 256 / d;   // rows a warp holds at once
  const int64_t warps = (int64_t)sms * 24;
  const int64_t want = (N * rows + warps - 1) / warps;
  const int64_t up = (want + gpw - 1) / gpw * gpw;
  return (int)(up < gpw ? gpw : (up > rows ? rows : up));
}

template <typename T>
Rows<T> rows_of(const vda_rows& r) {
  return Rows<T>{static_cast<T*>(r.data), r.token_stride, r.head_stride};
}

template <typename T, int D>
int launch_fwd(const vda_qk_args& s, float eps, int sms) {
  FwdArgs<T> a{};
  a.q = rows_of<const T>(s.q_in);
  a.k = rows_of<const T>(s.k_in);
  a.v = rows_of<const T>(s.v_in);
  a.qo = rows_of<T>(s.q_out);
  a.ko = rows_of<T>(s.k_out);
  a.kc = static_cast<T*>(s.k_cache);
  a.vc = static_cast<T*>(s.v_cache);
  a.slots = s.slots;
  a.wq = s.q_weight;
  a.wk = s.k_weight;
  a.turn = Turn{s.positions, s.frequencies, s.axis, s.axes, s.rot};
  a.slot_end = s.slots ? (int64_t)s.pages * s.page_size : 0;
  a.N = s.N; a.Hq = s.Hq; a.Hk = s.Hk;
  a.page = s.slots ? s.page_size : 1;
  a.rows = s.Hq + s.Hk + (s.slots ? s.Hk : 0);
  a.rpw = rows_per_warp(s.N, a.rows, D, sms);
  a.segs = (a.rows + a.rpw - 1) / a.rpw;
  a.eps = eps;
  const int64_t blocks = ((int64_t)s.N * a.segs + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 2147483647) return VDA_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), block(kThreads);
  cudaStream_t st = static_cast<cudaStream_t>(s.stream);
  return s.interleaved ? tc::launch_pdl("k_qk_norm_rope", k_qk_norm_rope<T, D, true>, grid, block, 0, st, a)
                       : tc::launch_pdl("k_qk_norm_rope", k_qk_norm_rope<T, D, false>, grid, block, 0, st, a);
}

template <typename T, int D>
int launch_bwd(const vda_qk_grad_args& s, float* part, float eps, int sms) {
  BwdArgs<T> a{};
  a.side[0] = BwdSide<T>{rows_of<const T>(s.q_in), rows_of<const T>(s.dq_out), rows_of<T>(s.dq_in), s.q_weight, s.Hq, 0, 0, 0};
  a.side[1] = BwdSide<T>{rows_of<const T>(s.k_in), rows_of<const T>(s.dk_out), rows_of<T>(s.dk_in), s.k_weight, s.Hk, 0, 0, 0};
  a.turn = Turn{s.positions, s.frequencies, s.axis, s.axes, s.rot};
  a.part = part;
  a.N = s.N;
  a.eps = eps;
  // the blocks are shared out by the rows of q and of k
  const int64_t most = std::min(kBwdMaxBlocks, sms * kBwdBlocksPerSm), nw = kThreads / 32;
  for (int i = 0; i < 2; ++i) {
    BwdSide<T>& sd = a.side[i];
    sd.rpw = std::min(rows_per_warp(s.N, s.Hq + s.Hk, D, sms), sd.H);
    sd.segs = (sd.H + sd.rpw - 1) / sd.rpw;
    const int64_t need = ((int64_t)s.N * sd.segs + nw - 1) / nw;
    const int64_t share = std::max<int64_t>(1, i == 0 ? (most * s.Hq + (s.Hq + s.Hk) / 2) / (s.Hq + s.Hk) : most - a.side[0].blocks);
    sd.blocks = (int)std::min(need, i == 0 ? std::min(share, most - 1) : share);
  }
  cudaStream_t st = static_cast<cudaStream_t>(s.stream);
  const dim3 grid((unsigned)(a.side[0].blocks + a.side[1].blocks)), block(kThreads);
  const int rc = s.interleaved
                     ? tc::launch_pdl("k_qk_norm_rope_bwd", k_qk_norm_rope_bwd<T, D, true>, grid, block, 0, st, a)
                     : tc::launch_pdl("k_qk_norm_rope_bwd", k_qk_norm_rope_bwd<T, D, false>, grid, block, 0, st, a);
  if (rc != VDA_OK || !part) return rc;
  return tc::launch_pdl("k_qk_weight_grad", k_qk_weight_grad, dim3(2 * D / 16), dim3(1024), 0, st, (const float*)part,
                        a.side[0].blocks, a.side[1].blocks, D, s.dq_weight, s.dk_weight);
}

}  // namespace qk
}  // namespace vda
