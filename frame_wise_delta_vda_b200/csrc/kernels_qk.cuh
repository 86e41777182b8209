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
// memory.  A warp takes consecutive rows of one token: the token's angles
// are computed once and stay in registers over all its rows.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "vda.h"

namespace vda {
namespace qk {

constexpr int kThreads = 256;
constexpr int kBatch = 4;   // rows in flight per lane group

// 8 consecutive channels as loaded
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_uint4(ptx::pack_bf16(x[0], x[1]), ptx::pack_bf16(x[2], x[3]), ptx::pack_bf16(x[4], x[5]),
                   ptx::pack_bf16(x[6], x[7]));
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&x)[8]) {
    a = make_float4(x[0], x[1], x[2], x[3]);
    b = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
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

// cos and sin of this lane's 8 channels, the sin with the sign that it takes
// in y_i = z_i cos_i + z_partner(i) sin_i; partner lane (offset in the row).
//
// The angle is held in turns as a 64-bit binary fraction: the frequency is
// brought to one once (53 significant bits), and its product with the integer
// position wraps without rounding, so a far position keeps its angle (to
// position * 2^-55 turns) where a 32-bit product of radians loses it.
template <bool INTER>
__device__ __forceinline__ void lane_angles(const Turn& t, int64_t token, int c0, float (&cs)[8], float (&sn)[8]) {
  const int half = t.rot >> 1;
  const bool turned = c0 < t.rot;
  const bool second = !INTER && c0 >= half;
  const int p0 = INTER ? c0 >> 1 : (second ? c0 - half : c0);
#pragma unroll
  for (int i = 0; i < (INTER ? 4 : 8); ++i) {
    float c = 1.f, s = 0.f;
    if (turned) {
      const int ax = __ldg(t.axis + p0 + i);
      if (ax >= 0 && ax < t.axes) {
        double turns = __ldg(t.freq + p0 + i) * 0.15915494309189533577;
        turns -= floor(turns);
        const unsigned long long step = __double2ull_rn(turns * 18446744073709551616.0);
        const long long pos = __ldg(t.pos + token * t.axes + ax);
        const int frac = (int)(((unsigned long long)pos * step) >> 32);   // signed: half a turn either way
        sincospif((float)frac * 4.656612873077392578125e-10f, &s, &c);
      }
    }
    if (INTER) {
      cs[2 * i] = cs[2 * i + 1] = c;
      sn[2 * i] = -s;
      sn[2 * i + 1] = s;
    } else {
      cs[i] = c;
      sn[i] = second ? s : -s;
    }
  }
}

// the value that each channel is paired with
template <bool INTER>
__device__ __forceinline__ void partner(const float (&z)[8], int src_lane, float (&zp)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) zp[i] = INTER ? z[i ^ 1] : __shfl_sync(0xffffffffu, z[i], src_lane);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

__device__ __forceinline__ void load_weight(const float* w, int c0, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = w ? __ldg(w + c0 + i) : 1.f;
}

// lane of the warp that holds the paired channels of this lane
__device__ __forceinline__ int partner_lane(int lane, int c0, int rot) {
  const int half = rot >> 1;
  if (c0 >= rot) return lane;
  return c0 < half ? lane + half / 8 : lane - half / 8;
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
__global__ void __launch_bounds__(kThreads)
k_qk_norm_rope(const FwdArgs<T> a) {
  constexpr int LPR = D / 8, GPW = 32 / LPR;
  const int lane = threadIdx.x & 31;
  const int64_t wid = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  ptx::grid_wait_prerequisites();
  ptx::grid_launch_dependents();
  const int64_t token = wid / a.segs;
  if (token >= a.N) return;
  const int r0 = (int)(wid - token * a.segs) * a.rpw, r1 = min(a.rows, r0 + a.rpw);
  const int g = lane / LPR, c0 = (lane % LPR) * 8;
  float wq[8], wk[8], cs[8], sn[8];
  load_weight(a.wq, c0, wq);
  load_weight(a.wk, c0, wk);
  lane_angles<INTER>(a.turn, token, c0, cs, sn);
  const int pl = partner_lane(lane, c0, a.turn.rot);
  int64_t slot = a.slots ? __ldg(a.slots + token) : -1;
  if (slot >= a.slot_end) slot = -1;
  // element offset of (page, head 0, offset) in the cache
  const int64_t cbase = slot < 0 ? 0 : ((slot / a.page) * a.Hk * a.page + slot % a.page) * D;

  for (int rb = r0; rb < r1; rb += GPW * kBatch) {
    Raw8<T> raw[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int r = rb + u * GPW + g;
      if (r >= r1) continue;
      const T* src = r < a.Hq ? a.q.at(token, r)
                              : (r < a.Hq + a.Hk ? a.k.at(token, r - a.Hq) : a.v.at(token, r - a.Hq - a.Hk));
      raw[u].load(src + c0);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (rb + u * GPW >= r1) break;   // the same for the whole warp
      const int r = rb + u * GPW + g;
      const bool live = r < r1;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (live) raw[u].get(x);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
      const float inv = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + a.eps);
      const bool isq = r < a.Hq;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= inv * (isq ? wq[i] : wk[i]);
      float xp[8];
      partner<INTER>(x, pl, xp);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], cs[i], xp[i] * sn[i]);
      if (!live) continue;
      if (isq) {
        raw[u].set(x);
        raw[u].store(a.qo.at(token, r) + c0);
      } else if (r < a.Hq + a.Hk) {
        const int h = r - a.Hq;
        raw[u].set(x);
        if (a.ko.p) raw[u].store(a.ko.at(token, h) + c0);
        if (slot >= 0) raw[u].store(a.kc + cbase + (int64_t)h * a.page * D + c0);
      } else if (slot >= 0) {   // V goes along as it is
        raw[u].store(a.vc + cbase + (int64_t)(r - a.Hq - a.Hk) * a.page * D + c0);
      }
    }
  }
}

template <typename T>
struct BwdArgs {
  Rows<const T> q, k, dqo, dko;
  Rows<T> dq, dk;
  const float *wq, *wk;
  Turn turn;
  float* part;             // [blocks][2][D] weight gradients of each block, or null: not wanted
  int N, Hq, Hk, rows, rpw, segs;
  float eps;
};

// Persistent: warps walk the (token, rows) units with the grid's stride and
// keep their share of the weight gradients in registers; each block leaves
// one partial sum, and k_qk_weight_grad adds the blocks' partials in a fixed
// order (no atomics: the same inputs give the same bits).
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads)
k_qk_norm_rope_bwd(const BwdArgs<T> a) {
  constexpr int LPR = D / 8, GPW = 32 / LPR, NW = kThreads / 32;
  constexpr int NB = 2;   // rows in flight per lane group (two tensors each)
  __shared__ float red[NW][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ptx::grid_wait_prerequisites();
  ptx::grid_launch_dependents();
  const int g = lane / LPR, c0 = (lane % LPR) * 8;
  float wq[8], wk[8], sq[8], sk[8];
  load_weight(a.wq, c0, wq);
  load_weight(a.wk, c0, wk);
#pragma unroll
  for (int i = 0; i < 8; ++i) sq[i] = sk[i] = 0.f;
  const int pl = partner_lane(lane, c0, a.turn.rot);
  const int64_t units = (int64_t)a.N * a.segs;
  for (int64_t wid = (int64_t)blockIdx.x * NW + warp; wid < units; wid += (int64_t)gridDim.x * NW) {
    const int64_t token = wid / a.segs;
    const int r0 = (int)(wid - token * a.segs) * a.rpw, r1 = min(a.rows, r0 + a.rpw);
    float cs[8], sn[8];
    lane_angles<INTER>(a.turn, token, c0, cs, sn);
    for (int rb = r0; rb < r1; rb += GPW * NB) {
      Raw8<T> rx[NB], rd[NB];
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        const int r = rb + u * GPW + g;
        if (r >= r1) continue;
        const bool isq = r < a.Hq;
        const int h = isq ? r : r - a.Hq;
        rx[u].load((isq ? a.q.at(token, h) : a.k.at(token, h)) + c0);
        rd[u].load((isq ? a.dqo.at(token, h) : a.dko.at(token, h)) + c0);
      }
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        if (rb + u * GPW >= r1) break;
        const int r = rb + u * GPW + g;
        const bool live = r < r1, isq = r < a.Hq;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, dp[8];
        if (live) {
          rx[u].get(x);
          rd[u].get(d);
        }
        partner<INTER>(d, pl, dp);
        float ss = 0.f, along = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
        const float inv = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float gi = fmaf(d[i], cs[i], -dp[i] * sn[i]);
          x[i] *= inv;
          const float t = gi * x[i];
          sq[i] += isq ? t : 0.f;
          sk[i] += isq ? 0.f : t;
          d[i] = gi * (isq ? wq[i] : wk[i]);
          along = fmaf(d[i], x[i], along);
        }
        along = row_sum<LPR>(along) * (1.f / D);
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = inv * fmaf(-x[i], along, d[i]);
        rd[u].set(d);
        const int h = isq ? r : r - a.Hq;
        rd[u].store((isq ? a.dq.at(token, h) : a.dk.at(token, h)) + c0);
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma unroll
    for (int off = 16; off >= LPR; off >>= 1) {
      sq[i] += __shfl_xor_sync(0xffffffffu, sq[i], off);
      sk[i] += __shfl_xor_sync(0xffffffffu, sk[i], off);
    }
    if (g == 0) {
      red[warp][0][c0 + i] = sq[i];
      red[warp][1][c0 + i] = sk[i];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * D; e += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += red[w][e / D][e % D];
    a.part[(size_t)blockIdx.x * 2 * D + e] = s;
  }
}

// dw[c] = sum over blocks of part[block][c]; 32 columns x 32 block strides per CTA
__global__ void __launch_bounds__(1024)
k_qk_weight_grad(const float* part, int blocks, int D, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  ptx::grid_wait_prerequisites();
  ptx::grid_launch_dependents();
  const int cx = threadIdx.x & 31, by = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;   // 2 D columns: q's, then k's
  float s = 0.f;
  for (int b = by; b < blocks; b += 32) s += part[(size_t)b * 2 * D + c];
  red[by][cx] = s;
  __syncthreads();
  s = red[cx][by];   // transposed: a warp adds one column
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (cx == 0) {
    const int o = blockIdx.x * 32 + by;
    float* dst = o < D ? dwq : dwk;
    if (dst) dst[o < D ? o : o - D] = s;
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
  a.q = rows_of<const T>(s.q_in);
  a.k = rows_of<const T>(s.k_in);
  a.dqo = rows_of<const T>(s.dq_out);
  a.dko = rows_of<const T>(s.dk_out);
  a.dq = rows_of<T>(s.dq_in);
  a.dk = rows_of<T>(s.dk_in);
  a.wq = s.q_weight;
  a.wk = s.k_weight;
  a.turn = Turn{s.positions, s.frequencies, s.axis, s.axes, s.rot};
  a.part = part;
  a.N = s.N; a.Hq = s.Hq; a.Hk = s.Hk;
  a.rows = s.Hq + s.Hk;
  a.rpw = rows_per_warp(s.N, a.rows, D, sms);
  a.segs = (a.rows + a.rpw - 1) / a.rpw;
  a.eps = eps;
  const int64_t units = (int64_t)s.N * a.segs, nw = kThreads / 32;
  int64_t blocks = (units + nw - 1) / nw;
  blocks = std::min<int64_t>(blocks, std::min(kBwdMaxBlocks, sms * kBwdBlocksPerSm));
  cudaStream_t st = static_cast<cudaStream_t>(s.stream);
  const dim3 grid((unsigned)blocks), block(kThreads);
  const int rc = s.interleaved
                     ? tc::launch_pdl("k_qk_norm_rope_bwd", k_qk_norm_rope_bwd<T, D, true>, grid, block, 0, st, a)
                     : tc::launch_pdl("k_qk_norm_rope_bwd", k_qk_norm_rope_bwd<T, D, false>, grid, block, 0, st, a);
  if (rc != VDA_OK || !part) return rc;
  return tc::launch_pdl("k_qk_weight_grad", k_qk_weight_grad, dim3(2 * D / 32), dim3(1024), 0, st,
                        (const float*)part, (int)blocks, D, s.dq_weight, s.dk_weight);
}

}  // namespace qk
}  // namespace vda
