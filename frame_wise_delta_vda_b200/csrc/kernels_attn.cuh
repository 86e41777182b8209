// Attention of new tokens over a paged cache (the Softmax branch: a chunk of
// new tokens sees its own block, a window of blocks before it and the
// anchors), B200 (sm_100a).
//
//   s_ij = scale q_i k_j over the keys that token i sees, o_i = sum_j
//   exp(s_ij - m_i) v_j / l_i,  l_i = sum_j exp(s_ij - m_i),  lse_i = m_i + log l_i
//
// in one pass over the keys with the running maximum m and sum l: a later,
// larger maximum scales what was summed.  Rows of a work item are (token,
// query head) pairs that share one KV head, so grouped heads read a key once.
//   k_attn_simt  any supported type and d, fp32 arithmetic
//   k_attn_join  joins the parts of items that several CTAs took
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include <atomic>

#include "attn_sched.cuh"
#include "common.cuh"
#include "tc_ptx.cuh"
#include "vda.h"

namespace vda {
namespace attn {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// Parts of split items: share g's first item (begun in an earlier share) in
// slot 0, its last (continued in a later one) in slot 1; per row the sums
// before division and (maximum in log2 units, sum).
struct Parts {
  float* o;      // [shares][2][rows][D]
  float2* ml;    // [shares][2][rows]
  Meta* meta;    // [shares]
  int rows;      // rows of a slot
};

struct CacheView {
  const int* table;        // [B, max_pages]
  int64_t table_stride;
  int pages;               // pages of the cache: ids outside [0, pages) are absent
  int page;                // tokens of a page
};

template <typename T>
struct OutView {
  T* out;                  // [N, Hq, D] by strides
  int64_t ts, hs;
  float* lse;              // [N, Hq] or null
  int Hq;
};

__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(ptx::pack_bf16(v.x, v.y), ptx::pack_bf16(v.z, v.w));
}
__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}

// ===========================================================================
// k_attn_simt: float32 I/O and head sizes without a tensor-core kernel.
// BM rows x 64 keys a tile; thread (ty, tx) of 16 x 16 has BM / 16 rows x 4 keys
// of the scores and BM / 16 rows x D / 16 channels of the output.  Bound by
// shared memory, not by the FMA pipe: at BM = 64 and D = 64 a thread reads eight
// 16-B words for 64 FMAs in the scores and again in P V, at BM = 16 five for 16.
// fp32, 4 x 256 tokens over 2000 keys, 8 / 2 heads: 160 us at d = 64 (24.6
// TFLOP/s of the pipe's 74) and 361 us at d = 128 (21.8), where 117 KB of shared
// memory let one CTA of the two per SM that the plan makes run at a time.
// ===========================================================================
template <int D, int BM>
struct SimtCfg {
  static constexpr int BN = 64, THREADS = 256;
  static constexpr int KS = D + 4;    // K row stride (floats): 16 rows hit different banks
  static constexpr int PS = BN + 4;   // P row stride
  static constexpr size_t SMEM = sizeof(float) * ((size_t)BM * D + (size_t)BN * KS + (size_t)BN * D + (size_t)BM * PS) +
                                 BN * sizeof(int) + sizeof(Plan) + 16;
};

template <typename T, int D, int BM>
__global__ void __launch_bounds__(SimtCfg<D, BM>::THREADS)
k_attn_simt(const T* __restrict__ q, int64_t q_ts, int64_t q_hs, const T* __restrict__ kc, const T* __restrict__ vc,
            CacheView cv, const __grid_constant__ Geom g, OutView<T> ov, Parts parts, float c2) {
  using C = SimtCfg<D, BM>;
  constexpr int BN = C::BN, R = BM / 16, V4 = D / 4, CPT = (V4 + 15) / 16;   // rows, 4-channel chunks a thread
  extern __shared__ __align__(16) uint8_t smem_raw[];
  float* Qs = reinterpret_cast<float*>(smem_raw);
  float* Ks = Qs + BM * D;
  float* Vs = Ks + BN * C::KS;
  float* Ps = Vs + BN * D;
  int* ok = reinterpret_cast<int*>(Ps + BM * C::PS);   // the key's page is there
  Plan* plan = reinterpret_cast<Plan*>((reinterpret_cast<uintptr_t>(ok + BN) + 15) & ~(uintptr_t)15);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  ptx::grid_wait_prerequisites();
  ptx::grid_launch_dependents();
  if (tid < 32) {
    const Plan p = plan_share<BN>(g, blockIdx.x, gridDim.x, tid);
    if (tid == 0) *plan = p;
  }
  __syncthreads();
  const Plan pl = *plan;
  Meta meta{0, 0, 0, 0};
  for (Walk<BN> w(g, pl); w.live; w.next()) {
    const int rows = w.ntok * g.group, tok0 = w.s.q0 + w.i0;
#pragma unroll
    for (int k = 0; k < (BM * V4 + C::THREADS - 1) / C::THREADS; ++k) {
      const int e = tid + k * C::THREADS, r = e / V4, v = e - r * V4;
      if (r >= BM) break;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) x = load4(q + (int64_t)(tok0 + r / g.group) * q_ts + (int64_t)(w.h * g.group + r % g.group) * q_hs + 4 * v);
      *reinterpret_cast<float4*>(Qs + r * D + 4 * v) = x;
    }
    Span sp[R];
    float m[R], l[R];
    float4 o[R][CPT];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = ty * R + i;
      sp[i] = r < rows ? span_of(g, w.s.len - w.s.n + w.i0 + r / g.group, w.s.len) : Span{0, 0, 0};
      m[i] = neg_inf();
      l[i] = 0.f;
#pragma unroll
      for (int v = 0; v < CPT; ++v) o[i][v] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int t = w.t0; t < w.t1; ++t) {
      const int j0 = key_tile(w.tiles, t) * BN;
#pragma unroll
      for (int k = 0; k < (BN * V4 + C::THREADS - 1) / C::THREADS; ++k) {   // unrolled: the loads overlap
        const int e = tid + k * C::THREADS, r = e / V4, v = e - r * V4, j = j0 + r;
        if (r >= BN) break;
        // keys that no row of the item sees read as zeros: what lies there may be anything
        float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
        int id = -1;
        if (j < w.tiles.anc || (j >= w.tiles.lo && j < w.tiles.end)) id = __ldg(cv.table + (int64_t)w.b * cv.table_stride + j / cv.page);
        const bool there = id >= 0 && id < cv.pages;
        if (there) {
          const int64_t at = (((int64_t)id * g.Hk + w.h) * cv.page + j % cv.page) * D + 4 * v;
          kx = load4(kc + at);
          vx = load4(vc + at);
        }
        *reinterpret_cast<float4*>(Ks + r * C::KS + 4 * v) = kx;
        *reinterpret_cast<float4*>(Vs + r * D + 4 * v) = vx;
        if (v == 0) ok[r] = there;
      }
      __syncthreads();
      float s[R][4];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[i][k] = 0.f;
#pragma unroll 4
      for (int v = 0; v < V4; ++v) {
        float4 a[R], b[4];
#pragma unroll
        for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4*>(Qs + (ty * R + i) * D + 4 * v);
#pragma unroll
        for (int k = 0; k < 4; ++k) b[k] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * k) * C::KS + 4 * v);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[i][k] = fmaf(a[i].x, b[k].x, s[i][k]);
            s[i][k] = fmaf(a[i].y, b[k].y, s[i][k]);
            s[i][k] = fmaf(a[i].z, b[k].z, s[i][k]);
            s[i][k] = fmaf(a[i].w, b[k].w, s[i][k]);
          }
      }
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float mx = neg_inf();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int j = j0 + tx + 16 * k;
          const bool see = j < sp[i].end && (j >= sp[i].lo || j < sp[i].anc) && ok[tx + 16 * k];
          s[i][k] = see ? s[i][k] * c2 : neg_inf();
          mx = fmaxf(mx, s[i][k]);
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float mn = fmaxf(m[i], mx);
        const float base = mn == neg_inf() ? 0.f : mn;   // nothing seen yet: every weight is 0
        const float alpha = exp2f(m[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float p = exp2f(s[i][k] - base);
          sum += p;
          Ps[(ty * R + i) * C::PS + tx + 16 * k] = p;
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l[i] = fmaf(l[i], alpha, sum);
        m[i] = mn;
#pragma unroll
        for (int v = 0; v < CPT; ++v) {
          o[i][v].x *= alpha; o[i][v].y *= alpha; o[i][v].z *= alpha; o[i][v].w *= alpha;
        }
      }
      __syncwarp();   // a row's P is written and read by the same half warp
#pragma unroll 2
      for (int k4 = 0; k4 < BN; k4 += 4) {
        float4 p[R];
#pragma unroll
        for (int i = 0; i < R; ++i) p[i] = *reinterpret_cast<const float4*>(Ps + (ty * R + i) * C::PS + k4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
#pragma unroll
          for (int v = 0; v < CPT; ++v) {
            const int ch = tx + 16 * v;
            if (ch >= V4) continue;
            const float4 x = *reinterpret_cast<const float4*>(Vs + (k4 + kk) * D + 4 * ch);
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const float pk = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
              o[i][v].x = fmaf(pk, x.x, o[i][v].x);
              o[i][v].y = fmaf(pk, x.y, o[i][v].y);
              o[i][v].z = fmaf(pk, x.z, o[i][v].z);
              o[i][v].w = fmaf(pk, x.w, o[i][v].w);
            }
          }
      }
      __syncthreads();   // K, V and Q are read: the next tile or item may replace them
    }
    const bool whole = w.whole();
    const int slot = w.t0 > 0 ? 0 : 1;
    if (!whole && slot == 1) {   // begun here, continued in later shares
      meta.parts = w.parts(pl, blockIdx.x);
      meta.tok0 = tok0;
      meta.h = w.h;
      meta.rows = rows;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = ty * R + i;
      if (r >= rows) continue;
      const int tok = tok0 + r / g.group, hd = w.h * g.group + r % g.group;
      const size_t prow = ((size_t)blockIdx.x * 2 + slot) * parts.rows + r;
      const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
      for (int v = 0; v < CPT; ++v) {
        const int ch = tx + 16 * v;
        if (ch >= V4) continue;
        float4 x = o[i][v];
        if (whole) {
          x.x *= inv; x.y *= inv; x.z *= inv; x.w *= inv;
          store4(ov.out + (int64_t)tok * ov.ts + (int64_t)hd * ov.hs + 4 * ch, x);
        } else {
          store4(parts.o + prow * D + 4 * ch, x);
        }
      }
      if (tx == 0) {
        if (!whole) parts.ml[prow] = make_float2(m[i], l[i]);
        else if (ov.lse) ov.lse[(int64_t)tok * ov.Hq + hd] = l[i] == 0.f ? neg_inf() : (m[i] + log2f(l[i])) * kLn2;
      }
    }
  }
  if (tid == 0) parts.meta[blockIdx.x] = meta;
}

// ===========================================================================
// k_attn_join: one warp a row of an item that several shares took.  The
// owner is the share in which the item begins: its slot 1, then slot 0 of the
// shares after it.
// ===========================================================================
template <typename T, int D>
__global__ void __launch_bounds__(256)
k_attn_join(Parts parts, OutView<T> ov, int group) {
  constexpr int CPL = D / 32 > 0 ? D / 32 : 1;   // channels a lane
  ptx::grid_wait_prerequisites();
  ptx::grid_launch_dependents();
  const Meta me = parts.meta[blockIdx.x];
  const int lane = threadIdx.x & 31;
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < me.rows; r += gridDim.y * 8) {
    auto row = [&](int i) -> size_t {
      return (((size_t)blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * parts.rows + r;
    };
    // lane i holds the maximum and sum of part i (of 32 at a time)
    float m = neg_inf(), l = 0.f, o[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) o[c] = 0.f;
    for (int i0 = 0; i0 < me.parts; i0 += 32) {
      const int n = imin(32, me.parts - i0);
      const float2 ml = lane < n ? parts.ml[row(i0 + lane)] : make_float2(neg_inf(), 0.f);
      float mn = fmaxf(m, ml.x);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
      const float base = mn == neg_inf() ? 0.f : mn;
      const float before = exp2f(m - base), a = exp2f(ml.x - base);
      float sum = ml.y * a;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l = fmaf(l, before, sum);
      m = mn;
#pragma unroll
      for (int c = 0; c < CPL; ++c) o[c] *= before;
#pragma unroll 8
      for (int i = 0; i < n; ++i) {
        const float ai = __shfl_sync(0xffffffffu, a, i);
        const float* src = parts.o + row(i0 + i) * D + lane * CPL;
        if constexpr (CPL == 4) {
          const float4 x = *reinterpret_cast<const float4*>(src);
          o[0] = fmaf(x.x, ai, o[0]); o[1] = fmaf(x.y, ai, o[1]);
          o[2] = fmaf(x.z, ai, o[2]); o[3] = fmaf(x.w, ai, o[3]);
        } else {
#pragma unroll
          for (int c = 0; c < CPL; ++c)
            if (lane * CPL + c < D) o[c] = fmaf(src[c], ai, o[c]);
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int tok = me.tok0 + r / group, hd = me.h * group + r % group;
    T* dst = ov.out + (int64_t)tok * ov.ts + (int64_t)hd * ov.hs + lane * CPL;
#pragma unroll
    for (int c = 0; c < CPL; ++c) o[c] *= inv;
    if constexpr (CPL == 4) {
      store4(dst, make_float4(o[0], o[1], o[2], o[3]));
    } else {
#pragma unroll
      for (int c = 0; c < CPL; ++c)
        if (lane * CPL + c < D) dst[c] = from_f32<T>(o[c]);
    }
    if (lane == 0 && ov.lse) ov.lse[(int64_t)tok * ov.Hq + hd] = l == 0.f ? neg_inf() : (m + log2f(l)) * kLn2;
  }
}

// ------------------------------------------------------------------- host
inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// What an item costs besides its key tiles, in tiles (Q's load, the first
// scores, the output).  32 / 8 heads of 128, with 0, 1, 3 and 6 in us: 64 single
// tokens over 246 to 8200 keys 176, 168, 150, 154; 200 over 100 to 600 keys 184,
// 168, 164, 166; 17 over 500 to 30000 keys 145, 135, 126, 127; 40 sequences of 1
// to 5 tokens over 50 to 3000 keys 96, 92, 88, 88; 6 prompts of 30 to 900 tokens
// over 900 to 4000 keys 133, 129, 121, 123.
constexpr int kTcItemCost = 3;

struct AttnPlan {
  bool tc;
  int ctas, rows, tpi;     // CTAs, rows of a part, tokens of an item
  int join_y;              // blocks of eight rows at a time that join one item
  size_t off_ml, off_meta, total;
};

// The tensor-core kernel takes bf16 of d = 64 and 128 in pages of a power of two
// from 8 tokens (a box of a TMA load: whole groups of 8 rows of the swizzle), up
// to 128 query heads a KV head; the SIMT kernel everything else, up to 64.
// bf16, 32 / 8 heads of 128, tensor cores and SIMT in us: 64 x 1 token over 4096
// keys 194 and 1588; 1 token over 100 keys 17.4 and 23.5; 2 x 512 tokens over
// 4096 keys 107 and 2649.
inline bool tc_supported(int dtype, int d, int group, int page) {
  return dtype == VDA_BF16 && (d == 64 || d == 128) && group <= 128 && page >= 8 && (page & (page - 1)) == 0;
}

inline AttnPlan make_attn_plan(int dtype, int Hq, int Hk, int d, int page, long long N, int B, int sms) {
  AttnPlan p{};
  const int G = Hq / Hk;
  p.tc = tc_supported(dtype, d, G, page);
  if (p.tc) {
    p.rows = 256;
    p.ctas = sms;
    p.tpi = 2 * (128 / G);
  } else {
    // 16-row tiles where a sequence has that few rows on average, else 64.
    // fp32, 8 / 2 heads of 64 over 2000 keys, 16 and 64 rows in us: 64 x 1 token
    // 134 and 179; 16 x 4 tokens 52 and 62; 16 x 8 tokens 75 and 67; 4 x 256
    // tokens 351 and 159
    p.rows = G <= 16 && N * G <= 16LL * B ? 16 : 64;
    p.ctas = 2 * sms;
    p.tpi = p.rows / G;
  }
  // rows that an item has on average
  const long long per = N * G / (B > 0 ? B : 1) + 1;
  p.join_y = (int)((per < p.rows ? per : p.rows) + 15) / 16;
  const size_t slots = (size_t)p.ctas * 2 * p.rows;
  p.off_ml = align256(slots * d * sizeof(float));
  p.off_meta = p.off_ml + align256(slots * sizeof(float2));
  p.total = p.off_meta + align256((size_t)p.ctas * sizeof(Meta));
  return p;
}

inline Geom geom_of(const vda_attn_args& a, const AttnPlan& p) {
  Geom g{};
  g.q_start = a.q_start;
  g.kv_len = a.kv_len;
  g.B = a.B; g.N = a.N; g.Hk = a.Hk;
  g.group = a.Hq / a.Hk;
  g.tpi = p.tpi;
  const long long keys = (long long)a.max_pages * a.page_size;
  g.max_keys = keys > 2147483647LL ? 2147483647 : (int)keys;
  g.block = a.block; g.window = a.window_blocks; g.anchors = a.anchors;
  g.item_cost = p.tc ? kTcItemCost : 0;
  return g;
}

template <typename T>
OutView<T> out_of(const vda_attn_args& a) {
  return OutView<T>{static_cast<T*>(a.out.data), a.out.token_stride, a.out.head_stride, a.lse, a.Hq};
}

inline Parts parts_of(char* ws, const AttnPlan& p) {
  return Parts{reinterpret_cast<float*>(ws), reinterpret_cast<float2*>(ws + p.off_ml),
               reinterpret_cast<Meta*>(ws + p.off_meta), p.rows};
}

template <typename T, int D>
int launch_join(const AttnPlan& p, const Parts& parts, const OutView<T>& ov, int group, cudaStream_t s) {
  return tc::launch_pdl("k_attn_join", k_attn_join<T, D>, dim3((unsigned)p.ctas, (unsigned)p.join_y), dim3(256), 0, s,
                        parts, ov, group);
}

// Shared memory of a kernel, set the first time that a device runs it.
template <typename K>
bool allow_smem(K kernel, size_t bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const bool known = dev >= 0 && dev < 64;
  if (known && done[dev].load(std::memory_order_relaxed)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) return false;
  if (known) done[dev].store(true, std::memory_order_relaxed);
  return true;
}

template <typename T, int D, int BM>
int launch_simt(const vda_attn_args& a, const AttnPlan& p, char* ws, float c2) {
  using C = SimtCfg<D, BM>;
  auto kernel = k_attn_simt<T, D, BM>;
  static std::atomic<bool> set[64];
  if (!allow_smem(kernel, C::SMEM, set)) return VDA_ERR_CUDA;
  const Geom g = geom_of(a, p);
  const OutView<T> ov = out_of<T>(a);
  const Parts parts = parts_of(ws, p);
  const CacheView cv{a.block_table, a.table_stride, a.pages, a.page_size};
  cudaStream_t s = static_cast<cudaStream_t>(a.stream);
  const int rc = tc::launch_pdl("k_attn_simt", kernel, dim3((unsigned)p.ctas), dim3(C::THREADS), C::SMEM, s,
                                static_cast<const T*>(a.q.data), a.q.token_stride, a.q.head_stride,
                                static_cast<const T*>(a.k_cache), static_cast<const T*>(a.v_cache), cv, g, ov, parts, c2);
  if (rc != VDA_OK) return rc;
  return launch_join<T, D>(p, parts, ov, g.group, s);
}

template <typename T, int D>
int launch_attn_simt(const vda_attn_args& a, const AttnPlan& p, char* ws, float c2) {
  return p.rows == 16 ? launch_simt<T, D, 16>(a, p, ws, c2) : launch_simt<T, D, 64>(a, p, ws, c2);
}

}  // namespace attn
}  // namespace vda
