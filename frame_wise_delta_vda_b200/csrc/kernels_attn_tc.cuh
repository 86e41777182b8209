// Paged attention on the tensor cores: bf16, d = 64 or 128, B200 (sm_100a).
//
// k_attn_tc: one persistent CTA an SM.  An item's rows fill two tiles of up to
// 128 rows; per key tile of 128 keys the MMA warp computes S = Q K^T into TMEM,
// four softmax warps turn it into P = exp(S - m) in bf16, written over S, and
// the MMA warp adds P V to the tile's output in TMEM with P as the operand in
// TMEM.  The two row tiles take turns, so one's softmax runs while the other's
// products do, and both share one stream of K and V through a ring of
// shared-memory stages filled by TMA, page by page.  Items of one row tile
// (few rows, as in single-token steps) give both turns to the same rows, even
// key tiles to one and odd ones to the other, and merge the two at the end.
//
// TMEM lane = row, so a thread holds whole rows: maximum and sum need no
// shuffles.  The maximum that exponents refer to is raised only when a row
// outgrows it by 2^8 (P stays in bf16's range and the quotient is the same),
// so the output in TMEM is rarely scaled.
//
// Warps 0-3 and 4-7: softmax and output of turn 0 and 1; warp 8: K, V loads;
// warp 9: MMA; warp 10: Q loads; warp 11 completes the warpgroup whose
// registers go to the softmax warps.
#pragma once

#include "kernels_attn.cuh"
#include "kernels_tc.cuh"

namespace vda {
namespace attn {

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16: A is 128 lanes x 8 columns of
// bf16 pairs (K-major).
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// bits of the keys j .. j + 31 that a row sees
__device__ __forceinline__ uint32_t below(int k) { return k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u; }
__device__ __forceinline__ uint32_t seen_word(const Span& sp, int j) {
  return below(sp.end - j) & (~below(sp.lo - j) | below(sp.anc - j));
}
// bits of the keys 32 c .. 32 c + 31 of a tile whose page (bit of `absent`, box keys each) does not exist
__device__ __forceinline__ uint32_t absent_word(uint32_t absent, int c, int box) {
  uint32_t w = 0u;
  if (box >= 32) return (absent >> (32 * c / box)) & 1u ? 0xffffffffu : 0u;
#pragma unroll 1
  for (int k = 0; k < 32; k += box)
    if ((absent >> ((32 * c + k) / box)) & 1u) w |= ((1u << box) - 1u) << k;
  return w;
}

template <int D>
struct TcCfg {
  static constexpr int BN = 128;                       // keys of a tile
  static constexpr int ROWS = 256;                     // rows of a part: two tiles of 128
  static constexpr int NB = D / 64;                    // 64-channel blocks
  static constexpr uint32_t BLK = 128 * 128;           // 128 rows x 64 bf16
  static constexpr uint32_t TILE = NB * BLK;
  static constexpr int NST = D == 128 ? 5 : 10;        // K / V stages
  static constexpr uint32_t OFF_Q = 0;                 // two row tiles; the second is also the merge's buffer
  static constexpr uint32_t OFF_KV = 2 * TILE;
  static constexpr uint32_t OFF_ML = OFF_KV + NST * TILE;   // merge: 64 rows x (m, l)
  static constexpr uint32_t OFF_BAR = OFF_ML + 64 * 8;
  // kvfull[NST], kvempty[NST], qfull, qempty, sfull[2], pfull[2], odone[2], ofree[2], handed, merged, drain
  static constexpr int NBAR = 2 * NST + 13;
  static constexpr uint32_t OFF_PLAN = OFF_BAR + NBAR * 8 + 16;
  static constexpr size_t SMEM = OFF_PLAN + sizeof(Plan) + 1024;
  static constexpr int WARP_KV = 8, WARP_MMA = 9, WARP_Q = 10, THREADS = 384;
  // registers: 384 threads x 168 at launch = 64512 >= 256 x 208 + 128 x 80 after the split
  static constexpr int REG_SOFTMAX = 208, REG_OTHER = 80;
  // TMEM columns: S (P over its first half) of turn 0, 1; output of turn 0, 1
  static constexpr uint32_t T_S = 0, T_O = 256, T_COLS = 512;
};

// The turns of an item: a unit is one key tile of one row tile.
template <int BN>
struct Units {
  Walk<BN> w;
  int u, nu;       // unit of the item, units
  int items;       // items before this one
  int base;        // key tiles of earlier items of this share
  __device__ __forceinline__ Units(const Geom& g, const Plan& p) : w(g, p), u(0), items(0), base(0) { size(); }
  // an item with at most half its tokens has one row tile
  __device__ __forceinline__ bool single() const { return 2 * w.ntok <= w.g->tpi; }
  // 64-row halves of a single tile whose two turns are merged
  __device__ __forceinline__ int halves() const {
    return !single() || w.n() < 2 ? 0 : w.ntok * w.g->group > 64 ? 2 : 1;
  }
  __device__ __forceinline__ void size() { nu = !w.live ? 0 : single() ? w.n() : 2 * w.n(); }
  __device__ __forceinline__ int turn() const { return u & 1; }
  __device__ __forceinline__ int tile() const { return single() ? u : u >> 1; }
  __device__ __forceinline__ bool tile_ends() const { return single() || (u & 1); }
  __device__ __forceinline__ void next() {
    if (++u < nu) return;
    u = 0;
    base += w.n();
    ++items;
    w.next();
    size();
  }
};

template <int D>
__global__ void __launch_bounds__(TcCfg<D>::THREADS, 1)
k_attn_tc(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
          const __grid_constant__ CUtensorMap tmV, CacheView cv, const __grid_constant__ Geom g,
          OutView<__nv_bfloat16> ov, Parts parts, float c2) {
  using namespace ptx;
  using C = TcCfg<D>;
  constexpr int BN = C::BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = tc::align1024(smem_raw);
  const uint32_t sbase = smem_u32(smem);
  auto BAR = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * (uint32_t)i; };
  constexpr int KVFULL = 0, KVEMPTY = C::NST, QFULL = 2 * C::NST, QEMPTY = QFULL + 1, SFULL = QFULL + 2, PFULL = SFULL + 2,
                ODONE = PFULL + 2, OFREE = ODONE + 2, HANDED = OFREE + 2, MERGED = HANDED + 1, DRAIN = MERGED + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + C::NBAR * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Plan* splan = reinterpret_cast<Plan*>(smem + C::OFF_PLAN);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(BAR(KVFULL + s), 1);
      mbar_init(BAR(KVEMPTY + s), 1);
    }
    mbar_init(BAR(QFULL), 1);
    mbar_init(BAR(QEMPTY), 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(BAR(SFULL + s), 1);
      mbar_init(BAR(PFULL + s), 128);
      mbar_init(BAR(ODONE + s), 1);
      mbar_init(BAR(OFREE + s), 128);
    }
    mbar_init(BAR(HANDED), 128);
    mbar_init(BAR(MERGED), 128);
    mbar_init(BAR(DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == C::WARP_MMA) {
    tmem_alloc(smem_u32(tmem_slot), C::T_COLS);
    tmem_relinquish();
  }
  grid_wait_prerequisites();
  grid_launch_dependents();
  if (warp == 0) {
    const Plan p = plan_share<BN>(g, blockIdx.x, gridDim.x, 1, lane);
    if (lane == 0) *splan = p;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Plan plan = *splan;
  const int tpt = g.tpi >> 1;   // tokens of a row tile

  if (warp >= C::WARP_KV) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_OTHER));
  if (warp == C::WARP_KV) {
    // ---------------- K and V tiles, page by page: lane i sends page i of the tile
    const int box = cv.page < BN ? cv.page : BN, boxes = BN / box;
    uint32_t idx = 0, sent = 0;
    bool ok = true;
    for (Walk<BN> w(g, plan); ok && w.live; w.next()) {
      for (int t = w.t0; t < w.t1; ++t, idx += 2) {
        const int j = key_tile(w.tiles, t) * BN + lane * box;
        // pages that no row of the item sees, or that do not exist, load as
        // zeros: their coordinate lies outside the map
        int row = -1;
        if (lane < boxes && ((j < w.tiles.anc) || (j < w.tiles.end && j + box > w.tiles.lo))) {
          const int id = __ldg(cv.table + (int64_t)w.b * cv.table_stride + j / cv.page);
          if (id >= 0 && id < cv.pages) row = id * g.Hk + w.h;
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t s = (idx + v) % C::NST, ph = ((idx + v) / C::NST) & 1u;
          if (!__all_sync(0xffffffffu, mbar_wait(BAR(KVEMPTY + s), ph ^ 1u, abort_flag))) { ok = false; break; }
          if (lane == 0) mbar_arrive_expect_tx(BAR(KVFULL + s), C::TILE);
          __syncwarp();
          if (lane < boxes) {
            const uint32_t dst = sbase + C::OFF_KV + s * C::TILE + (uint32_t)(lane * box) * 128u;
#pragma unroll
            for (int cb = 0; cb < C::NB; ++cb)
              tma_load_3d(dst + cb * C::BLK, v ? &tmV : &tmK, 64 * cb, j % cv.page, row, BAR(KVFULL + s));
          }
          __syncwarp();
          ++sent;
        }
        if (!ok) break;
      }
    }
    if (*abort_flag && lane == 0) {   // let issued copies land
      const uint32_t n = sent < (uint32_t)C::NST ? sent : (uint32_t)C::NST;
      for (uint32_t k = sent - n; k < sent; ++k) mbar_wait_drain(BAR(KVFULL + k % C::NST), (k / C::NST) & 1u);
    }
  } else if (warp == C::WARP_Q) {
    // ---------------- Q tiles
    if (lane == 0) {
      int merges = 0, sent = 0;
      for (Units<BN> un(g, plan); un.w.live;) {
        const bool one = un.single();
        if (!mbar_wait(BAR(QEMPTY), (uint32_t)(un.items & 1) ^ 1u, abort_flag)) break;
        // the second tile's place has been the buffer of the last merge
        if (!one && merges > 0 && !mbar_wait(BAR(MERGED), (uint32_t)(merges - 1) & 1u, abort_flag)) break;
        const uint32_t bytes = (uint32_t)(tpt * g.group) * 128u * C::NB;
        mbar_arrive_expect_tx(BAR(QFULL), one ? bytes : 2 * bytes);
        for (int s = 0; s < (one ? 1 : 2); ++s)
#pragma unroll
          for (int cb = 0; cb < C::NB; ++cb)
            tma_load_3d(sbase + C::OFF_Q + s * C::TILE + cb * C::BLK, &tmQ, 64 * cb, un.w.h * g.group,
                        un.w.s.q0 + un.w.i0 + s * tpt, BAR(QFULL));
        ++sent;
        merges += un.halves();
        un.u = un.nu - 1;   // to the next item
        un.next();
      }
      if (*abort_flag && sent > 0) mbar_wait_drain(BAR(QFULL), (uint32_t)(sent - 1) & 1u);
    }
  } else if (warp == C::WARP_MMA) {
    // ---------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t kIdQK = idesc_bf16(128, BN, 0, 0);   // both K-major
      constexpr uint32_t kIdPV = idesc_bf16(128, D, 0, 1);    // V: channels contiguous
      Units<BN> qk(g, plan), pv(g, plan);
      int nqk[2] = {0, 0}, npv[2] = {0, 0}, nitem[2] = {0, 0}, ahead = 0;
      bool ok = true;
      while (ok && pv.w.live) {
        // scores run up to two units ahead, once the turn's P has been used
        while (ok && qk.w.live && ahead < 2 && nqk[qk.turn()] == npv[qk.turn()]) {
          const int tn = qk.turn();
          if (qk.u == 0 && !mbar_wait(BAR(QFULL), (uint32_t)qk.items & 1u, abort_flag)) { ok = false; break; }
          const uint32_t k = 2u * (uint32_t)(qk.base + qk.tile()), s = k % C::NST;
          if (!mbar_wait(BAR(KVFULL + s), (k / C::NST) & 1u, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t qa = sbase + C::OFF_Q + (qk.single() ? 0u : (uint32_t)tn * C::TILE);
          const uint32_t kb = sbase + C::OFF_KV + s * C::TILE;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = (uint32_t)(ks >> 2) * C::BLK + (uint32_t)(ks & 3) * 32u;
            mma_bf16_ss(tmem + C::T_S + tn * 128u, desc_sw128(qa + off, 16, 1024), desc_sw128(kb + off, 16, 1024), kIdQK,
                        ks != 0);
          }
          mma_commit(BAR(SFULL + tn));
          if (qk.tile_ends()) mma_commit(BAR(KVEMPTY + s));
          if (qk.u + 1 == qk.nu) mma_commit(BAR(QEMPTY));
          ++nqk[tn];
          ++ahead;
          qk.next();
        }
        if (!ok) break;
        const int tn = pv.turn();
        const uint32_t k = 2u * (uint32_t)(pv.base + pv.tile()) + 1u, s = k % C::NST;
        const bool first = pv.u < 2;   // of this turn in the item
        if (!mbar_wait(BAR(KVFULL + s), (k / C::NST) & 1u, abort_flag)) break;
        if (!mbar_wait(BAR(PFULL + tn), (uint32_t)npv[tn] & 1u, abort_flag)) break;
        if (first) {   // the output of the last item has been read
          if (!mbar_wait(BAR(OFREE + tn), (uint32_t)(nitem[tn] & 1) ^ 1u, abort_flag)) break;
          ++nitem[tn];
        }
        tc_fence_after();
        const uint32_t vb = sbase + C::OFF_KV + s * C::TILE;
#pragma unroll
        for (int ks = 0; ks < BN / 16; ++ks)
          mma_bf16_ts(tmem + C::T_O + (uint32_t)tn * D, tmem + C::T_S + tn * 128u + 8u * ks,
                      desc_sw128(vb + (uint32_t)ks * 2048u, C::BLK, 1024), kIdPV, !(first && ks == 0));
        mma_commit(BAR(ODONE + tn));
        if (pv.tile_ends()) mma_commit(BAR(KVEMPTY + s));
        ++npv[tn];
        --ahead;
        pv.next();
      }
      mma_commit(BAR(DRAIN));
      mbar_wait_drain(BAR(DRAIN), 0);
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REG_SOFTMAX));
    // ---------------- softmax and output: thread = row of its turn's tile
    const int tn = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + C::T_S + tn * 128u, tO = tmem + lanes + C::T_O + (uint32_t)tn * D;
    const int box = cv.page < BN ? cv.page : BN;
    const int npg = BN / box;
    const int ri = r / g.group, rg = r % g.group;   // token of the tile, head of the group
    uint32_t cnt = 0;
    int merges = 0;   // 64-row halves merged so far
    bool ok = true;
    Meta meta{0, 0, 0, 0};
    for (Units<BN> un(g, plan); ok && un.w.live;) {
      const Walk<BN>& w = un.w;
      const bool one = un.single();
      const int tok = (one ? 0 : tn * tpt) + ri;      // of the item
      const bool valid = ri < tpt && tok < w.ntok;
      const bool busy = __any_sync(0xffffffffu, valid);
      Span sp{0, 0, 0};
      if (valid) sp = span_of(g, w.s.len - w.s.n + w.i0 + tok, w.s.len);
      float m = neg_inf(), l = 0.f;
      const int n = w.n();
      int done = 0;   // units of this turn
      for (int t = one ? tn : 0; t < n; t += one ? 2 : 1, ++cnt, ++done) {
        const int j0 = key_tile(w.tiles, w.t0 + t) * BN;
        // pages of the tile that do not exist
        bool gone = false;
        if (lane < npg && j0 + lane * box < w.s.len) {
          const int id = __ldg(cv.table + (int64_t)w.b * cv.table_stride + (j0 + lane * box) / cv.page);
          gone = id < 0 || id >= cv.pages;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(BAR(SFULL + tn), cnt & 1u, abort_flag))) { ok = false; break; }
        tc_fence_after();
        const unsigned absent = __ballot_sync(0xffffffffu, gone);
        // keys of the tile that no row of the item sees: their values may be
        // anything (0 x NaN would reach the sums), so they become zeros
        const bool inside = j0 + BN <= w.tiles.anc || (j0 >= w.tiles.lo && j0 + BN <= w.tiles.end);
        if (!inside) {
          const uint32_t k = 2u * (uint32_t)(un.base + t) + 1u, s = k % C::NST;
          if (!__all_sync(0xffffffffu, mbar_wait(BAR(KVFULL + s), (k / C::NST) & 1u, abort_flag))) { ok = false; break; }
          const int j = j0 + r;
          if (!(j < w.tiles.anc || (j >= w.tiles.lo && j < w.tiles.end))) {
            const uint32_t at = sbase + C::OFF_KV + s * C::TILE + (uint32_t)r * 128u;
#pragma unroll
            for (int cb = 0; cb < C::NB; ++cb)
#pragma unroll
              for (int c = 0; c < 8; ++c) st_shared_v4(at + cb * C::BLK + 16u * c, make_uint4(0u, 0u, 0u, 0u));
          }
          fence_proxy_async_smem();
        }
        if (busy) {
          uint32_t v[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32u * c, v[c]);
          tmem_wait_ld();
          const bool all = !valid || j0 + BN <= sp.anc || (j0 >= sp.lo && j0 + BN <= sp.end);
          if (absent || !__all_sync(0xffffffffu, all)) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t see = seen_word(sp, j0 + 32 * c) & ~absent_word(absent, c, box);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((see >> i) & 1u)) v[c][i] = 0xff800000u;
            }
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            mx[c] = __uint_as_float(v[c][0]);
#pragma unroll
            for (int i = 1; i < 32; ++i) mx[c] = fmaxf(mx[c], __uint_as_float(v[c][i]));
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // a row's first keys set its maximum; later it moves when outgrown
          const bool grow = m != neg_inf() && (top - m) * c2 > 8.f;
          if (__any_sync(0xffffffffu, grow)) {
            const float alpha = grow ? ex2((m - top) * c2) : 1.f;
            l *= alpha;
            if (!__all_sync(0xffffffffu, mbar_wait(BAR(ODONE + tn), (cnt - 1u) & 1u, abort_flag))) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + 32u * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + 32u * c, o);
            }
          }
          if (grow || m == neg_inf()) m = top;
          const float base = m == neg_inf() ? 0.f : m * c2;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t p[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int e = 64 * h + 2 * i;
              const float a = ex2(fmaf(__uint_as_float(v[e >> 5][e & 31]), c2, -base));
              const float b = ex2(fmaf(__uint_as_float(v[(e + 1) >> 5][(e + 1) & 31]), c2, -base));
              sum[2 * (i & 1)] += a;
              sum[2 * (i & 1) + 1] += b;
              p[i] = pack_bf16(a, b);
            }
            tmem_st32(tS + 32u * h, p);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(BAR(PFULL + tn));
      }
      if (!ok) break;
      if (done > 0) {   // the turn's last product
        if (!__all_sync(0xffffffffu, mbar_wait(BAR(ODONE + tn), (cnt - 1u) & 1u, abort_flag))) break;
        tc_fence_after();
      }
      const bool whole = w.whole();
      const int slot = w.t0 > 0 ? 0 : 1;
      const int tok0 = w.s.q0 + w.i0;
      if (!whole && slot == 1) {   // begun here, continued in later shares
        const long long start = plan.w1 - n;
        meta.parts = share_of(plan.W, start + w.tiles.count - 1, plan.shares) - (int)blockIdx.x + 1;
        meta.tok0 = tok0;
        meta.h = w.h;
        meta.rows = w.ntok * g.group;
      }
      // rows of a single tile: turn 1 hands its sums to turn 0 in shared
      // memory, 64 rows at a time
      const int halves = un.halves();
      const uint32_t xr = (uint32_t)(r & 63) * 16u, xb = sbase + C::OFF_Q + C::TILE, xml = sbase + C::OFF_ML + 8u * (uint32_t)(r & 63);
      if (one && tn == 1) {
        for (int half = 0; half < halves; ++half, ++merges) {
          if (merges > 0 && !__all_sync(0xffffffffu, mbar_wait(BAR(MERGED), (uint32_t)(merges - 1) & 1u, abort_flag))) { ok = false; break; }
          if ((r >> 6) == half && busy) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + 32u * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                st_shared_v4(xb + (uint32_t)(8 * c + i) * 1024u + xr, make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
            }
            st_shared_f1(xml, m);
            st_shared_f1(xml + 4u, l);
          }
          fence_proxy_async_smem();
          mbar_arrive(BAR(HANDED));
        }
      } else {
        const int tokg = tok0 + tok, hd = w.h * g.group + rg;
        const size_t prow = ((size_t)blockIdx.x * 2 + slot) * parts.rows + (one ? 0 : tn * tpt * g.group) + r;
        const int passes = halves > 0 ? halves : 1;
        for (int half = 0; half < passes; ++half) {
          float ms = m, lt = l, f0 = 1.f, f1 = 0.f;   // maximum and sum of both turns; scales of this turn's and the other's output
          if (halves > 0) {
            if (!__all_sync(0xffffffffu, mbar_wait(BAR(HANDED), (uint32_t)merges & 1u, abort_flag))) { ok = false; break; }
            ++merges;
            const float m1 = ld_shared_f1(xml), l1 = ld_shared_f1(xml + 4u);
            ms = fmaxf(m, m1);
            const float b = ms == neg_inf() ? 0.f : ms;
            f0 = ex2((m - b) * c2);
            f1 = ex2((m1 - b) * c2);
            lt = l * f0 + l1 * f1;
          }
          if ((halves == 0 || (r >> 6) == half) && busy) {
            const float inv = whole ? 1.f / lt : 1.f;
            const bool none = lt == 0.f;   // a row that sees nothing
            f0 *= inv;
            f1 *= inv;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + 32u * c, o);
              tmem_wait_ld();
              float x[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(o[i]) * f0;
              if (halves > 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float4 y = ld_shared_f4(xb + (uint32_t)(8 * c + i) * 1024u + xr);
                  x[4 * i] = fmaf(y.x, f1, x[4 * i]);
                  x[4 * i + 1] = fmaf(y.y, f1, x[4 * i + 1]);
                  x[4 * i + 2] = fmaf(y.z, f1, x[4 * i + 2]);
                  x[4 * i + 3] = fmaf(y.w, f1, x[4 * i + 3]);
                }
              }
              if (none) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = 0.f;
              }
              if (valid) {
                if (whole) {
                  uint4* dst = reinterpret_cast<uint4*>(ov.out + (int64_t)tokg * ov.ts + (int64_t)hd * ov.hs + 32 * c);
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    dst[i] = make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                                        pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
                } else {
                  float4* dst = reinterpret_cast<float4*>(parts.o + prow * D + 32 * c);
#pragma unroll
                  for (int i = 0; i < 8; ++i) dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                }
              }
            }
            if (valid) {
              const float m2 = ms == neg_inf() ? neg_inf() : ms * c2;
              if (!whole) parts.ml[prow] = make_float2(m2, lt);
              else if (ov.lse) ov.lse[(int64_t)tokg * ov.Hq + hd] = none ? neg_inf() : (m2 + log2f(lt)) * kLn2;
            }
          }
          if (halves > 0) {   // the buffer is free for the next rows, or the next Q tile
            fence_proxy_async_smem();
            mbar_arrive(BAR(MERGED));
          }
        }
      }
      if (!ok) break;
      tc_fence_before();
      if (done > 0) mbar_arrive(BAR(OFREE + tn));
      un.u = un.nu - 1;   // to the next item
      un.next();
    }
    if (tid == 0) parts.meta[blockIdx.x] = meta;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::T_COLS);
  }
}

// ------------------------------------------------------------------- host
// [tokens][heads][d] by strides, a box of 64 channels x heads x tokens
inline bool encode_q(CUtensorMap* m, const vda_rows& q, uint64_t N, uint64_t Hq, uint32_t d, uint32_t heads, uint32_t tokens) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {d, Hq, N};
  // a stride that nothing steps over may be anything
  const cuuint64_t hs = Hq > 1 ? (cuuint64_t)q.head_stride * 2 : 2ull * d;
  cuuint64_t strides[2] = {hs, N > 1 ? (cuuint64_t)q.token_stride * 2 : hs * Hq};
  cuuint32_t box[3] = {64, heads, tokens};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q.data, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
int launch_attn_tc(const vda_attn_args& a, const AttnPlan& p, char* ws, float c2) {
  using C = TcCfg<D>;
  const Geom g = geom_of(a, p);
  CUtensorMap tmQ, tmK, tmV;
  const uint32_t box = (uint32_t)(a.page_size < C::BN ? a.page_size : C::BN);
  const uint64_t heads = (uint64_t)a.pages * a.Hk;
  if (!encode_q(&tmQ, a.q, (uint64_t)a.N, (uint64_t)a.Hq, D, (uint32_t)g.group, (uint32_t)(g.tpi / 2)) ||
      !tc::encode_bf16_3d(&tmK, a.k_cache, (uint64_t)a.page_size, heads, box, D) ||
      !tc::encode_bf16_3d(&tmV, a.v_cache, (uint64_t)a.page_size, heads, box, D))
    return VDA_ERR_CUDA;
  auto kernel = k_attn_tc<D>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM) != cudaSuccess)
    return VDA_ERR_CUDA;
  const OutView<__nv_bfloat16> ov = out_of<__nv_bfloat16>(a);
  const Parts parts = parts_of(ws, p);
  const CacheView cv{a.block_table, a.table_stride, a.pages, a.page_size};
  cudaStream_t s = static_cast<cudaStream_t>(a.stream);
  const int rc = tc::launch_pdl("k_attn_tc", kernel, dim3((unsigned)p.ctas), dim3(C::THREADS), C::SMEM, s, tmQ, tmK, tmV, cv, g,
                                ov, parts, c2);
  if (rc != VDA_OK) return rc;
  return launch_join<__nv_bfloat16, D>(p, parts, ov, g.group, s);
}

}  // namespace attn
}  // namespace vda
