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
// P is rounded to bf16 (its sum l is not): both operands of a product have one
// type, and V is bf16.  A weight is off by at most 2^-8 of itself, so the result
// by at most that of sum_j p_j |v_j|; measured against 64 bits, 2.1e-3 to 2.3e-3
// of the result's norm, where rounding the result alone gives 1.7e-3.  P as two
// bf16 terms would take the difference away, for twice the products of P V.
//
// Measured, 32 / 8 heads of 128: 4096 tokens over 16400 keys 1004 to 1017 us (58%
// of the measured bf16 rate), bound by the chain of a turn (scores, maximum,
// exponentials, product: 2285 cycles a tile, 1024 of either pipe); 64 steps over
// 246 to 8200 keys 154 to 157 us (70% of a plain copy's rate) and 2 over 131000
// keys 189 to 193 us (85%), bound by memory and by the items' begin and end.
// 4096 tokens over 16400 keys with 32 / 8 heads of 64: 826 us (583 TFLOP/s), the
// same chain for half the products.
//
// Registers: three values that are set once at the start live in local memory
// (12 bytes stored) and are read again at some 150 places (624 bytes of reloads
// in the code), more than half of them in the loops of waits that go on: with
// those compiled out 296 bytes are left.
//
// Warps 0-3 and 4-7: softmax and output of turn 0 and 1; warp 8: K, V loads;
// warps 9 and 10: MMA of turn 0 and 1; warp 11: the list of items and Q loads.
#pragma once

#include "kernels_attn.cuh"
#include "kernels_tc.cuh"

namespace vda {
namespace attn {

// Matrix descriptors as 32-bit halves, so that the addresses of a product's
// steps are one 32-bit add each: the high half holds SBO = 1024, version 1 and
// the 128-B swizzle (see ptx::desc_sw128), the low half address and LBO.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
// D[tmem] (+)= A[smem] * B[smem], kind::f16
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}"
      ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem], kind::f16: A is 128 lanes x 8 columns of
// bf16 pairs (K-major).
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(kDescHi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// True for one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
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

// ptx::mbar_wait by a whole converged warp, with one answer for all lanes; a
// phase that is over already costs one poll and one vote.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort));
}
// A count in shared memory that several warps add to (release) and one waits
// for (acquire), with the bounds of ptx::mbar_wait: for a waiter that does not
// see every phase, where a barrier's parity would be ambiguous.
__device__ __forceinline__ void count_add(uint32_t* c) {
  asm volatile("red.release.cta.shared::cta.add.u32 [%0], 1;" ::"r"(ptx::smem_u32(c)) : "memory");
}
__device__ __forceinline__ bool count_wait(const uint32_t* c, uint32_t n, volatile int* abort) {
  const long long t0 = clock64();
  while (true) {
    uint32_t v;
    asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(v) : "r"(ptx::smem_u32(c)) : "memory");
    if (v >= n) return true;
    if (*abort) return false;
    if (clock64() - t0 > ptx::kWaitCycles) {
      raise_device_error(kErrWaitTimeout);
      *abort = 1;
      return false;
    }
  }
}

template <int D>
struct TcCfg {
  static constexpr int BN = 128;                       // keys of a tile
  static constexpr int ROWS = 256;                     // rows of a part: two tiles of 128
  static constexpr int NB = D / 64;                    // 64-channel blocks
  static constexpr uint32_t BLK = 128 * 128;           // 128 rows x 64 bf16
  static constexpr uint32_t TILE = NB * BLK;
  static constexpr int NST = D == 128 ? 5 : 10;        // K / V stages
  static constexpr int NIT = 4;                        // items ahead
  static constexpr int NGONE = 16;                     // key tiles whose absent pages are kept (> NST / 2 + 1)
  static constexpr uint32_t OFF_Q = 0;                 // two row tiles; the second is also the merge's buffer
  static constexpr uint32_t OFF_KV = 2 * TILE;
  static constexpr uint32_t OFF_ML = OFF_KV + NST * TILE;   // merge: 64 rows x (m, l)
  static constexpr uint32_t OFF_ITEM = OFF_ML + 64 * 8;
  static constexpr uint32_t OFF_GONE = OFF_ITEM + NIT * 64;
  static constexpr uint32_t OFF_BAR = OFF_GONE + NGONE * 4;
  // kvfull[NST], kvempty[NST], itfull[NIT], itempty[NIT], qfull, qempty, sfull[2], pfull[2][2], odone[2], ofree[2],
  // handed, merged, drain[2], exped[2][4]
  static constexpr int NBAR = 2 * NST + 2 * NIT + 24;
  static constexpr size_t SMEM = OFF_BAR + NBAR * 8 + 16 + 1024;   // + TMEM address, abort flag, merge count
  static constexpr int WARP_KV = 8, WARP_MMA = 9, WARP_ITEM = 11, THREADS = 384;
  // registers: 384 threads x 168 at launch = 64512 >= 256 x 200 + 128 x 96 after the split
  static constexpr int REG_SOFTMAX = 200, REG_OTHER = 96;
  // TMEM columns: S (P over its first half) of turn 0, 1; output of turn 0, 1
  static constexpr uint32_t T_S = 0, T_O = 256, T_COLS = 512;
};

// One item of this CTA's share, published in shared memory by the item warp.
struct Item {
  int b, h;              // sequence, KV head
  int tok0, ntok;        // first token of the batch, tokens
  int pos0, len;         // position of the first token, keys of the sequence
  int lo, end, anc;      // keys that any of its rows sees: [lo, end) and [0, anc)
  int n_anchor, first;   // see Tiles
  int t0, n;             // this share's key tiles of the item; n = 0 ends the list
  int flags;
  int pad[2];
};
static_assert(sizeof(Item) == 64, "ring stride");
constexpr int kSingle = 1;     // one row tile: the turns alternate over the key tiles
constexpr int kWhole = 2;      // no other share has a part of it
constexpr int kLast = 4;       // continued in later shares: part slot 1
constexpr int kHalfShift = 4;  // 64-row halves that the turns' merge takes (0-2)

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
  constexpr int KVFULL = 0, KVEMPTY = C::NST, ITFULL = 2 * C::NST, ITEMPTY = ITFULL + C::NIT, QFULL = ITEMPTY + C::NIT,
                QEMPTY = QFULL + 1, SFULL = QFULL + 2, PFULL = SFULL + 2, ODONE = PFULL + 4, OFREE = ODONE + 2,
                HANDED = OFREE + 2, MERGED = HANDED + 1, DRAIN = MERGED + 1,
                EXPED = DRAIN + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + C::NBAR * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile Item* items = reinterpret_cast<volatile Item*>(smem + C::OFF_ITEM);
  uint32_t* merged = tmem_slot + 2;   // 64-row halves of merges that are read, times four warps
  volatile uint32_t* gone = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_GONE);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(BAR(KVFULL + s), 1);
      mbar_init(BAR(KVEMPTY + s), 2);    // both MMA warps
    }
    for (int s = 0; s < C::NIT; ++s) {
      mbar_init(BAR(ITFULL + s), 1);
      mbar_init(BAR(ITEMPTY + s), 11);   // eight softmax warps, K/V, two MMA
    }
    mbar_init(BAR(QFULL), 1);
    mbar_init(BAR(QEMPTY), 2);
    for (int s = 0; s < 2; ++s) {
      mbar_init(BAR(SFULL + s), 1);
      for (int p = 0; p < 2; ++p) mbar_init(BAR(PFULL + 2 * s + p), 4);
      mbar_init(BAR(ODONE + s), 1);
      mbar_init(BAR(OFREE + s), 4);
    }
    mbar_init(BAR(HANDED), 4);
    mbar_init(BAR(MERGED), 4);
    mbar_init(BAR(DRAIN), 1);
    mbar_init(BAR(DRAIN + 1), 1);
    for (int s = 0; s < 8; ++s) mbar_init(BAR(EXPED + s), 1);
    *abort_flag = 0;
    *merged = 0u;
    fence_mbar_init();
  }
  if (tid == 32) {
    for (const CUtensorMap* m : {&tmQ, &tmK, &tmV})
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  if (warp == C::WARP_MMA) {
    tmem_alloc(smem_u32(tmem_slot), C::T_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_wait_prerequisites();
  grid_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const int tpt = g.tpi >> 1;   // tokens of a row tile
  // A barrier's parity tells a phase only from the one before and the one after
  // it, so every waiter here either sees each phase in its turn (and the
  // phase after it cannot end before the waiter's own arrival), or waits for a
  // phase whose predecessor a barrier that it has passed implies.
  // wait for item i of the share; the same for a whole warp
  auto item_ready = [&](int i) -> bool {
    return mbar_wait(BAR(ITFULL + i % C::NIT), (uint32_t)(i / C::NIT) & 1u, abort_flag);
  };

  if (warp >= C::WARP_KV) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_OTHER));
    if (warp == C::WARP_ITEM) {
      // ---------------- the share's items, published one ahead of their Q tiles
      const Plan plan = plan_share<BN>(g, blockIdx.x, gridDim.x, lane);
      if (lane == 0) {
        Meta meta{0, 0, 0, 0};
        Walk<BN> w(g, plan);
        int merges = 0, sent = 0, listed = 0;
        bool more = true;   // items to list
        while (true) {
          // one item is listed ahead of the Q tile that is sent, for K and V to
          // follow without a gap; the first Q tile goes at once
          if (more && (listed == 0 || (sent > 0 && listed <= sent + 1))) {
            const int s = listed % C::NIT;
            if (!mbar_wait(BAR(ITEMPTY + s), ((uint32_t)(listed / C::NIT) & 1u) ^ 1u, abort_flag)) break;
            volatile Item& it = items[s];
            it.n = w.live ? w.n() : 0;
            if (w.live) {
              const bool single = 2 * w.ntok <= g.tpi, last = !w.whole() && w.t0 == 0;
              const int rows = w.ntok * g.group;
              it.b = w.b;
              it.h = w.h;
              it.tok0 = w.s.q0 + w.i0;
              it.ntok = w.ntok;
              it.pos0 = w.s.len - w.s.n + w.i0;
              it.len = w.s.len;
              it.lo = w.tiles.lo;
              it.end = w.tiles.end;
              it.anc = w.tiles.anc;
              it.n_anchor = w.tiles.n_anchor;
              it.first = w.tiles.first;
              it.t0 = w.t0;
              it.flags = (single ? kSingle : 0) | (w.whole() ? kWhole : 0) | (last ? kLast : 0) |
                         ((single && w.n() > 1 ? (rows > 64 ? 2 : 1) : 0) << kHalfShift);
              if (last) {
                meta.parts = w.parts(plan, blockIdx.x);
                meta.tok0 = w.s.q0 + w.i0;
                meta.h = w.h;
                meta.rows = rows;
              }
            }
            mbar_arrive(BAR(ITFULL + s));
            ++listed;
            more = w.live;
            if (more) w.next();
            continue;
          }
          const volatile Item& it = items[sent % C::NIT];   // its place is not used again before item sent + NIT
          if (it.n == 0) break;
          const int flags = it.flags, h = it.h, tok0 = it.tok0;
          const bool one = flags & kSingle;
          if (!mbar_wait(BAR(QEMPTY), (uint32_t)(sent & 1) ^ 1u, abort_flag)) break;
          // the second tile's place has been the buffer of the last merge
          if (!one && !count_wait(merged, 4u * (uint32_t)merges, abort_flag)) break;
          const uint32_t bytes = (uint32_t)(tpt * g.group) * 128u * C::NB;
          mbar_arrive_expect_tx(BAR(QFULL), one ? bytes : 2 * bytes);
#pragma unroll 1
          for (int s = 0; s < (one ? 1 : 2); ++s)
#pragma unroll
            for (int cb = 0; cb < C::NB; ++cb)
              tma_load_3d(sbase + C::OFF_Q + s * C::TILE + cb * C::BLK, &tmQ, 64 * cb, h * g.group, tok0 + s * tpt, BAR(QFULL));
          ++sent;
          merges += flags >> kHalfShift;
        }
        if (*abort_flag && sent > 0) mbar_wait_drain(BAR(QFULL), (uint32_t)(sent - 1) & 1u);
        parts.meta[blockIdx.x] = meta;
      }
      __syncwarp();
    } else if (warp == C::WARP_KV) {
      // ---------------- K and V tiles, page by page: lane i sends page i of the tile
      const int page_log2 = 31 - __clz(cv.page), page_mask = cv.page - 1;   // a power of two
      const int box = cv.page < BN ? cv.page : BN, boxes = BN / box;
      uint32_t idx = 0, sent = 0;
      bool ok = true;
      for (int i = 0; ok; ++i) {
        if (!__all_sync(0xffffffffu, item_ready(i))) break;
        const volatile Item& it = items[i % C::NIT];
        const int n = it.n;
        if (n == 0) break;
        const int lo = it.lo, end = it.end, anc = it.anc, n_anchor = it.n_anchor, first = it.first, t0 = it.t0, h = it.h;
        const int* row_of = cv.table + (int64_t)it.b * cv.table_stride;
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(ITEMPTY + i % C::NIT));
        // pages that no row of the item sees, or that do not exist, load as
        // zeros: their coordinate lies outside the map.  -1: such a page,
        // -2: one that is seen but does not exist.
        auto page_row = [&](int t) -> int {
          if (lane >= boxes) return -1;
          const int kt = t < n_anchor ? t : first + (t - n_anchor), j = kt * BN + lane * box;
          if (!run_any_seen(lo, end, anc, j, box)) return -1;
          const int id = __ldg(row_of + (j >> page_log2));
          return id >= 0 && id < cv.pages ? id * g.Hk + h : -2;
        };
        int row = page_row(t0);
        for (int t = 0; t < n; ++t, idx += 2) {
          const int here = row;
          if (t + 1 < n) row = page_row(t0 + t + 1);
          const int kt = t0 + t < n_anchor ? t0 + t : first + (t0 + t - n_anchor);
          const int off = (int)(((uint32_t)kt * BN + (uint32_t)(lane * box)) & (uint32_t)page_mask);
          const uint32_t absent = __ballot_sync(0xffffffffu, here == -2);
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint32_t s = (idx + v) % C::NST, ph = ((idx + v) / C::NST) & 1u;
            if (!warp_wait(BAR(KVEMPTY + s), ph ^ 1u, abort_flag)) { ok = false; break; }
            if (lane == 0) {
              if (v == 0) gone[(idx >> 1) % C::NGONE] = absent;
              mbar_arrive_expect_tx(BAR(KVFULL + s), C::TILE);
            }
            __syncwarp();
            if (lane < boxes) {
              const uint32_t dst = sbase + C::OFF_KV + s * C::TILE + (uint32_t)(lane * box) * 128u;
#pragma unroll
              for (int cb = 0; cb < C::NB; ++cb)
                tma_load_3d(dst + cb * C::BLK, v ? &tmV : &tmK, 64 * cb, off, here < 0 ? -1 : here, BAR(KVFULL + s));
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
      __syncwarp();
    } else {
      // ---------------- MMA issuers, one warp a turn: P V of a unit (a key tile
      // of the turn's rows) as its P comes, then the next unit's scores over S
      // and P.  An issuing warp spends as long again on waits and commits as
      // its products take; two of them fill each other's gaps (one warp for
      // both turns kept the tensor cores busy 45% of the time).  The whole warp
      // walks the units, so that addresses stay in uniform registers, and one
      // lane issues.
      constexpr uint32_t kIdQK = idesc_bf16(128, BN, 0, 0);   // both K-major
      constexpr uint32_t kIdPV = idesc_bf16(128, D, 0, 1);    // V: channels contiguous
      const int tn = __shfl_sync(0xffffffffu, warp, 0) - C::WARP_MMA;
      const uint32_t k_lo = desc_lo(sbase + C::OFF_KV, 16), v_lo = desc_lo(sbase + C::OFF_KV, C::BLK);
      const uint32_t tS = tmem + C::T_S + (uint32_t)tn * 128u, tO = tmem + C::T_O + (uint32_t)(tn * D);
      const bool leader = elect_one();
      auto wait = [&](int bar, uint32_t parity) -> bool {
        return warp_wait(BAR(bar), parity & 1u, abort_flag);
      };
      uint32_t stage = 0, phase = 0;      // of the next K or V
      uint32_t units = 0, begun = 0;      // of this turn: units with V's product issued; items begun
      bool ok = true;
      auto advance = [&]() {
        if (++stage == C::NST) {
          stage = 0;
          phase ^= 1u;
        }
      };
      // the unit whose scores are issued and whose product with V is not
      bool due = false, due_first = false, due_last = false;   // ... of this turn in its item
      uint32_t due_stage = 0, due_phase = 0;
      // its product with V, in two parts as P comes: keys 0-63, 64-127
      auto pv = [&](int part) -> bool {
        if (part == 0) {
          if (!wait(KVFULL + due_stage, due_phase)) return false;
          if (due_first && !wait(OFREE + tn, begun++ ^ 1u)) return false;   // the output of the last item has been read
        }
        if (!wait(PFULL + 2 * tn + part, units)) return false;
        tc_fence_after();
        if (leader) {
          const uint32_t vb = v_lo + due_stage * (C::TILE >> 4);
#pragma unroll
          for (int ks = 4 * part; ks < 4 * part + 4; ++ks)
              mma_ts(tO, tS + 8u * ks, vb + (uint32_t)ks * (2048u >> 4), kIdPV, !(due_first && ks == 0));
        }
        __syncwarp();
        return true;
      };
      auto pv_done = [&]() {
        if (leader) {
          mma_commit(BAR(KVEMPTY + due_stage));
          if (due_last) mma_commit(BAR(ODONE + tn));
        }
        __syncwarp();
        ++units;
        due = false;
      };
      for (int i = 0; ok; ++i) {
        if (due) {
          if (!(pv(0) && pv(1))) break;
          pv_done();
        }
        if (!__all_sync(0xffffffffu, item_ready(i))) break;
        const volatile Item& it = items[i % C::NIT];
        const int n = __shfl_sync(0xffffffffu, it.n, 0), flags = __shfl_sync(0xffffffffu, it.flags, 0);
        if (n == 0) break;
        const bool one = flags & kSingle;
        if (leader) mbar_arrive(BAR(ITEMPTY + i % C::NIT));
        if (!wait(QFULL, (uint32_t)i)) break;
        const uint32_t q_lo = desc_lo(sbase + C::OFF_Q, 16) + (one ? 0u : (uint32_t)tn * (C::TILE >> 4));
        const int end = one ? n - ((n - 1 - tn) & 1) : n;   // one past this turn's last tile
        if (end <= 0 && leader) mbar_arrive(BAR(QEMPTY));   // no unit for this turn
        bool first = true;
        for (int t = 0; t < n; ++t) {
          if (due && !pv(0)) { ok = false; break; }
          if (one) {
            if (due) {
              if (!pv(1)) { ok = false; break; }
              pv_done();
            }
            if ((t & 1) != tn) {   // the other turn's tile: seen and passed over
              for (int v = 0; v < 2 && ok; ++v) {
                ok = wait(KVFULL + stage, phase);
                if (leader) mbar_arrive(BAR(KVEMPTY + stage));
                advance();
              }
              if (!ok) break;
              continue;
            }
          }
          // what the scores need is waited for before the last of P, so that
          // they follow the product without a gap; the commits come after both
          if (due) {
            if (!pv(1)) { ok = false; break; }
            pv_done();
          }
          if (!wait(KVFULL + stage, phase)) { ok = false; break; }
          tc_fence_after();
          if (leader) {
            const uint32_t kb = k_lo + stage * (C::TILE >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = ((uint32_t)(ks >> 2) * C::BLK + (uint32_t)(ks & 3) * 32u) >> 4;
              mma_ss(tS, q_lo + off, kb + off, kIdQK, ks != 0);
            }
            mma_commit(BAR(SFULL + tn));
            mma_commit(BAR(KVEMPTY + stage));
            if (t + 1 == end) mma_commit(BAR(QEMPTY));
          }
          __syncwarp();
          advance();
          due = true;
          due_first = first;
          due_last = t + 1 == end;
          due_stage = stage;
          due_phase = phase;
          advance();
          first = false;
        }
      }
      if (leader) {
        mma_commit(BAR(DRAIN + tn));
        mbar_wait_drain(BAR(DRAIN + tn), 0);
      }
      __syncwarp();
    }
  } else {
    // ---------------- softmax and output: thread = row of its turn's tile
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REG_SOFTMAX));
    const int tn = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + C::T_S + tn * 128u, tO = tmem + lanes + C::T_O + (uint32_t)tn * D;
    const int box = cv.page < BN ? cv.page : BN;
    const int ri = r / g.group;   // token of the tile
    uint32_t cnt = 0, outs = 0;   // units of this turn so far, items with units
    uint32_t base = 0;            // key tiles before the item
    int merges = 0;               // 64-row halves merged so far
    auto arrive = [&](int bar) {   // the warp's one arrival, after its lanes' TMEM and shared-memory accesses
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(bar));
    };
    auto wait = [&](int bar, uint32_t phase) -> bool {
      return warp_wait(BAR(bar), phase & 1u, abort_flag);
    };
    // The turns' exponentials alternate: left alone, the two warps of an SM
    // quarter end up in step, share the XU pipe and then leave it idle together
    // (4500 cycles for 128 keys of both turns).  Round k of turn 0 follows
    // round k - 1 of turn 1, round k of turn 1 follows round k of turn 0.
    uint32_t rounds = 0;
    auto exp_begin = [&](bool one) -> bool {
      if (one || (tn == 0 && rounds == 0)) return true;
      return wait(EXPED + (tn ^ 1) * 4 + (warp & 3), tn ? rounds : rounds - 1u);
    };
    auto exp_end = [&](bool one) {
      if (one) return;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(EXPED + tn * 4 + (warp & 3)));
      ++rounds;
    };
    bool ok = true;
    for (int i = 0; ok; ++i) {
      if (!__all_sync(0xffffffffu, item_ready(i))) break;
      const volatile Item& it = items[i % C::NIT];
      const int n = it.n;
      if (n == 0) break;
      const int flags = it.flags;
      const bool one = flags & kSingle;
      const int tok = (one ? 0 : tn * tpt) + ri;      // of the item
      const bool valid = ri < tpt && tok < it.ntok;
      const bool busy = __any_sync(0xffffffffu, valid);
      Span sp{0, 0, 0};
      if (valid) sp = span_of(g, it.pos0 + tok, it.len);
      float m = neg_inf(), l = 0.f;
      int done = 0;   // units of this turn
      for (int t = one ? tn : 0; ok && t < n; t += one ? 2 : 1, ++cnt, ++done) {
        const int kt = it.t0 + t, na = it.n_anchor;
        const int j0 = (kt < na ? kt : it.first + (kt - na)) * BN;
        if (!wait(SFULL + tn, cnt)) { ok = false; break; }
        tc_fence_after();
        // keys of the tile that no row of the item sees: their values may be
        // anything (0 x NaN would reach the sums), so they become zeros
        if (!run_all_seen(it.lo, it.end, it.anc, j0, BN)) {
          const uint32_t k = 2u * (base + (uint32_t)t) + 1u, s = k % C::NST;
          if (!wait(KVFULL + s, k / C::NST)) { ok = false; break; }
          const int j = j0 + r;
          if (!(j < it.anc || (j >= it.lo && j < it.end))) {
            const uint32_t at = sbase + C::OFF_KV + s * C::TILE + (uint32_t)r * 128u;
#pragma unroll
            for (int cb = 0; cb < C::NB; ++cb)
#pragma unroll
              for (int c = 0; c < 8; ++c) st_shared_v4(at + cb * C::BLK + 16u * c, make_uint4(0u, 0u, 0u, 0u));
          }
          fence_proxy_async_smem();
        }
        if (!busy) {
          if (!exp_begin(one)) { ok = false; break; }
          exp_end(one);
#pragma unroll
          for (int p = 0; p < 2; ++p) arrive(PFULL + 2 * tn + p);
          continue;
        }
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32u * c, v[c]);
        const uint32_t absent = gone[(base + (uint32_t)t) % C::NGONE];   // pages of the tile that do not exist
        const bool all = !valid || run_all_seen(sp.lo, sp.end, sp.anc, j0, BN);
        const bool masked = !__all_sync(0xffffffffu, all && absent == 0u);
        tmem_wait_ld();
        if (masked) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t see = seen_word(sp, j0 + 32 * c) & ~absent_word(absent, c, box);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((see >> e) & 1u)) v[c][e] = 0xff800000u;
          }
        }
        float mx[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t* x = v[c >> 1] + 16 * (c & 1);
          mx[c] = __uint_as_float(x[0]);
#pragma unroll
          for (int e = 1; e < 15; e += 2) mx[c] = fmaxf(fmaxf(mx[c], __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
          mx[c] = fmaxf(mx[c], __uint_as_float(x[15]));
        }
        const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
        // a row's first keys set its maximum; later it moves when outgrown (the
        // products so far are complete: the scores came after them)
        const bool grow = m != neg_inf() && (top - m) * c2 > 8.f;
        if (__any_sync(0xffffffffu, grow)) {
          const float alpha = grow ? ex2((m - top) * c2) : 1.f;
          l *= alpha;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(tO + 16u * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(tO + 16u * c, o);
          }
        }
        if (grow || m == neg_inf()) m = top;
        const float nb = m == neg_inf() ? 0.f : -m * c2;
        if (!exp_begin(one)) { ok = false; break; }
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            // scalar, not paired, arithmetic: with one warp of an SM quarter at
            // work 64 keys take 592 cycles instead of 765 (512 of the XU pipe)
            const float a = ex2(fmaf(__uint_as_float(v[c][2 * e]), c2, nb));
            const float b = ex2(fmaf(__uint_as_float(v[c][2 * e + 1]), c2, nb));
            sum[2 * (e & 1)] += a;
            sum[2 * (e & 1) + 1] += b;
            p[e] = pack_bf16(a, b);
          }
          tmem_st16(tS + 16u * c, p);
          if (c == 3) exp_end(one);
          if (c & 1) {   // a half of P is there for its product with V
            tmem_wait_st();
            arrive(PFULL + 2 * tn + (c >> 1));
          }
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      if (!ok) break;
      base += (uint32_t)n;
      if (done > 0) {   // the turn's last product
        if (!wait(ODONE + tn, outs++)) break;
        tc_fence_after();
      }
      // rows of a single tile: turn 1 hands its sums to turn 0 in shared
      // memory, 64 rows at a time
      const int halves = flags >> kHalfShift;
      const uint32_t xr = (uint32_t)(r & 63) * 16u, xb = sbase + C::OFF_Q + C::TILE, xml = sbase + C::OFF_ML + 8u * (uint32_t)(r & 63);
      if (one && tn == 1) {
        for (int half = 0; half < halves; ++half, ++merges) {
          if (merges > 0 && !wait(MERGED, (uint32_t)(merges - 1))) { ok = false; break; }
          if ((r >> 6) == half && busy) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + 32u * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e)
                st_shared_v4(xb + (uint32_t)(8 * c + e) * 1024u + xr, make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
            }
            st_shared_f1(xml, m);
            st_shared_f1(xml + 4u, l);
          }
          fence_proxy_async_smem();
          arrive(HANDED);
        }
      } else {
        const bool whole = flags & kWhole;
        const int tokg = it.tok0 + tok, hd = it.h * g.group + r % g.group;
        const size_t prow = ((size_t)blockIdx.x * 2 + (flags & kLast ? 1 : 0)) * parts.rows + (one ? 0 : tn * tpt * g.group) + r;
        const int passes = halves > 0 ? halves : 1;
        for (int half = 0; half < passes; ++half) {
          float ms = m, lt = l, f0 = 1.f, f1 = 0.f;   // maximum and sum of both turns; scales of this turn's and the other's output
          if (halves > 0) {
            if (!wait(HANDED, (uint32_t)merges)) { ok = false; break; }
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
              for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(o[e]) * f0;
              if (halves > 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 y = ld_shared_f4(xb + (uint32_t)(8 * c + e) * 1024u + xr);
                  x[4 * e] = fmaf(y.x, f1, x[4 * e]);
                  x[4 * e + 1] = fmaf(y.y, f1, x[4 * e + 1]);
                  x[4 * e + 2] = fmaf(y.z, f1, x[4 * e + 2]);
                  x[4 * e + 3] = fmaf(y.w, f1, x[4 * e + 3]);
                }
              }
              if (none) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = 0.f;
              }
              if (valid) {
                if (whole) {
                  uint4* dst = reinterpret_cast<uint4*>(ov.out + (int64_t)tokg * ov.ts + (int64_t)hd * ov.hs + 32 * c);
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    dst[e] = make_uint4(pack_bf16(x[8 * e], x[8 * e + 1]), pack_bf16(x[8 * e + 2], x[8 * e + 3]),
                                        pack_bf16(x[8 * e + 4], x[8 * e + 5]), pack_bf16(x[8 * e + 6], x[8 * e + 7]));
                } else {
                  float4* dst = reinterpret_cast<float4*>(parts.o + prow * D + 32 * c);
#pragma unroll
                  for (int e = 0; e < 8; ++e) dst[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
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
            arrive(MERGED);
            if (lane == 0) count_add(merged);
          }
        }
      }
      if (!ok) break;
      if (done > 0) arrive(OFREE + tn);
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(ITEMPTY + i % C::NIT));
    }
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
  static std::atomic<bool> set[64];
  if (!allow_smem(kernel, C::SMEM, set)) return VDA_ERR_CUDA;
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
