// Work of the paged attention: which keys a token sees, the items (sequence,
// KV head, run of tokens) with the key tiles that each needs, and the equal
// shares of all tiles that the CTAs take.  Host and device code, so that the
// arithmetic is tested without a GPU.
//
// New tokens and cached keys differ from sequence to sequence and are known
// on the device only.  All items' key tiles, in the order sequence, run of
// tokens, KV head, form one line of W tiles; CTA g of G takes the tiles
// [W g / G, W (g + 1) / G) or so, which may begin and end inside an item.  Every
// item counts Geom::item_cost tiles more, before its own, for what it costs to begin and
// end one (without it, the CTAs with the short sequences of a ragged batch end a
// third later than the others).  The parts
// of an item that several CTAs took are joined afterwards (their running
// maximum and sum say how).  So long and short sequences, one token or
// thousands of them, load every SM alike, without a plan made on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define VDA_HD __host__ __device__ __forceinline__
#else
#define VDA_HD inline
#endif

namespace vda {
namespace attn {

// The token at position p sees the keys j < end with j >= lo or j < anc.
struct Span {
  int lo, end, anc;
};

struct Geom {
  const int* q_start;   // [B + 1]
  const int* kv_len;    // [B]
  int B, N, Hk;
  int group;            // query heads of a KV head
  int tpi;              // tokens of an item
  int max_keys;         // places in a row of the block table
  int block, window, anchors;
  int item_cost;        // what an item costs besides its key tiles, in tiles
};

VDA_HD int imin(int a, int b) { return a < b ? a : b; }
VDA_HD int imax(int a, int b) { return a > b ? a : b; }

// Keys seen from position p of a sequence of len keys.  Anchors behind the end
// of the token's own block are not seen.
VDA_HD Span span_of(const Geom& g, int p, int len) {
  Span s;
  if (p < 0) {
    s.lo = s.end = s.anc = 0;
    return s;
  }
  if (g.block == 0) {
    s.lo = s.anc = 0;
    s.end = len;
    return s;
  }
  const int bs = g.block, d = p - g.anchors;
  // floor(d / bs); block and anchors are at most 2^30
  const long long blk = bs == 1 ? d : d >= 0 ? d / bs : -((-d + bs - 1) / bs);
  const long long e = (blk + 1) * bs + g.anchors;
  s.end = e < len ? (int)e : len;
  long long lo = g.window < 0 ? 0 : (blk - g.window) * bs + g.anchors;
  if (lo < 0) lo = 0;
  s.lo = lo < s.end ? (int)lo : s.end;
  s.anc = imin(g.anchors, s.lo);
  return s;
}

// One sequence as its kernel sees it; whatever the arrays hold, tokens stay in
// [0, N) and keys within the block table's row.
struct Seq {
  int q0, n, len;
};
VDA_HD Seq make_seq(const Geom& g, int a, int b, int len) {
  Seq s;
  s.q0 = imin(imax(a, 0), g.N);
  s.n = imax(0, imin(b, g.N) - s.q0);
  s.len = imin(imax(len, 0), g.max_keys);
  return s;
}

VDA_HD int items_of(const Geom& g, int n) { return (n + g.tpi - 1) / g.tpi; }

// Key tiles of BN keys that tokens [i0, i0 + ntok) of a sequence see: first
// the tiles of the anchors below the window, then those of the window.
struct Tiles {
  int lo, end, anc;     // union of the tokens' keys: [lo, end) and [0, anc)
  int n_anchor, first;  // anchor tiles; first window tile
  int count;            // at least 1: an item that sees nothing still writes its rows
};
template <int BN>
VDA_HD Tiles tiles_of(const Geom& g, const Seq& s, int i0, int ntok) {
  Tiles t;
  const int p1 = s.len - s.n + i0 + ntok - 1;
  const Span a = span_of(g, imax(0, s.len - s.n + i0), s.len), b = span_of(g, p1, s.len);
  t.lo = imin(a.lo, b.end);
  t.end = b.end;
  t.anc = b.anc;
  t.first = t.lo / BN;
  // unsigned: a length of up to 2^31 - 1 is rounded up past 31 bits
  const auto upto = [](int k) { return (int)(((unsigned)k + BN - 1u) / BN); };
  t.n_anchor = imin(upto(t.anc), t.first);
  const int count = t.n_anchor + upto(t.end) - t.first;
  t.count = count > 1 ? count : 1;
  return t;
}
// key tile number of the item's tile t
VDA_HD int key_tile(const Tiles& t, int i) { return i < t.n_anchor ? i : t.first + (i - t.n_anchor); }

// Whether the n keys from j0 on lie all in [0, anc), or all in [lo, end); and
// whether any of them lies in either.  j0 + n may pass 31 bits, so it is not formed.
VDA_HD bool run_all_seen(int lo, int end, int anc, int j0, int n) {
  return j0 <= anc - n || (j0 >= lo && j0 <= end - n);
}
VDA_HD bool run_any_seen(int lo, int end, int anc, int j0, int n) {
  return j0 < anc || (j0 < end && j0 > lo - n);
}

// first tile of share g, and the share that holds tile x
// (the first W % G shares have one tile more)
VDA_HD int share_begin(int W, int g, int G) { return g * (W / G) + imin(g, W % G); }
VDA_HD int share_of(int W, int x, int G) {
  const int per = W / G, rem = W % G, longer = rem * (per + 1);
  return x < longer ? x / (per + 1) : rem + (x - longer) / per;
}

// ------------------------------------------------------------------- device
#ifdef __CUDACC__
__device__ __forceinline__ Seq load_seq(const Geom& g, int b) {
  return make_seq(g, __ldg(g.q_start + b), __ldg(g.q_start + b + 1), __ldg(g.kv_len + b));
}

// Where a CTA's share begins.
struct Plan {
  int W, w0, w1;         // all items' costs; this share
  int shares;            // CTAs with work
  int b, h, r;           // item in which the share begins
  int t;                 // of that item's cost, what lies before it
};

// One warp finds share `cta` of `ctas`.  It walks the runs of tokens of all
// sequences twice, 32 at a time: for their total cost, and for the run in which
// the share begins.  This runs once a CTA, on code that no cache holds yet,
// where a fetch of instructions costs as much as a load of data: one small loop
// body for both passes.  (Counted by sequences, with a branch for long ones and
// called functions, it took 4 to 11 us.)
//
// The host bounds W below 2^31 for ascending q_start, and any one sequence's
// tiles whatever it holds; overlapping sequences may pass it together and get
// wrong results, but the clamps here and in Walk keep them within the tensors.
template <int BN>
__device__ __forceinline__ Plan plan_share(const Geom& g, int cta, int ctas, int lane) {
  Plan p;
  p.W = p.w0 = p.w1 = p.shares = p.b = p.h = p.r = p.t = 0;
  int sum = 0, rest = 0;   // pass 0: this lane's costs; pass 1: cost still to pass
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int b0 = 0; b0 < g.B; b0 += 32) {
      Seq s{0, 0, 0};
      if (b0 + lane < g.B) s = load_seq(g, b0 + lane);
      const int runs = items_of(g, s.n);
      int upto = runs;   // runs of the sequences up to this lane's
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += v;
      }
      const int all = __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll 1
      for (int k0 = 0; k0 < all; k0 += 32) {
        const int k = k0 + lane;
        int l = 0;   // the sequence of run k: as many as end at or before it
#pragma unroll
        for (int step = 16; step > 0; step >>= 1)
          if (__shfl_sync(0xffffffffu, upto, l + step - 1) <= k) l += step;
        l = imin(l, 31);
        Seq o;
        o.q0 = 0;
        o.n = __shfl_sync(0xffffffffu, s.n, l);
        o.len = __shfl_sync(0xffffffffu, s.len, l);
        const int r = k - (__shfl_sync(0xffffffffu, upto, l) - __shfl_sync(0xffffffffu, runs, l));
        int cost = 0;   // of one head
        if (k < all) cost = tiles_of<BN>(g, o, r * g.tpi, imin(g.tpi, o.n - r * g.tpi)).count + g.item_cost;
        if (pass == 0) {
          sum += cost;
          continue;
        }
        int pre = cost * g.Hk;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, pre, off);
          if (lane >= off) pre += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, pre > rest);
        if (hit) {
          const int at = __ffs(hit) - 1;
          const int one = imax(1, __shfl_sync(0xffffffffu, cost, at));
          rest = imax(0, rest - (__shfl_sync(0xffffffffu, pre, at) - one * g.Hk));
          p.b = b0 + __shfl_sync(0xffffffffu, l, at);
          p.r = __shfl_sync(0xffffffffu, r, at);
          p.h = imin(rest / one, g.Hk - 1);
          p.t = imin(rest - p.h * one, one - 1);
          return p;
        }
        rest -= __shfl_sync(0xffffffffu, pre, 31);
      }
    }
    if (pass == 1) break;
    p.W = imax(0, __reduce_add_sync(0xffffffffu, sum) * g.Hk);
    p.shares = imin(p.W, ctas);
    if (cta >= p.shares) return p;
    rest = p.w0 = share_begin(p.W, cta, p.shares);
    p.w1 = share_begin(p.W, cta + 1, p.shares);
  }
  p.w1 = p.w0;   // not found: nothing to do
  return p;
}

// Walks the items of a share.  After the constructor and after every next()
// that returns true, the fields describe the present item.
template <int BN>
struct Walk {
  const Geom* g;
  int left;              // cost of the share from this item's part on
  int b, h, r;
  Seq s;
  int i0, ntok;          // tokens [i0, i0 + ntok) of the sequence
  Tiles tiles;
  int c0, c1;            // this share's part of the item's cost
  int t0, t1;            // its key tiles
  bool live;

  __device__ __forceinline__ Walk(const Geom& geom, const Plan& p)
      : g(&geom), left(p.w1 - p.w0), b(p.b), h(p.h), r(p.r), c0(p.t) {
    live = left > 0;
    if (!live) return;
    s = load_seq(*g, b);
    item();
  }
  __device__ __forceinline__ void item() {
    i0 = r * g->tpi;
    ntok = imin(g->tpi, s.n - i0);
    tiles = tiles_of<BN>(*g, s, i0, ntok);
    const int all = tiles.count + g->item_cost;
    c1 = left < all - c0 ? c0 + left : all;
    t0 = imax(0, c0 - g->item_cost);
    t1 = imax(0, c1 - g->item_cost);
    live = t1 > t0;   // a share that ends before the item's first tile leaves it to the next one
  }
  __device__ __forceinline__ int n() const { return t1 - t0; }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles.count; }
  // of an item that begins in share `cta` and goes on: the shares with a part of it
  __device__ __forceinline__ int parts(const Plan& p, int cta) const {
    const int last = share_of(p.W, p.w1 - (c1 - c0) - c0 + tiles.count + g->item_cost - 1, p.shares);
    return imin(last, p.shares - 1) - cta + 1;
  }
  __device__ __forceinline__ bool next() {
    left -= c1 - c0;
    live = left > 0;
    if (!live) return false;
    c0 = 0;
    if (++h == g->Hk) {
      h = 0;
      if (++r == items_of(*g, s.n)) {
        r = 0;
        do {   // some is left, so a sequence with new tokens follows
          if (++b >= g->B) return live = false;
          s = load_seq(*g, b);
        } while (s.n == 0);
      }
    }
    item();
    return live;
  }
};

// What the join needs of an item whose parts lie in several shares; written
// by the share in which the item begins.
struct Meta {
  int parts;     // 0: nothing to join
  int tok0;      // token of row 0
  int h;         // KV head
  int rows;      // rows of the item
};
#endif   // __CUDACC__

}  // namespace attn
}  // namespace vda
