// Work of the paged attention: which keys a token sees, the items (sequence,
// KV head, run of tokens) with the key tiles that each needs, and the equal
// shares of all tiles that the CTAs take.  Host and device code, so that the
// arithmetic is tested without a GPU.
//
// New tokens and cached keys differ from sequence to sequence and are known
// on the device only.  All items' key tiles, in the order sequence, KV head,
// run of tokens, form one line of W tiles; CTA g of G takes the tiles
// [W g / G, W (g + 1) / G) or so, which may begin and end inside an item.  The parts
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
};

VDA_HD int imin(int a, int b) { return a < b ? a : b; }
VDA_HD int imax(int a, int b) { return a > b ? a : b; }

// keys seen from position p of a sequence of len keys
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
  t.n_anchor = imin((t.anc + BN - 1) / BN, t.first);
  const int count = t.n_anchor + (t.end + BN - 1) / BN - t.first;
  t.count = count > 1 ? count : 1;
  return t;
}
// key tile number of the item's tile t
VDA_HD int key_tile(const Tiles& t, int i) { return i < t.n_anchor ? i : t.first + (i - t.n_anchor); }

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

// Tiles of one head of a sequence, computed by one lane.
template <int BN>
__device__ __forceinline__ int seq_tiles_serial(const Geom& g, const Seq& s) {
  int w = 0;
  const int n = items_of(g, s.n);
  for (int r = 0; r < n; ++r) w += tiles_of<BN>(g, s, r * g.tpi, imin(g.tpi, s.n - r * g.tpi)).count;
  return w;
}
// ... and by a whole warp.
template <int BN>
__device__ __forceinline__ int seq_tiles_warp(const Geom& g, const Seq& s, int lane) {
  int w = 0;
  const int n = items_of(g, s.n);
  for (int r = lane; r < n; r += 32) w += tiles_of<BN>(g, s, r * g.tpi, imin(g.tpi, s.n - r * g.tpi)).count;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) w += __shfl_xor_sync(0xffffffffu, w, off);
  return w;
}

// Where a CTA's share begins.
struct Plan {
  int W, w0, w1;         // all tiles; this share
  int shares;            // CTAs with work
  int b, h, r;           // item in which the share begins
  int t;                 // tiles of that item before it
};

constexpr int kSerialItems = 4;   // longer sequences are counted by the whole warp

// One head's tiles of sequences 32 c .. 32 c + 31, one a lane.
template <int BN>
__device__ __forceinline__ int chunk_tiles(const Geom& g, int c, int lane) {
  const int b = c * 32 + lane;
  Seq s{0, 0, 0};
  if (b < g.B) s = load_seq(g, b);
  int w = 0;
  const bool longer = items_of(g, s.n) > kSerialItems;
  if (!longer) w = seq_tiles_serial<BN>(g, s);
  unsigned todo = __ballot_sync(0xffffffffu, longer);
  while (todo) {
    const int l = __ffs(todo) - 1;
    todo &= todo - 1;
    Seq o;
    o.q0 = 0;
    o.n = __shfl_sync(0xffffffffu, s.n, l);
    o.len = __shfl_sync(0xffffffffu, s.len, l);
    const int v = seq_tiles_warp<BN>(g, o, lane);
    if (lane == l) w = v;
  }
  return w;
}

// One warp finds share `cta` of `ctas`.  The first kKeep chunks of 32
// sequences are counted once and kept in registers.  The host bounds W for
// ascending q_start; sequences that overlap so that W passes 2^31 get nothing.
template <int BN>
__device__ __forceinline__ Plan plan_share(const Geom& g, int cta, int ctas, int lane) {
  constexpr int kKeep = 4;
  int keep[kKeep];
  long long total = 0;
  const int chunks = (g.B + 31) / 32;
#pragma unroll
  for (int c = 0; c < kKeep; ++c) {
    keep[c] = c < chunks ? chunk_tiles<BN>(g, c, lane) : 0;
    total += keep[c];
  }
#pragma unroll 1
  for (int c = kKeep; c < chunks; ++c) total += chunk_tiles<BN>(g, c, lane);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  total *= g.Hk;
  Plan p;
  p.W = total > 2147483647LL ? 0 : (int)total;
  p.w0 = p.w1 = p.b = p.h = p.r = p.t = 0;
  p.shares = imin(p.W, ctas);
  if (cta >= p.shares) return p;
  p.w0 = share_begin(p.W, cta, p.shares);
  p.w1 = share_begin(p.W, cta + 1, p.shares);
  int rest = p.w0;   // tiles still to pass
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    int w = 0;
    if (c < kKeep) {
#pragma unroll
      for (int k = 0; k < kKeep; ++k)
        if (c == k) w = keep[k];
    } else {
      w = chunk_tiles<BN>(g, c, lane);
    }
    int upto = w * g.Hk;   // inclusive prefix over the lanes
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, upto > rest);
    if (!hit) {
      rest -= __shfl_sync(0xffffffffu, upto, 31);
      continue;
    }
    const int l = __ffs(hit) - 1;
    const int per_head = __shfl_sync(0xffffffffu, w, l);
    rest -= __shfl_sync(0xffffffffu, upto, l) - per_head * g.Hk;
    p.b = c * 32 + l;
    p.h = rest / per_head;
    rest -= p.h * per_head;
    // the run of tokens that holds tile `rest` of this head
    const Seq s = load_seq(g, p.b);
    const int n = items_of(g, s.n);
#pragma unroll 1
    for (int r0 = 0; r0 < n; r0 += 32) {
      const int r = r0 + lane;
      const int k = r < n ? tiles_of<BN>(g, s, r * g.tpi, imin(g.tpi, s.n - r * g.tpi)).count : 0;
      int pre = k;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, pre, off);
        if (lane >= off) pre += v;
      }
      const unsigned at = __ballot_sync(0xffffffffu, pre > rest);
      if (at) {
        const int rl = __ffs(at) - 1;
        p.r = r0 + rl;
        p.t = rest - (__shfl_sync(0xffffffffu, pre, rl) - __shfl_sync(0xffffffffu, k, rl));
        break;
      }
      rest -= __shfl_sync(0xffffffffu, pre, 31);
    }
    break;
  }
  return p;
}

// Walks the items of a share.  After the constructor and after every next()
// that returns true, the fields describe the present item.
template <int BN>
struct Walk {
  const Geom* g;
  int left;              // tiles of the share from this item's on
  int b, h, r;
  Seq s;
  int i0, ntok;          // tokens [i0, i0 + ntok) of the sequence
  Tiles tiles;
  int t0, t1;            // this share's tiles of the item
  bool live;

  __device__ __forceinline__ Walk(const Geom& geom, const Plan& p)
      : g(&geom), left(p.w1 - p.w0), b(p.b), h(p.h), r(p.r), t0(p.t) {
    live = left > 0;
    if (!live) return;
    s = load_seq(*g, b);
    item();
  }
  __device__ __forceinline__ void item() {
    i0 = r * g->tpi;
    ntok = imin(g->tpi, s.n - i0);
    tiles = tiles_of<BN>(*g, s, i0, ntok);
    t1 = left < tiles.count - t0 ? t0 + left : tiles.count;
  }
  __device__ __forceinline__ int n() const { return t1 - t0; }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles.count; }
  __device__ __forceinline__ bool next() {
    left -= n();
    live = left > 0;
    if (!live) return false;
    t0 = 0;
    if (++r == items_of(*g, s.n)) {
      r = 0;
      if (++h == g->Hk) {
        h = 0;
        do {   // tiles are left, so a sequence with new tokens follows
          if (++b >= g->B) return live = false;
          s = load_seq(*g, b);
        } while (s.n == 0);
      }
    }
    item();
    return true;
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
