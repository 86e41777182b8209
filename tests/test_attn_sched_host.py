"""The schedule of the paged attention (which keys a token sees, key tiles of
an item, equal shares) compiled for the host: against the mask's definition,
and at the largest lengths that 32 bits hold."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from frame_wise_delta_vda_b200 import build
from oracle import softmax_ref as ref

CXX = shutil.which("g++") or shutil.which("c++")
pytestmark = pytest.mark.skipif(CXX is None, reason="needs a host C++ compiler")

SOURCE = r"""
#include "attn_sched.cuh"
using namespace vda::attn;
static Geom geom(int tpi, int block, int window, int anchors) {
  Geom g{};
  g.B = 1; g.N = 1 << 30; g.Hk = 1; g.group = 1; g.tpi = tpi; g.max_keys = 2147483647;
  g.block = block; g.window = window; g.anchors = anchors;
  return g;
}
extern "C" {
void span(int p, int len, int block, int window, int anchors, int* o) {
  const Span s = span_of(geom(1, block, window, anchors), p, len);
  o[0] = s.lo; o[1] = s.end; o[2] = s.anc;
}
void tiles(int bn, int n, int len, int i0, int ntok, int block, int window, int anchors, int* o) {
  const Geom g = geom(ntok, block, window, anchors);
  const Seq s = make_seq(g, 0, n, len);
  const Tiles t = bn == 128 ? tiles_of<128>(g, s, i0, ntok) : tiles_of<64>(g, s, i0, ntok);
  o[0] = t.lo; o[1] = t.end; o[2] = t.anc; o[3] = t.n_anchor; o[4] = t.first; o[5] = t.count;
}
int begin_of(int W, int g, int G) { return share_begin(W, g, G); }
int share(int W, int x, int G) { return share_of(W, x, G); }
int all_seen(int lo, int end, int anc, int j0, int n) { return run_all_seen(lo, end, anc, j0, n); }
int any_seen(int lo, int end, int anc, int j0, int n) { return run_any_seen(lo, end, anc, j0, n); }
}
"""


@pytest.fixture(scope="module")
def S(tmp_path_factory):
    d = tmp_path_factory.mktemp("sched")
    (d / "s.cpp").write_text(SOURCE)
    # -fwrapv: an overflow, were there one, gives what the GPU gives
    subprocess.run([CXX, "-O1", "-std=c++17", "-fwrapv", "-shared", "-fPIC", "-I", build.CSRC, "-o", str(d / "s.so"), str(d / "s.cpp")],
                   check=True)
    return ctypes.CDLL(os.fspath(d / "s.so"))


def call(f, n, *a):
    o = (ctypes.c_int * n)()
    f(*a, o)
    return list(o)


def test_spans_are_the_mask(S):
    rng = np.random.default_rng(1)
    for _ in range(300):
        L = int(rng.integers(1, 300))
        block = int(rng.choice([0, 1, 1, 2, 7, 64, 500, 1 << 30]))
        window = int(rng.choice([-1, 0, 1, 30, 2 ** 31 - 1]))
        anchors = int(rng.choice([0, 3, 90, 700, 1 << 30]))
        pos = np.arange(-2, L)
        see = ref.visible(pos, L, block, window, anchors)
        j = np.arange(L)
        for i, p in enumerate(pos):
            lo, end, anc = call(S.span, 3, int(p), L, block, window, anchors)
            assert ((j < end) & ((j >= lo) | (j < anc)) == see[i]).all(), (p, L, block, window, anchors)


@pytest.mark.parametrize("bn", [64, 128])
def test_tiles_hold_every_seen_key_once(S, bn):
    rng = np.random.default_rng(2)
    for _ in range(300):
        L, n = int(rng.integers(0, 900)), int(rng.integers(1, 200))
        block = int(rng.choice([0, 1, 1, 5, 80, 1 << 30]))
        window = int(rng.choice([-1, 0, 2, 100, 2 ** 31 - 1]))
        anchors = int(rng.choice([0, 4, 200, 1 << 30]))
        i0 = int(rng.integers(0, n))
        ntok = int(rng.integers(1, n - i0 + 1))
        lo, end, anc, n_anchor, first, count = call(S.tiles, 6, bn, n, L, i0, ntok, block, window, anchors)
        kt = [t if t < n_anchor else first + t - n_anchor for t in range(count)]
        assert count >= 1 and kt == sorted(set(kt))
        see = ref.visible(np.arange(L - n + i0, L - n + i0 + ntok), L, block, window, anchors).any(0)
        j = np.flatnonzero(see)
        assert set(j // bn) <= set(kt)
        assert ((j < anc) | ((j >= lo) & (j < end))).all()
        assert end == 0 or max(kt) * bn < end
        for t in kt:
            for w in (8, 32, bn):
                for j0 in range(t * bn, (t + 1) * bn, w):
                    inside = [(k < anc) or (lo <= k < end) for k in range(j0, j0 + w)]
                    assert S.all_seen(lo, end, anc, j0, w) <= all(inside)
                    assert S.any_seen(lo, end, anc, j0, w) == any(inside)


def test_shares_split_the_line(S):
    for W in (1, 2, 147, 148, 149, 1000, 12345, 2 ** 31 - 1):
        for G in (1, 3, 148, 296):
            G = min(W, G)
            b = [S.begin_of(W, g, G) for g in range(G + 1)]
            assert b[0] == 0 and b[-1] == W and all(x < y for x, y in zip(b, b[1:]))
            for g in range(G):
                assert S.share(W, b[g], G) == g and S.share(W, b[g + 1] - 1, G) == g


@pytest.mark.parametrize("L", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 128, 2 ** 31 - 129, 2 ** 31 - 300])
@pytest.mark.parametrize("bn", [64, 128])
def test_the_longest_sequences(S, L, bn):
    """Keys whose tile ends past 2^31 - 1 are in a tile like any other."""
    lo, end, anc, n_anchor, first, count = call(S.tiles, 6, bn, 1, L, 0, 1, 0, -1, 0)
    assert (lo, end, anc, n_anchor, first, count) == (0, L, 0, 0, 0, -(-L // bn))
    lo, end, anc, n_anchor, first, count = call(S.tiles, 6, bn, 1, L, 0, 1, 1, 200, 70)
    assert (lo, end, anc) == (L - 201, L, 70) and first == lo // bn
    assert (n_anchor, count) == (-(-70 // bn), -(-70 // bn) + -(-L // bn) - first)
    j0 = (L - 1) // bn * bn
    assert S.all_seen(0, L, 0, j0, bn) == (L % bn == 0)
    assert S.all_seen(0, L, 0, j0 - bn, bn) == 1
    assert S.all_seen(L - 1, L, 70, j0, bn) == 0 and S.any_seen(L - 1, L, 70, j0, bn) == 1
    assert S.any_seen(0, j0, 0, j0, bn) == 0
