"""The check that results lie apart from inputs: its arithmetic against sets of
bytes, and what the Softmax branch's entry points refuse.  Without a GPU."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from frame_wise_delta_vda_b200 import _lib, build
from frame_wise_delta_vda_b200._lib import VdaRows
from test_softmax_refusals_host import INVALID, P, attn_args, grad_args, qk_args

CXX = shutil.which("g++") or shutil.which("c++")

SOURCE = r"""
#include "overlap.cuh"
extern "C" int overlap(const int64_t* a, const int64_t* b) {
  const auto r = [](const int64_t* x) { return vda::make_region((const void*)x[0], x[1], x[2], x[3], x[4], x[5]); };
  return vda::overlap(r(a), r(b));
}
"""


def held(a):
    at = a[0] + (np.arange(a[2]) * a[3])[:, None, None] + (np.arange(a[4]) * a[5])[None, :, None] + np.arange(a[1])
    return set(at.ravel().tolist())


@pytest.mark.skipif(CXX is None, reason="needs a host C++ compiler")
def test_overlap_is_that_of_the_bytes(tmp_path):
    (tmp_path / "o.cpp").write_text(SOURCE)
    subprocess.run([CXX, "-O1", "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, "-o", str(tmp_path / "o.so"),
                    str(tmp_path / "o.cpp")], check=True)
    L = ctypes.CDLL(os.fspath(tmp_path / "o.so"))
    rng = np.random.default_rng(3)
    seen = [0, 0]
    pick = lambda *v: int(rng.choice(v))  # noqa: E731
    for _ in range(6000):
        d = pick(2, 4)
        kind = pick(0, 1, 2)
        if kind == 0:       # views of one tensor [tokens, width] or [width, tokens]
            s1, s0 = pick(24, 40), d * pick(1, 1, 2, 3)
            a = [1000, d, pick(1, 2, 7), s1, pick(1, 2, 3), s0]
            b = [1000 + int(rng.integers(-60, 200)), d, pick(1, 2, 9), s1, pick(1, 2, 4), pick(s0, s0, d)]
        elif kind == 1:     # a contiguous tensor, or one row, and a view
            a = [1000, pick(1, 8, 50), 1, 0, 1, 0]
            b = [1000 + int(rng.integers(-90, 90)), d, pick(1, 6), pick(0, 12, 20), pick(1, 2, 3), pick(0, 4, 5)]
        else:               # one axis each
            a = [1000, d, pick(1, 5), pick(0, 6, 10), 1, 0]
            b = [1000 + int(rng.integers(-60, 60)), d, 1, 0, pick(1, 6), pick(0, 7, 10)]
        if rng.random() < 0.5:
            a, b = b, a
        if rng.random() < 0.5:
            a = a[:2] + a[4:] + a[2:4]      # the order of the axes does not matter
        if rng.random() < 0.5:
            b = b[:2] + b[4:] + b[2:4]
        want = bool(held(a) & held(b))
        arr = lambda x: (ctypes.c_int64 * 6)(*x)  # noqa: E731
        assert bool(L.overlap(arr(a), arr(b))) == want, (a, b, want)
        seen[want] += 1
    assert min(seen) > 1000


def at(k):
    """The k-th of many places far apart."""
    return P + (k << 24)


APART = dict(q_in=VdaRows(at(1), 256, 64), k_in=VdaRows(at(2), 128, 64), v_in=VdaRows(at(3), 128, 64),
             q_out=VdaRows(at(4), 256, 64), k_out=VdaRows(at(5), 128, 64), q_weight=at(6), k_weight=at(7), positions=at(8),
             frequencies=at(9), axis=at(10), slots=at(11), k_cache=at(12), v_cache=at(13))


@pytest.mark.parametrize("over", [
    dict(q_out=VdaRows(at(1), 256, 64)),                 # in place
    dict(k_out=VdaRows(at(2), 128, 64)),
    dict(q_out=VdaRows(at(1) + 128, 256, 64)),           # a head further
    dict(q_out=VdaRows(at(1) + 64, 1024, 256)),          # between the heads, 16 channels short
    dict(q_out=VdaRows(at(3), 256, 64)),                 # on v
    dict(k_out=VdaRows(at(4) + 512, 256, 64)),           # on the second token of q_out
    dict(k_cache=at(3)), dict(v_cache=at(12)), dict(v_cache=at(12) + 1024), dict(k_cache=at(4)),
    dict(q_out=VdaRows(at(6), 256, 64)), dict(k_out=VdaRows(at(8), 128, 64)), dict(k_cache=at(11)),
    dict(q_in=VdaRows(at(4), 0, 0)),                     # a broadcast input under the results
])
def test_norm_and_rotation_refuses_results_on_inputs(over):
    assert _lib.lib().vda_qk_norm_rope(ctypes.byref(qk_args(**{**APART, **over}))) == INVALID


GRAD = dict(dq_out=VdaRows(at(1), 256, 64), dk_out=VdaRows(at(2), 128, 64), q_in=VdaRows(at(3), 256, 64),
            k_in=VdaRows(at(4), 128, 64), dq_in=VdaRows(at(5), 256, 64), dk_in=VdaRows(at(6), 128, 64), q_weight=at(7),
            k_weight=at(8), dq_weight=at(9), dk_weight=at(10), positions=at(11), frequencies=at(12), axis=at(13))


@pytest.mark.parametrize("over,ws", [
    (dict(dq_in=VdaRows(at(1), 256, 64)), at(20)), (dict(dq_in=VdaRows(at(3), 256, 64)), at(20)),
    (dict(dk_in=VdaRows(at(5) + 128, 256, 64)), at(20)), (dict(dq_weight=at(10)), at(20)), (dict(dk_weight=at(8)), at(20)),
    (dict(dq_out=VdaRows(at(6), 0, 0)), at(20)), (dict(), at(5)), (dict(), at(1)), (dict(), at(9)),
])
def test_gradient_refuses_results_on_inputs(over, ws):
    assert _lib.lib().vda_qk_norm_rope_backward(ctypes.byref(grad_args(**{**GRAD, **over})), ws, 1 << 22) == INVALID


ATTN = dict(q=VdaRows(at(1), 256, 64), out=VdaRows(at(2), 256, 64), k_cache=at(3), v_cache=at(4), block_table=at(5),
            kv_len=at(6), q_start=at(7), lse=at(8))


@pytest.mark.parametrize("over,ws", [
    (dict(out=VdaRows(at(1), 256, 64)), at(20)), (dict(out=VdaRows(at(1) + 128, 256, 64)), at(20)),
    (dict(out=VdaRows(at(4) + 1024, 256, 64)), at(20)), (dict(out=VdaRows(at(5), 256, 64)), at(20)), (dict(lse=at(2)), at(20)),
    (dict(lse=at(6)), at(20)), (dict(lse=at(1)), at(20)), (dict(), at(2)), (dict(), at(3)), (dict(), at(8)),
])
def test_attention_refuses_results_on_inputs(over, ws):
    assert _lib.lib().vda_paged_attention(ctypes.byref(attn_args(**{**ATTN, **over})), ws, 1 << 40) == INVALID
