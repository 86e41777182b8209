"""Empty calls of the paged attention, without a GPU: nothing is launched and no
pointer of an empty tensor is needed."""

import ctypes

import pytest

from frame_wise_delta_vda_b200 import _lib
from frame_wise_delta_vda_b200._lib import VdaRows
from test_softmax_refusals_host import INVALID, UNSUPPORTED, P, attn_args


@pytest.mark.parametrize("over", [
    dict(),
    dict(q_start=P, block_table=None, kv_len=None, B=0),     # no sequences
    dict(max_pages=0, block_table=None),                     # sequences without a page yet
    dict(dtype=1, B=0, kv_len=None, block_table=None, max_pages=0),
], ids=str)
def test_a_batch_without_tokens_is_a_valid_call(over):
    z = VdaRows()
    a = attn_args(**{**dict(N=0, q=z, out=z, lse=None), **over})
    assert _lib.lib().vda_paged_attention(ctypes.byref(a), None, 0) == 0


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), INVALID), (dict(d=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(B=-1), INVALID), (dict(Hq=3), INVALID),
    (dict(block=-1), INVALID), (dict(anchors=-1), INVALID), (dict(scale=float("nan")), INVALID), (dict(pages=0), INVALID),
    (dict(max_pages=-1), INVALID), (dict(k_cache=None), INVALID),
])
def test_an_empty_batch_of_what_is_not_supported_is_still_refused(over, status):
    z = VdaRows()
    a = attn_args(**{**dict(N=0, q=z, out=z), **over})
    assert _lib.lib().vda_paged_attention(ctypes.byref(a), None, 0) == status


@pytest.mark.parametrize("over", [dict(B=0), dict(max_pages=0), dict(block_table=None), dict(kv_len=None)])
def test_tokens_need_sequences_and_tables(over):
    assert _lib.lib().vda_paged_attention(ctypes.byref(attn_args(**over)), P, 1 << 40) == INVALID


def test_workspace_of_an_empty_batch():
    L = _lib.lib()
    assert L.vda_paged_attention_workspace_bytes(0, 0, 0, 4, 2, 64, 16) >= 0
    assert L.vda_paged_attention_workspace_bytes(0, 1, 0, 4, 2, 64, 16) == 0
