"""Masks of the paged attention written out by hand: which keys a token sees,
for the oracle, the schedule's code and the kernels.  Anchors before the end of
a token's own block are seen, those behind it are not."""

import numpy as np
import pytest

from oracle import softmax_ref as ref
from test_attn_sched_host import CXX, S, call  # noqa: F401

# block, window, anchors, keys, and the keys that each position sees
PINS = [
    # causal by token, four anchors: a token among them does not see the later ones
    (1, 0, 4, 8, ["0", "01", "012", "0123", "01234", "01235", "01236", "01237"]),
    (1, 1, 2, 6, ["0", "01", "012", "0123", "0134", "0145"]),
    # more anchors than keys: causal alone
    (1, 0, 9, 4, ["0", "01", "012", "0123"]),
    # blocks of two behind three anchors: the anchors are blocks {0}, {1, 2}
    (2, 0, 3, 9, ["0", "012", "012", "01234", "01234", "01256", "01256", "01278", "01278"]),
    # blocks of four behind two anchors, one block before: the last is cut off by the keys there are
    (4, 1, 2, 11, ["01"] * 2 + ["012345"] * 4 + ["0123456789"] * 4 + ["016789a"]),
    # every block before, so the anchors change where blocks begin and nothing else
    (3, -1, 1, 8, ["0"] + ["0123"] * 3 + ["0123456"] * 3 + ["01234567"]),
    (0, -1, 5, 4, ["0123"] * 4),
]


def table(rows, keys):
    see = np.zeros((len(rows), keys), bool)
    for i, r in enumerate(rows):
        see[i, [int(c, 16) for c in r]] = True
    return see


@pytest.mark.parametrize("block,window,anchors,keys,rows", PINS)
def test_oracle(block, window, anchors, keys, rows):
    assert (ref.visible(np.arange(keys), keys, block, window, anchors) == table(rows, keys)).all()


@pytest.mark.skipif(CXX is None, reason="needs a host C++ compiler")
@pytest.mark.parametrize("block,window,anchors,keys,rows", PINS)
def test_schedule(S, block, window, anchors, keys, rows):  # noqa: F811
    j = np.arange(keys)
    for p, want in enumerate(table(rows, keys)):
        lo, end, anc = call(S.span, 3, p, keys, block, window, anchors)
        assert (((j < end) & ((j >= lo) | (j < anc))) == want).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16-64", "bf16-128", "f32-32"])
@pytest.mark.parametrize("block,window,anchors,keys,rows", PINS)
def test_kernels(block, window, anchors, keys, rows, kind):
    """With equal scores and the unit vectors as values, channel j of a token's
    result is 1 / (keys seen) where key j is seen: half a step of the type, the
    weights' rounding and 2^-21 of the quotient."""
    torch = pytest.importorskip("torch")
    from frame_wise_delta_vda_b200 import api
    name, d = kind.split("-")
    dtype, d = (torch.bfloat16 if name == "bf16" else torch.float32), int(d)
    q = torch.ones(keys, 2, d, dtype=dtype, device="cuda")
    kc = torch.zeros(1, 2, 16, d, dtype=dtype, device="cuda")
    vc = torch.eye(16, d, dtype=dtype, device="cuda").expand(1, 2, 16, d).contiguous()
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    out = api.vda_paged_attention(q, kc, vc, ints(0).view(1, 1), ints(keys), ints(0, keys), block=block,
                                  window_blocks=window, anchors=anchors)
    see = table(rows, keys)
    want = np.zeros((keys, 2, d))
    want[:, :, :keys] = (see / see.sum(1, keepdims=True))[:, None]
    u = 2.0 ** -8 if name == "bf16" else 2.0 ** -24
    got = out.double().cpu().numpy()
    assert ((got > 0) == (want > 0)).all()
    assert (np.abs(got - want) <= (2 * u + 2.0 ** -21) * want).all()
