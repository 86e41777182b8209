"""What the Softmax branch's entry points refuse, without a GPU: every check
happens before any launch, so the pointers here are never followed."""

import ctypes
import re

import pytest

from frame_wise_delta_vda_b200 import _lib
from frame_wise_delta_vda_b200._lib import VdaAttnArgs, VdaQkArgs, VdaQkGradArgs, VdaRows

P = 1 << 20   # an aligned address that nothing reads


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def header_fields(struct):
    text = open(_lib.HEADER).read()
    body = re.search(r"typedef struct " + struct + r" \{(.*?)\} " + struct + ";", text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    fields = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        fields += [n.strip().lstrip("*") for n in re.sub(r"^(const\s+)?\w+\s*\**", "", decl).split(",")]
    return fields


@pytest.mark.parametrize("struct,mirror", [("vda_rows", VdaRows), ("vda_qk_args", VdaQkArgs),
                                           ("vda_qk_grad_args", VdaQkGradArgs), ("vda_attn_args", VdaAttnArgs)])
def test_argument_structs_mirror_the_header(struct, mirror):
    assert header_fields(struct) == [f[0] for f in mirror._fields_]


def rows(heads, d, n=10, data=P):
    return VdaRows(data, heads * d, d)


def qk_args(**over):
    a = VdaQkArgs()
    a.dtype, a.N, a.Hq, a.Hk, a.d, a.axes, a.rot = 0, 10, 4, 2, 64, 1, 64
    a.q_in, a.k_in, a.v_in, a.q_out, a.k_out = rows(4, 64), rows(2, 64), rows(2, 64), rows(4, 64), rows(2, 64)
    a.q_weight = a.k_weight = a.positions = a.frequencies = a.axis = P
    a.pages, a.page_size = 3, 16
    for k, v in over.items():
        setattr(a, k, v)
    return a


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
SIZES = [
    (dict(dtype=2), INVALID), (dict(N=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID),
    (dict(d=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(rot=-16), INVALID),
    (dict(rot=80), INVALID), (dict(rot=24), UNSUPPORTED), (dict(axes=0), INVALID), (dict(axes=9), UNSUPPORTED),
    (dict(positions=None), INVALID), (dict(frequencies=None), INVALID), (dict(axis=None), INVALID),
    (dict(positions=P + 2), INVALID), (dict(frequencies=P + 4), INVALID), (dict(q_weight=P + 1), INVALID),
    (dict(Hq=70000), UNSUPPORTED),
]


@pytest.mark.parametrize("over,status", SIZES + [
    (dict(q_in=rows(4, 64, data=0)), INVALID), (dict(k_in=rows(2, 64, data=P + 8)), INVALID),
    (dict(q_in=VdaRows(P, 260, 64)), INVALID),           # a token stride that is no multiple of 16 bytes
    (dict(q_in=VdaRows(P, 256, -64)), INVALID),
    (dict(q_in=VdaRows(P, 1 << 60, 64)), INVALID),       # an extent past every address
    (dict(k_out=rows(2, 64, data=0)), INVALID),          # no cache to go to instead
    (dict(q_out=VdaRows(P, 256, 0)), INVALID),           # results on top of one another
    (dict(q_out=VdaRows(P, 0, 64)), INVALID),
    (dict(q_out=VdaRows(P, 192, 64)), INVALID),
    (dict(q_out=VdaRows(P, 64, 576)), INVALID),          # head-major: 10 tokens of 64 need 640
    (dict(slots=P), INVALID),                            # no cache
    (dict(slots=P + 4, k_cache=P, v_cache=P), INVALID),
    (dict(slots=P, k_cache=P, v_cache=P + 8), INVALID),
    (dict(slots=P, k_cache=P, v_cache=P, pages=0), INVALID),
    (dict(slots=P, k_cache=P, v_cache=P, page_size=0), INVALID),
    (dict(slots=P, k_cache=P, v_cache=P, v_in=rows(2, 64, data=0)), INVALID),
])
def test_qk_norm_rope_refuses(L, over, status):
    assert L.vda_qk_norm_rope(ctypes.byref(qk_args(**over))) == status


def test_qk_norm_rope_takes_an_empty_batch_and_no_null_block(L):
    assert L.vda_qk_norm_rope(None) == INVALID
    z = VdaRows()
    assert L.vda_qk_norm_rope(ctypes.byref(qk_args(N=0, q_in=z, k_in=z, q_out=z, k_out=z, positions=None))) == 0


def grad_args(**over):
    a = VdaQkGradArgs()
    a.dtype, a.N, a.Hq, a.Hk, a.d, a.axes, a.rot = 0, 10, 4, 2, 64, 1, 64
    a.dq_out, a.dk_out, a.q_in, a.k_in, a.dq_in, a.dk_in = (rows(4, 64), rows(2, 64)) * 3
    a.q_weight = a.k_weight = a.positions = a.frequencies = a.axis = a.dq_weight = a.dk_weight = P
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", SIZES + [
    (dict(dq_weight=P + 2), INVALID), (dict(dk_out=rows(2, 64, data=0)), INVALID),
    (dict(dq_in=VdaRows(P, 256, 0)), INVALID), (dict(dk_in=VdaRows(P, 0, 64)), INVALID),
])
def test_qk_backward_refuses(L, over, status):
    n = L.vda_qk_grad_workspace_bytes(64)
    assert L.vda_qk_norm_rope_backward(ctypes.byref(grad_args(**over)), P, n) == status


def test_qk_backward_workspace(L):
    assert L.vda_qk_grad_workspace_bytes(96) == 0
    n = L.vda_qk_grad_workspace_bytes(64)
    assert n > 0
    for ws, size in ((None, n), (P, n - 1), (P + 128, n)):
        assert L.vda_qk_norm_rope_backward(ctypes.byref(grad_args()), ws, size) == WORKSPACE
    assert L.vda_qk_norm_rope_backward(None, P, n) == INVALID


def attn_args(**over):
    a = VdaAttnArgs()
    a.dtype, a.N, a.B, a.Hq, a.Hk, a.d = 0, 10, 2, 4, 2, 64
    a.q, a.out = rows(4, 64), rows(4, 64)
    a.k_cache = a.v_cache = a.block_table = a.kv_len = a.q_start = a.lse = P
    a.table_stride, a.pages, a.page_size, a.max_pages = 5, 9, 16, 5
    a.block, a.window_blocks = 1, -1
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(dtype=2), INVALID), (dict(N=-1), INVALID), (dict(B=0), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID),
    (dict(Hq=3), INVALID), (dict(d=0), INVALID), (dict(d=96), UNSUPPORTED), (dict(pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(max_pages=0), INVALID), (dict(table_stride=-1), INVALID),
    (dict(block=-1), INVALID), (dict(anchors=-1), INVALID), (dict(block=(1 << 30) + 1), UNSUPPORTED),
    (dict(anchors=(1 << 30) + 1), UNSUPPORTED), (dict(pages=1 << 30), UNSUPPORTED),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(k_cache=None), INVALID), (dict(v_cache=P + 8), INVALID), (dict(block_table=None), INVALID),
    (dict(kv_len=P + 2), INVALID), (dict(q_start=None), INVALID), (dict(lse=P + 1), INVALID),
    (dict(q=rows(4, 64, data=0)), INVALID), (dict(q=VdaRows(P, 260, 64)), INVALID),
    (dict(q=VdaRows(P, 0, 64)), UNSUPPORTED), (dict(q=VdaRows(P, 256, 0)), UNSUPPORTED),
    (dict(q=VdaRows(P, 1 << 40, 64)), UNSUPPORTED),
    (dict(out=VdaRows(P, 256, 0)), INVALID), (dict(out=VdaRows(P, 192, 64)), INVALID),
    (dict(Hq=129, Hk=1), UNSUPPORTED), (dict(Hq=65, Hk=1, dtype=1), UNSUPPORTED),
    (dict(Hq=65, Hk=1, page_size=17), UNSUPPORTED), (dict(N=1 << 30), UNSUPPORTED),
])
def test_paged_attention_refuses(L, over, status):
    n = 1 << 40
    assert L.vda_paged_attention(ctypes.byref(attn_args(**over)), P, n) == status


def test_paged_attention_workspace(L):
    assert L.vda_paged_attention_workspace_bytes(0, 10, 2, 4, 2, 96, 16) == 0
    assert L.vda_paged_attention_workspace_bytes(0, 10, 2, 5, 2, 64, 16) == 0
    for dtype, page in ((0, 16), (0, 17), (1, 16)):
        n = L.vda_paged_attention_workspace_bytes(dtype, 10, 2, 4, 2, 64, page)
        assert n > 0
        for ws, size in ((None, n), (P, n - 1), (P + 128, n)):
            a = attn_args(dtype=dtype, page_size=page)
            assert L.vda_paged_attention(ctypes.byref(a), ws, size) == WORKSPACE
    assert L.vda_paged_attention(None, P, 1) == INVALID
    z = VdaRows()
    assert L.vda_paged_attention(ctypes.byref(attn_args(N=0, q=z, out=z)), None, 0) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    torch = pytest.importorskip("torch")
    from frame_wise_delta_vda_b200 import api
    q, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        api.vda_qk_norm_rope(q, k)
    with pytest.raises(ValueError, match="CUDA"):
        api.vda_qk_norm_rope_backward(q, k, q, k)
    with pytest.raises(ValueError, match="heads"):
        api.vda_qk_norm_rope(q[0], k)
    with pytest.raises(ValueError, match="CUDA"):
        api.vda_paged_attention(q, None, None, None, None, None)
    with pytest.raises(ValueError, match="Hq"):
        api.vda_paged_attention(q[0], None, None, None, None, None)


def test_rope_frequencies():
    torch = pytest.importorskip("torch")
    from frame_wise_delta_vda_b200 import api
    f, a = api.rope_frequencies(16, 100.0, [4, 2, 2], device="cpu")
    assert f.dtype == torch.float64 and a.dtype == torch.int32
    assert a.tolist() == [0, 0, 0, 0, 1, 1, 2, 2]
    assert f.tolist() == pytest.approx([1, 100 ** -0.25, 0.1, 100 ** -0.75, 1, 0.1, 1, 0.1])
    assert api.rope_frequencies(8, device="cpu")[0].tolist() == pytest.approx([1, 0.1, 0.01, 0.001])
    for bad in ((7, None), (16, [4, 2]), (16, [10, -2])):
        with pytest.raises(ValueError):
            api.rope_frequencies(bad[0], sections=bad[1], device="cpu")


@pytest.mark.parametrize("mirror,pack", [(VdaQkArgs, _lib.pack_qk), (VdaQkGradArgs, _lib.pack_qk_grad),
                                         (VdaAttnArgs, _lib.pack_attn)])
def test_packed_arguments_are_the_struct(mirror, pack):
    """Every field, packed in order, is found in the struct's place."""
    leaves = []

    def fill(m, base):
        for name, t in m._fields_:
            if issubclass(t, ctypes.Structure):
                fill(t, base + getattr(m, name).offset)
            else:
                leaves.append((base + getattr(m, name).offset, t))

    fill(mirror, 0)
    values = [float(i) if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(leaves)]
    raw = pack(*values)
    assert len(raw) == ctypes.sizeof(mirror)
    for v, (off, t) in zip(values, leaves):
        assert (t.from_buffer_copy(raw, off).value or 0) == v
