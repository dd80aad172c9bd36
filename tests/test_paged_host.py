"""The paged-cache and packed-prompt calls without a GPU: sizes, and the
refusal of bad arguments before anything is launched."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def R():
    from top_kv_span_b200 import build
    build.build()
    from top_kv_span_b200 import reatt
    return reatt


def dims(R, **kw):
    base = dict(B=3, Hq=32, Hkv=8, d=128, dtype="bf16", N=3, page=16, max_pages=100, n_pages=300,
                rope_base=5e5)
    base.update(kw)
    return R.make_paged_dims(**base)


A, M = 0x10000, 0x10008   # aligned / misaligned addresses, never dereferenced


def append(R, d, **kw):
    a = dict(q=A, k=A + 4096, v=A, cu=A, past=A, table=A, q_rot=A + 16, k_rot=None, k_pages=A,
             v_pages=A, seq_len=A + 16, ws=A)
    a.update(kw)
    return R.reatt_paged_append(d, a["q"], a["k"], a["v"], a["cu"], a["past"], a["table"],
                                a["q_rot"], a["k_rot"], a["k_pages"], a["v_pages"], a["seq_len"],
                                a["ws"], stream=0, check=False)


def decode(R, d, **kw):
    a = dict(q=A, k_pages=A, v_pages=A, table=A, lens=A, out=A, ws=A)
    a.update(kw)
    return R.reatt_paged_decode(d, a["q"], a["k_pages"], a["v_pages"], a["table"], a["lens"],
                                a["out"], a["ws"], stream=0, check=False)


def prompt(R, d, **kw):
    a = dict(q=A, k=A, v=A, cu=A, out=A, ws=A)
    a.update(kw)
    return R.reatt_prompt_attend(d, a["q"], a["k"], a["v"], a["cu"], a["out"], a["ws"], stream=0,
                                 check=False)


def test_struct_layout_and_workspace(R):
    # int32 x 8, int64 x 7, double
    assert ctypes.sizeof(R.reatt_paged_dims) == 96
    assert R.reatt_paged_dims.N.offset == 32 and R.reatt_paged_dims.rope_base.offset == 88
    ws = R.reatt_paged_workspace_bytes(dims(R))
    assert ws % 256 == 0 and ws >= 256
    # neither the lengths nor the pools change it
    assert ws == R.reatt_paged_workspace_bytes(dims(R, N=4000, max_pages=9000, n_pages=1 << 20))
    assert R.status_string(R.EPAGE) != R.status_string(99)


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), 1), (dict(Hq=30), 1), (dict(Hkv=0), 1), (dict(Hq=0), 1), (dict(N=-1), 1),
    (dict(page=0), 1), (dict(page=24), 1), (dict(page=-16), 1), (dict(max_pages=0), 1),
    (dict(n_pages=0), 1), (dict(rope_base=-1.0), 1), (dict(rope_base=float("inf")), 1),
    (dict(rope_base=float("nan")), 1), (dict(q_stride=32 * 128 - 8), 1),
    (dict(q_stride=32 * 128 + 4), 1), (dict(k_stride=8 * 128 - 8), 1), (dict(v_stride=-1024), 1),
    (dict(q_rot_stride=8), 1), (dict(k_rot_stride=1025), 1),
    (dict(d=96), 2), (dict(d=256), 2), (dict(dtype=7), 2), (dict(B=65537, N=65537), 2),
    (dict(Hq=129, Hkv=1), 2), (dict(max_pages=(1 << 20) + 1), 2), (dict(N=1 << 28), 2),
    (dict(n_pages=1 << 31), 2),
])
def test_bad_dims_rejected_everywhere(R, bad, code):
    d = dims(R, **bad)
    v = ctypes.c_size_t()
    assert R.lib.reatt_paged_workspace_bytes(ctypes.byref(d), ctypes.byref(v)) == code
    assert append(R, d) == code
    assert decode(R, d) == code
    assert prompt(R, d) == code


def test_reserved_field_and_null_dims(R):
    d = dims(R)
    d.reserved = 1
    assert append(R, d) == R.EINVAL and decode(R, d) == R.EINVAL and prompt(R, d) == R.EINVAL
    v = ctypes.c_size_t()
    assert R.lib.reatt_paged_workspace_bytes(None, ctypes.byref(v)) == R.EINVAL
    assert R.lib.reatt_paged_workspace_bytes(ctypes.byref(dims(R)), None) == R.EINVAL
    assert R.lib.reatt_paged_append(None, *[A] * 13) == R.EINVAL
    assert R.lib.reatt_paged_decode(None, *[A] * 8) == R.EINVAL
    assert R.lib.reatt_prompt_attend(None, *[A] * 7) == R.EINVAL


@pytest.mark.parametrize("name", ["k", "v", "cu", "past", "table", "k_pages", "v_pages", "ws"])
def test_append_needs_its_pointers(R, name):
    assert append(R, dims(R), **{name: None}) == R.EINVAL
    assert append(R, dims(R), **{name: M}) == R.EINVAL


def test_append_optional_pointers(R):
    d = dims(R)
    # q and q_rot come together; seq_len is not past_len; aligned like all
    assert append(R, d, q=None) == R.EINVAL
    assert append(R, d, q_rot=None) == R.EINVAL
    assert append(R, d, seq_len=A) == R.EINVAL
    for name in ("q", "q_rot", "k_rot", "seq_len"):
        assert append(R, d, **{name: M}) == R.EINVAL
    # in place needs the same stride
    wide = dims(R, q_stride=6144, k_stride=6144)
    assert append(R, wide, q_rot=A) == R.EINVAL
    assert append(R, wide, k_rot=A + 4096) == R.EINVAL


@pytest.mark.parametrize("name", ["q", "k_pages", "v_pages", "table", "lens", "out", "ws"])
def test_decode_needs_its_pointers(R, name):
    assert decode(R, dims(R), **{name: None}) == R.EINVAL
    assert decode(R, dims(R), **{name: M}) == R.EINVAL


def test_decode_needs_one_row_per_sequence(R):
    assert decode(R, dims(R, N=2)) == R.EINVAL
    assert decode(R, dims(R, N=4)) == R.EINVAL


@pytest.mark.parametrize("name", ["q", "k", "v", "cu", "out", "ws"])
def test_prompt_needs_its_pointers(R, name):
    assert prompt(R, dims(R), **{name: None}) == R.EINVAL
    assert prompt(R, dims(R), **{name: M}) == R.EINVAL


def test_nothing_to_do_needs_no_rows(R):
    # no packed rows: nothing is launched, row pointers may be null
    d = dims(R, N=0)
    assert prompt(R, d, q=None, k=None, v=None, out=None) == R.OK
    assert append(R, d, q=None, k=None, v=None, q_rot=None, seq_len=None) == R.OK


def test_host_tensors_are_refused(R):
    d = dims(R)
    x = torch.zeros((3, 32, 128), dtype=torch.bfloat16)
    with pytest.raises(R.ReattError) as e:
        R.reatt_paged_decode(d, x, A, A, A, A, A, A, stream=0)
    assert e.value.code == R.EINVAL
    with pytest.raises(R.ReattError):
        R.reatt_prompt_attend(d, A, A, A, torch.zeros(4, dtype=torch.int32), A, A, stream=0)
    with pytest.raises(R.ReattError):
        append(R, d, ws=torch.zeros(1 << 20, dtype=torch.uint8))


def test_more_prompt_blocks_than_a_grid(R):
    # one token a block and thousands of heads: refused before any CUDA call
    d = dims(R, Hq=4096, Hkv=32, d=64, N=(1 << 28) - 1)
    assert prompt(R, d) == R.EUNSUPPORTED
    d = dims(R, Hq=4096, Hkv=4096, d=64, N=(1 << 28) - 1, dtype="f32")
    assert prompt(R, d) == R.EUNSUPPORTED


def test_unknown_dtypes_are_refused(R):
    for dtype in ("fp16", torch.float16, torch.float64):
        with pytest.raises(R.ReattError) as e:
            dims(R, dtype=dtype)
        assert e.value.code == R.EUNSUPPORTED
    assert dims(R, dtype=torch.float32).dtype == R.F32 and dims(R, dtype="bf16").dtype == R.BF16
