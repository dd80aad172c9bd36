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


# ------------------------------------------------------------------ the binding's look at tensors
@pytest.fixture
def on_host(R, monkeypatch):
    """The binding with the host as its device and calls that only note their arguments."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # get_device() of a host tensor
    R._paged_plan.cache_clear()
    calls = []
    for name in ("reatt_paged_append", "reatt_paged_decode", "reatt_prompt_attend"):
        monkeypatch.setattr(R.lib, name, lambda *a: calls.append(a) or R.OK)
    yield calls
    R._paged_plan.cache_clear()


B, HQ, HKV, D, PAGE, PAGES, COLS, ROWS = 3, 8, 2, 64, 16, 11, 4, 20


def operands(call, dtype=torch.bfloat16):
    """Well-formed operands of a call, q, k and v as slices of one projection."""
    N = B if call == "decode" else ROWS
    row = torch.zeros((N, HQ + 2 * HKV, D), dtype=dtype)
    i32 = torch.int32
    x = dict(q=row[:, :HQ], k=row[:, HQ:HQ + HKV], v=row[:, HQ + HKV:],
             cu=torch.zeros(B + 1, dtype=i32), past=torch.zeros(B, dtype=i32),
             table=torch.zeros((B, COLS), dtype=i32), q_rot=torch.zeros((N, HQ, D), dtype=dtype),
             k_rot=torch.zeros((N, HKV, D), dtype=dtype),
             k_pages=torch.zeros((PAGES, HKV, PAGE, D), dtype=dtype),
             v_pages=torch.zeros((PAGES, HKV, PAGE, D), dtype=dtype),
             lens=torch.zeros(B, dtype=i32), out=torch.zeros((N, HQ, D), dtype=dtype))
    return x


def call_with(R, call, x, dtype="bf16", **kw):
    s = (HQ + 2 * HKV) * D
    d = R.make_paged_dims(B=B, Hq=HQ, Hkv=HKV, d=D, dtype=dtype, N=B if call == "decode" else ROWS,
                          page=PAGE, max_pages=COLS, n_pages=PAGES, q_stride=s, k_stride=s,
                          v_stride=s, **kw)
    if "ws" not in x:
        x = dict(x, ws=torch.zeros(R.reatt_paged_workspace_bytes(d), dtype=torch.uint8))
    if call == "append":
        return R.reatt_paged_append(d, x["q"], x["k"], x["v"], x["cu"], x["past"], x["table"],
                                    x["q_rot"], x["k_rot"], x["k_pages"], x["v_pages"], x["lens"],
                                    x["ws"], stream=0)
    if call == "decode":
        return R.reatt_paged_decode(d, x["q"], x["k_pages"], x["v_pages"], x["table"], x["lens"],
                                    x["out"], x["ws"], stream=0)
    return R.reatt_prompt_attend(d, x["q"], x["k"], x["v"], x["cu"], x["out"], x["ws"], stream=0)


CALLS = {"append": ("q", "k", "v", "cu", "past", "table", "q_rot", "k_rot", "k_pages", "v_pages", "lens"),
         "decode": ("q", "k_pages", "v_pages", "table", "lens", "out"),
         "prompt": ("q", "k", "v", "cu", "out")}


@pytest.mark.parametrize("call", CALLS)
def test_well_formed_tensors_pass_with_their_addresses(R, on_host, call):
    x = operands(call)
    for _ in range(2):
        assert call_with(R, call, x) == R.OK
    got = on_host[-1][1:]
    order = {"append": ("q", "k", "v", "cu", "past", "table", "q_rot", "k_rot", "k_pages", "v_pages", "lens"),
             "decode": ("q", "k_pages", "v_pages", "table", "lens", "out"),
             "prompt": ("q", "k", "v", "cu", "out")}[call]
    assert list(got[:len(order)]) == [x[n].data_ptr() for n in order]


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in CALLS[c]])
@pytest.mark.parametrize("after", [False, True])
def test_short_tensors_are_refused(R, on_host, call, name, after):
    """One row, page or entry too few would be read or written past its end; also after
    a call whose operands fitted."""
    x = operands(call)
    if after:
        call_with(R, call, x)
    short = x[name][:-1]
    with pytest.raises(R.ReattError) as e:
        call_with(R, call, dict(x, **{name: short}))
    assert e.value.code == R.EINVAL
    assert call_with(R, call, x) == R.OK


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in CALLS[c]])
@pytest.mark.parametrize("after", [False, True])
def test_other_layouts_are_refused(R, on_host, call, name, after):
    """The same elements in another order: transposed, every second one, or dense rows
    where the dims say that they lie apart."""
    x = operands(call)
    if after:
        call_with(R, call, x)
    t = x[name]
    wrong = [torch.zeros([2 * n for n in t.shape], dtype=t.dtype)[tuple([slice(None, None, 2)] * t.dim())]]
    if t.dim() > 1:
        wrong.append(torch.zeros(t.transpose(0, 1).shape, dtype=t.dtype).transpose(0, 1))
    if t.dim() == 3:
        wrong.append(torch.zeros((t.shape[0], D, t.shape[1]), dtype=t.dtype).transpose(1, 2))
        wrong.append(torch.zeros((t.shape[1], t.shape[0], D), dtype=t.dtype))   # heads before tokens
    if t.dim() == 4:   # tokens before heads
        wrong.append(torch.zeros((PAGES, PAGE, HKV, D), dtype=t.dtype))
        wrong.append(torch.zeros((PAGES, PAGE, HKV, D), dtype=t.dtype).transpose(1, 2))
    if name in ("q", "k", "v"):
        wrong.append(t.contiguous())
    if name in ("q_rot", "k_rot", "out"):
        wrong.append(torch.zeros((t.shape[0], 12, D), dtype=t.dtype)[:, :t.shape[1]])
    for w in wrong:
        with pytest.raises(R.ReattError) as e:
            call_with(R, call, dict(x, **{name: w}))
        assert e.value.code == R.EINVAL, (tuple(w.shape), w.stride())
    assert call_with(R, call, x) == R.OK


def test_other_dtypes_and_small_workspaces_are_refused(R, on_host):
    x = operands("prompt")
    assert call_with(R, "prompt", operands("prompt", torch.float32), dtype="f32") == R.OK
    for bad in (dict(cu=x["cu"].long()), dict(q=x["q"].float()), dict(out=x["out"].half()),
                dict(ws=torch.zeros(256, dtype=torch.uint8))):
        with pytest.raises(R.ReattError) as e:
            call_with(R, "prompt", dict(x, **bad))
        assert e.value.code == R.EINVAL


def test_other_ways_to_hold_the_same_rows_pass(R, on_host):
    """Flat buffers, rows without a dimension for the heads, padded buffers, tokens in two
    dimensions, and fp32 words as a workspace."""
    s, N = (HQ + 2 * HKV) * D, ROWS
    x = operands("prompt")
    row = torch.zeros((N + 5, HQ + 2 * HKV, D), dtype=torch.bfloat16)
    need = R.reatt_paged_workspace_bytes(R.make_paged_dims(B=B, Hq=HQ, Hkv=HKV, d=D, dtype="bf16",
                                                           N=N))
    for ok in (dict(q=row, k=row[:, HQ:], v=row.flatten()[(HQ + HKV) * D:]),
               dict(q=row.flatten(1)[:, :HQ * D], out=torch.zeros(N * HQ * D, dtype=torch.bfloat16)),
               dict(q=row[:N].view(4, 5, HQ + 2 * HKV, D)[:, :, :HQ],
                    out=torch.zeros((4, 5, HQ * D), dtype=torch.bfloat16)),
               dict(cu=torch.zeros(B + 9, dtype=torch.int32)),
               dict(ws=torch.zeros(need // 4, dtype=torch.float32))):
        assert call_with(R, "prompt", dict(x, **ok)) == R.OK
    # one row: the distance to the next one does not matter
    d = R.make_paged_dims(B=1, Hq=1, Hkv=1, d=D, dtype="bf16", N=1, q_stride=s)
    ws = torch.zeros(need, dtype=torch.uint8)
    for q in (row[3:4, :1], row[0, 0], row[:, 0]):
        k = torch.zeros((1, 1, D), dtype=torch.bfloat16)
        assert R.reatt_prompt_attend(d, q, k, k, torch.zeros(2, dtype=torch.int32), k, ws,
                                     stream=0) == R.OK
