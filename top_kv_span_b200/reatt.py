"""Thin ctypes binding of ``libreatt.so`` (the C ABI in ``include/reatt.h``).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  Functions keep the C names; tensors are passed as device pointers,
the stream defaults to torch's current stream.  Missing library -> ImportError
(there is no fallback of any kind).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libreatt.so")

OK, EINVAL, EUNSUPPORTED, ECUDA, ETIMEOUT, EPAGE = 0, 1, 2, 3, 4, 5
F32, BF16 = 0, 1

EXPORTS = ["reatt_status_string", "reatt_num_spans", "reatt_window_max", "reatt_workspace_bytes",
           "reatt_workspace_status", "reatt_score_spans", "reatt_topk", "reatt_gather_rope",
           "reatt_attend", "reatt_step", "reatt_append_kv", "reatt_selftest_bounded_wait",
           "reatt_step_fixed_scratch", "reatt_fixed_scratch_address", "reatt_shard_plan", "reatt_shard_workspace_bytes",
           "reatt_shard_candidates", "reatt_shard_select", "reatt_shard_attend",
           "reatt_merge_partials", "reatt_paged_workspace_bytes", "reatt_paged_append",
           "reatt_paged_decode", "reatt_prompt_attend"]


class reatt_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("C", ctypes.c_int32), ("G", ctypes.c_int32),
                ("L", ctypes.c_int32), ("S", ctypes.c_int32), ("k", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("T", ctypes.c_int64), ("rope_base", ctypes.c_double),
                ("T_cap", ctypes.c_int64)]


class reatt_shard(ctypes.Structure):
    _fields_ = [("t_begin", ctypes.c_int64), ("t_end", ctypes.c_int64),
                ("rows_cap", ctypes.c_int64), ("owns_current", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class reatt_paged_dims(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dtype", ctypes.c_int32), ("page", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("N", ctypes.c_int64), ("n_pages", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("q_rot_stride", ctypes.c_int64),
                ("k_rot_stride", ctypes.c_int64), ("rope_base", ctypes.c_double)]


class ReattError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (status {code})")


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m top_kv_span_b200.build` "
                      "(nvcc, sm_100a); there is no fallback path")

lib = ctypes.CDLL(LIB_PATH)
_vp, _dp = ctypes.c_void_p, ctypes.POINTER(reatt_dims)
lib.reatt_status_string.restype = ctypes.c_char_p
lib.reatt_status_string.argtypes = [ctypes.c_int]
lib.reatt_num_spans.argtypes = [_dp, ctypes.POINTER(ctypes.c_int64)]
lib.reatt_window_max.argtypes = [_dp, ctypes.POINTER(ctypes.c_int64)]
lib.reatt_workspace_bytes.argtypes = [_dp, ctypes.POINTER(ctypes.c_size_t)]
lib.reatt_workspace_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_int), _vp]
lib.reatt_score_spans.argtypes = [_dp, _vp, _vp, _vp, _vp, _vp]
lib.reatt_topk.argtypes = [_dp, _vp, _vp, _vp, _vp]
lib.reatt_gather_rope.argtypes = [_dp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.reatt_attend.argtypes = [_dp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.reatt_step.argtypes = [_dp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.reatt_step_fixed_scratch.argtypes = [_dp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.reatt_selftest_bounded_wait.argtypes = [_vp, ctypes.c_int64, _vp]
lib.reatt_append_kv.argtypes = [_dp, _vp, _vp, _vp, _vp, _vp]
_sp = ctypes.POINTER(reatt_shard)
lib.reatt_shard_plan.argtypes = [_dp, ctypes.c_int32, _sp]
lib.reatt_shard_workspace_bytes.argtypes = [_dp, _sp, ctypes.c_int32,
                                            ctypes.POINTER(ctypes.c_size_t)]
lib.reatt_shard_candidates.argtypes = [_dp, _sp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.reatt_shard_select.argtypes = [_dp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp]
lib.reatt_shard_attend.argtypes = [_dp, _sp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
lib.reatt_merge_partials.argtypes = [_dp, ctypes.c_int32, _vp, _vp, _vp, _vp]
_pp = ctypes.POINTER(reatt_paged_dims)
lib.reatt_paged_workspace_bytes.argtypes = [_pp, ctypes.POINTER(ctypes.c_size_t)]
lib.reatt_paged_append.argtypes = [_pp] + [_vp] * 13
lib.reatt_paged_decode.argtypes = [_pp] + [_vp] * 8
lib.reatt_prompt_attend.argtypes = [_pp] + [_vp] * 7
for _name in EXPORTS[1:]:
    getattr(lib, _name).restype = ctypes.c_int


def status_string(code: int) -> str:
    return lib.reatt_status_string(int(code)).decode()


def make_dims(B, Hq, Hkv, d, C, T, G, L, S, k, dtype, rope_base, T_cap=0) -> reatt_dims:
    if isinstance(dtype, str):
        dtype = F32 if dtype == "f32" else BF16
    elif isinstance(dtype, torch.dtype):
        dtype = F32 if dtype == torch.float32 else BF16
    return reatt_dims(int(B), int(Hq), int(Hkv), int(d), int(C), int(G), int(L), int(S), int(k),
                      int(dtype), int(T), float(rope_base), int(T_cap))


def dims_of(w, **override) -> reatt_dims:
    """Dims of a ``workloads.Workload`` (fields may be overridden)."""
    f = dict(B=w.B, Hq=w.Hq, Hkv=w.Hkv, d=w.d, C=w.C, T=w.T, G=w.G, L=w.L, S=w.S, k=w.k,
             dtype=w.dtype, rope_base=w.rope_base)
    f.update(override)
    return make_dims(**f)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:   # torch.cuda.current_stream() without building a Stream object (3 us)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc, where):
    if rc != OK:
        raise ReattError(rc, where)


def reatt_num_spans(dims) -> int:
    v = ctypes.c_int64()
    _check(lib.reatt_num_spans(ctypes.byref(dims), ctypes.byref(v)), "reatt_num_spans")
    return v.value


def reatt_window_max(dims) -> int:
    v = ctypes.c_int64()
    _check(lib.reatt_window_max(ctypes.byref(dims), ctypes.byref(v)), "reatt_window_max")
    return v.value


def reatt_workspace_bytes(dims) -> int:
    v = ctypes.c_size_t()
    _check(lib.reatt_workspace_bytes(ctypes.byref(dims), ctypes.byref(v)),
           "reatt_workspace_bytes")
    return v.value


def reatt_workspace_status(ws, stream=None) -> int:
    v = ctypes.c_int()
    _check(lib.reatt_workspace_status(_ptr(ws), ctypes.byref(v), _stream(stream)),
           "reatt_workspace_status")
    return v.value


def reatt_score_spans(dims, q, k_cache, span_scores, ws, stream=None, check=True):
    rc = lib.reatt_score_spans(ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(span_scores),
                               _ptr(ws), _stream(stream))
    if check:
        _check(rc, "reatt_score_spans")
    return rc


def reatt_topk(dims, span_scores, sel, ws, stream=None, check=True):
    rc = lib.reatt_topk(ctypes.byref(dims), _ptr(span_scores), _ptr(sel), _ptr(ws),
                        _stream(stream))
    if check:
        _check(rc, "reatt_topk")
    return rc


def reatt_gather_rope(dims, k_cache, v_cache, k_cur, v_cur, sel, k_win, v_win, win_len,
                      stream=None, check=True):
    rc = lib.reatt_gather_rope(ctypes.byref(dims), _ptr(k_cache), _ptr(v_cache), _ptr(k_cur),
                               _ptr(v_cur), _ptr(sel), _ptr(k_win), _ptr(v_win), _ptr(win_len),
                               _stream(stream))
    if check:
        _check(rc, "reatt_gather_rope")
    return rc


def reatt_attend(dims, q, k_win, v_win, win_len, out, ws, stream=None, check=True):
    rc = lib.reatt_attend(ctypes.byref(dims), _ptr(q), _ptr(k_win), _ptr(v_win), _ptr(win_len),
                          _ptr(out), _ptr(ws), _stream(stream))
    if check:
        _check(rc, "reatt_attend")
    return rc


def reatt_step(dims, q, k_cache, v_cache, k_cur, v_cur, sel_out, out, ws, stream=None,
               check=True):
    rc = lib.reatt_step(ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_cur),
                        _ptr(v_cur), _ptr(sel_out), _ptr(out), _ptr(ws), _stream(stream))
    if check:
        _check(rc, "reatt_step")
    return rc


def reatt_append_kv(dims, k_cache, v_cache, k_cur, v_cur, stream=None, check=True):
    rc = lib.reatt_append_kv(ctypes.byref(dims), _ptr(k_cache), _ptr(v_cache), _ptr(k_cur),
                             _ptr(v_cur), _stream(stream))
    if check:
        _check(rc, "reatt_append_kv")
    return rc


def reatt_selftest_bounded_wait(ws, limit_ns, stream=None, check=True):
    """Run one bounded wait that nothing completes; the timeout lands in the
    workspace status word (read it with reatt_workspace_status)."""
    rc = lib.reatt_selftest_bounded_wait(_ptr(ws), int(limit_ns), _stream(stream))
    if check:
        _check(rc, "reatt_selftest_bounded_wait")
    return rc


def reatt_step_fixed_scratch(dims, q, k_cache, v_cache, k_cur, v_cur, sel_out, out, stream=None,
                             check=True):
    """reatt_step with the library's fixed 16 MiB device scratch instead of a
    caller workspace (for callers that cannot allocate device memory)."""
    rc = lib.reatt_step_fixed_scratch(ctypes.byref(dims), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                      _ptr(k_cur), _ptr(v_cur), _ptr(sel_out), _ptr(out),
                                      _stream(stream))
    if check:
        _check(rc, "reatt_step_fixed_scratch")
    return rc


def reatt_fixed_scratch_address() -> int:
    """Device address of the fixed scratch on the current device, for
    reatt_workspace_status (its status word) and the bounded-wait selftest."""
    p = ctypes.c_void_p()
    _check(lib.reatt_fixed_scratch_address(ctypes.byref(p)), "reatt_fixed_scratch_address")
    return int(p.value)


def reatt_shard_plan(dims, n):
    """n contiguous shards of the sequence's tokens (list of reatt_shard)."""
    arr = (reatt_shard * int(n))()
    _check(lib.reatt_shard_plan(ctypes.byref(dims), int(n), arr), "reatt_shard_plan")
    return list(arr)


def reatt_shard_workspace_bytes(dims, shard, n_shards) -> int:
    v = ctypes.c_size_t()
    _check(lib.reatt_shard_workspace_bytes(ctypes.byref(dims), ctypes.byref(shard),
                                           int(n_shards), ctypes.byref(v)),
           "reatt_shard_workspace_bytes")
    return v.value


def reatt_shard_candidates(dims, shard, q, k_cache, cand_score, cand_id, ws, stream=None,
                           check=True):
    rc = lib.reatt_shard_candidates(ctypes.byref(dims), ctypes.byref(shard), _ptr(q),
                                    _ptr(k_cache), _ptr(cand_score), _ptr(cand_id), _ptr(ws),
                                    _stream(stream))
    if check:
        _check(rc, "reatt_shard_candidates")
    return rc


def reatt_shard_select(dims, n_shards, cand_score_all, cand_id_all, sel, ws, stream=None,
                       check=True):
    rc = lib.reatt_shard_select(ctypes.byref(dims), int(n_shards), _ptr(cand_score_all),
                                _ptr(cand_id_all), _ptr(sel), _ptr(ws), _stream(stream))
    if check:
        _check(rc, "reatt_shard_select")
    return rc


def reatt_shard_attend(dims, shard, q, k_cache, v_cache, k_cur, v_cur, sel, part_ml, part_acc,
                       ws, stream=None, check=True):
    rc = lib.reatt_shard_attend(ctypes.byref(dims), ctypes.byref(shard), _ptr(q), _ptr(k_cache),
                                _ptr(v_cache), _ptr(k_cur), _ptr(v_cur), _ptr(sel),
                                _ptr(part_ml), _ptr(part_acc), _ptr(ws), _stream(stream))
    if check:
        _check(rc, "reatt_shard_attend")
    return rc


def reatt_merge_partials(dims, n_parts, part_ml_all, part_acc_all, out, stream=None,
                         check=True):
    rc = lib.reatt_merge_partials(ctypes.byref(dims), int(n_parts), _ptr(part_ml_all),
                                  _ptr(part_acc_all), _ptr(out), _stream(stream))
    if check:
        _check(rc, "reatt_merge_partials")
    return rc


# ----------------------------------------------------------------- paged cache, packed prompts
def make_paged_dims(B, Hq, Hkv, d, dtype, N, page=1, max_pages=1, n_pages=1, rope_base=0.0,
                    q_stride=0, k_stride=0, v_stride=0, q_rot_stride=0,
                    k_rot_stride=0) -> reatt_paged_dims:
    """Dims of the paged calls (strides in elements between packed rows, 0 = dense).
    dtype: "f32", "bf16", the torch dtypes of these, or a reatt_dtype code."""
    codes = {"f32": F32, "bf16": BF16, torch.float32: F32, torch.bfloat16: BF16}
    if not isinstance(dtype, int):
        if dtype not in codes:
            raise ReattError(EUNSUPPORTED, f"make_paged_dims: dtype {dtype}")
        dtype = codes[dtype]
    return reatt_paged_dims(int(B), int(Hq), int(Hkv), int(d), int(dtype), int(page),
                            int(max_pages), 0, int(N), int(n_pages), int(q_stride), int(k_stride),
                            int(v_stride), int(q_rot_stride), int(k_rot_stride), float(rope_base))


def _rows_fit(shape, strides, N, H, d, stride) -> bool:
    """Whether a tensor of this shape and these strides holds N packed rows of H heads of
    d elements, dense, that lie `stride` elements apart.  The inner dimensions make up a
    row; the outer ones, together, are the rows.  A flat buffer only has to be long
    enough."""
    width = H * d
    if N == 0:
        return True
    if len(shape) < 2:
        return len(shape) == 1 and (strides[0] == 1 or shape[0] == 1) and \
            shape[0] >= (N - 1) * stride + width
    held, rows = 1, 0
    for size, step in zip(reversed(shape), reversed(strides)):
        if size == 1:
            continue
        if not rows and step == held and held * size <= stride:
            held *= size
        elif step == stride * (rows or 1):
            rows = (rows or 1) * size
        elif N == 1:     # what lies beyond the one row does not matter
            break
        else:
            return False
    return held >= width and (rows or 1) >= N


def _dense_fit(shape, strides, *want) -> bool:
    """Whether a tensor is dense and holds an array of the shape `want`: as many
    dimensions with the inner ones alike, or a flat or otherwise shaped buffer that is
    long enough."""
    n = 1
    for size, step in zip(reversed(shape), reversed(strides)):
        if size != 1 and step != n:
            return False
        n *= size
    return n >= math.prod(want) and (len(shape) != len(want) or tuple(shape[1:]) == want[1:])


class _PagedPlan:
    """What a call asks of its operands, in the order of its list: dtype, and packed rows
    (N, H, d, stride) or a dense array's shape; of the workspace, last, its bytes.  In
    `fitted`, the dtype, shape and strides (None: dense) with which each one last fitted."""

    def __init__(self, call, d, need):
        want = torch.bfloat16 if d.dtype == BF16 else torch.float32

        def rows(H, stride):
            return want, _rows_fit, (d.N, H, d.d, stride or H * d.d)

        q, out, q_rot = rows(d.Hq, d.q_stride), rows(d.Hq, 0), rows(d.Hq, d.q_rot_stride)
        k, v, k_rot = (rows(d.Hkv, s) for s in (d.k_stride, d.v_stride, d.k_rot_stride))
        pages = want, _dense_fit, (d.n_pages, d.Hkv, d.page, d.d)
        table = torch.int32, _dense_fit, (d.B, d.max_pages)
        cu, each = (torch.int32, _dense_fit, (d.B + 1,)), (torch.int32, _dense_fit, (d.B,))
        self.call, self.ws_bytes = call, need
        self.operands = {
            "reatt_paged_append": (q, k, v, cu, each, table, q_rot, k_rot, pages, pages, each),
            "reatt_paged_decode": (q, pages, pages, table, each, out),
            "reatt_prompt_attend": (q, k, v, cu, out)}[call]
        self.fitted = [(None, None, None)] * (len(self.operands) + 1)

    def check(self, tensors, dev):
        for i, t in enumerate(tensors):
            if t is None or t.__class__ is int:
                continue
            # the workspace may have any dtype
            dt, fit, want = self.operands[i] if i < len(self.operands) else (t.dtype, None, None)
            if t.dtype is not dt or t.get_device() != dev:
                raise ReattError(EINVAL, f"{self.call}: a tensor of {t.dtype} on {t.device}, "
                                         f"wanted {dt} on the current CUDA device")
            if fit is None:
                ok = t.is_contiguous() and t.numel() * t.element_size() >= self.ws_bytes
                what = f"{self.ws_bytes} bytes, dense"
            elif fit is _rows_fit:
                ok = fit(t.shape, t.stride(), *want)
                what = "{} rows of {} x {}, {} elements apart".format(*want)
            else:
                ok, what = fit(t.shape, t.stride(), *want), f"{want}, dense"
            if not ok:
                raise ReattError(EINVAL, f"{self.call}: a tensor of shape {tuple(t.shape)} and "
                                         f"strides {t.stride()}, wanted {what}")
            self.fitted[i] = (dt, t.shape, None if t.is_contiguous() else t.stride())


@functools.lru_cache(maxsize=256)
def _paged_plan(call, raw):
    """The plan for dims of these bytes; None where the call itself refuses them, before it
    looks at any address."""
    d, need = reatt_paged_dims.from_buffer_copy(raw), ctypes.c_size_t()
    if lib.reatt_paged_workspace_bytes(ctypes.byref(d), ctypes.byref(need)) != OK:
        return None
    return _PagedPlan(call, d, need.value)


def _paged_args(call, dims, *tensors):
    """Device addresses of a paged call's operands, its workspace last.  What the library
    cannot see is checked on the way: each tensor lives on the current device, has its
    dtype and holds what the dims say where they say it.  Addresses (int) and None
    pass.  An operand of the shape and strides that last fitted in its place fits; looking
    at all of them anew takes 10 us."""
    plan = _paged_plan(call, bytes(dims))
    if plan is None:
        return [*map(_ptr, tensors)]
    # without an initialised CUDA there is no tensor that could be on the device
    dev, out = torch.cuda.current_device() if torch.cuda.is_initialized() else None, []
    for t, (dt, shape, strides) in zip(tensors, plan.fitted):
        if t is None or t.__class__ is int:
            out.append(t)
        elif t.dtype is dt and t.get_device() == dev and t.shape == shape and (
                t.is_contiguous() if strides is None else t.stride() == strides):
            out.append(t.data_ptr())
        else:
            plan.check(tensors, dev)
            return [*map(_ptr, tensors)]
    return out


def reatt_paged_workspace_bytes(dims) -> int:
    v = ctypes.c_size_t()
    _check(lib.reatt_paged_workspace_bytes(ctypes.byref(dims), ctypes.byref(v)),
           "reatt_paged_workspace_bytes")
    return v.value


def reatt_paged_append(dims, q, k, v, cu_seqlens, past_len, page_table, q_rot, k_rot, k_pages,
                       v_pages, seq_len, ws, stream=None, check=True):
    """Append packed new tokens to the paged caches, k (and q) rotated at their
    positions; q/q_rot, k_rot and seq_len may be None."""
    pq, pk, pv, pcu, ppast, ptab, pqr, pkr, pkp, pvp, plen, pws = _paged_args(
        "reatt_paged_append", dims, q, k, v, cu_seqlens, past_len, page_table, q_rot, k_rot,
        k_pages, v_pages, seq_len, ws)
    rc = lib.reatt_paged_append(ctypes.byref(dims), pq, pk, pv, pcu, ppast, ptab, pqr, pkr, pkp,
                                pvp, plen, pws, _stream(stream))
    if check:
        _check(rc, "reatt_paged_append")
    return rc


def reatt_paged_decode(dims, q, k_pages, v_pages, page_table, seq_len, out, ws, stream=None,
                       check=True):
    """Attention of one new token per sequence over its pages."""
    pq, pkp, pvp, ptab, plen, pout, pws = _paged_args(
        "reatt_paged_decode", dims, q, k_pages, v_pages, page_table, seq_len, out, ws)
    rc = lib.reatt_paged_decode(ctypes.byref(dims), pq, pkp, pvp, ptab, plen, pout, pws,
                                _stream(stream))
    if check:
        _check(rc, "reatt_paged_decode")
    return rc


def reatt_prompt_attend(dims, q, k, v, cu_seqlens, out, ws, stream=None, check=True):
    """Causal attention of whole prompts, packed."""
    pq, pk, pv, pcu, pout, pws = _paged_args("reatt_prompt_attend", dims, q, k, v,
                                             cu_seqlens, out, ws)
    rc = lib.reatt_prompt_attend(ctypes.byref(dims), pq, pk, pv, pcu, pout, pws, _stream(stream))
    if check:
        _check(rc, "reatt_prompt_attend")
    return rc


# ----------------------------------------------------------------- convenience
def alloc_outputs(dims, device="cuda"):
    """Caller-side buffers for one call of every entry point (torch allocates)."""
    NS = reatt_num_spans(dims)
    Wmax = reatt_window_max(dims)
    BH = dims.B * dims.Hkv
    ws_bytes = reatt_workspace_bytes(dims)
    return dict(
        span_scores=torch.empty((dims.B, dims.Hkv, NS), dtype=torch.float32, device=device),
        sel=torch.empty((dims.B, dims.Hkv, dims.k), dtype=torch.int32, device=device),
        k_win=torch.zeros((dims.B, dims.Hkv, Wmax, dims.d), dtype=torch.float32, device=device),
        v_win=torch.zeros((dims.B, dims.Hkv, Wmax, dims.d), dtype=torch.float32, device=device),
        win_len=torch.empty((dims.B, dims.Hkv), dtype=torch.int32, device=device),
        out=torch.empty((dims.B, dims.Hq, dims.C, dims.d), dtype=torch.float32, device=device),
        ws=torch.zeros(max(ws_bytes, 256), dtype=torch.uint8, device=device),
    )
