"""The paged-cache and packed-prompt operators on the GPU against their
definition in 64 bits: head layouts, widths, types, page sizes, lengths from
none to long, strides, NaN in every place that is not a token's, streams, graphs,
and a whole generation (append, prompt attention, decode steps)."""
import math

import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def R():
    from top_kv_span_b200 import build
    build.build()
    from top_kv_span_b200 import reatt
    return reatt


def workspace(R, d):
    # nothing in it has to be zero but the status word
    ws = torch.full((R.reatt_paged_workspace_bytes(d),), 0xA5, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    return ws


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(lens, before=0):
    cu = [before]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


# ------------------------------------------------------------------ decode
def run_decode(R, Hq, Hkv, d, dtype, page, lens, seed=1, std=1.0, wide=0):
    pool = ref.Pool(lens, Hkv, d, page, dtype, seed, std=std)
    gen = torch.Generator().manual_seed(seed + 100)
    B = len(lens)
    q = torch.randn((B, Hq + wide, d), generator=gen).to(dtype)
    dims = R.make_paged_dims(B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=B, page=page,
                             max_pages=pool.max_pages, n_pages=pool.n_pages,
                             q_stride=(Hq + wide) * d)
    ws = workspace(R, dims)
    out = torch.full((B, Hq, d), math.nan, dtype=dtype, device="cuda")
    args = (q.cuda(), pool.k.cuda(), pool.v.cuda(), pool.table.cuda(), ints(lens))
    R.reatt_paged_decode(dims, *args, out, ws)
    torch.cuda.synchronize()
    assert R.reatt_workspace_status(ws) == R.OK
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all()
            continue
        k, v = (x.transpose(0, 1) for x in pool.rows[b])
        o, tol = ref.attend(q[b, :Hq].unsqueeze(1), k, v, torch.tensor([n - 1]))
        ref.check(out[b].cpu(), o[:, 0], tol[:, 0], f"sequence {b} of {n}")
    again = torch.empty_like(out)
    R.reatt_paged_decode(dims, *args, again, ws)
    torch.cuda.synchronize()
    assert torch.equal(again, out)   # no order of atomics decides a result


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 1), (8, 2), (12, 2), (5, 5), (7, 1), (9, 1),
                                    (33, 3), (40, 2), (128, 1)])
def test_decode_heads(R, Hq, Hkv, d, dtype):
    run_decode(R, Hq, Hkv, d, dtype, 16, [33, 1, 0, 150, 16], seed=Hq)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 2, 8, 16, 64, 256, 2048])
def test_decode_pages(R, page, dtype):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 0, 31, 32, 33]
    run_decode(R, 8, 2, 128, dtype, page, lens, seed=page)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)])
def test_decode_one_long_sequence(R, dtype, d):
    run_decode(R, 4, 1, d, dtype, 64, [20011], std=2.0)      # split over every range
    run_decode(R, 12, 2, d, dtype, 128, [0, 9001, 0], std=2.0)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_decode_many_sequences(R, dtype):
    gen = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 90, (1100,), generator=gen).tolist()
    lens[500] = 3000
    run_decode(R, 4, 2, 64, dtype, 32, lens, wide=3)


def test_decode_all_empty(R):
    run_decode(R, 8, 2, 128, BF16, 16, [0, 0, 0])


def test_decode_shared_pages(R):
    """Two sequences with the same prefix pages, read by both."""
    pool = ref.Pool([100, 40], 2, 128, 16, BF16, 9)
    pool.table[1] = pool.table[0]
    q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(1)).to(BF16)
    dims = R.make_paged_dims(B=2, Hq=8, Hkv=2, d=128, dtype=BF16, N=2, page=16,
                             max_pages=pool.max_pages, n_pages=pool.n_pages)
    out = torch.empty((2, 8, 128), dtype=BF16, device="cuda")
    R.reatt_paged_decode(dims, q.cuda(), pool.k.cuda(), pool.v.cuda(), pool.table.cuda(),
                         ints([100, 37]), out, workspace(R, dims))
    k, v = (x.transpose(0, 1) for x in pool.rows[0])
    for b, n in enumerate([100, 37]):
        o, tol = ref.attend(q[b].unsqueeze(1), k[:, :n], v[:, :n], torch.tensor([n - 1]))
        ref.check(out[b].cpu(), o[:, 0], tol[:, 0])


def test_decode_infinite_logit_is_nan_and_stays_in_its_row(R):
    for dtype in (BF16, F32):
        pool = ref.Pool([50, 50], 1, 64, 16, dtype, 4)
        pool.put(0, 7, torch.full((1, 1, 64), math.nan, dtype=dtype), pool.rows[0][1][7:8])
        q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(2)).to(dtype)
        dims = R.make_paged_dims(B=2, Hq=4, Hkv=1, d=64, dtype=dtype, N=2, page=16,
                                 max_pages=pool.max_pages, n_pages=pool.n_pages)
        out = torch.empty((2, 4, 64), dtype=dtype, device="cuda")
        R.reatt_paged_decode(dims, q.cuda(), pool.k.cuda(), pool.v.cuda(), pool.table.cuda(),
                             ints([50, 50]), out, workspace(R, dims))
        assert out[0].isnan().all() and out[1].isfinite().all()


def test_decode_bad_pages_and_lengths_are_left_out(R):
    """The kernels check every id and length themselves: nothing is read outside
    the pools, the status says so, other sequences are untouched by it."""
    for dtype in (BF16, F32):
        pool = ref.Pool([100, 60, 30, 20], 2, 128, 16, dtype, 5)
        table = pool.table.clone()
        table[0, 2] = pool.n_pages
        table[0, 4] = -1
        q = torch.randn((4, 8, 128), generator=torch.Generator().manual_seed(2)).to(dtype)
        dims = R.make_paged_dims(B=4, Hq=8, Hkv=2, d=128, dtype=dtype, N=4, page=16,
                                 max_pages=pool.max_pages, n_pages=pool.n_pages)
        ws = workspace(R, dims)
        out = torch.empty((4, 8, 128), dtype=dtype, device="cuda")

        def call(tab, lens):
            R.reatt_paged_decode(dims, q.cuda(), pool.k.cuda(), pool.v.cuda(), tab.cuda(),
                                 ints(lens), out, ws)
            torch.cuda.synchronize()
            k, v = (x.transpose(0, 1) for x in pool.rows[1])
            o, tol = ref.attend(q[1].unsqueeze(1), k, v, torch.tensor([59]))
            ref.check(out[1].cpu(), o[:, 0], tol[:, 0])
            return R.reatt_workspace_status(ws)

        assert call(table, [100, 60, 30, 20]) == R.EPAGE
        assert call(pool.table, [100, 60, 30, 20]) == R.OK
        assert call(pool.table, [100, 60, -5, 20]) == R.EPAGE
        assert (out[2] == 0).all()
        assert call(pool.table, [100, 60, 30, 1 << 30]) == R.EPAGE
        assert call(pool.table, [100, 60, 30, 20]) == R.OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (16, 2), (40, 2)])
def test_decode_weights_keep_their_precision(R, Hq, Hkv, d):
    """bf16: a weight meets v as a sum of two bf16 terms.  The first is cut off, within
    2^-7 of the weight, the second is off by 2^-8 of that and has 2^-16 of the weight
    added: under 2^-14.  Sums of many values of either sign show it: they are much
    smaller than their terms."""
    lens = [150, 33, 7, 1, 90]
    pool = ref.Pool(lens, Hkv, d, 16, BF16, 71)
    q = torch.randn((len(lens), Hq, d), generator=torch.Generator().manual_seed(72)).to(BF16)
    dims = R.make_paged_dims(B=len(lens), Hq=Hq, Hkv=Hkv, d=d, dtype=BF16, N=len(lens), page=16,
                             max_pages=pool.max_pages, n_pages=pool.n_pages)
    out = torch.empty((len(lens), Hq, d), dtype=BF16, device="cuda")
    R.reatt_paged_decode(dims, q.cuda(), pool.k.cuda(), pool.v.cuda(), pool.table.cuda(), ints(lens),
                         out, workspace(R, dims))
    for b, n in enumerate(lens):
        k, v = (x.transpose(0, 1) for x in pool.rows[b])
        o, tol = ref.attend(q[b].unsqueeze(1), k, v, torch.tensor([n - 1]), p_step=2.0 ** -14)
        ref.check(out[b].cpu(), o[:, 0], tol[:, 0], f"sequence {b} of {n}")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("what", [math.inf, -math.inf])
def test_decode_infinite_value_stays_infinite(R, dtype, what):
    """An infinity in V that the token sees has a weight above zero: the column is that
    infinity; other columns and sequences are as without it."""
    for lens, at in (([50, 50], 7), ([3000, 50], 2999), ([3000, 50], 16)):
        pool = ref.Pool(lens, 2, 128, 16, dtype, 6)
        q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(3)).to(dtype)
        dims = R.make_paged_dims(B=2, Hq=8, Hkv=2, d=128, dtype=dtype, N=2, page=16,
                                 max_pages=pool.max_pages, n_pages=pool.n_pages)
        ws, outs = workspace(R, dims), []
        for _ in range(2):
            out = torch.empty((2, 8, 128), dtype=dtype, device="cuda")
            R.reatt_paged_decode(dims, q.cuda(), pool.k.cuda(), pool.v.cuda(), pool.table.cuda(),
                                 ints(lens), out, ws)
            outs.append(out)
            v = pool.rows[0][1][at:at + 1].clone()
            v[0, :, 5] = what
            pool.put(0, at, pool.rows[0][0][at:at + 1], v)
        clean, got = outs
        assert (got[0, :, 5] == what).all()
        got[0, :, 5] = clean[0, :, 5]
        assert torch.equal(got, clean)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_keys_without_weight_still_count(R, dtype, d):
    """A key whose logit is -inf has weight 0, and 0 times an infinity in its V is NaN,
    whichever keys share its warp or range; a finite V of it adds nothing."""
    for n, none in ((200, 16), (200, 200), (2500, 1300)):
        pool = ref.Pool([n, 60], 1, d, 16, dtype, 7)
        q = torch.rand((2, 4, d), generator=torch.Generator().manual_seed(4)).add(0.1).to(dtype)
        k0, v0 = pool.rows[0]
        pool.put(0, 0, torch.full((none, 1, d), -math.inf, dtype=dtype), v0[:none])
        dims = R.make_paged_dims(B=2, Hq=4, Hkv=1, d=d, dtype=dtype, N=2, page=16,
                                 max_pages=pool.max_pages, n_pages=pool.n_pages)
        ws, outs = workspace(R, dims), []
        for _ in range(2):
            out = torch.empty((2, 4, d), dtype=dtype, device="cuda")
            R.reatt_paged_decode(dims, q.cuda(), pool.k.cuda(), pool.v.cuda(), pool.table.cuda(),
                                 ints([n, 60]), out, ws)
            outs.append(out)
            v = v0[3:4].clone()
            v[0, 0, 9] = math.inf
            pool.put(0, 3, k0[3:4] * -math.inf * k0[3:4].sign(), v)
        clean, got = outs
        assert torch.equal(got[1], clean[1])
        if none == n:
            assert clean[0].isnan().all() and got[0].isnan().all()
            continue
        o, tol = ref.attend(q[0].unsqueeze(1), k0[none:].transpose(0, 1), v0[none:].transpose(0, 1),
                            torch.tensor([n - none - 1]))
        ref.check(clean[0].cpu(), o[:, 0], tol[:, 0])
        assert got[0, :, 9].isnan().all()
        got[0, :, 9] = clean[0, :, 9]
        assert torch.equal(got, clean)


# ------------------------------------------------------------------ append
def run_append(R, Hq, Hkv, d, dtype, page, past, new, base, *, keep_k=True, in_place=False,
               fused=True, before=0, after=0, with_q=True, seed=1):
    gen = torch.Generator().manual_seed(seed)
    N = before + sum(new) + after
    H = Hq + 2 * Hkv if fused else Hq
    row = torch.randn((N, Hq + 2 * Hkv, d), generator=gen).to(dtype)
    pool = ref.Pool([p + n for p, n in zip(past, new)], Hkv, d, page, dtype, seed)
    cu = starts(new, before)
    dev = row.cuda()
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    kw = {}
    if in_place:
        q_rot, k_rot = q, k
        kw = dict(q_rot_stride=q.stride(0), k_rot_stride=k.stride(0))
    else:
        q_rot = torch.full((N, Hq, d), 5.0, dtype=dtype, device="cuda")
        k_rot = torch.full((N, Hkv, d), 5.0, dtype=dtype, device="cuda")
    dims = R.make_paged_dims(B=len(new), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=N, page=page,
                             max_pages=pool.max_pages, n_pages=pool.n_pages, rope_base=base,
                             q_stride=q.stride(0), k_stride=k.stride(0), v_stride=v.stride(0), **kw)
    ws = workspace(R, dims)
    kp, vp = pool.k.cuda(), pool.v.cuda()
    seq = torch.full((len(new),), -9, dtype=torch.int32, device="cuda")
    R.reatt_paged_append(dims, q if with_q else None, k, v, ints(cu), ints(past), pool.table.cuda(),
                         q_rot if with_q else None, k_rot if keep_k else None, kp, vp, seq, ws)
    torch.cuda.synchronize()
    assert R.reatt_workspace_status(ws) == R.OK
    assert seq.tolist() == [p + n for p, n in zip(past, new)]
    want_k, want_v = pool.k.clone(), pool.v.clone()
    tol_k = torch.zeros_like(want_k, dtype=torch.float64)
    want_k = want_k.double()
    for b, (p, n) in enumerate(zip(past, new)):
        if n == 0:
            continue
        r = slice(cu[b], cu[b + 1])
        pos = torch.arange(p, p + n)
        if base:
            yq, tq = ref.rotate(row[r, :Hq], pos, base)
            yk, tk = ref.rotate(row[r, Hq:Hq + Hkv], pos, base)
        else:
            yq, yk = row[r, :Hq].double(), row[r, Hq:Hq + Hkv].double()
            tq, tk = torch.zeros_like(yq), torch.zeros_like(yk)
        if with_q:
            ref.check(q_rot[r].cpu(), yq, tq, f"q of sequence {b}")
        if keep_k:
            ref.check(k_rot[r].cpu(), yk, tk, f"k of sequence {b}")
        where, slot = pool.table[b][pos // page].long(), pos % page
        want_k[where, :, slot] = yk
        tol_k[where, :, slot] = tk
        want_v[where, :, slot] = row[r, Hq + Hkv:]
        if keep_k:   # the same rounding in both places
            assert torch.equal(kp[where.cuda(), :, slot.cuda()], k_rot[r])
    same = torch.nan_to_num(want_k, nan=77.0)
    got = torch.nan_to_num(kp.cpu().double(), nan=77.0)
    assert ((got - same).abs() <= tol_k).all()
    assert torch.equal(torch.nan_to_num(vp.cpu().double(), nan=77.0),
                       torch.nan_to_num(want_v.double(), nan=77.0))
    # rows of no sequence are left as they were
    for r in (slice(0, before), slice(N - after, N)):
        if in_place:
            assert torch.equal(q_rot[r].cpu(), row[r, :Hq])
        else:
            assert (q_rot[r] == 5.0).all() and (k_rot[r] == 5.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (12, 2), (5, 5), (32, 8), (71, 1)])
def test_append_heads(R, Hq, Hkv, d, dtype):
    run_append(R, Hq, Hkv, d, dtype, 16, [0, 5, 31, 100, 7], [3, 0, 18, 1, 40], 5e5, before=2,
               after=3)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 4, 16, 64, 512])
def test_append_pages(R, page, dtype):
    run_append(R, 8, 2, 128, dtype, page, [0, 1, 15, 16, 17, 63, 500], [65, 1, 1, 1, 2, 130, 0], 1e4,
               fused=False)


def test_append_one_token_each(R):
    gen = torch.Generator().manual_seed(8)
    past = torch.randint(0, 300, (333,), generator=gen).tolist()
    run_append(R, 12, 2, 128, BF16, 64, past, [1] * 333, 1e6, keep_k=False)
    run_append(R, 4, 1, 64, F32, 32, [4096], [1], 1e4, keep_k=False)


def test_append_long_prompts(R):
    run_append(R, 8, 2, 128, BF16, 64, [0, 0, 0], [1500, 1, 2001], 5e5, in_place=True, after=1)


def test_append_far_positions(R):
    # positions up to the last one that the table may hold (2^24 tokens)
    far = (1 << 24) - 40
    for dtype in (BF16, F32):
        Hq, Hkv, d, page = 4, 1, 128, 1 << 15
        k = torch.randn((40, Hkv, d), generator=torch.Generator().manual_seed(1)).to(dtype)
        q = torch.randn((40, Hq, d), generator=torch.Generator().manual_seed(2)).to(dtype)
        dims = R.make_paged_dims(B=1, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=40, page=page,
                                 max_pages=512, n_pages=2, rope_base=5e5)
        table = torch.full((1, 512), -1, dtype=torch.int32)
        table[0, 511] = 1
        kp = torch.zeros((2, Hkv, page, d), dtype=dtype, device="cuda")
        vp, qr = torch.zeros_like(kp), torch.empty((40, Hq, d), dtype=dtype, device="cuda")
        ws = workspace(R, dims)
        R.reatt_paged_append(dims, q.cuda(), k.cuda(), k.cuda(), ints([0, 40]), ints([far]),
                             table.cuda(), qr, None, kp, vp, None, ws)
        torch.cuda.synchronize()
        assert R.reatt_workspace_status(ws) == R.OK
        pos = torch.arange(far, far + 40)
        ref.check(qr.cpu(), *ref.rotate(q, pos, 5e5))
        y, t = ref.rotate(k, pos, 5e5)
        ref.check(kp[1, :, page - 40:].cpu().transpose(0, 1), y, t)
        assert torch.equal(vp[1, :, page - 40:].cpu().transpose(0, 1), k)


def test_append_without_rotation_or_queries(R):
    for dtype in (BF16, F32):
        run_append(R, 8, 2, 128, dtype, 16, [3, 0], [20, 33], 0.0)
        run_append(R, 8, 2, 64, dtype, 16, [3, 0], [20, 33], 1e4, with_q=False)


def test_append_nothing_still_writes_lengths(R):
    run_append(R, 8, 2, 128, BF16, 16, [3, 0], [0, 0], 1e4)


def test_append_bad_pages_and_offsets_are_left_out(R):
    pool = ref.Pool([50, 50], 2, 64, 16, BF16, 6)
    x = torch.randn((60, 4, 64), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    k = x[:, :2].contiguous()
    dims = R.make_paged_dims(B=2, Hq=2, Hkv=2, d=64, dtype=BF16, N=60, page=16,
                             max_pages=pool.max_pages, n_pages=pool.n_pages, rope_base=1e4)
    ws = workspace(R, dims)

    def call(cu, past, table):
        kp, vp = pool.k.cuda(), pool.v.cuda()
        R.reatt_paged_append(dims, None, k, k, ints(cu), ints(past), table.cuda(), None, None, kp,
                             vp, None, ws)
        torch.cuda.synchronize()
        changed = (torch.nan_to_num(vp, nan=77.0) != torch.nan_to_num(pool.v.cuda(), nan=77.0))
        return R.reatt_workspace_status(ws), set(changed.flatten(1).any(1).nonzero().flatten().tolist())

    good = pool.table.clone()
    bad = good.clone()
    bad[0, 0] = pool.n_pages + 5
    st, pages = call([0, 30, 60], [0, 0], good)
    assert st == R.OK and pages == set(good[:, :2].flatten().tolist())
    st, pages = call([0, 30, 60], [0, 0], bad)
    assert st == R.EPAGE and pages == set(good[:, :2].flatten().tolist()) - {int(good[0, 0])}
    st, pages = call([0, 30, 60], [0, pool.max_pages * 16 - 3], good)   # past the table
    assert st == R.EPAGE
    st, pages = call([0, 30, 60], [-100, 0], good)
    assert st == R.EPAGE and pages == set(good[1, :2].tolist())
    # offsets that run backwards or past the rows stay inside the rows
    call([0, 90, 60], [0, 0], good)
    call([-20, 10, 1 << 30], [0, 0], good)
    call([50, 20, 10], [0, 0], good)


# ------------------------------------------------------------------ prompts
def run_prompt(R, Hq, Hkv, d, dtype, lens, *, fused=False, before=0, after=0, seed=1, std=1.0,
               q_dev=None):
    gen = torch.Generator().manual_seed(seed)
    N = before + sum(lens) + after
    row = (torch.randn((N, Hq + 2 * Hkv, d), generator=gen) * std).to(dtype)
    cu = starts(lens, before)
    row[:before] = math.nan
    row[cu[-1]:] = math.nan
    dev = row.cuda()
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    dims = R.make_paged_dims(B=len(lens), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=N,
                             q_stride=q.stride(0), k_stride=k.stride(0), v_stride=v.stride(0))
    ws = workspace(R, dims)
    out = torch.full((N, Hq, d), 5.0, dtype=dtype, device="cuda")
    R.reatt_prompt_attend(dims, q, k, v, ints(cu), out, ws)
    torch.cuda.synchronize()
    assert R.reatt_workspace_status(ws) == R.OK
    for b, n in enumerate(lens):
        if n == 0:
            continue
        r = slice(cu[b], cu[b + 1])
        qb, kb, vb = (x.transpose(0, 1) for x in (row[r, :Hq], row[r, Hq:Hq + Hkv], row[r, Hq + Hkv:]))
        o, tol = ref.attend(qb, kb, vb, torch.arange(n))
        ref.check(out[r].cpu(), o.transpose(0, 1), tol.transpose(0, 1), f"sequence {b} of {n}")
    assert (out[:before] == 5.0).all() and (out[cu[-1]:] == 5.0).all()
    again = torch.full_like(out, 5.0)
    R.reatt_prompt_attend(dims, q, k, v, ints(cu), again, ws)
    torch.cuda.synchronize()
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 1), (8, 2), (12, 2), (3, 3), (7, 1), (10, 2),
                                    (33, 1), (128, 1)])
def test_prompt_heads(R, Hq, Hkv, d, dtype):
    run_prompt(R, Hq, Hkv, d, dtype, [5, 0, 130, 1, 67], seed=Hq, before=3, after=5)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 383,
                               384, 385, 511, 513, 700])
def test_prompt_lengths(R, n, dtype):
    run_prompt(R, 4, 1, 128, dtype, [n], seed=n, fused=True)
    run_prompt(R, 2, 2, 64, dtype, [n], seed=n, after=1)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (BF16, 64), (F32, 128), (F32, 64)])
def test_prompt_long(R, dtype, d):
    run_prompt(R, 4, 1, d, dtype, [2500, 17, 1100], std=1.5, fused=True, after=200)


def test_prompt_many_sequences(R):
    gen = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 40, (150,), generator=gen).tolist()
    lens[70] = 600
    for dtype in (BF16, F32):
        run_prompt(R, 6, 2, 64, dtype, lens, before=1)


def test_prompt_all_empty(R):
    run_prompt(R, 4, 1, 128, BF16, [0, 0], after=3)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("operand", ["k", "v"])
@pytest.mark.parametrize("d,Hq", [(128, 4), (64, 1)])
def test_prompt_later_token_reaches_no_earlier_one(R, dtype, what, operand, d, Hq):
    """A NaN or infinity in token t changes no row before t and no other
    sequence; in V it makes row t and the later ones non-finite in that column."""
    lens, t = [70, 200, 90], 133
    gen = torch.Generator().manual_seed(11)
    N = sum(lens)
    q, k, v = (torch.randn((N, h, d), generator=gen).to(dtype) for h in (Hq, 1, 1))
    dims = R.make_paged_dims(B=3, Hq=Hq, Hkv=1, d=d, dtype=dtype, N=N)
    ws, cu = workspace(R, dims), ints(starts(lens))

    def call():
        out = torch.empty((N, Hq, d), dtype=dtype, device="cuda")
        R.reatt_prompt_attend(dims, q.cuda(), k.cuda(), v.cuda(), cu, out, ws)
        return out

    clean = call()
    at = 70 + t
    if operand == "k":
        k[at] = what
    else:
        v[at, 0, 3] = what
    got = call()
    torch.cuda.synchronize()
    assert torch.equal(got[:at], clean[:at])
    assert torch.equal(got[270:], clean[270:])
    if operand == "v":
        hit = got[at:270, :, 3]
        assert hit.isnan().all() if math.isnan(what) else (~hit.isfinite()).all()
        rest = [c for c in range(d) if c != 3]
        assert torch.equal(got[at:270][..., rest], clean[at:270][..., rest])
    elif math.isnan(what):
        assert got[at:270].isnan().all()


def test_prompt_logits_of_minus_infinity(R):
    """A row whose every logit is -inf has no softmax: NaN, as the formula gives."""
    for dtype in (BF16, F32):
        q = torch.ones((2, 1, 64), dtype=dtype, device="cuda")
        k = torch.full((2, 1, 64), -math.inf, dtype=dtype, device="cuda")
        dims = R.make_paged_dims(B=1, Hq=1, Hkv=1, d=64, dtype=dtype, N=2)
        out = torch.empty_like(q)
        R.reatt_prompt_attend(dims, q, k, q, ints([0, 2]), out, workspace(R, dims))
        assert out.isnan().all()


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_of_equal_values_returns_them(R, d):
    """Weights that sum to one give back a value that all tokens share: the sums in fp32
    are off by (m + 8) steps of 2^-23 at most, each, which is far from half a step."""
    lens = [1, 2, 5, 64, 65, 130, 300]
    gen = torch.Generator().manual_seed(81)
    N = sum(lens)
    q, k = (torch.randn((N, h, d), generator=gen).mul(1.5).to(BF16).cuda() for h in (8, 2))
    v = torch.cat([torch.randn((1, 2, d), generator=gen).to(BF16).expand(n, 2, d) for n in lens]).cuda()
    dims = R.make_paged_dims(B=len(lens), Hq=8, Hkv=2, d=d, dtype=BF16, N=N)
    out = torch.empty_like(q)
    R.reatt_prompt_attend(dims, q, k, v, ints(starts(lens)), out, workspace(R, dims))
    assert torch.equal(out, v.repeat_interleave(4, 1))


@pytest.mark.parametrize("d", [64, 128])
def test_prompt_rounded_weights_still_sum_to_one(R, d):
    """bf16: rounding a weight p_t by half a step moves the row by that of p_t (v_t - o)
    only, as the sum takes the rounded weights: little where the values are alike."""
    n, Hq = 150, 4
    gen = torch.Generator().manual_seed(82)
    q, k, v = (torch.randn((n, h, d), generator=gen) for h in (Hq, 1, 1))
    q, k, v = q.to(BF16), k.to(BF16), (4 + v / 32).to(BF16)
    dims = R.make_paged_dims(B=1, Hq=Hq, Hkv=1, d=d, dtype=BF16, N=n)
    out = torch.empty((n, Hq, d), dtype=BF16, device="cuda")
    R.reatt_prompt_attend(dims, q.cuda(), k.cuda(), v.cuda(), ints([0, n]), out, workspace(R, dims))
    qt, kt, vt = (x.transpose(0, 1) for x in (q, k, v))
    o, tol = ref.attend(qt, kt, vt, torch.arange(n), p_step=0.0)
    x = (qt.double() @ kt.double().transpose(-1, -2)) / math.sqrt(d)
    p = torch.softmax(x.masked_fill(torch.ones(n, n).triu(1) > 0, -math.inf), -1)
    apart = torch.stack([(p[:, r, :, None] * (vt.double() - o[:, r, None]).abs()).sum(1)
                         for r in range(n)], 1)
    tol = tol + 2.0 ** -8 * (1 + 2.0 ** -6) * apart
    ref.check(out.cpu(), o.transpose(0, 1), tol.transpose(0, 1))


def test_prompt_malformed_offsets_stay_inside(R):
    q = torch.randn((60, 4, 64), device="cuda").to(BF16)
    k = torch.randn((60, 1, 64), device="cuda").to(BF16)
    for dtype in (BF16, F32):
        dims = R.make_paged_dims(B=2, Hq=4, Hkv=1, d=64, dtype=dtype, N=60)
        ws = workspace(R, dims)
        for cu in ([0, 90, 60], [-20, 10, 1 << 30], [50, 20, 10], [0, 60, 60]):
            out = torch.zeros((60, 4, 64), dtype=dtype, device="cuda")
            R.reatt_prompt_attend(dims, q.to(dtype), k.to(dtype), k.to(dtype), ints(cu), out, ws)
            torch.cuda.synchronize()
            assert R.reatt_workspace_status(ws) == R.OK


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,d,Hq,Hkv,page", [(BF16, 128, 8, 2, 16), (F32, 64, 4, 1, 32),
                                                 (BF16, 64, 6, 1, 64)])
def test_generation(R, dtype, d, Hq, Hkv, page):
    """Ragged prompts are appended (rotated in place in the projection's output)
    and attended; then decode steps append and attend one token each, eagerly and
    from one captured graph; all of it matches causal attention over the whole
    sequences, and a side stream and a dirty workspace change nothing."""
    base, lens, steps = 5e5, [37, 1, 150, 64], 6
    B, N = len(lens), sum(lens)
    gen = torch.Generator().manual_seed(21)
    H = Hq + 2 * Hkv
    rows = [torch.randn((n + steps, H, d), generator=gen).to(dtype) for n in lens]
    pool = ref.Pool([0] * B, Hkv, d, page, dtype, 3, room=max(lens) + steps)
    kp, vp, table = pool.k.cuda(), pool.v.cuda(), pool.table.cuda()
    common = dict(B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, page=page, max_pages=pool.max_pages,
                  n_pages=pool.n_pages, rope_base=base, q_stride=H * d, k_stride=H * d,
                  v_stride=H * d, q_rot_stride=H * d, k_rot_stride=H * d)
    pre, dec = R.make_paged_dims(N=N, **common), R.make_paged_dims(N=B, **common)
    ws = workspace(R, pre)
    x = torch.cat([r[:n] for r, n in zip(rows, lens)]).cuda()
    lens_a, zero = torch.empty(B, dtype=torch.int32, device="cuda"), ints([0] * B)
    out_p = torch.empty((N, Hq, d), dtype=dtype, device="cuda")
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cu_p, cu_d = ints(starts(lens)), ints(list(range(B + 1)))
    R.reatt_paged_append(pre, q, k, v, cu_p, zero, table, q, k, kp, vp, lens_a, ws)
    R.reatt_prompt_attend(pre, q, k, v, cu_p, out_p, ws)
    assert lens_a.tolist() == lens

    def step_rows(i):
        return torch.stack([r[n + i] for r, n in zip(rows, lens)]).cuda()

    y = step_rows(0).clone()
    qd, kd, vd = y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]
    past, now = lens_a.clone(), torch.empty_like(lens_a)
    out_d = torch.empty((B, Hq, d), dtype=dtype, device="cuda")

    def step(stream=None):
        R.reatt_paged_append(dec, qd, kd, vd, cu_d, past, table, qd, kd, kp, vp, now, ws,
                             stream=stream)
        R.reatt_paged_decode(dec, qd, kp, vp, table, now, out_d, ws, stream=stream)
        past.copy_(now)

    k_end, v_end, eager = kp.clone(), vp.clone(), []
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for i in range(steps):
            y.copy_(step_rows(i))
            step()
            eager.append(out_d.clone())
    torch.cuda.synchronize()
    assert past.tolist() == [n + steps for n in lens]
    k_eager, v_eager = kp.clone(), vp.clone()
    kp.copy_(k_end)
    vp.copy_(v_end)
    past.copy_(lens_a)
    graph = torch.cuda.CUDAGraph()
    y.copy_(step_rows(0))
    with torch.cuda.graph(graph):
        step()
    past.copy_(lens_a)
    kp.copy_(k_end)
    vp.copy_(v_end)
    for i in range(steps):
        y.copy_(step_rows(i))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out_d, eager[i])
    same = [torch.nan_to_num(t, nan=77.0) for t in (kp, k_eager, vp, v_eager)]
    assert torch.equal(same[0], same[1]) and torch.equal(same[2], same[3])
    assert R.reatt_workspace_status(ws) == R.OK

    cu = starts(lens)
    for b, n in enumerate(lens):
        pos = torch.arange(n + steps)
        qb, _ = ref.rotate(rows[b][:, :Hq], pos, base)
        kb, _ = ref.rotate(rows[b][:, Hq:Hq + Hkv], pos, base)
        # the rotated rows round to dtype (half a step each, and the rotation's
        # own 2^-20): the logits move by that of |q|.|k|, twice
        o, tol = ref.attend(qb.to(dtype).transpose(0, 1), kb.to(dtype).transpose(0, 1),
                            rows[b][:, Hq + Hkv:].transpose(0, 1), pos)
        moved = 2 * (2 * ref.half_step(dtype) + 2.0 ** -19)
        mag = (qb.abs().transpose(0, 1) @ kb.abs().transpose(0, 1).repeat_interleave(
            Hq // Hkv, 0).transpose(-1, -2)).amax((-1, -2)) / math.sqrt(d)
        tol = tol + 2 * moved * mag[:, None, None] * rows[b][:, Hq + Hkv:].double().abs().max()
        got = torch.cat([out_p[cu[b]:cu[b + 1]], torch.stack([e[b] for e in eager])])
        ref.check(got.cpu(), o.transpose(0, 1), tol.transpose(0, 1), f"sequence {b}")


def test_two_graphs_share_a_workspace(R):
    """Two captured decode calls of different shapes on one workspace, replayed
    in turn, give what each gives alone."""
    cases = []
    for Hq, Hkv, d, dtype, lens in [(8, 2, 128, BF16, [3000, 5, 0, 70]), (4, 4, 64, F32, [900, 31])]:
        pool = ref.Pool(lens, Hkv, d, 16, dtype, 31)
        dims = R.make_paged_dims(B=len(lens), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=len(lens), page=16,
                                 max_pages=pool.max_pages, n_pages=pool.n_pages)
        q = torch.randn((len(lens), Hq, d), device="cuda").to(dtype)
        cases.append((dims, q, pool.k.cuda(), pool.v.cuda(), pool.table.cuda(), ints(lens),
                      torch.empty_like(q)))
    ws = max((workspace(R, c[0]) for c in cases), key=lambda t: t.numel())
    alone, graphs = [], []
    for c in cases:
        R.reatt_paged_decode(*c, workspace(R, c[0]))
        torch.cuda.synchronize()
        alone.append(c[-1].clone())
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            R.reatt_paged_decode(*c, ws)
        graphs.append(g)
    for _ in range(3):
        for c in cases:
            c[-1].fill_(math.nan)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, a in zip(cases, alone):
            assert torch.equal(c[-1], a)


def test_wrong_dtypes_are_refused(R):
    dims = R.make_paged_dims(B=1, Hq=4, Hkv=1, d=64, dtype=BF16, N=1)
    q = torch.zeros((1, 4, 64), dtype=F32, device="cuda")
    ws = workspace(R, dims)
    with pytest.raises(R.ReattError):
        R.reatt_paged_decode(dims, q, q, q, ints([0]), ints([1]), q, ws)
    with pytest.raises(R.ReattError):
        R.reatt_prompt_attend(dims, q.to(BF16), q.to(BF16), q.to(BF16),
                              torch.zeros(2, dtype=torch.int64, device="cuda"), q.to(BF16), ws)


# ------------------------------------------------------------------ large and concurrent
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_pool_offsets_beyond_32_bits(R, dtype):
    """Pools of more than 2^32 elements: the tokens sit in the last pages."""
    Hq, Hkv, d, page, n_pages = 16, 8, 128, 64, 66000      # 4.3e9 elements a pool
    kp = torch.empty((n_pages, Hkv, page, d), dtype=dtype, device="cuda")
    vp = torch.empty_like(kp)
    gen = torch.Generator().manual_seed(41)
    n = 150
    x = torch.randn((n, Hq + 2 * Hkv, d), generator=gen).to(dtype)
    dev = x.cuda()
    q, k, v = dev[:, :Hq], dev[:, Hq:Hq + Hkv], dev[:, Hq + Hkv:]
    table = torch.tensor([[n_pages - 1, n_pages - 3, n_pages - 2]], dtype=torch.int32)
    strides = dict(q_stride=x.stride(0), k_stride=x.stride(0), v_stride=x.stride(0))
    dims = R.make_paged_dims(B=1, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=n, page=page, max_pages=3,
                             n_pages=n_pages, **strides)
    ws, seq = workspace(R, dims), ints([0])
    R.reatt_paged_append(dims, None, k, v, ints([0, n]), ints([0]), table.cuda(), None, None, kp, vp,
                         seq, ws)
    pos = torch.arange(n)
    where, slot = table[0][pos // page].long().cuda(), (pos % page).cuda()
    assert torch.equal(kp[where, :, slot], k) and torch.equal(vp[where, :, slot], v)
    one = R.make_paged_dims(B=1, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=1, page=page, max_pages=3,
                            n_pages=n_pages, **strides)
    out = torch.empty((1, Hq, d), dtype=dtype, device="cuda")
    R.reatt_paged_decode(one, q[n - 1:], kp, vp, table.cuda(), seq, out, ws)
    torch.cuda.synchronize()
    assert R.reatt_workspace_status(ws) == R.OK
    o, tol = ref.attend(x[n - 1:, :Hq].transpose(0, 1), x[:, Hq:Hq + Hkv].transpose(0, 1),
                        x[:, Hq + Hkv:].transpose(0, 1), torch.tensor([n - 1]))
    ref.check(out.cpu(), o.transpose(0, 1), tol.transpose(0, 1))


@pytest.mark.parametrize("dtype,N", [(BF16, 600_064), (F32, 540_672)])
def test_prompt_offsets_beyond_31_bits(R, dtype, N):
    """Packed rows of more than 2^31 elements in q and out; many sequences."""
    Hq, Hkv, d, n = 32, 2, 128, 128
    lens = [n] * (N // n - 1) + [n - 5]
    gen = torch.Generator("cuda").manual_seed(43)
    q = torch.empty((N, Hq, d), dtype=dtype, device="cuda")
    k, v = (torch.randn((N, Hkv, d), generator=gen, device="cuda").to(dtype) for _ in range(2))
    picks = [0, 1, len(lens) // 2, len(lens) - 2, len(lens) - 1]
    cu = starts(lens)
    q.zero_()
    for b in picks:
        q[cu[b]:cu[b + 1]] = torch.randn((lens[b], Hq, d), generator=gen, device="cuda").to(dtype)
    dims = R.make_paged_dims(B=len(lens), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=N)
    out = torch.empty_like(q)
    ws = workspace(R, dims)
    R.reatt_prompt_attend(dims, q, k, v, ints(cu), out, ws)
    torch.cuda.synchronize()
    assert R.reatt_workspace_status(ws) == R.OK
    for b in picks:
        r = slice(cu[b], cu[b + 1])
        o, tol = ref.attend(*(t[r].cpu().transpose(0, 1) for t in (q, k, v)), torch.arange(lens[b]))
        ref.check(out[r].cpu(), o.transpose(0, 1), tol.transpose(0, 1), f"sequence {b}")


def test_calls_on_two_streams_at_once(R):
    """Prompt attention and decode on two streams, each with its own workspace, many
    times over: every result equals the one alone."""
    gen = torch.Generator().manual_seed(51)
    lens = [700, 90, 1300]
    N = sum(lens)
    q, k, v = (torch.randn((N, h, 128), generator=gen).to(BF16).cuda() for h in (8, 2, 2))
    pd = R.make_paged_dims(B=3, Hq=8, Hkv=2, d=128, dtype=BF16, N=N)
    cu = ints(starts(lens))
    pool = ref.Pool([4000, 77, 900], 2, 128, 32, BF16, 5)
    dd = R.make_paged_dims(B=3, Hq=8, Hkv=2, d=128, dtype=BF16, N=3, page=32,
                           max_pages=pool.max_pages, n_pages=pool.n_pages)
    dq = torch.randn((3, 8, 128), generator=gen).to(BF16).cuda()
    args = (dq, pool.k.cuda(), pool.v.cuda(), pool.table.cuda(), ints([4000, 77, 900]))
    w = [workspace(R, pd), workspace(R, pd), workspace(R, dd), workspace(R, dd)]
    want_p, want_d = torch.empty_like(q), torch.empty_like(dq)
    R.reatt_prompt_attend(pd, q, k, v, cu, want_p, w[0])
    R.reatt_paged_decode(dd, *args, want_d, w[2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [[torch.full_like(want_p if i < 2 else want_d, math.nan) for _ in range(10)] for i in range(4)]
    torch.cuda.synchronize()
    for j in range(10):
        for i, s in enumerate(streams):
            if i < 2:
                R.reatt_prompt_attend(pd, q, k, v, cu, outs[i][j], w[i], stream=s)
            else:
                R.reatt_paged_decode(dd, *args, outs[i][j], w[i], stream=s)
    torch.cuda.synchronize()
    for i in range(4):
        for o in outs[i]:
            assert torch.equal(o, want_p if i < 2 else want_d)
        assert R.reatt_workspace_status(w[i]) == R.OK


def test_prompt_captured_with_lengths_that_change(R):
    """Offsets are read when the kernel runs: one captured call, replayed with other
    offsets in the same buffer."""
    for dtype in (BF16, F32):
        gen = torch.Generator().manual_seed(61)
        N = 900
        x = [torch.randn((N, h, 64), generator=gen).to(dtype) for h in (6, 2, 2)]
        q, k, v = (t.cuda() for t in x)
        dims = R.make_paged_dims(B=4, Hq=6, Hkv=2, d=64, dtype=dtype, N=N)
        cu, ws = ints([0, 0, 0, 0, 0]), workspace(R, dims)
        out = torch.empty_like(q)
        R.reatt_prompt_attend(dims, q, k, v, cu, out, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            R.reatt_prompt_attend(dims, q, k, v, cu, out, ws)
        for lens in ([900, 0, 0, 0], [1, 400, 99, 400], [0, 0, 30, 200], [0, 0, 0, 0]):
            cu.copy_(ints(starts(lens)))
            out.fill_(5.0)
            graph.replay()
            torch.cuda.synchronize()
            at = 0
            for n in lens:
                if n:
                    o, tol = ref.attend(*(t[at:at + n].transpose(0, 1) for t in x), torch.arange(n))
                    ref.check(out[at:at + n].cpu(), o.transpose(0, 1), tol.transpose(0, 1))
                at += n
            assert (out[at:] == 5.0).all()
        assert R.reatt_workspace_status(ws) == R.OK


def test_thousands_of_sequences(R):
    """More sequences than any table in a kernel keeps at hand, most of them empty."""
    B = 9000
    lens = [0] * B
    for b, n in ((0, 3), (17, 70), (4095, 1), (4096, 200), (8191, 64), (8998, 33), (8999, 5)):
        lens[b] = n
    run_decode(R, 4, 1, 64, BF16, 16, lens)
    for dtype in (BF16, F32):
        run_prompt(R, 4, 1, 64, dtype, lens, before=2, after=2)
    run_append(R, 4, 1, 64, BF16, 16, [0] * B, lens, 1e4, before=1, after=2)
