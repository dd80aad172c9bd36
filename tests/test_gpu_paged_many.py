"""The paged operators with as many sequences as they take: results against plain torch
and the definition in 64 bits, and times that grow with the tokens, not with tokens times
sequences."""
import math

import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_paged import BF16, F32, R, ints, starts, workspace  # noqa: F401 (R is a fixture)
from tests.test_gpu_paged_steady import guarded, outside_is

pytestmark = pytest.mark.gpu

MOST = 65536


def best_us(call, n=7):
    times = []
    for _ in range(n):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return min(times)


def random_lengths(B, most, seed):
    return torch.randint(0, most + 1, (B,), generator=torch.Generator().manual_seed(seed)).tolist()


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("B", [256, 257, 1000, 8191, 8193, MOST])
@pytest.mark.parametrize("most", [1, 3])
def test_append_finds_every_token_its_sequence(R, B, most):
    """Un-rotated rows land in the slots that the table names, wherever their sequence is
    among the offsets; empty sequences lie in between."""
    lens = random_lengths(B, most, B)
    cu, N, page, Hkv, d = starts(lens, 2), sum(lens) + 5, 4, 1, 64
    gen = torch.Generator("cuda").manual_seed(1)
    k, v = (torch.randn((N, Hkv, d), generator=gen, device="cuda").to(BF16) for _ in range(2))
    past = torch.randint(0, page * 2 - 3, (B,), generator=torch.Generator().manual_seed(2)).int()
    table = torch.randperm(2 * B, generator=torch.Generator().manual_seed(3)).int().view(B, 2)
    dims = R.make_paged_dims(B=B, Hq=1, Hkv=Hkv, d=d, dtype=BF16, N=N, page=page, max_pages=2,
                             n_pages=2 * B)
    ws = workspace(R, dims)
    pools = [torch.full((2 * B, Hkv, page, d), 7.0, dtype=BF16, device="cuda") for _ in range(2)]
    want = [p.clone() for p in pools]
    now = torch.empty(B, dtype=torch.int32, device="cuda")
    R.reatt_paged_append(dims, None, k, v, ints(cu), past.cuda(), table.cuda(), None, None, *pools,
                         now, ws)
    n = torch.tensor(lens)
    seq = torch.repeat_interleave(torch.arange(B), n)
    row = torch.arange(len(seq)) + cu[0]
    pos = past[seq] + (row - torch.tensor(cu)[seq])
    where, slot = table[seq, (pos // page).long()].long().cuda(), (pos % page).cuda()
    for w, x in zip(want, (k, v)):
        w[where, :, slot.long()] = x[row.cuda()]
    torch.cuda.synchronize()
    assert R.reatt_workspace_status(ws) == R.OK
    assert torch.equal(pools[0], want[0]) and torch.equal(pools[1], want[1])
    assert torch.equal(now.cpu(), past + n.int())


def test_append_time_does_not_grow_with_the_sequences(R):
    """65536 tokens of as many sequences or of 64: the same bytes, and about the same time
    (ten times as much when every token's warp read all offsets)."""
    N, Hq, Hkv, d, page = MOST, 8, 2, 64, 16
    q, k = (torch.zeros((N, h, d), dtype=BF16, device="cuda") for h in (Hq, Hkv))
    pools = [torch.zeros((N, Hkv, page, d), dtype=BF16, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(q), torch.empty_like(k)]
    times = []
    for B in (64, MOST):
        dims = R.make_paged_dims(B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=BF16, N=N, page=page,
                                 max_pages=N // B // page + 1, n_pages=N, rope_base=1e4)
        cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * (N // B)
        past, now = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))
        table = torch.arange(B * dims.max_pages, dtype=torch.int32, device="cuda").view(B, -1) % N
        ws = workspace(R, dims)
        times.append(best_us(lambda: R.reatt_paged_append(dims, q, k, k, cu, past, table, *outs,
                                                          *pools, now, ws)))
        assert R.reatt_workspace_status(ws) == R.OK
    assert times[1] < 4 * times[0], times


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hkv,d", [(n, *h) for n in (40, 41, 300, 301, 1000)
                                         for h in ((8, 2, 64), (8, 2, 128), (16, 1, 64), (9, 1, 128))] +
                         [(9001, 8, 2, 64), (9001, 32, 8, 128), (MOST, 8, 2, 64)])
def test_decode_passes_over_empty_sequences(R, dtype, B, Hq, Hkv, d):
    """A batch of fixed size with few live sequences, runs of empty ones of every length
    between them, more tiles than CTAs: every live one is found, the others are zeros."""
    page = 128
    gen = torch.Generator().manual_seed(B)
    gaps = [0, 0, 1, 30, 31, 32, 33, 63, 64, 65, 200, 7000]
    live, at = [], 0
    for g in gaps:
        at += g
        if at >= B:
            break
        live.append(at)
        at += 1
    live = sorted({*live, B - 1})
    n = {b: 3000 + 100 * i for i, b in enumerate(live)}
    n[live[1]] = 1
    pool = ref.Pool([n[b] for b in live], Hkv, d, page, dtype, 61)
    table = torch.full((B, pool.max_pages), -7, dtype=torch.int32)
    table[live] = pool.table
    lens = torch.zeros(B, dtype=torch.int32)
    lens[live] = torch.tensor([n[b] for b in live], dtype=torch.int32)
    q = torch.randn((B, Hq, d), generator=gen).to(dtype)
    dims = R.make_paged_dims(B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=B, page=page,
                             max_pages=pool.max_pages, n_pages=pool.n_pages)
    ws = workspace(R, dims)
    out = torch.full((B, Hq, d), math.nan, dtype=dtype, device="cuda")
    R.reatt_paged_decode(dims, q.cuda(), pool.k.cuda(), pool.v.cuda(), table.cuda(), lens.cuda(),
                         out, ws)
    torch.cuda.synchronize()
    assert R.reatt_workspace_status(ws) == R.OK
    got = out[live].cpu()
    out[live] = 0
    assert (out == 0).all()
    for i, b in enumerate(live):
        k, v = (x.transpose(0, 1) for x in pool.rows[i])
        o, tol = ref.attend(q[b].unsqueeze(1), k, v, torch.tensor([n[b] - 1]))
        ref.check(got[i], o[:, 0], tol[:, 0], f"sequence {b}")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_decode_time_does_not_grow_with_a_gap(R, dtype):
    """Two live sequences among 65536, side by side or at either end: the same tiles, and
    about the same time (66 times as much when the gap was walked one by one)."""
    B, Hq, Hkv, d, page, n = MOST, 32, 8, 128, 128, 8000
    need = -(-n // page)
    q = torch.zeros((B, Hq, d), dtype=dtype, device="cuda")
    pools = [torch.zeros((2 * need, Hkv, page, d), dtype=dtype, device="cuda") for _ in range(2)]
    dims = R.make_paged_dims(B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=B, page=page, max_pages=need,
                             n_pages=2 * need)
    ws, out, times = workspace(R, dims), torch.empty_like(q), []
    table = torch.zeros((B, need), dtype=torch.int32, device="cuda")
    for live in ([0, 1], [0, B - 1]):
        table[live] = torch.arange(2 * need, dtype=torch.int32, device="cuda").view(2, need)
        lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        lens[live] = ints([n, n - 3000])   # so that some CTA's share holds the gap
        times.append(best_us(lambda: R.reatt_paged_decode(dims, q, *pools, table, lens, out, ws)))
        assert R.reatt_workspace_status(ws) == R.OK
    assert times[1] < 4 * times[0], times


# ------------------------------------------------------------------ prompts
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hkv,d", [(128, 4, 1, 64), (129, 8, 2, 64), (512, 6, 2, 128), (513, 6, 2, 128),
                                        (1024, 3, 1, 64), (1025, 8, 8, 64), (5000, 8, 2, 128), (MOST, 4, 1, 64)])
def test_prompts_of_many_sequences(R, dtype, B, Hq, Hkv, d):
    """Prompts of 0 to 3 tokens, a few of hundreds among them, first and last too: every row
    against the definition, rows of no sequence left alone."""
    lens = random_lengths(B, 3, B + d)
    long = {0: 300, 1: 65, B // 3: 1000, B // 2: 64, B - 2: 129, B - 1: 513}
    for b, n in long.items():
        lens[b] = n
    cu, N, g = starts(lens, 3), sum(lens) + 7, Hq // Hkv
    gen = torch.Generator("cuda").manual_seed(B)
    row = torch.randn((N, Hq + 2 * Hkv, d), generator=gen, device="cuda").to(dtype)
    row[:3] = math.nan
    row[cu[-1]:] = math.nan
    q, k, v = row[:, :Hq], row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:]
    s = row.stride(0)
    dims = R.make_paged_dims(B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=N, q_stride=s, k_stride=s,
                             v_stride=s)
    ws = workspace(R, dims)
    outs = [torch.full((N, Hq, d), 5.0, dtype=dtype, device="cuda") for _ in range(2)]
    for out in outs:
        R.reatt_prompt_attend(dims, q, k, v, ints(cu), out, ws)
    torch.cuda.synchronize()
    assert R.reatt_workspace_status(ws) == R.OK
    assert torch.equal(*outs)
    out = outs[0]
    assert (out[:3] == 5.0).all() and (out[cu[-1]:] == 5.0).all()
    for b in long:
        r = slice(cu[b], cu[b + 1])
        o, tol = ref.attend(*(x[r].transpose(0, 1) for x in (q, k, v)),
                            torch.arange(lens[b], device="cuda"))
        ref.check(out[r].cpu(), o.transpose(0, 1).cpu(), tol.transpose(0, 1).cpu(), f"sequence {b}")
    # the short ones of one length at a time: [H, sequences * n, ...] as a batch of sequences
    n_of, at = torch.tensor(lens), torch.tensor(cu)
    short = torch.ones(B, dtype=torch.bool)
    short[list(long)] = False
    for n in (1, 2, 3):
        rows = (at[:-1][short & (n_of == n)][:, None] + torch.arange(n)).cuda()   # [S, n]
        for r0 in range(0, rows.shape[0], 4096):
            r = rows[r0:r0 + 4096]
            S = r.shape[0]
            flat = [x[r].transpose(1, 2).reshape(-1, n, d) for x in (q, k, v)]    # [S * H, n, d]
            o, tol = ref.attend(*flat, torch.arange(n, device="cuda"))
            back = [x.reshape(S, Hq, n, d).transpose(1, 2).cpu() for x in (o, tol)]
            ref.check(out[r].cpu(), *back, f"sequences of {n}")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_prompt_time_grows_with_the_sequences_not_their_square(R, dtype):
    """One-token prompts: 65536 of them take about 16 times as long as 4096 (400 times when
    every block passed over all sequences)."""
    Hq, Hkv, d, times = 8, 2, 64, []
    for B in (4096, MOST):
        q, k = (torch.zeros((B, h, d), dtype=dtype, device="cuda") for h in (Hq, Hkv))
        dims = R.make_paged_dims(B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=B)
        ws, out = workspace(R, dims), torch.empty_like(q)
        cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        times.append(best_us(lambda: R.reatt_prompt_attend(dims, q, k, k, cu, out, ws), 3))
        assert R.reatt_workspace_status(ws) == R.OK
    assert times[1] < 40 * times[0], times


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B", [129, 300, 4000])
def test_malformed_offsets_of_many_sequences(R, dtype, B):
    """Offsets in any order, before and behind the rows too, overlapping: nothing outside
    the rows is written, and no row of q, k or v from outside (all NaN) reaches a result."""
    N, Hq, Hkv, d, page = 500, 4, 2, 64, 512
    rgen = torch.Generator().manual_seed(B)
    gen = torch.Generator("cuda").manual_seed(B)
    rows = []
    for h in (Hq, Hkv, Hkv):
        _, t = guarded((N, h, d), dtype, math.nan)
        t.copy_(torch.randn((N, h, d), generator=gen, device="cuda"))
        rows.append(t)
    dims = R.make_paged_dims(B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=N, page=page, max_pages=1,
                             n_pages=B, rope_base=1e4)
    ws = workspace(R, dims)
    table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    past = torch.zeros(B, dtype=torch.int32, device="cuda")
    for spread in (N + 50, 1 << 31, 3):
        cu = torch.randint(-spread, spread, (B + 1,), generator=rgen).int().cuda()
        big, out = guarded((N, Hq, d), dtype, 5.0)
        R.reatt_prompt_attend(dims, *rows, cu, out, ws)
        torch.cuda.synchronize()
        assert R.reatt_workspace_status(ws) == R.OK
        assert outside_is(big, N, 5.0) and out.isfinite().all()
        bufs = [guarded(s, dtype, 5.0) for s in ((N, Hq, d), (N, Hkv, d), (B, Hkv, page, d),
                                                 (B, Hkv, page, d))]
        R.reatt_paged_append(dims, *rows, cu, past, table, *(b[1] for b in bufs), None, ws)
        torch.cuda.synchronize()
        R.reatt_workspace_status(ws)
        for big, t in bufs:
            assert outside_is(big, t.shape[0], 5.0) and t.isfinite().all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_prompts_of_many_sequences_captured(R, dtype):
    """One captured call, replayed with other offsets, beside a decode on the same workspace."""
    B, Hq, Hkv, d, N = 3000, 4, 2, 64, 4000
    gen = torch.Generator("cuda").manual_seed(7)
    q, k, v = (torch.randn((N, h, d), generator=gen, device="cuda").to(dtype) for h in (Hq, Hkv, Hkv))
    dims = R.make_paged_dims(B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=N)
    one = R.make_paged_dims(B=B, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=B, page=8, max_pages=1, n_pages=B)
    pools = [torch.randn((B, Hkv, 8, d), generator=gen, device="cuda").to(dtype) for _ in range(2)]
    table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    seq = torch.randint(0, 9, (B,), generator=torch.Generator().manual_seed(8)).int().cuda()
    ws, cu, out = workspace(R, dims), ints([0] * (B + 1)), torch.empty_like(q)
    dec = torch.empty((B, Hq, d), dtype=dtype, device="cuda")
    want_dec = torch.empty_like(dec)
    R.reatt_paged_decode(one, q[:B], *pools, table, seq, want_dec, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.reatt_prompt_attend(dims, q, k, v, cu, out, ws)
        R.reatt_paged_decode(one, q[:B], *pools, table, seq, dec, ws)
    for lens in (random_lengths(B, 2, 1), [0] * (B - 1) + [N], [1] * B, [N - 2] + [0] * (B - 2) + [2],
                 [0] * B):
        while sum(lens) > N:
            lens.pop()
            lens.insert(0, 0)
        cu.copy_(ints(starts(lens)))
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert R.reatt_workspace_status(ws) == R.OK
        assert torch.equal(dec, want_dec)
        # the same prompts alone, without the empty ones: few enough to be found without a list
        some = [(b, n) for b, n in enumerate(lens) if n]
        at = starts(lens)
        for c in range(0, len(some), 100):
            part = some[c:c + 100]
            lo, hi = at[part[0][0]], at[part[-1][0] + 1]
            few = R.make_paged_dims(B=len(part), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=hi - lo)
            alone = torch.empty((hi - lo, Hq, d), dtype=dtype, device="cuda")
            R.reatt_prompt_attend(few, q[lo:hi], k[lo:hi], v[lo:hi], ints(starts([n for _, n in part])),
                                  alone, workspace(R, few))
            assert torch.equal(out[lo:hi], alone)
        assert (out[at[-1]:] == 5.0).all()
