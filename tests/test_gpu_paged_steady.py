"""The paged operators in their steady state: decode ranges of many tiles of a unit whose
maximum moves on the way, prompt CTAs that take many blocks of different lengths one
after the other, malformed offsets between guarded rows, infinite logits.  Against the
definition in 64 bits, or bit for bit against an equal call."""
import math

import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_paged import BF16, F32, R, ints, starts, workspace  # noqa: F401 (R is a fixture)

pytestmark = pytest.mark.gpu


def resident_ctas():
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count   # of a decode, at most


# ------------------------------------------------------------------ decode
def uneven_keys(n, Hkv, d, dtype, u, gen):
    """Keys whose logits under the query u stand near 0 but for a few high ones, more than
    2^8 in weight over the others (5.6 in the exponent), and as many low ones, high under
    -u: the many and the few add up to sums of one size.  An odd n has a few keys
    another such step higher in its later half."""
    c = torch.zeros(n)
    c[torch.randperm(n, generator=gen)[:n // 250]] = 6.3
    c[torch.randperm(n, generator=gen)[:n // 250]] = -6.3
    if n % 2:
        late = n - 1 - torch.randperm(n // 2, generator=gen)[:2 + n // 4000]
        c[late] = torch.tensor([12.5, -12.5]).repeat(len(late))[:len(late)]
    k = c[:, None, None] * u / math.sqrt(d) + torch.randn((n, Hkv, d), generator=gen) / 2
    return k.to(dtype)


@pytest.mark.parametrize("dtype,d,Hq,Hkv,lens", [
    (BF16, 128, 32, 8, [3001, 2500, 4096, 17, 0, 3333, 2600, 1999, 3700]),
    (BF16, 64, 32, 8, [6001, 5500, 8000, 17, 0, 5333, 3600, 81, 5003]),
    (BF16, 128, 40, 2, [20011, 0, 9001, 333]),       # two chunks: 16 heads and 4
    (BF16, 64, 16, 1, [50003, 60001]),               # one unit of 16 heads a sequence
    (BF16, 128, 5, 1, [60007]),
    (F32, 128, 16, 4, [1501, 2500, 2048, 17, 0, 1333, 1600]),
    (F32, 64, 24, 2, [9001, 0, 5000, 12345]),        # two chunks: 8 heads and 4
])
def test_decode_ranges_of_many_tiles(R, dtype, d, Hq, Hkv, lens):
    gen = torch.Generator().manual_seed(Hq + d)
    u = torch.randint(0, 2, (d,), generator=gen).mul(2).sub(1).float()
    pool = ref.Pool(lens, Hkv, d, 64, dtype, 17)
    for b, n in enumerate(lens):
        if n:
            pool.rows[b] = (uneven_keys(n, Hkv, d, dtype, u, gen), pool.rows[b][1])
            pool.put(b, 0, *pool.rows[b])
    # a tile: 4096 bytes of K for each of five warps; a unit: 16 query heads, or 8 in fp32
    size, most = (2, 16 if Hq // Hkv > 8 else 8) if dtype == BF16 else (4, 8 if Hq // Hkv > 4 else 4)
    tile = 5 * 4096 // (d * size)
    units = Hkv * -(-(Hq // Hkv) // most)
    assert sum(-(-n // tile) for n in lens) * units > 2 * resident_ctas()
    q = torch.randn((len(lens), Hq, d), generator=gen) / 4
    q = (q + u * torch.tensor([1.0, -1.0]).repeat(Hq)[:Hq, None]).to(dtype)
    dims = R.make_paged_dims(B=len(lens), Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=len(lens), page=64,
                             max_pages=pool.max_pages, n_pages=pool.n_pages)
    ws = workspace(R, dims)
    args = (q.cuda(), pool.k.cuda(), pool.v.cuda(), pool.table.cuda(), ints(lens))
    out = torch.full((len(lens), Hq, d), math.nan, dtype=dtype, device="cuda")
    R.reatt_paged_decode(dims, *args, out, ws)
    torch.cuda.synchronize()
    assert R.reatt_workspace_status(ws) == R.OK
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all()
            continue
        k, v = (x.cuda().transpose(0, 1) for x in pool.rows[b])
        o, tol = ref.attend(q[b].cuda().unsqueeze(1), k, v, torch.tensor([n - 1], device="cuda"),
                            p_step=2.0 ** -14)
        ref.check(out[b].cpu(), o[:, 0].cpu(), tol[:, 0].cpu(), f"sequence {b} of {n}")
    again = torch.empty_like(out)
    R.reatt_paged_decode(dims, *args, again, ws)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,at", [(50, 7), (700, 0), (9000, 8765)])
def test_decode_infinite_logits(R, dtype, n, at):
    """A logit of +inf makes its rows NaN (inf - inf), as the formula does; one of -inf has
    no weight.  K holds one infinity, q a positive element beside it in the even heads
    and a negative one in the odd heads."""
    d, Hq = 128, 4
    pool = ref.Pool([n, 60], 1, d, 16, dtype, 23)
    gen = torch.Generator().manual_seed(24)
    q = torch.randn((2, Hq, d), generator=gen)
    q[:, :, 11] = torch.tensor([0.5, -0.5, 0.25, -2.0])
    q = q.to(dtype)
    k = pool.rows[0][0][at:at + 1].clone()
    k[0, 0, 11] = math.inf
    pool.put(0, at, k, pool.rows[0][1][at:at + 1])
    dims = R.make_paged_dims(B=2, Hq=Hq, Hkv=1, d=d, dtype=dtype, N=2, page=16,
                             max_pages=pool.max_pages, n_pages=pool.n_pages)
    out = torch.empty((2, Hq, d), dtype=dtype, device="cuda")
    R.reatt_paged_decode(dims, q.cuda(), pool.k.cuda(), pool.v.cuda(), pool.table.cuda(),
                         ints([n, 60]), out, workspace(R, dims))
    assert out[0, 0::2].isnan().all()
    keep = [t for t in range(n) if t != at]
    k, v = (x[keep].transpose(0, 1) for x in pool.rows[0])
    o, tol = ref.attend(q[0].unsqueeze(1), k, v, torch.tensor([n - 2]))
    ref.check(out[0, 1::2].cpu(), o[1::2, 0], tol[1::2, 0])
    k, v = (x.transpose(0, 1) for x in pool.rows[1])
    o, tol = ref.attend(q[1].unsqueeze(1), k, v, torch.tensor([59]))
    ref.check(out[1].cpu(), o[:, 0], tol[:, 0])


# ------------------------------------------------------------------ prompts
# heads, widths and prompts that give every CTA several blocks of different step counts
MANY = [(32, 8, 128, [1, 700, 2, 63, 1500, 64, 65, 0, 300, 129, 1000, 31, 128, 517]),
        (32, 8, 64, [400, 1, 1, 1200, 90, 255, 256, 257, 0, 0, 800, 5, 640]),
        (30, 10, 128, [333, 84, 85, 86, 1400, 168, 169, 1, 42, 43, 900]),
        (24, 24, 64, [1100, 7, 128, 129, 256, 900, 257, 1, 1300, 500]),
        (48, 8, 128, [600, 42, 41, 43, 3, 1200, 21, 777, 84])]


def prompts(Hq, Hkv, d, lens, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    N = sum(lens)
    row = torch.randn((N, Hq + 2 * Hkv, d), generator=gen, device="cuda").to(BF16)
    return row, row[:, :Hq], row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:]


def blocks(Hq, Hkv, lens):
    per = 2 * (128 // (Hq // Hkv))
    return Hkv * sum(-(-n // per) for n in lens)


@pytest.mark.parametrize("Hq,Hkv,d,lens", MANY)
def test_prompt_ctas_of_many_blocks(R, Hq, Hkv, d, lens):
    assert blocks(Hq, Hkv, lens) > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    row, q, k, v = prompts(Hq, Hkv, d, lens, 31)
    N = sum(lens)
    s = row.stride(0)
    dims = R.make_paged_dims(B=len(lens), Hq=Hq, Hkv=Hkv, d=d, dtype=BF16, N=N, q_stride=s,
                             k_stride=s, v_stride=s)
    ws, cu = workspace(R, dims), starts(lens)
    outs = []
    for _ in range(3):
        out = torch.full((N, Hq, d), math.nan, dtype=BF16, device="cuda")
        R.reatt_prompt_attend(dims, q, k, v, ints(cu), out, ws)
        outs.append(out)
    torch.cuda.synchronize()
    assert R.reatt_workspace_status(ws) == R.OK
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    for b, n in enumerate(lens):
        if n:
            r = slice(cu[b], cu[b + 1])
            o, tol = ref.attend(*(x[r].transpose(0, 1) for x in (q, k, v)),
                                torch.arange(n, device="cuda"))
            ref.check(outs[0][r].cpu(), o.transpose(0, 1).cpu(), tol.transpose(0, 1).cpu(),
                      f"sequence {b} of {n}")


@pytest.mark.parametrize("Hq,Hkv,d,lens", MANY)
def test_prompt_values_behind_the_mask_in_many_blocks(R, Hq, Hkv, d, lens):
    """NaN and infinities in V of tokens all over the list of blocks, one or two in each
    prompt and KV head: the rows that see one have it in its column, everything else is as
    without it, bit for bit."""
    row, q, k, v = prompts(Hq, Hkv, d, lens, 37)
    N, s, g = sum(lens), row.stride(0), Hq // Hkv
    dims = R.make_paged_dims(B=len(lens), Hq=Hq, Hkv=Hkv, d=d, dtype=BF16, N=N, q_stride=s,
                             k_stride=s, v_stride=s)
    ws, cu = workspace(R, dims), starts(lens)
    clean, got = torch.empty((N, Hq, d), dtype=BF16, device="cuda"), None
    R.reatt_prompt_attend(dims, q, k, v, ints(cu), clean, ws)
    gen = torch.Generator().manual_seed(38)
    hit = torch.zeros((N, Hq, d), dtype=torch.bool)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            for _ in range(0 if n == 0 else 1 + (b + h) % 2):
                t, c = (int(torch.randint(0, x, (1,), generator=gen)) for x in (n, d))
                v[cu[b] + t, h, c] = (math.nan, math.inf, -math.inf)[(b + h) % 3]
                hit[cu[b] + t:cu[b + 1], h * g:(h + 1) * g, c] = True
    for _ in range(2):
        got = torch.empty_like(clean)
        R.reatt_prompt_attend(dims, q, k, v, ints(cu), got, ws)
    torch.cuda.synchronize()
    assert R.reatt_workspace_status(ws) == R.OK
    hit = hit.cuda()
    assert not got[hit].isfinite().any()
    assert torch.equal(got[~hit], clean[~hit])


# ------------------------------------------------------------------ malformed offsets
BAD = [[0, 90, 60, 60], [-20, 10, 30, 1 << 30], [50, 20, 10, 0], [0, 50, 20, 60], [60, 0, 60, 0],
       [-(1 << 31), 0, (1 << 31) - 1, -1], [70, 80, 90, 95]]


def guarded(shape, dtype, fill, room=64):
    """A tensor of this shape between `room` rows of the same fill on either side."""
    big = torch.full((shape[0] + 2 * room, *shape[1:]), fill, dtype=dtype, device="cuda")
    return big, big[room:room + shape[0]]


def outside_is(big, n, fill, room=64):
    both = torch.cat([big[:room], big[room + n:]])
    return bool(both.isnan().all() if math.isnan(fill) else (both == fill).all())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_malformed_offsets_between_guards(R, dtype, d):
    """Offsets that run backwards or leave the rows: nothing outside the rows is written,
    and no row of q, k or v from outside (all NaN) reaches a result."""
    N, Hq, Hkv = 60, 4, 2
    gen = torch.Generator("cuda").manual_seed(41)
    rows = []
    for h in (Hq, Hkv, Hkv):
        _, t = guarded((N, h, d), dtype, math.nan)
        t.copy_(torch.randn((N, h, d), generator=gen, device="cuda"))
        rows.append(t)
    dims = R.make_paged_dims(B=3, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=N)
    ws = workspace(R, dims)
    for cu in BAD:
        big, out = guarded((N, Hq, d), dtype, 5.0)
        R.reatt_prompt_attend(dims, *rows, ints(cu), out, ws)
        torch.cuda.synchronize()
        assert R.reatt_workspace_status(ws) == R.OK
        assert outside_is(big, N, 5.0) and out.isfinite().all(), cu


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_append_malformed_offsets_between_guards(R, dtype):
    N, Hq, Hkv, d, page = 60, 4, 2, 64, 16
    gen = torch.Generator("cuda").manual_seed(43)
    rows = []
    for h in (Hq, Hkv, Hkv):
        _, t = guarded((N, h, d), dtype, math.nan)
        t.copy_(torch.randn((N, h, d), generator=gen, device="cuda"))
        rows.append(t)
    table = torch.randperm(12, generator=torch.Generator().manual_seed(44)).int().view(3, 4).cuda()
    dims = R.make_paged_dims(B=3, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, N=N, page=page, max_pages=4,
                             n_pages=12, rope_base=1e4)
    ws = workspace(R, dims)
    for cu in BAD:
        for past in ([0, 0, 0], [30, 64, 1], [-5, 1 << 30, 3]):
            bufs = [guarded(s, dtype, 5.0) for s in ((N, Hq, d), (N, Hkv, d), (12, Hkv, page, d),
                                                     (12, Hkv, page, d))]
            lens_big, lens = guarded((3,), torch.int32, -9)
            R.reatt_paged_append(dims, *rows, ints(cu), ints(past), table,
                                 *(b[1] for b in bufs), lens, ws)
            torch.cuda.synchronize()
            R.reatt_workspace_status(ws)
            for big, t in bufs:
                assert outside_is(big, t.shape[0], 5.0) and t.isfinite().all(), (cu, past)
            assert outside_is(lens_big, 3, -9)
            clip = [min(max(c, 0), N) for c in cu]
            want = [p + max(clip[i + 1] - clip[i], 0) for i, p in enumerate(past)]
            assert lens.tolist() == want
