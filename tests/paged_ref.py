"""The paged operators in 64 bits on the host, and the bounds that their fp32
arithmetic and roundings allow (each written where it is computed)."""
import math

import torch


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rotate(x, pos, base):
    """[n, H, d] at positions [n] -> (rotated, bound)."""
    half = x.shape[-1] // 2
    w = base ** (-torch.arange(half, dtype=torch.float64) / half)
    ang = pos.double()[:, None, None] * w
    a, b = x.double()[..., :half], x.double()[..., half:]
    y = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    # The angle in half-turns is within two steps of 2^-24 of a value in [-1, 1]
    # and is turned by pi; sincospif is off by at most two steps (2^-22), the
    # product and the sum round by half a step each: under 8 * 2^-23 of |a| + |b|.
    s = (a.abs() + b.abs()) * 2.0 ** -20
    return y, torch.cat([s, s], -1) + half_step(x.dtype) * y.abs()


def attend(q, k, v, last, p_step=None):
    """q [Hq, n, d] over k, v [Hkv, m, d]; row r sees keys 0..last[r] ->
    (out [Hq, n, d], bound).  k, v are taken only where some row sees them.  p_step:
    how far a weight may be rounded before it meets v (half a step of bf16 for bf16)."""
    Hq, n, d = q.shape
    g, m = Hq // k.shape[0], k.shape[1]
    dt = q.dtype
    q = q.double()
    kk = k.double().repeat_interleave(g, 0)
    vv = v.double().repeat_interleave(g, 0)
    off = torch.arange(m, device=last.device) > last[:, None]
    x = (q @ kk.transpose(-1, -2)) / math.sqrt(d)
    x = x.masked_fill(off, -math.inf)
    p = torch.softmax(x, -1)
    o = p @ vv
    # A logit is a sum of d products in fp32 (any order: d half steps of the sum
    # of magnitudes), scaled (two more); the exponential adds 2^-22 and its
    # argument's rounding (half a step of the largest magnitude of a logit and
    # of the maximum).  Each weight is then off by at most e = 2 * (that), and so
    # is the sum of weights: 2 e of sum p |v|.  The sums over keys in fp32, in
    # any order, add (m + 8) half steps; for bf16 the weights may be rounded to
    # bf16 before they meet v: half a step each.  The result rounds once.
    mag = ((q.abs() @ kk.abs().transpose(-1, -2)) / math.sqrt(d)).masked_fill(off, 0)
    big = mag.amax(-1, keepdim=True)
    e = 2 * ((d + 4) * 2.0 ** -24 * big + 2.0 ** -22)
    pv = p @ vv.abs()
    tol = (2 * e + (m + 8) * 2.0 ** -23) * pv + half_step(dt) * o.abs()
    if dt != torch.float32:
        tol = tol + (half_step(dt) if p_step is None else p_step) * pv
    return o, tol * (1 + 2.0 ** -6) + 1e-30


def check(got, want, tol, what=""):
    err = (got.double().cpu() - want).abs()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst " \
                          f"{float((err / tol).max()):.3g} of the bound"


class Pool:
    """Pages of a batch in a shuffled pool; everything that no token owns is NaN
    and unused table entries are out of range."""

    def __init__(self, lens, Hkv, d, page, dtype, seed, room=0, std=1.0):
        gen = torch.Generator().manual_seed(seed)
        need = [-(-(n + room) // page) for n in lens]
        self.n_pages = sum(need) + 3
        self.max_pages = max(max(need), 1) + 2
        order = torch.randperm(self.n_pages, generator=gen)
        self.table = torch.full((len(lens), self.max_pages), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n].int()
            at += n
        shape = (self.n_pages, Hkv, page, d)
        self.page = page
        self.k = torch.full(shape, math.nan, dtype=dtype)
        self.v = torch.full(shape, math.nan, dtype=dtype)
        self.rows = []
        for b, n in enumerate(lens):
            kb = (torch.randn((n, Hkv, d), generator=gen) * std).to(dtype)
            vb = (torch.randn((n, Hkv, d), generator=gen) * std).to(dtype)
            self.put(b, 0, kb, vb)
            self.rows.append((kb, vb))

    def put(self, b, start, kb, vb):
        t = torch.arange(start, start + kb.shape[0])
        where, slot = self.table[b][t // self.page].long(), t % self.page
        self.k[where, :, slot] = kb
        self.v[where, :, slot] = vb
