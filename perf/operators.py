"""Cases of the paged key-value cache operators: append with rotation, attention
of one new token over the pages, and causal attention over packed prompts.

``own`` false runs the operators as plain torch operations; ``own`` true makes
the calls of ``top_kv_span_b200.reatt``.  Head layouts are those of the
workloads in ``top_kv_span_b200/workloads.py``: 32 query / 8 KV heads of width
128 (RoPE base 5e5), 12 / 2 of width 128 (base 1e6), 4 / 1 of width 64 (1e4).
"""
import math
import random

import torch

own = False

HEADS = {  # query heads, KV heads, head width, RoPE base
    "llama3_8b": (32, 8, 128, 5e5),
    "qwen2_1p5b": (12, 2, 128, 1e6),
    "tiny": (4, 1, 64, 1e4),
}


def listed():
    return [
        # one request decoding: a single token joins its cache (launch latency)
        dict(name="append_one_token", op="append", heads="llama3_8b", dtype="bf16", page=16, B=1,
             total=1, past=4096, mix=1, keep_k=False),
        # a decoding step of a full serving batch: one token for each of 256 requests
        dict(name="append_batch_step", op="append", heads="qwen2_1p5b", dtype="bf16", page=64,
             B=256, total=256, past=1500, mix=2, keep_k=False),
        # a prefill step: ragged prompts, the rotated keys also kept for the prompt's attention
        dict(name="append_prompts", op="append", heads="llama3_8b", dtype="bf16", page=64, B=9,
             total=16001, past=0, mix=3, keep_k=True),
        # the fp32 shape of the repository's small workload, odd sizes
        dict(name="append_f32", op="append", heads="tiny", dtype="f32", page=32, B=5, total=777,
             past=301, mix=4, keep_k=True),
        # the small workload's one fp32 sequence of 4096 tokens (latency)
        dict(name="decode_one_f32", op="decode", heads="tiny", dtype="f32", page=32, B=1,
             total=4096, mix=5),
        # one long request: all of the card on one sequence of 128K tokens
        dict(name="decode_one_128k", op="decode", heads="llama3_8b", dtype="bf16", page=64, B=1,
             total=131073, mix=6),
        # requests of very different age in one batch
        dict(name="decode_ragged", op="decode", heads="llama3_8b", dtype="bf16", page=16, B=61,
             total=140003, mix=7),
        # a full serving batch with few KV heads
        dict(name="decode_batch", op="decode", heads="qwen2_1p5b", dtype="bf16", page=64, B=256,
             total=400011, mix=8),
        # one short prompt (latency)
        dict(name="prompt_short", op="prompt", heads="llama3_8b", dtype="bf16", B=1, total=133,
             mix=9),
        # a prefill batch of ragged prompts
        dict(name="prompt_ragged", op="prompt", heads="llama3_8b", dtype="bf16", B=7, total=8191,
             mix=10),
        # one long prompt: the largest case
        dict(name="prompt_16k", op="prompt", heads="llama3_8b", dtype="bf16", B=1, total=16384,
             mix=11),
        # fp32 prompts of the small workload's shape
        dict(name="prompt_f32", op="prompt", heads="tiny", dtype="f32", B=2, total=4131, mix=12),
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))

    case = dict(op=rng.choice(("append", "decode", "prompt")), heads=rng.choice(sorted(HEADS)),
                dtype="f32" if rng.random() < 0.25 else "bf16", mix=rng.randrange(1 << 20))
    if case["op"] == "append":
        case["B"] = log(1, 512)
        case["total"] = case["B"] if rng.random() < 0.4 else max(case["B"], log(1, 16000))
        case["past"] = rng.choice((0, log(1, 6000)))
        case["keep_k"] = rng.random() < 0.5
    elif case["op"] == "decode":
        case["B"] = log(1, 256)
        # up to about 500 MB of pages
        Hkv, d, size = HEADS[case["heads"]][1], HEADS[case["heads"]][2], _size(case)
        case["total"] = log(case["B"], min(500_000_000 // (2 * Hkv * d * size), 600_000))
    else:
        # a prompt of up to 12000 tokens, fp32 up to 5000
        case["total"] = log(1, 5000 if case["dtype"] == "f32" else 12000)
        case["B"] = min(case["total"], log(1, 12))
    if case["op"] != "prompt":
        case["page"] = rng.choice((1, 8, 16, 32, 64, 128, 256))
    return case


def _size(case):
    return 4 if case["dtype"] == "f32" else 2


def _lengths(case):
    """B sequence lengths of at least one token with the given sum, spread over
    about a factor of sixteen (one token each where there are no more)."""
    B, total = case["B"], case["total"]
    rng = random.Random(case["mix"])
    share = [math.exp(rng.uniform(0.0, math.log(16.0))) for _ in range(B)]
    left, weight, lens = total - B, sum(share), []
    for s in share[:-1]:
        lens.append(1 + int((total - B) * s / weight))
        left -= lens[-1] - 1
    return lens + [1 + left]


def _past(case):
    """Cached tokens of each sequence before an append."""
    rng = random.Random(case["mix"] + 1)
    return [rng.randint(case["past"] // 2, case["past"]) for _ in range(case["B"])]


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _channels(gen, Hkv, d):
    """Standard deviations of K's or V's channels."""
    return torch.rand((Hkv, d), generator=gen, device="cuda") * 3.5 + 0.5


def _table(gen, lens, page):
    """Pages of each sequence in a shuffled pool, and the pool's size."""
    need = [-(-n // page) for n in lens]
    total = sum(need)
    n_pages = total + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda")[:total].to(torch.int32).cpu()
    table = torch.zeros((len(lens), max(need)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.cuda(), n_pages


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return _ints(cu)


def prepare(case, seed):
    Hq, Hkv, d, base = HEADS[case["heads"]]
    dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    gen = torch.Generator("cuda").manual_seed(seed)
    lens = _lengths(case)
    s = dict(case=dict(case), heads=(Hq, Hkv, d), base=base, kept={})
    ks, vs = _channels(gen, Hkv, d), _channels(gen, Hkv, d)
    if case["op"] == "decode":
        s["table"], s["n_pages"] = _table(gen, lens, case["page"])
        shape = (s["n_pages"], Hkv, case["page"], d)
        # the rotated keys as an append leaves them: the same variances, position by position
        s["k_pages"] = (_normal(gen, *shape) * ks[:, None]).to(dt)
        s["v_pages"] = (_normal(gen, *shape) * vs[:, None]).to(dt)
        s["q"] = _normal(gen, case["B"], Hq, d).to(dt)
        s["lens"] = _ints(lens)
        s["out"] = torch.empty_like(s["q"])
        return s
    N = sum(lens)
    # one projection's output holds q, k and v of a token side by side
    row = torch.cat([_normal(gen, N, Hq, d), _normal(gen, N, Hkv, d) * ks,
                     _normal(gen, N, Hkv, d) * vs], 1).to(dt)
    s["q"], s["k"], s["v"] = row[:, :Hq], row[:, Hq:Hq + Hkv], row[:, Hq + Hkv:]
    s["cu"], s["max_len"] = _starts(lens), max(lens)
    if case["op"] == "prompt":
        s["out"] = torch.empty((N, Hq, d), dtype=dt, device="cuda")
        return s
    past = _past(case)
    s["past"] = _ints(past)
    s["table"], s["n_pages"] = _table(gen, [p + n for p, n in zip(past, lens)], case["page"])
    shape = (s["n_pages"], Hkv, case["page"], d)
    s["k_pages"] = _normal(gen, *shape).to(dt)
    s["v_pages"] = _normal(gen, *shape).to(dt)
    s["q_rot"] = torch.empty((N, Hq, d), dtype=dt, device="cuda")
    s["k_rot"] = torch.empty((N, Hkv, d), dtype=dt, device="cuda") if case["keep_k"] else None
    s["seq_len"] = torch.empty_like(s["past"])
    return s


# ------------------------------------------------------------------ plain forms
def _token_places(s):
    """Sequence and position of every packed token."""
    n = s["cu"][1:] - s["cu"][:-1]
    at = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n,
                                  output_size=at.numel())
    return seq, at - s["cu"][seq]


def _rotate(x, pos, base):
    half = x.shape[-1] // 2
    freq = base ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = pos.double()[:, None, None] * freq
    c, n = angle.cos().float(), angle.sin().float()
    a, b = x.float()[..., :half], x.float()[..., half:]
    return torch.cat([a * c - b * n, b * c + a * n], -1).to(x.dtype)


def _append_plain(s):
    seq, at = _token_places(s)
    pos = s["past"][seq] + at
    page = s["case"]["page"]
    where, slot = s["table"][seq, pos // page].long(), pos % page
    s["q_rot"].copy_(_rotate(s["q"], pos, s["base"]))
    k = _rotate(s["k"], pos, s["base"])
    if s["k_rot"] is not None:
        s["k_rot"].copy_(k)
    s["k_pages"][where, :, slot] = k
    s["v_pages"][where, :, slot] = s["v"]
    s["seq_len"].copy_(s["past"] + s["cu"][1:] - s["cu"][:-1])


def _decode_plain(s):
    Hq, Hkv, d = s["heads"]
    B = s["q"].shape[0]
    table = s["table"].long()
    k = s["k_pages"][table].float().transpose(1, 2).reshape(B, Hkv, -1, d)
    v = s["v_pages"][table].float().transpose(1, 2).reshape(B, Hkv, -1, d)
    x = s["q"].float().view(B, Hkv, Hq // Hkv, d) @ k.transpose(-1, -2) / math.sqrt(d)
    off = torch.arange(k.shape[2], device="cuda") >= s["lens"][:, None]
    x = x.masked_fill(off[:, None, None], -math.inf)
    p = (x - x.amax(-1, keepdim=True)).exp()
    s["out"].copy_(((p @ v) / p.sum(-1, keepdim=True)).view(B, Hq, d))


def _prompt_plain(s):
    Hq, Hkv, d = s["heads"]
    B, L, g = s["cu"].numel() - 1, s["max_len"], Hq // Hkv
    seq, at = _token_places(s)

    def padded(x):
        y = torch.zeros((B, L, x.shape[1], d), device="cuda")
        y[seq, at] = x.float()
        return y.transpose(1, 2)

    q = padded(s["q"]).reshape(B, Hkv, g * L, d)
    x = q @ padded(s["k"]).transpose(-1, -2)
    t = torch.arange(L, device="cuda")
    x = x.view(B, Hkv, g, L, L).div_(math.sqrt(d))
    x.masked_fill_(t[None, :] > t[:, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = (x.view(B, Hkv, g * L, L) @ padded(s["v"])).view(B, Hq, L, d)
    o = o / x.sum(-1).view(B, Hq, L, 1)
    s["out"].copy_(o.transpose(1, 2)[seq, at])


# ------------------------------------------------------------------ the framework's calls
def _handle(s):
    """What a program keeps between calls: the dims and a workspace."""
    if not s["kept"]:
        from top_kv_span_b200 import reatt as R
        Hq, Hkv, d = s["heads"]
        c = s["case"]
        N, paged = s["q"].shape[0], "table" in s
        strides = dict(q_stride=s["q"].stride(0))
        if "k" in s:
            strides.update(k_stride=s["k"].stride(0), v_stride=s["v"].stride(0))
        dims = R.make_paged_dims(B=c["B"], Hq=Hq, Hkv=Hkv, d=d, dtype=c["dtype"], N=N,
                                 page=c["page"] if paged else 1,
                                 max_pages=s["table"].shape[1] if paged else 1,
                                 n_pages=s["n_pages"] if paged else 1, rope_base=s["base"],
                                 **strides)
        s["kept"] = dict(R=R, dims=dims,
                         ws=torch.zeros(R.reatt_paged_workspace_bytes(dims), dtype=torch.uint8,
                                        device="cuda"))
    return s["kept"]["R"], s["kept"]["dims"], s["kept"]["ws"]


def run(s):
    op = s["case"]["op"]
    if own:
        R, dims, ws = _handle(s)
        if op == "append":
            R.reatt_paged_append(dims, s["q"], s["k"], s["v"], s["cu"], s["past"], s["table"],
                                 s["q_rot"], s["k_rot"], s["k_pages"], s["v_pages"],
                                 s["seq_len"], ws)
        elif op == "decode":
            R.reatt_paged_decode(dims, s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                 s["out"], ws)
        else:
            R.reatt_prompt_attend(dims, s["q"], s["k"], s["v"], s["cu"], s["out"], ws)
    else:
        {"append": _append_plain, "decode": _decode_plain, "prompt": _prompt_plain}[op](s)
    return _outputs(s)


def _outputs(s):
    if s["case"]["op"] == "append":
        return {n: s[n] for n in ("q_rot", "k_rot", "k_pages", "v_pages", "seq_len")}
    return s["out"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    Hq, Hkv, d, _ = HEADS[case["heads"]]
    e, lens = _size(case), _lengths(case)
    N = sum(lens)
    if case["op"] == "append":
        rows = 2 * (Hq + 2 * Hkv) + (Hkv if case["keep_k"] else 0)
        return dict(bytes=N * rows * d * e, flops=3 * N * (Hq + Hkv) * d)
    if case["op"] == "decode":
        return dict(bytes=2 * N * Hkv * d * e + 2 * case["B"] * Hq * d * e, flops=4 * N * Hq * d)
    return dict(bytes=2 * N * (Hq + Hkv) * d * e,
                flops=sum(2 * n * (n + 1) * Hq * d for n in lens))


# ------------------------------------------------------------------ the definition in 64 bits
def _turn64(x, pos, base):
    """Rotation as a product of complex numbers."""
    half = x.shape[-1] // 2
    i = torch.arange(half, device="cuda", dtype=torch.float64)
    w = torch.polar(torch.ones_like(i).expand(pos.numel(), half),
                    pos.double()[:, None] * torch.exp(i * (-math.log(base) / half)))
    z = torch.complex(x[..., :half].double(), x[..., half:].double()) * w[:, None]
    return torch.cat([z.real, z.imag], -1)


def _softmax64(q, k, v, last):
    """Rows of q [H, n, d] over k, v [H, m, d]; row r sees keys 0..last[r]."""
    x = torch.einsum("hnd,hmd->hnm", q, k) * q.shape[-1] ** -0.5
    x.masked_fill_(torch.arange(k.shape[1], device="cuda") > last[:, None], -math.inf)
    return torch.einsum("hnm,hmd->hnd", torch.softmax(x, -1), v)


def exact(case, seed):
    s = prepare(case, seed)
    Hq, Hkv, d = s["heads"]
    g, lens = Hq // Hkv, _lengths(case)
    if case["op"] == "append":
        past, page = _past(case), case["page"]
        pos = torch.cat([torch.arange(p, p + n) for p, n in zip(past, lens)]).cuda()
        q, k = _turn64(s["q"], pos, s["base"]), _turn64(s["k"], pos, s["base"])
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        at = 0
        for b, n in enumerate(lens):
            t = pos[at:at + n]
            where, slot = s["table"][b].long()[t // page], t % page
            for h in range(Hkv):
                kp[where, h, slot] = k[at:at + n, h]
                vp[where, h, slot] = s["v"][at:at + n, h].double()
            at += n
        return {"q_rot": q, "k_rot": k if case["keep_k"] else None, "k_pages": kp,
                "v_pages": vp, "seq_len": None}
    if case["op"] == "decode":
        out = []
        for b, n in enumerate(lens):
            rows = s["table"][b].long()[: -(-n // case["page"])]
            k = s["k_pages"][rows].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].double()
            v = s["v_pages"][rows].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].double()
            q = s["q"][b].double().view(Hkv, g, d)
            out.append(_softmax64(q, k, v, torch.full((g,), n, device="cuda")).reshape(Hq, d))
        return torch.stack(out)
    out, at = [], 0
    for n in lens:
        q, k, v = (s[x][at:at + n].double().transpose(0, 1) for x in ("q", "k", "v"))
        parts = []
        for r in range(0, n, 1024):  # a block of queries at a time, all heads of one KV head
            last = torch.arange(r, min(n, r + 1024), device="cuda")
            m = int(last[-1]) + 1
            parts.append(torch.cat([
                _softmax64(q[h:h + 1, r:m], k[h // g:h // g + 1, :m], v[h // g:h // g + 1, :m],
                           last) for h in range(Hq)]))
        out.append(torch.cat(parts, 1).transpose(0, 1))
        at += n
    return torch.cat(out)
