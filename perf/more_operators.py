"""Cases of the operators that serve grouped heads beside the latent heads, on the same page tables.

Each case names one operator and its sizes:

* ``append``: new keys and values go to their pages in 8 bits, with one power-of-two scale for each block of 16 tokens
  and head; keys and queries are rotated by their positions on the way;
* ``cache``: attention of each request's new tokens over that cache;
* ``prompt``: causal attention of packed prompts on their fresh keys and values.

``run`` is one pass in plain torch operations, or, where ``own`` is true, through the library's calls.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
PAGE, BLOCK = 64, 16
E_MIN, E_MAX = -24, 24
BASE = 10000.0


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one request of a chat, one new token: the call's latency
        dict(name="append 1x1", op="append", batch=1, rows=1, ctx=8192, jitter=0.0, kv=8, group=8, dim=128, rope=128, halves=True),
        # a decode batch on ragged contexts
        dict(name="append 128x1", op="append", batch=128, rows=1, ctx=32768, jitter=0.25, kv=8, group=8, dim=128, rope=64, halves=False),
        # prompts of different lengths, far into long contexts
        dict(name="append 7x1024", op="append", batch=7, rows=1024, ctx=1000003, jitter=0.1, kv=8, group=8, dim=128, rope=128, halves=True),
        # one request of a chat, one new token
        dict(name="cache decode 1x8192", op="cache", batch=1, rows=1, ctx=8192, jitter=0.0, kv=8, group=8, dim=128),
        # an ordinary decode batch on ragged contexts
        dict(name="cache decode 64x32768", op="cache", batch=64, rows=1, ctx=32768, jitter=0.25, kv=8, group=8, dim=128),
        # a draft of five tokens and the one before them are verified, wide heads
        dict(name="cache verify 16x6 dim 256", op="cache", batch=16, rows=6, ctx=16381, jitter=0.25, kv=4, group=4, dim=256),
        # a prompt's next chunk behind what the cache holds
        dict(name="cache prefill 2048", op="cache", batch=1, rows=2048, ctx=16384, jitter=0.0, kv=8, group=8, dim=128),
        # one short question
        dict(name="prompt 1x129", op="prompt", batch=1, rows=129, past=0, jitter=0.0, kv=8, group=8, dim=128),
        # many prompts of different lengths in one batch
        dict(name="prompt 16x512", op="prompt", batch=16, rows=512, past=0, jitter=0.9, kv=8, group=8, dim=128),
        # small heads without groups
        dict(name="prompt 4x2048 dim 64", op="prompt", batch=4, rows=2048, past=0, jitter=0.25, kv=16, group=1, dim=64),
        # one long prompt
        dict(name="prompt 1x8192", op="prompt", batch=1, rows=8192, past=0, jitter=0.0, kv=8, group=8, dim=128),
        # latent attention with its keys and values written out: 64 heads of 256 dims
        dict(name="prompt 2x4096 dim 256", op="prompt", batch=2, rows=4096, past=0, jitter=0.1, kv=64, group=1, dim=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))


def draw(rng: random.Random):
    while True:
        op = rng.choice(["append", "cache", "cache", "prompt", "prompt"])
        dim = rng.choice([64, 128, 128, 256])
        kv, group = rng.choice([(8, 8), (4, 4), (8, 4), (2, 7), (1, 64), (16, 1), (8, 5), (4, 12), (64, 1), (3, 3)])
        c = dict(op=op, jitter=rng.choice([0.0, 0.25, 0.9]), kv=kv, group=group, dim=dim)
        if op == "append":
            rope = rng.choice([0, 32, 64, 64, dim])
            c.update(batch=_log(rng, 1, 256), rows=rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 4096)]), ctx=_log(rng, 4096, 1000003), rope=rope,
                     halves=rng.random() < 0.5)
            if c["batch"] * c["rows"] * (kv * (group + 2)) * dim > 8192 * 80 * 128:
                continue
        elif op == "cache":
            rows = rng.choice([1, 1, 1, rng.randint(2, 8), _log(rng, 9, 2048)])
            c.update(batch=_log(rng, 1, 128), rows=rows, ctx=_log(rng, max(rows, 33), 131072))
        else:
            c.update(batch=_log(rng, 1, 64), rows=_log(rng, 1, 8192), past=rng.choice([0, 0, 0, _log(rng, 1, 2048)]))
        if op != "append":
            w = work(c)
            span = max(x for x, _ in _lens(c))
            heads = kv * group
            if w["flops"] > 1.1e12 or w["bytes"] > 4.4e9 or c["batch"] * c["rows"] * span * heads > 4.3e9 or c["batch"] * span * kv * dim > 2.7e9:
                continue
        return c


def _lens(c):
    """(context, new tokens) of each request, from the case alone."""
    got = []
    for r in range(c["batch"]):
        f = (r * 0.6180339887) % 1.0
        much = 1.0 + c["jitter"] * (2.0 * f - 1.0)
        if c["op"] == "prompt":
            n = max(1, min(c["rows"], int(c["rows"] * (1.0 - c["jitter"] * f))))
            got.append((c["past"] + n, n))
        elif c["op"] == "append":
            n = max(1, int(c["rows"] * (1.0 - c["jitter"] * f)))
            got.append((max(n, int(c["ctx"] * much)), n))
        else:
            L = max(1, int(c["ctx"] * much))
            got.append((L, min(L, c["rows"])))
    return got


def work(c):
    rows = sum(n for _, n in _lens(c))
    kv, heads, dim = c["kv"], c["kv"] * c["group"], c["dim"]
    if c["op"] == "append":
        # k, v and q read; codes, scales of the touched blocks, rotated q and k written
        blocks = sum((L - 1) // BLOCK - (L - n) // BLOCK + 1 for L, n in _lens(c))
        return dict(bytes=rows * dim * (2 * kv * (2 + 1) + 2 * kv + heads * 4) + blocks * kv * 8, flops=rows * (kv + heads) * c["rope"] * 3)
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in _lens(c))
    tokens = sum(L for L, _ in _lens(c))
    io = rows * heads * (4 * dim + 4)
    per_token = kv * (2 * dim + 8 / BLOCK) if c["op"] == "cache" else kv * 4 * dim
    return dict(bytes=tokens * per_token + io, flops=pairs * heads * 4 * dim)


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(7654321 + seed)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _head_bytes(dim):
    return 2 * PAGE * dim + 32


def _views(cache, kv, dim):
    """K codes [pages, kv, 4, 16, dim], V codes [pages, kv, 4, dim, 16] and the scales [pages, kv, 2, 4] of a cache."""
    heads = cache.view(-1, kv, _head_bytes(dim))
    return (heads[..., : PAGE * dim].unflatten(-1, (4, BLOCK, dim)), heads[..., PAGE * dim: 2 * PAGE * dim].unflatten(-1, (4, dim, BLOCK)),
            heads[..., 2 * PAGE * dim:].view(torch.float32).unflatten(-1, (2, 4)))


def _pow2(e):
    """2^e for whole e in [-126, 127], exactly."""
    return (e.to(torch.int32) + 127 << 23).view(torch.float32)


def _cache(pages, kv, dim, g):
    """Pages as appends leave them: values N(0, 1) times a size of each block, 8 bits, one power of two for a block and head."""
    cache = torch.empty(pages, kv * _head_bytes(dim), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (kv * PAGE * dim))
    for a in range(0, pages, step):
        part = _views(cache[a: a + step], kv, dim)
        for i in (0, 1):
            x = torch.randn(part[i].shape, generator=g, device=DEV)
            x *= torch.exp(0.3 * torch.randn(x.shape[:3], generator=g, device=DEV))[..., None, None]
            e = torch.ceil(torch.log2(x.abs().amax((-2, -1)) / 448.0))
            part[i].copy_((x * _pow2(-e)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8))
            part[2][:, :, i] = _pow2(e)
    return cache


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def prepare(case, seed):
    c, g = case, _gen(seed)
    lens = _lens(c)
    L, n = [x for x, _ in lens], [x for _, x in lens]
    B, T, kv, heads, dim = c["batch"], sum(n), c["kv"], c["kv"] * c["group"], c["dim"]
    start = [sum(n[:r]) for r in range(B + 1)]
    st = dict(case=c, T=T, max_len=max(L), max_q=max(n), q_start=_ints(start), q=_randn((T, heads, dim), g))
    if c["op"] == "prompt":
        ends = [sum(L[:r]) for r in range(B + 1)]
        st.update(k_start=_ints(ends), TK=ends[-1], k=_randn((ends[-1], kv, dim), g), v=_randn((ends[-1], kv, dim), g))
    else:
        width = (max(L) + PAGE - 1) // PAGE
        # an append needs the pages of the new tokens alone, attention needs all of them
        held = torch.zeros(B, width, dtype=torch.bool)
        for r in range(B):
            held[r, ((L[r] - n[r]) // PAGE if c["op"] == "append" else 0): (L[r] + PAGE - 1) // PAGE] = True
        total = int(held.sum())
        pages = total + 3
        perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        table[held.to(DEV)] = perm[:total]
        st.update(seq_len=_ints(L), table=table, pages=pages, cache=_cache(pages, kv, dim, g))
    if c["op"] == "append":
        # what a projection gives: q, k and v side by side in one row of each token
        rows = _randn((T, heads + 2 * kv, dim), g)
        # tokens of different sizes, so that a block's scale grows at times
        rows *= torch.exp(0.5 * torch.randn(T, 1, 1, generator=g, device=DEV)).to(torch.bfloat16)
        st.update(q=rows[:, :heads], k=rows[:, heads: heads + kv], v=rows[:, heads + kv:],
                  q_out=torch.empty(T, heads, dim, dtype=torch.bfloat16, device=DEV), k_out=torch.empty(T, kv, dim, dtype=torch.bfloat16, device=DEV))
    else:
        st.update(out=torch.empty(T, heads, dim, dtype=torch.bfloat16, device=DEV), lse=torch.empty(T, heads, dtype=torch.float32, device=DEV))
    return st


# ------------------------------------------------------------------------------------------------ plain forms
def _request(st):
    """Request and place in it of every row."""
    start = st["q_start"].long()
    t = torch.arange(st["T"], device=DEV)
    r = torch.searchsorted(start[1:], t, right=True)
    return r, t - start[r]


def _rotate(x, pos, c):
    """x [T, heads, dim] rotated by its positions: angles in 64 bits, products in 32."""
    R = c["rope"]
    x = x.float()
    if R == 0:
        return x
    freq = BASE ** (-2.0 * torch.arange(R // 2, dtype=torch.float64, device=DEV) / R)
    angle = pos.double()[:, None] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    y = x.clone()
    if c["halves"]:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        y[..., : R // 2], y[..., R // 2: R] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_append(st):
    c, B = st["case"], st["case"]["batch"]
    kv, dim = c["kv"], c["dim"]
    seq, start = st["seq_len"].long(), st["q_start"].long()
    r, t = _request(st)
    first = seq - (start[1:] - start[:-1])
    pos = first[r] + t
    q, k, v = _rotate(st["q"], pos, c), _rotate(st["k"], pos, c), st["v"].float()
    # blocks that get new tokens: [B, N] from each request's first one on
    N = (st["max_q"] + BLOCK - 2) // BLOCK + 1
    block = first[:, None] // BLOCK + torch.arange(N, device=DEV)
    live = block * BLOCK < seq[:, None]
    page = torch.gather(st["table"].long(), 1, (block // 4).clamp(max=st["table"].shape[1] - 1))
    page, at = page[live], (block % 4)[live]
    place = block[live][:, None] * BLOCK + torch.arange(BLOCK, device=DEV)
    req = torch.arange(B, device=DEV)[:, None].expand(B, N)[live]
    new = (place >= first[req][:, None]) & (place < seq[req][:, None])
    old = place < first[req][:, None]
    row = (start[req][:, None] + place - first[req][:, None]).clamp(0, st["T"] - 1)
    views = _views(st["cache"], kv, dim)
    for i, x in enumerate((k, v)):
        codes, scales = views[i], views[2][:, :, i]
        was = codes[page, :, at]                                    # [blocks, kv, 16, dim], V's transposed
        was = (was if i == 0 else was.transpose(-1, -2)).contiguous()
        fresh = torch.where(new[:, None, :, None], x[row].transpose(1, 2), torch.zeros((), device=DEV))
        amax = fresh.abs().amax((-2, -1))
        m, e = torch.frexp(amax / 448.0)
        need = torch.where(amax > 0, torch.where(m == 0.5, e - 1, e), torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
        e_was = torch.frexp(scales[page, :, at])[1] - 1
        now = torch.where(old.any(1)[:, None], torch.maximum(need, e_was), need)
        kept = (was.view(torch.float8_e4m3fn).float() * _pow2((e_was - now).clamp(min=-126))[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        put = (fresh * _pow2(-now)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        got = torch.where(new[:, None, :, None], put, torch.where(old[:, None, :, None], kept, was))
        codes[page, :, at] = got if i == 0 else got.transpose(-1, -2)
        scales[page, :, at] = _pow2(now)
    st["q_out"].copy_(q.to(torch.bfloat16))
    st["k_out"].copy_(k.to(torch.bfloat16))
    return _append_outputs(st)


def _append_outputs(st):
    k, v, s = _views(st["cache"], st["case"]["kv"], st["case"]["dim"])
    return dict(k=k.view(torch.float8_e4m3fn), v=v.view(torch.float8_e4m3fn), scale=s, q=st["q_out"], k_out=st["k_out"])


def _attend(q, k, v, see, st):
    """q [B, Q, heads, dim], k and v [B, kv, S, dim] in 32 bits, see [B, Q, S]: outputs and log-sums of the batch's rows."""
    c = st["case"]
    B, Q, heads, dim = q.shape
    kv, G = c["kv"], c["group"]
    q = q.view(B, Q, kv, G, dim).permute(0, 2, 1, 3, 4).reshape(B * kv, Q * G, dim) * dim ** -0.5
    x = torch.bmm(q, k.flatten(0, 1).transpose(1, 2)).view(B, kv, Q, G, -1)
    x.masked_fill_(~see[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.bmm(x.view(B * kv, Q * G, -1), v.flatten(0, 1)).view(B, kv, Q, G, dim)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    r, t = _request(st)
    out = o.permute(0, 2, 1, 3, 4).reshape(B, Q, heads, dim)[r, t]
    lse = (m + total.log()).permute(0, 2, 1, 3, 4).reshape(B, Q, heads)[r, t]
    return dict(out=out.to(torch.bfloat16), lse=lse)


def _padded(x, start, width):
    """[B, width, ...] of a packed x [rows, ...]: sequence r's rows, then others."""
    at = (start[:-1, None] + torch.arange(width, device=DEV)).clamp(max=x.shape[0] - 1)
    return x[at]


def _plain_cache(st):
    c = st["case"]
    kv, dim, B = c["kv"], c["dim"], c["batch"]
    seq, start, Q = st["seq_len"].long(), st["q_start"].long(), st["max_q"]
    W = st["table"].shape[1]
    k, v, s = _views(st["cache"], kv, dim)
    page = st["table"].long()
    held = page >= 0
    page = page.clamp(min=0)
    x = s[page].transpose(1, 2)[..., None, None] * held[:, None, :, None, None, None, None]      # [B, kv, W, 2, 4, 1, 1]
    k = (k[page].transpose(1, 2).contiguous().view(torch.float8_e4m3fn).float() * x[:, :, :, 0]).reshape(B, kv, W * PAGE, dim)
    v = (v[page].transpose(1, 2).contiguous().view(torch.float8_e4m3fn).float() * x[:, :, :, 1]).transpose(-1, -2).reshape(B, kv, W * PAGE, dim)
    p = (seq - (start[1:] - start[:-1]))[:, None] + torch.arange(Q, device=DEV)
    see = torch.arange(W * PAGE, device=DEV) <= p[..., None]
    return _attend(_padded(st["q"].float(), start, Q), k, v, see, st)


def _plain_prompt(st):
    start, ends, Q, S = st["q_start"].long(), st["k_start"].long(), st["max_q"], st["max_len"]
    n, L = start[1:] - start[:-1], ends[1:] - ends[:-1]
    k, v = (_padded(st[x].float(), ends, S).transpose(1, 2) for x in ("k", "v"))
    j = torch.arange(S, device=DEV)
    see = (j <= ((L - n)[:, None] + torch.arange(Q, device=DEV))[..., None]) & (j < L[:, None, None])
    return _attend(_padded(st["q"].float(), start, Q), k, v, see, st)


# ------------------------------------------------------------------------------------------------ the library's calls
def _own(st):
    import dsa_sparse_attention_indexer_gb300 as D
    c = st["case"]
    if "handle" not in st:                               # what a program keeps from step to step
        h = st["handle"] = {}
        if c["op"] == "prompt":
            h["batch"] = D.PromptBatch(st["q_start"], st["k_start"], max_q_len=st["max_q"], max_k_len=st["max_len"], total_q=st["T"], total_k=st["TK"])
            h["ws"] = D.workspace(D.dsa_prompt_attention_workspace_size(h["batch"], c["kv"] * c["group"], c["kv"], c["dim"]), DEV)
        else:
            h["batch"] = D.Batch(st["seq_len"], st["q_start"], st["table"], st["pages"], max_seq_len=st["max_len"], max_q_len=st["max_q"], total_q=st["T"])
        if c["op"] == "cache":
            h["ws"] = D.workspace(D.dsa_kv8_attention_workspace_size(h["batch"], c["kv"] * c["group"], c["kv"], c["dim"]), DEV)
    h = st["handle"]
    if c["op"] == "append":
        D.dsa_kv8_append(st["k"], st["v"], st["cache"], h["batch"], q=st["q"], rope_dims=c["rope"], rope_style=D.ROPE_HALVES if c["halves"] else D.ROPE_INTERLEAVED,
                         rope_base=BASE, q_out=st["q_out"], k_out=st["k_out"])
        return _append_outputs(st)
    if c["op"] == "cache":
        D.dsa_kv8_attention(st["q"], st["cache"], h["batch"], kv_heads=c["kv"], out=st["out"], lse=st["lse"], ws=h["ws"])
    else:
        D.dsa_prompt_attention(st["q"], st["k"], st["v"], h["batch"], out=st["out"], lse=st["lse"], ws=h["ws"])
    return dict(out=st["out"], lse=st["lse"])


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "cache": _plain_cache, "prompt": _plain_prompt}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ 64 bits
def _e4m3_values():
    v = []
    for code in range(256):
        e, m = code >> 3 & 15, code & 7
        x = math.nan if e == 15 and m == 7 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-x if code & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _nearest_e4m3(x, values):
    """The codes' values nearest to x (64 bits), ties to the even code."""
    grid = values[:127]
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - grid[lo], grid[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.copysign(torch.where(up, grid[hi], grid[lo]), x)


def _turned(x, pos, c):
    """Rotation as a product of complex numbers, in 64 bits."""
    x, R = x.double(), c["rope"]
    if R == 0:
        return x
    angle = torch.outer(pos.double(), torch.exp(torch.arange(R // 2, dtype=torch.float64, device=DEV) * (-2.0 * math.log(BASE) / R)))
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    pairs = x[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2) if c["halves"] else x[..., :R].unflatten(-1, (R // 2, 2))
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z.transpose(-1, -2) if c["halves"] else z
    return torch.cat([z.flatten(-2), x[..., R:]], -1)


def exact(case, seed):
    """Request by request from the definition, in 64 bits."""
    st = prepare(case, seed)
    values = _e4m3_values()
    every = torch.tensor([2.0 ** e for e in range(2 * E_MIN, E_MAX + 1)], dtype=torch.float64, device=DEV)
    powers, power = every[-E_MIN:], lambda e: every[e - 2 * E_MIN]
    c, kv, G, dim = case, case["kv"], case["group"], case["dim"]
    lens = _lens(case)
    if c["op"] == "append":
        pos = torch.cat([torch.arange(L - n, L, device=DEV) for L, n in lens])
        q, k, v = _turned(st["q"], pos, c), _turned(st["k"], pos, c), st["v"].double()
        K, V, S = _views(st["cache"], kv, dim)
        K, V, S = values[K.long()], values[V.long()].transpose(-1, -2).contiguous(), S.double().clone()
        begin = 0
        table = st["table"].cpu()
        for r, (L, n) in enumerate(lens):
            for b in range((L - n) // BLOCK, (L - 1) // BLOCK + 1):
                page, at = int(table[r, b // 4]), b % 4
                lo, hi = max(L - n, b * BLOCK), min(L, (b + 1) * BLOCK)
                for X, src, i in ((K, k, 0), (V, v, 1)):
                    x = src[begin + lo - (L - n): begin + hi - (L - n)].transpose(0, 1)      # [kv, tokens, dim]
                    amax = x.abs().amax((1, 2))
                    # the first power of two that holds the largest value (E_MIN for zeros), by comparison
                    e = torch.searchsorted(448.0 * powers[: E_MAX - E_MIN], amax) + E_MIN
                    held = lo - b * BLOCK
                    if held:
                        was = torch.searchsorted(powers, S[page, :, i, at].contiguous()) + E_MIN
                        e = torch.maximum(e, was)
                        X[page, :, at, :held] = _nearest_e4m3(X[page, :, at, :held] * power(was - e)[:, None, None], values)
                    X[page, :, at, held: held + hi - lo] = _nearest_e4m3(x * power(-e)[:, None, None], values)
                    S[page, :, i, at] = power(e)
            begin += n
        return dict(k=K, v=V.transpose(-1, -2), scale=S, q=q, k_out=k)
    if work(case)["flops"] > 4e12:
        return None
    out, lse, begin, held = [], [], 0, 0
    for r, (L, n) in enumerate(lens):
        if c["op"] == "prompt":
            K, V = st["k"][held: held + L].double().transpose(0, 1), st["v"][held: held + L].double().transpose(0, 1)
            held += L
        else:
            j = torch.arange(L, device=DEV)
            page, at, row = st["table"][r, j // PAGE].long(), j % PAGE // BLOCK, j % BLOCK
            k, v, s = _views(st["cache"], kv, dim)
            h = torch.arange(kv, device=DEV)[:, None]
            K = values[k[page, h, at, row].long()] * s[page, h, 0, at].double()[..., None]
            V = values[v[page, h, at, :, row].long()] * s[page, h, 1, at].double()[..., None]
        q = st["q"][begin: begin + n].double().view(n, kv, G, dim).transpose(0, 1)
        o = torch.empty(n, kv * G, dim, dtype=torch.float64, device=DEV)
        z = torch.empty(n, kv * G, dtype=torch.float64, device=DEV)
        step = max(1, (1 << 27) // (kv * G * L))
        for a in range(0, n, step):
            b = min(n, a + step)
            top = L - n + b                                   # keys that the piece's last row sees
            x = torch.matmul(q[:, a:b].reshape(kv, -1, dim), K[:, :top].transpose(1, 2)).view(kv, b - a, G, top) / math.sqrt(dim)
            x.masked_fill_(torch.arange(top, device=DEV) > torch.arange(L - n + a, top, device=DEV)[:, None, None], -math.inf)
            part = torch.logsumexp(x, -1, keepdim=True)
            y = torch.matmul(torch.exp(x - part).view(kv, -1, top), V[:, :top]).view(kv, b - a, G, dim)
            o[a:b] = y.transpose(0, 1).reshape(b - a, -1, dim)
            z[a:b] = part[..., 0].transpose(0, 1).reshape(b - a, -1)
        out.append(o)
        lse.append(z)
        begin += n
    return dict(out=torch.cat(out), lse=torch.cat(lse))
