"""Cases of the operators that serve drafted, windowed and forked requests over the paged caches.

Each case names one operator and its sizes:

* ``window``: sparse-MLA heads over a sliding window of each row's context and its first tokens;
* ``tree``: the same heads for a tree of drafted tokens behind a cached prefix;
* ``commit``: the accepted path of a tree moves to the front of its tokens, in every layer's cache;
* ``fork``: requests share their parent's full pages and get a copy of the last, partial one;
* ``turnover``: finished requests give their pages back, new ones take theirs.

``run`` is one pass in plain torch operations, or, where ``own`` is true, through the library's calls.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
PAGE, HEADS, QK, LATENT, ROPE = 64, 64, 576, 512, 64
KV_ROW, KV_PAGE = 656, 41984
IDX_PAGE, IDX_PAYLOAD = 8448, 8192
SCALE = 1.0 / 16


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one request of a chat, one new token: the call's latency
        dict(name="window decode 1x512", op="window", batch=1, rows=1, ctx=8192, jitter=0.0, window=512, sinks=4),
        # an ordinary decode batch on ragged contexts
        dict(name="window decode 64x4096", op="window", batch=64, rows=1, ctx=32768, jitter=0.25, window=4096, sinks=64),
        # few requests of about a million tokens whose middle pages were given back
        dict(name="window decode 4x131072", op="window", batch=4, rows=1, ctx=1000003, jitter=0.02, window=131072, sinks=16),
        # a prefill chunk behind a cached prefix
        dict(name="window prefill 2048x2048", op="window", batch=1, rows=2048, ctx=8192, jitter=0.0, window=2048, sinks=16),
        # one request verifies a small tree
        dict(name="tree 1x8 ctx 2048", op="tree", batch=1, nodes=8, ctx=2048, jitter=0.0),
        # a batch verifies wide trees on long contexts
        dict(name="tree 8x64 ctx 32768", op="tree", batch=8, nodes=64, ctx=32768, jitter=0.25),
        # after a verify step: one request on a four-layer group, and a batch on a whole model's 78 + 21 caches
        dict(name="commit 1x8 4 layers", op="commit", batch=1, nodes=8, ctx=2048, kv=4, idx=1),
        dict(name="commit 128x16 78 layers", op="commit", batch=128, nodes=16, ctx=2085, kv=78, idx=21),
        # parallel samples of one prompt: a few on a layer group, many on a whole model
        dict(name="fork 4 4 layers", op="fork", n=4, ctx=8229, kv=4, idx=1),
        dict(name="fork 64 78 layers", op="fork", n=64, ctx=8229, kv=78, idx=21),
        # requests finish and others begin: a small pool, and a GPU full of pages
        dict(name="turnover 8 of 1024 pages", op="turnover", n=8, ctx=4096, pages=1024),
        dict(name="turnover 256 of 131072 pages", op="turnover", n=256, ctx=32768, pages=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.499)))))


def draw(rng: random.Random):
    while True:
        op = rng.choice(["window", "window", "tree", "tree", "commit", "fork", "turnover"])
        if op == "window":
            rows = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 2048)])
            c = dict(op=op, batch=_log(rng, 1, 128), rows=rows, ctx=_log(rng, max(rows, 33), 131072),
                     jitter=rng.choice([0.0, 0.25]), window=_log(rng, 1, 65536), sinks=rng.choice([0, rng.randint(1, 256)]))
        elif op == "tree":
            c = dict(op=op, batch=_log(rng, 1, 64), nodes=rng.randint(1, 64), ctx=_log(rng, 64, 32768), jitter=rng.choice([0.0, 0.25]))
        elif op == "commit":
            c = dict(op=op, batch=_log(rng, 1, 128), nodes=rng.randint(1, 64), ctx=_log(rng, 64, 4096), kv=rng.randint(1, 78), idx=rng.randint(1, 21))
        elif op == "fork":
            c = dict(op=op, n=_log(rng, 1, 64), ctx=_log(rng, 1, 8229), kv=rng.randint(1, 78), idx=rng.randint(1, 21))
        else:
            c = dict(op=op, n=_log(rng, 1, 256), ctx=_log(rng, 64, 32768), pages=_log(rng, 1024, 131072))
            if c["n"] * (c["ctx"] // PAGE + 2) > c["pages"]:
                continue
        if op in ("window", "tree"):
            w = work(c)
            span = _span(c)
            if w["flops"] > 2.2e12 or w["bytes"] > 9e8 or c["batch"] * _rows(c) * HEADS * span > 1.05e9 or c["batch"] * span > 4e6:
                continue
        return c


def _rows(c):
    return c["rows"] if c["op"] == "window" else c["nodes"]


def _lens(c):
    """(context, new tokens) of each request, from the case alone: contexts ctx (1 +- jitter), trees of 3/4 to all of the nodes."""
    got = []
    for r in range(c["batch"]):
        f = (r * 0.6180339887) % 1.0
        L = max(1, int(c["ctx"] * (1.0 + c.get("jitter", 0.0) * (2.0 * f - 1.0))))
        if c["op"] == "window":
            n = min(c["rows"], L)
        else:
            n = c["nodes"] - int(f * (c["nodes"] // 4 + 1))
            L += n
        got.append((L, n))
    return got


def _span(c):
    """Positions that the rows of one request see together, at most."""
    L = max(x for x, _ in _lens(c))
    return L if c["op"] == "tree" else min(L, c["sinks"] + c["window"] + c["rows"] - 1)


def _tree(c, r):
    """Parent of each node of request r's tree, -1 for the root's children; half of the nodes extend the newest branch."""
    rng = random.Random(1000 + r)
    n = _lens(c)[r][1]
    return [-1 if u == 0 else (u - 1 if rng.random() < 0.5 else rng.randrange(-1, u)) for u in range(n)]


def _path(parents):
    """The longest path from the root, the one a commit keeps (ties: the lowest leaf)."""
    best, at = [], {-1: []}
    for u, p in enumerate(parents):
        at[u] = at[p] + [u]
        if len(at[u]) > len(best):
            best = at[u]
    return best


def work(c):
    op = c["op"]
    if op in ("window", "tree"):
        tokens = pairs = rows = 0
        for r, (L, n) in enumerate(_lens(c)):
            rows += n
            if op == "window":
                s, w = c["sinks"], c["window"]
                seen = lambda p: min(p + 1, min(p + 1, w) + min(s, max(0, p + 1 - w)))  # noqa: E731
                pairs += sum(seen(p) for p in range(L - n, L))
                tokens += min(L, min(s, max(0, L - n + 1 - w)) + min(L, w + n - 1))
            else:
                depth = [0] * n
                for u, p in enumerate(_tree(c, r)):
                    depth[u] = 1 if p < 0 else depth[p] + 1
                pairs += n * (L - n) + sum(depth)
                tokens += L
        io = rows * HEADS * (QK * 2 + LATENT * 2 + 4)
        return dict(bytes=tokens * KV_ROW + io, flops=pairs * HEADS * 2 * (QK + LATENT))
    row = c.get("kv", 0) * KV_ROW + c.get("idx", 0) * 132
    if op == "commit":
        moved = sum(sum(a != k for k, a in enumerate(_path(_tree(c, r)))) for r in range(c["batch"]))
        return dict(bytes=2 * moved * row + 8 * c["batch"] * c["nodes"], flops=0)
    if op == "fork":
        full, part = divmod(c["ctx"], PAGE)
        # each child: the shared pages' table entries given back and taken again, the counts, the partial page's rows
        return dict(bytes=c["n"] * (2 * part * row + 5 * 4 * (full + 1)) + 8 * full, flops=0)
    held = c["n"] * ((c["ctx"] + PAGE - 1) // PAGE)
    return dict(bytes=held * 2 * (3 * 4), flops=0)


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(1234567 + seed)


def _latent_pages(n_pages, g):
    """Latent pages as the store leaves them: 512 values N(0, 1) times a per-token size, four FP8 blocks with power-of-two scales, 64 bf16."""
    cache = torch.empty(n_pages * PAGE, KV_ROW, dtype=torch.uint8, device=DEV)
    step = 1 << 19
    for a in range(0, cache.shape[0], step):
        b = min(cache.shape[0], a + step)
        c = torch.randn(b - a, 4, 128, generator=g, device=DEV)
        c *= torch.exp(0.3 * torch.randn(b - a, 1, 1, generator=g, device=DEV))
        e = torch.ceil(torch.log2(c.abs().amax(2, keepdim=True) / 448.0))
        s = torch.exp2(e)
        cache[a:b, :512] = (c / s).to(torch.float8_e4m3fn).view(torch.uint8).reshape(b - a, 512)
        cache[a:b, 512:528] = s.reshape(b - a, 4).contiguous().view(torch.uint8)
        cache[a:b, 528:] = torch.randn(b - a, 64, generator=g, device=DEV).to(torch.bfloat16).view(torch.uint8)
    return cache.reshape(-1)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _prepare_attention(c, seed):
    g = _gen(seed)
    lens = _lens(c)
    B, rows = c["batch"], _rows(c)
    L = [x for x, _ in lens]
    n = [x for _, x in lens]
    T = sum(n)
    width = (max(L) + PAGE - 1) // PAGE
    need = torch.zeros(B, width, dtype=torch.bool)
    for r in range(B):
        last = (L[r] + PAGE - 1) // PAGE
        if c["op"] == "tree":
            need[r, :last] = True
        else:
            need[r, : (min(c["sinks"], L[r]) + PAGE - 1) // PAGE] = True
            need[r, max(0, L[r] - n[r] - c["window"] + 1) // PAGE: last] = True
    total = int(need.sum())
    pages = total + 3
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[need.to(DEV)] = perm[:total]
    st = dict(case=c, q=torch.randn(T, HEADS, QK, generator=g, device=DEV).to(torch.bfloat16), kv=_latent_pages(pages, g),
              pages=pages, table=table, seq_len=_ints(L), q_start=_ints([sum(n[:r]) for r in range(B + 1)]), T=T,
              max_len=max(L), max_q=max(n), span=_span(c))
    if c["op"] == "tree":
        masks = []
        for r in range(B):
            m = []
            for u, p in enumerate(_tree(c, r)):
                m.append((m[p] if p >= 0 else 0) | 1 << u)
            masks += [x - (1 << 64) if x >> 63 else x for x in m]
        st["mask"] = torch.tensor(masks, dtype=torch.int64, device=DEV)
    st["out"] = torch.empty(T, HEADS, LATENT, dtype=torch.bfloat16, device=DEV)
    st["lse"] = torch.empty(T, HEADS, dtype=torch.float32, device=DEV)
    return st


def _raw(layers, pages, page_bytes, g):
    """Whole pages of bytes for `layers` layers: what a copy moves has no say in it."""
    if layers == 0:
        return torch.zeros(0, pages, page_bytes, dtype=torch.uint8, device=DEV)
    words = torch.empty(layers * pages * page_bytes // 4, dtype=torch.int32, device=DEV)
    words.random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    return words.view(torch.uint8).view(layers, pages, page_bytes)


def prepare(case, seed):
    c, op = case, case["op"]
    if op in ("window", "tree"):
        return _prepare_attention(c, seed)
    g = _gen(seed)
    if op == "commit":
        # every request reads the same cached prompt; its tree's tokens lie in pages of its own
        B, n = c["batch"], [x for _, x in _lens(c)]
        first = c["ctx"] // PAGE
        width = (c["ctx"] + max(n) + PAGE - 1) // PAGE
        pages = first + B * (width - first)
        perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.cat([perm[:first].expand(B, first), perm[first:].view(B, width - first)], 1).contiguous()
        # a request keeps its longest path, or the first tokens of it: the seed says how many of them the model accepted
        rng = random.Random(seed)
        accept = torch.full((B, c["nodes"]), -1, dtype=torch.int32)
        for r in range(B):
            path = _path(_tree(c, r))
            path = path[: rng.randint(max(1, len(path) - 2), len(path))]
            accept[r, : len(path)] = torch.tensor(path, dtype=torch.int32)
        return dict(case=c, table=table, seq_len=_ints([c["ctx"] + x for x in n]), q_start=_ints([sum(n[:r]) for r in range(B + 1)]),
                    T=sum(n), max_len=c["ctx"] + max(n), max_q=max(n), pages=pages, accept=accept.to(DEV),
                    kv=_raw(c["kv"], pages, KV_PAGE, g), idx=_raw(c["idx"], pages, IDX_PAGE, g),
                    new_len=torch.empty(B, dtype=torch.int32, device=DEV))
    if op == "fork":
        n, held = c["n"], (c["ctx"] + PAGE - 1) // PAGE
        pages = held + n + 5
        perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((n + 1, held + 1), -1, dtype=torch.int32, device=DEV)
        table[0, :held] = perm[:held]
        ref = torch.zeros(pages, dtype=torch.int32, device=DEV)
        ref[perm[:held].long()] = 1
        return dict(case=c, table=table, ref=ref, pages=pages, src=_ints([0] * n), dst=_ints(list(range(1, n + 1))), length=_ints([c["ctx"]] * n),
                    zero=_ints([0] * n), end=_ints([held + 1] * n), kv=_raw(c["kv"], pages, KV_PAGE, g), idx=_raw(c["idx"], pages, IDX_PAGE, g))
    # turnover: n requests hold pages all over the pool, others hold some of the rest
    n, held = c["n"], (c["ctx"] + PAGE - 1) // PAGE
    pages = c["pages"]
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((n, held + 1), -1, dtype=torch.int32, device=DEV)
    table[:, :held] = perm[: n * held].view(n, held)
    ref = torch.zeros(pages, dtype=torch.int32, device=DEV)
    ref[perm[: n * held + (pages - n * held) // 3].long()] = 1
    want = (torch.rand(n, generator=g, device=DEV) * 0.5 + 0.5) * c["ctx"]
    return dict(case=c, table=table, ref=ref, pages=pages, rows=_ints(list(range(n))), zero=_ints([0] * n), end=_ints([held + 1] * n),
                want=want.to(torch.int32).clamp_(1))


# ------------------------------------------------------------------------------------------------ plain forms
def _rows_fp32(kv, pages, table, pos, ok):
    """Dequantised latent rows [B, N, 576] at positions `pos` of each request."""
    page = torch.where(ok, torch.gather(table.long(), 1, pos // PAGE), torch.zeros_like(pos))
    ok = ok & (page >= 0)
    raw = kv.view(pages, PAGE, KV_ROW)[page.clamp(min=0), pos % PAGE]
    c = raw[..., :512].contiguous().view(torch.float8_e4m3fn).float()
    s = raw[..., 512:528].contiguous().view(torch.float32)
    k = torch.cat([c * s.repeat_interleave(128, -1), raw[..., 528:].contiguous().view(torch.bfloat16).float()], -1)
    return torch.where(ok[..., None], k, torch.zeros_like(k)), ok


def _plain_attention(st):
    c = st["case"]
    seq, start, T, Q = st["seq_len"].long(), st["q_start"].long(), st["T"], st["max_q"]
    n = start[1:] - start[:-1]
    first = seq - n
    t = torch.arange(Q, device=DEV)
    row = (start[:-1, None] + t).clamp(max=T - 1)
    p = first[:, None] + t
    at = torch.arange(st["span"], device=DEV)
    if c["op"] == "window":
        s, w = c["sinks"], c["window"]
        s_here = min(s, st["span"])
        lo = (first - w + 1).clamp(min=s)
        pos = torch.cat([at[:s_here].expand(len(seq), -1), lo[:, None] + at[: st["span"] - s_here]], 1)
        see = (pos[:, None] <= p[..., None]) & ((pos[:, None] < s) | (pos[:, None] > p[..., None] - w))
    else:
        pos = at.expand(len(seq), -1)
        bit = (pos - first[:, None]).clamp(0, 63)
        see = (pos < first[:, None])[:, None] | ((st["mask"][row][..., None] >> bit[:, None]) & 1).bool() & (pos >= first[:, None])[:, None]
    ok = pos < seq[:, None]
    k, ok = _rows_fp32(st["kv"], st["pages"], st["table"], torch.where(ok, pos, torch.zeros_like(pos)), ok)
    see = see & ok[:, None]
    q = st["q"][row].float().reshape(len(seq), Q * HEADS, QK)
    x = torch.bmm(q, k.transpose(1, 2)).view(len(seq), Q, HEADS, -1) * SCALE
    x = x.masked_fill_(~see[:, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.bmm(x.view(len(seq), Q * HEADS, -1), k[..., :LATENT]).view(len(seq), Q, HEADS, LATENT)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    at = torch.searchsorted(start[1:], torch.arange(T, device=DEV), right=True)
    mine = at * Q + torch.arange(T, device=DEV) - start[at]
    lse = (m + total.log()).view(-1, HEADS)
    return dict(out=o.view(-1, HEADS, LATENT)[mine].to(torch.bfloat16), lse=lse[mine])


def _plain_commit(st):
    seq, start, accept = st["seq_len"].long(), st["q_start"].long(), st["accept"].long()
    n = start[1:] - start[:-1]
    first = seq - n
    k = torch.arange(accept.shape[1], device=DEV)
    ok = accept >= 0
    stay = torch.minimum(k[None], n[:, None] - 1)
    src = first[:, None] + torch.where(ok, accept, stay)
    dst = first[:, None] + torch.where(ok, k[None].expand_as(accept), stay)
    sp, dp = torch.gather(st["table"].long(), 1, src // PAGE), torch.gather(st["table"].long(), 1, dst // PAGE)
    kv, idx = st["kv"].view(-1, st["pages"], PAGE, KV_ROW), st["idx"]
    kv[:, dp, dst % PAGE] = kv[:, sp, src % PAGE]
    keys, scales = idx[..., :IDX_PAYLOAD].unflatten(-1, (PAGE, 128)), idx[..., IDX_PAYLOAD:].unflatten(-1, (PAGE, 4))
    keys[:, dp, dst % PAGE] = keys[:, sp, src % PAGE]
    scales[:, dp, dst % PAGE] = scales[:, sp, src % PAGE]
    return dict(kv=st["kv"].view(torch.int32), idx=st["idx"].view(torch.int32), seq_len=(first + ok.sum(1)).to(torch.int32))


def _plain_release(ref, table, rows, lo, hi):
    k = torch.arange(table.shape[1], device=DEV)
    held = table[rows.long()]
    mine = (k >= lo[:, None]) & (k < hi[:, None])
    drop = mine & (held >= 0)
    ref.index_add_(0, held.clamp(min=0).flatten().long(), -drop.flatten().to(torch.int32))
    table[rows.long()] = torch.where(mine, torch.full_like(held, -1), held)


def _plain_free(ref):
    """The pool's pages, free ones first, each part in ascending order."""
    return torch.sort((ref > 0).to(torch.int8), stable=True).indices


def _plain_fork(st):
    ref, table = st["ref"], st["table"]
    src, dst, full, part = st["src"].long(), st["dst"].long(), st["length"].long() // PAGE, st["length"].long() % PAGE
    _plain_release(ref, table, st["dst"], st["zero"], st["end"])
    k = torch.arange(table.shape[1], device=DEV)
    held = table[src]
    fresh = part > 0
    new = _plain_free(ref)[(fresh.long().cumsum(0) - 1).clamp(min=0)]
    shared = (k < full[:, None]) & (held >= 0)
    ref.index_add_(0, held.clamp(min=0).flatten().long(), shared.flatten().to(torch.int32))
    ref.index_add_(0, new, fresh.to(torch.int32))
    last = torch.gather(held, 1, full.clamp(max=held.shape[1] - 1)[:, None])[:, 0].clamp(min=0).long()
    table[dst] = torch.where(shared, held, torch.where((k == full[:, None]) & fresh[:, None], new[:, None].to(torch.int32), torch.full_like(held, -1)))
    copy = (torch.arange(PAGE, device=DEV) < part[:, None])[None, ..., None]
    new, last = torch.where(fresh, new, last), last
    kv, idx = st["kv"].view(-1, st["pages"], PAGE, KV_ROW), st["idx"]
    kv[:, new] = torch.where(copy, kv[:, last], kv[:, new])
    keys, scales = idx[..., :IDX_PAYLOAD].unflatten(-1, (PAGE, 128)), idx[..., IDX_PAYLOAD:].unflatten(-1, (PAGE, 4))
    keys[:, new] = torch.where(copy, keys[:, last], keys[:, new])
    scales[:, new] = torch.where(copy, scales[:, last], scales[:, new])
    return dict(kv=st["kv"].view(torch.int32), idx=st["idx"].view(torch.int32), table=table, ref=ref)


def _plain_turnover(st):
    ref, table = st["ref"], st["table"]
    _plain_release(ref, table, st["rows"], st["zero"], st["end"])
    k = torch.arange(table.shape[1], device=DEV)
    take = k < ((st["want"].long() + PAGE - 1) // PAGE)[:, None]
    rank = take.flatten().long().cumsum(0) - 1
    new = _plain_free(ref)[rank.clamp(min=0)]
    ref.index_add_(0, new, take.flatten().to(torch.int32))
    rows = st["rows"].long()
    table[rows] = torch.where(take, new.view(take.shape).to(torch.int32), table[rows])
    return dict(table=table, ref=ref)


# ------------------------------------------------------------------------------------------------ the library's calls
def _own(st):
    import dsa_sparse_attention_indexer_gb300 as D
    op = st["case"]["op"]
    if "handle" not in st:                               # what a program keeps from step to step
        h = st["handle"] = {}
        if op in ("window", "tree", "commit"):
            h["batch"] = D.Batch(st["seq_len"], st["q_start"], st["table"], st["pages"], max_seq_len=st["max_len"], max_q_len=st["max_q"], total_q=st["T"])
        if op in ("window", "tree"):
            h["ws"] = D.workspace(D.dsa_dense_mla_workspace_size(h["batch"]), DEV)
        if op in ("commit", "fork"):
            h["caches"] = D.CacheSet([(x, D.CACHE_KV) for x in st["kv"]] + [(x, D.CACHE_IDXK) for x in st["idx"]], st["pages"])
    h = st["handle"]
    if op == "window":
        D.dsa_window_mla(st["q"], st["kv"], h["batch"], window=st["case"]["window"], sinks=st["case"]["sinks"], softmax_scale=SCALE,
                         out=st["out"], lse=st["lse"], ws=h["ws"])
        return dict(out=st["out"], lse=st["lse"])
    if op == "tree":
        D.dsa_tree_mla(st["q"], st["mask"], st["kv"], h["batch"], softmax_scale=SCALE, out=st["out"], lse=st["lse"], ws=h["ws"])
        return dict(out=st["out"], lse=st["lse"])
    if op == "commit":
        D.dsa_tree_commit(st["accept"], h["batch"], h["caches"], new_seq_len=st["new_len"])
        return dict(kv=st["kv"].view(torch.int32), idx=st["idx"].view(torch.int32), seq_len=st["new_len"])
    if op == "fork":
        D.dsa_pages_release(st["ref"], st["table"], st["dst"], st["zero"], st["end"])
        D.dsa_pages_fork(st["ref"], st["table"], st["src"], st["dst"], st["length"], h["caches"])
        return dict(kv=st["kv"].view(torch.int32), idx=st["idx"].view(torch.int32), table=st["table"], ref=st["ref"])
    D.dsa_pages_release(st["ref"], st["table"], st["rows"], st["zero"], st["end"])
    D.dsa_pages_reserve(st["ref"], st["table"], st["rows"], st["zero"], st["want"])
    return dict(table=st["table"], ref=st["ref"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("window", "tree"):
        return _plain_attention(state)
    return {"commit": _plain_commit, "fork": _plain_fork, "turnover": _plain_turnover}[op](state)


# ------------------------------------------------------------------------------------------------ 64 bits
def _e4m3_values():
    v = []
    for code in range(256):
        e, m = code >> 3 & 15, code & 7
        x = math.nan if e == 15 and m == 7 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v.append(-x if code & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def exact(case, seed):
    """Row by row from the definition, in 64 bits; the paged operators move whole numbers only."""
    if case["op"] not in ("window", "tree"):
        return None
    st = prepare(case, seed)
    values = _e4m3_values()
    cache = st["kv"].view(-1, KV_ROW)
    out, lse = [], []
    begin = 0
    for r, (L, n) in enumerate(_lens(case)):
        P = L - n
        j = torch.arange(L, device=DEV)
        if case["op"] == "window":
            j = j[(j < case["sinks"]) | (j > P - case["window"])]
        slot = st["table"][r, j // PAGE].long() * PAGE + j % PAGE
        raw = cache[slot]
        latent = values[raw[:, :512].long()].view(-1, 4, 128) * raw[:, 512:528].contiguous().view(torch.float32).double()[..., None]
        latent = latent.view(-1, 512)
        rope = raw[:, 528:].contiguous().view(torch.bfloat16).double()
        for a in range(0, n, 64):
            b = min(n, a + 64)
            p = torch.arange(P + a, P + b, device=DEV)
            if case["op"] == "window":
                see = (j <= p[:, None]) & ((j < case["sinks"]) | (p[:, None] - j < case["window"]))
                use = see.any(0)
            else:
                anc = torch.zeros(b - a, L, dtype=torch.bool)
                anc[:, :P] = True
                parents = _tree(case, r)
                for u in range(a, b):
                    v = u
                    while v >= 0:
                        anc[u - a, P + v] = True
                        v = parents[v]
                see = anc.to(DEV)
                use = torch.ones(len(j), dtype=torch.bool, device=DEV)
            see = see[:, use]
            q = st["q"][begin + a: begin + b].double().view(-1, QK)
            s = (q[:, :512] @ latent[use].T + q[:, 512:] @ rope[use].T) / 16.0
            s = s.view(b - a, HEADS, -1).masked_fill(~see[:, None], -math.inf)
            z = torch.logsumexp(s, -1)
            w = torch.exp(s - z[..., None])
            out.append((w.view(-1, w.shape[-1]) @ latent[use]).view(b - a, HEADS, LATENT))
            lse.append(z)
        begin += n
    return dict(out=torch.cat(out), lse=torch.cat(lse))
