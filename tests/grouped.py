"""What the tests of attention on grouped heads share: random KV8 caches and the bounds on outputs.

With A the largest sum of a row's products |q_d k_d| times the softmax scale, a score is off by at most D steps of its
fp32 sum, 2 D 2^-24 A for a sum that cuts off, and 2^-22 of the score in the exponent (log2 units and the power of
two's approximation): at most OFF = (2 D 2^-24 + 2^-21) A.  A probability is off by that, by its rounding P and, in fp16
and where it is small, by 2^-25: with the largest contribution at 2^6.5 or more, and codes of up to twice its block's largest
one, by less than 2^-30 of the largest value; sums over n positions and their merge are off by (n + 64) 2^-23 of the sum of sizes W.
Numerator and denominator both count the scores' error:
  |out - exact| <= W (P + 2 OFF + (n + 64) 2^-23) + n 2^-30 max|v| (+ half a step of the output)
  |lse - exact| <= 2 OFF + (n + 64) 2^-23 + 2^-21 (1 + |lse|)
"""

import numpy as np
import torch

import dsa_sparse_attention_indexer_gb300 as D
from oracle import dsa_oracle as O

DEV = "cuda"


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def random_cache(pages, kv, dim, g, spread=2):
    """Random codes (no NaN) and scales 2^e, e in [-6 - spread, -6 + spread]."""
    cache = torch.randint(0, 256, (pages, D.kv8_page_bytes(kv, dim)), generator=g, dtype=torch.uint8)
    k, v, s = D.kv8_views(cache, kv, dim)
    for i, x in ((0, k), (1, v)):
        y = torch.randn(x.shape, generator=g) * 90.0
        x.copy_(y.clamp(-448, 448).to(torch.float8_e4m3fn))
        s[:, :, i] = torch.exp2(torch.randint(-6 - spread, -5 + spread, s[:, :, i].shape, generator=g).float())
    return cache


def cache_case(seq, n, kv, group, dim, seed=0, pad_rows=0, spread=2, q_size=1.0, max_pages=None):
    g = torch.Generator().manual_seed(77 + seed)
    B, T = len(seq), sum(n)
    width = max(1, max((L + 63) // 64 for L in seq)) if max_pages is None else max_pages
    used = [min(width, (max(L, 0) + 63) // 64) for L in seq]
    pages = sum(used) + 3
    perm = torch.randperm(pages, generator=g)[: sum(used)].to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for r, u in enumerate(used):
        table[r, :u] = perm[at:at + u]
        at += u
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    q = (torch.randn(T + pad_rows, kv * group, dim, generator=g) * q_size).to(torch.bfloat16)
    cache = random_cache(pages, kv, dim, g, spread)
    c = dict(seq=list(seq), n=list(n), kv=kv, group=group, dim=dim, heads=kv * group, T=T, start=start, table=table, pages=pages, q=q.to(DEV),
             cache=cache, pad=pad_rows)
    return place(c)


def place(c):
    """(Re)makes the batch and the device's copy of the cache from the case's host side."""
    c["dev_cache"] = c["cache"].to(DEV)
    c["batch"] = D.Batch(torch.tensor(c["seq"], dtype=torch.int32, device=DEV), torch.tensor(c["start"], device=DEV), c["table"].to(DEV),
                         c["pages"], max_seq_len=c["table"].shape[1] * 64, max_q_len=max(c["n"] + [-(-(c["T"] + c["pad"]) // len(c["n"]))]), total_q=c["T"] + c["pad"])
    return c


def expected(c, scale=None):
    """(out, lse, bound of out without rounding, bound of lse) of every row, for probabilities rounded to `P`."""
    scale = c["dim"] ** -0.5 if scale is None else scale
    cache = c["cache"].numpy().reshape(-1)
    got = []
    for r, (L, n) in enumerate(zip(c["seq"], c["n"])):
        if n:
            k, v, ok = O.kv8_read(cache, c["kv"], c["dim"], c["table"][r].numpy(), max(L, 0), c["pages"])
            got.append(bounds(f64(c["q"][c["start"][r]:c["start"][r] + n]), k, v, L - n, scale, 2.0 ** -11, ok))
    return [np.concatenate(x) for x in zip(*got)]


def bounds(q, k, v, first, scale, P, ok=None):
    out, lse, W = O.grouped_attention(q, k, v, first, scale, ok)
    n, heads, dim = q.shape
    G = heads // k.shape[1]
    L = len(k)
    A, top = np.zeros((n, heads)), np.zeros((heads, dim))
    fine = np.nan_to_num(np.abs(k), nan=0.0, posinf=0.0)
    fv = np.nan_to_num(np.abs(v), nan=0.0, posinf=0.0)
    if ok is not None:
        fine, fv = fine * ok[:, None, None], fv * ok[:, None, None]
    for h in range(heads):
        if L:
            A[:, h] = scale * (np.abs(q[:, h]) @ fine[:, h // G].T).max(1)
            top[h] = fv[:, h // G].max()
    off = (2 * dim * 2.0 ** -24 + 2.0 ** -21) * A
    tol = W * (P + 2 * off + (L + 64) * 2.0 ** -23)[..., None] + (L * 2.0 ** -30 if P < 2.0 ** -10 else 0.0) * top
    lse_tol = 2 * off + (L + 64) * 2.0 ** -23 + 2.0 ** -21 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))
    return out, lse, tol, lse_tol


def check(got, lse, want, what=""):
    out, z, tol, lse_tol = want
    T = len(out)
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    got, lse = f64(got[:T]), f64(lse[:T])
    fine = np.isfinite(out)
    assert np.array_equal(np.isnan(got), ~fine), f"{what}: NaN in other places"
    err, lim = np.abs(got[fine] - out[fine]), (tol * (1 + half) + half * np.abs(out))[fine]
    assert np.all(err <= lim + 1e-37), f"{what}: out off by {np.max(err / (lim + 1e-37)):.2f} of the bound"
    assert np.array_equal(np.isneginf(lse), np.isneginf(z)) and np.array_equal(np.isnan(lse), np.isnan(z)), f"{what}: lse"
    f = np.isfinite(z)
    err = np.abs(lse[f] - z[f])
    assert np.all(err <= lse_tol[f]), f"{what}: lse off by {np.max(err / lse_tol[f]):.2f} of the bound"
