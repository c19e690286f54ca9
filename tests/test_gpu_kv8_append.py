"""dsa_kv8_append against the 64-bit oracle: rotation, scales, codes, and every byte that it must leave alone.

Values go straight from bf16 to E4M3: their codes and scales are the oracle's.  Rotated numbers are formed in fp32:
with |cos|, |sin| <= 1 the angle's rounding to 24 bits (pi 2^-25 < 2^-23), the error of the sine (2 ulp, 2^-23) and
the two products and the sum (each 2^-24 of at most |a| + |b|) stay within TURN (|a| + |b|) of the exact ones, so a
key's code is that of some number within that of the exact one, and a bf16 output within that and half a step, 2^-8.
"""

import numpy as np
import pytest
import torch

import dsa_sparse_attention_indexer_gb300 as D
from oracle import dsa_oracle as O
from tests.oracle_side import f64

pytestmark = pytest.mark.gpu

DEV = "cuda"
TURN = 2.0 ** -21


def _case(seq_len, q_len, kv, group, dim, seed=0, pad_rows=0, size=1.0, extra_pages=2):
    """A batch, its random tensors and a cache of random codes; pages in random order."""
    g = torch.Generator().manual_seed(1000 + seed)
    B = len(seq_len)
    width = max(1, max((L + 63) // 64 for L in seq_len))
    pages = B * width + extra_pages
    perm = torch.randperm(pages, generator=g)[: B * width].to(torch.int32).view(B, width)
    T = sum(q_len)
    start = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
    x = torch.randn(T + pad_rows, kv * (group + 2), dim, generator=g) * size
    x *= torch.exp(torch.randn(T + pad_rows, 1, 1, generator=g))
    x = x.to(torch.bfloat16).to(DEV)
    heads = kv * group
    cache = torch.randint(0, 256, (pages, D.kv8_page_bytes(kv, dim)), generator=g, dtype=torch.uint8)
    scale = D.kv8_views(cache, kv, dim)[2]
    scale.copy_(torch.exp2(torch.randint(-9, -3, scale.shape, generator=g).float()))
    batch = D.Batch(torch.tensor(seq_len, dtype=torch.int32, device=DEV), torch.tensor(start, device=DEV), perm.to(DEV), pages,
                    max_seq_len=width * 64, max_q_len=max(q_len + [1]), total_q=T + pad_rows)
    return dict(seq=seq_len, n=q_len, start=start, table=perm.numpy().copy(), pages=pages, q=x[:, :heads], k=x[:, heads:heads + kv],
                v=x[:, heads + kv:], cache=cache.to(DEV), batch=batch, kv=kv, heads=heads, dim=dim, T=T)


def _blocks(cache, kv, dim):
    """Numpy copies: K codes and V codes [pages, kv, 4, 16, dim], scales [pages, kv, 2, 4]."""
    k, v, s = D.kv8_views(cache, kv, dim)
    return (k.view(torch.uint8).cpu().numpy().copy(), v.view(torch.uint8).transpose(-1, -2).cpu().numpy().copy(), s.cpu().numpy().copy())


def _check(c, before, rope, halves, q_out=None, k_out=None, inv_freq=None, base=10000.0):
    kv, dim = c["kv"], c["dim"]
    now = _blocks(c["cache"], kv, dim)
    want = [x.copy() for x in before]
    pos = np.concatenate([np.arange(L - n, L) for L, n in zip(c["seq"], c["n"])] + [np.zeros(0, int)]).astype(np.int64)
    T = c["T"]

    def turned(x):
        x = f64(x[:T])
        size = np.abs(x).copy()
        if rope:
            i = np.arange(rope // 2)
            a, b = (i, i + rope // 2) if halves else (2 * i, 2 * i + 1)
            size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
            off = TURN * size
            off[..., rope:] = 0.0
            with np.errstate(invalid="ignore"):
                return O.rope_pairs(x, pos, rope, halves, inv_freq, base), off
        return x, np.zeros_like(x)

    k, k_off = turned(c["k"])
    v = f64(c["v"][:T])
    for got, x, off in ((q_out, *(turned(c["q"]) if q_out is not None else (None, None))), (k_out, k, k_off)):
        if got is not None:
            got = f64(got[:T])
            fine = np.isfinite(x)
            assert np.all(np.abs(got - x)[fine] <= (2.0 ** -8 * np.abs(x) + off * (1 + 2.0 ** -8))[fine] + 1e-38)
            assert not np.any(np.isfinite(got[~fine]))
    limit = 448.0 * 2.0 ** 24
    for r, (L, n) in enumerate(zip(c["seq"], c["n"])):
        for p in range(L - n, L):
            if p < 0 or p // 64 >= c["table"].shape[1] or (p != max(0, L - n) and p % 16):
                continue
            pg, at = int(c["table"][r, p // 64]), p % 64 // 16
            if pg < 0 or pg >= c["pages"]:
                continue
            row, held, m = c["start"][r] + p - (L - n), p % 16, min(16 - p % 16, L - p)
            for h in range(kv):
                e_was = int(np.frexp(before[2][pg, h, 1, at])[1]) - 1
                want[1][pg, h, at], e = O.kv8_block_append(before[1][pg, h, at], e_was, held, v[row:row + m, h])
                want[2][pg, h, 1, at] = 2.0 ** e
                # keys: the scale of some number near the largest, then codes of numbers near the exact ones
                x, off = k[row:row + m, h], k_off[row:row + m, h]
                e_was = int(np.frexp(before[2][pg, h, 0, at])[1]) - 1
                with np.errstate(invalid="ignore"):
                    good = np.abs(x) <= limit
                lo, hi = (O.kv8_exponent(float(np.max(np.maximum(0.0, np.abs(x[good]) + s * off[good]), initial=0.0))) for s in (-1, 1))
                e = int(np.frexp(now[2][pg, h, 0, at])[1]) - 1
                assert (max(lo, e_was) if held else lo) <= e <= (max(hi, e_was) if held else hi)
                assert now[2][pg, h, 0, at] == 2.0 ** e
                want[2][pg, h, 0, at] = 2.0 ** e
                if held and e > e_was:
                    grown = O.kv8_block_append(before[0][pg, h, at], e_was, held, np.full((1, dim), 448.0 * 2.0 ** e))[0]
                    want[0][pg, h, at, :held] = grown[:held]
                codes = now[0][pg, h, at, held:held + m]
                value = O.e4m3_decode(codes)
                top = 448.0
                near = [np.clip(np.where(good, x + s * off, 0.0) * 2.0 ** -e, -top, top) for s in (-1, 1)]
                ok = np.where(good, (value >= O.e4m3_decode(O.e4m3_encode(near[0]))) & (value <= O.e4m3_decode(O.e4m3_encode(near[1]))), codes == 0x7f)
                assert ok.all(), (r, p, h, np.argwhere(~ok)[:4])
                want[0][pg, h, at, held:held + m] = codes
    for got, exp, name in zip(now, want, ("keys", "values", "scales")):
        bad = np.argwhere(got.view(np.uint8 if got.dtype == np.uint8 else np.uint32) != exp.view(np.uint8 if exp.dtype == np.uint8 else np.uint32))
        assert len(bad) == 0, (name, len(bad), bad[:4])


SHAPES = [
    # seq_len, q_len, kv_heads, group, dim, rope, halves
    ([1], [1], 1, 1, 128, 128, True),
    ([8192], [1], 8, 8, 128, 128, True),
    ([16, 17, 64, 65, 1, 100], [1, 1, 1, 1, 1, 1], 2, 4, 128, 64, False),
    ([70, 5, 0, 31, 200], [7, 5, 0, 20, 0], 3, 5, 64, 64, True),
    ([300, 10003], [300, 133], 2, 2, 128, 32, True),
    ([129, 47], [129, 31], 4, 1, 256, 256, False),
    ([640, 90], [333, 64], 2, 7, 256, 128, True),
    ([50, 51, 52], [50, 2, 17], 5, 3, 64, 0, True),
    ([2200], [2177], 1, 2, 128, 128, True),
]


@pytest.mark.parametrize("seq,n,kv,group,dim,rope,halves", SHAPES)
def test_append(seq, n, kv, group, dim, rope, halves):
    c = _case(seq, n, kv, group, dim, seed=len(seq))
    before = _blocks(c["cache"], kv, dim)
    k_out = torch.empty(c["T"], kv, dim, dtype=torch.bfloat16, device=DEV)
    st = D.new_device_status(DEV)
    q_out = D.dsa_kv8_append(c["k"], c["v"], c["cache"], c["batch"], q=c["q"], rope_dims=rope,
                             rope_style=D.ROPE_HALVES if halves else D.ROPE_INTERLEAVED, k_out=k_out, dev_status=st)
    _check(c, before, rope, halves, q_out, k_out)
    assert D.dsa_device_status_read(st)[0] == 0


def test_append_one_by_one_grows_scales():
    """Tokens of growing sizes, one call each: earlier codes of a block are rounded again to its new scale."""
    kv, dim = 2, 128
    c = _case([40], [40], kv, 1, dim)
    for t in range(40):
        one = dict(c, seq=[t + 1], n=[1], start=np.array([0, 1]), T=1)
        one["k"], one["v"] = c["k"][t:t + 1] * 2.0 ** (t % 19 - 9), c["v"][t:t + 1] * 2.0 ** (t % 17 - 9)
        b = c["batch"]
        one["batch"] = D.Batch(torch.tensor([t + 1], dtype=torch.int32, device=DEV), torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                               b.page_table, c["pages"])
        before = _blocks(c["cache"], kv, dim)
        D.dsa_kv8_append(one["k"], one["v"], c["cache"], one["batch"])
        _check(one, before, dim, True)


def test_append_extreme_values():
    """Zeros, the smallest and largest numbers, infinities and NaN: a scale within its limits, NaN codes, others' codes unharmed."""
    kv, dim = 4, 64
    c = _case([37, 20], [37, 9], kv, 2, dim)
    c["k"], c["v"] = c["k"].clone(), c["v"].clone()
    for x in (c["k"], c["v"]):
        x[:16, 0] = 0.0
        x[16:20, 1] = 1e-38
        x[3, 2] = float("inf")
        x[20, 2, 5] = float("nan")
        x[21, 2, 7] = -float("inf")
        x[30:, 3] = 3e38
        x[40, 3] = -2.0 ** 33
    before = _blocks(c["cache"], kv, dim)
    D.dsa_kv8_append(c["k"], c["v"], c["cache"], c["batch"], rope_dims=0)
    _check(c, before, 0, True)


def test_append_held_nan_codes_stay():
    kv, dim = 1, 128
    c = _case([9], [1], kv, 1, dim)
    k, v, s = D.kv8_views(c["cache"], kv, dim)
    pg = int(c["table"][0, 0])
    k.view(torch.uint8)[pg, 0, 0, 2, :] = 0xff
    v.view(torch.uint8)[pg, 0, 0, :, 3] = 0x7f
    c["k"], c["v"] = c["k"] * 64, c["v"] * 64
    before = _blocks(c["cache"], kv, dim)
    D.dsa_kv8_append(c["k"], c["v"], c["cache"], c["batch"], rope_dims=0)
    _check(c, before, 0, True)


def test_append_scale_words_of_any_bits():
    """A block whose scale word was never written by an append: its exponent is cut to the cache's, nothing else happens."""
    kv, dim = 1, 64
    for bits, e_was in ((0, -24), (0x7f800000, 24), (0x7fc00000, 24), (0x3fc00000, 0)):
        c = _case([9], [1], kv, 1, dim)
        s = D.kv8_views(c["cache"], kv, dim)[2]
        s.view(torch.int32).fill_(bits)
        D.dsa_kv8_append(c["k"], c["v"], c["cache"], c["batch"], rope_dims=0)
        pg = int(c["table"][0, 0])
        for i, x in ((0, c["k"]), (1, c["v"])):
            e = max(e_was, O.kv8_exponent(float(x.abs().max())))
            assert float(s[pg, 0, i, 0]) == 2.0 ** e


@pytest.mark.parametrize("halves", [True, False])
def test_append_far_positions_and_given_frequencies(halves):
    """Positions near 2^20 in a table that holds their pages alone; scaled frequencies."""
    kv, dim, rope = 2, 128, 96
    L, n = 1048576 - 5, 40
    c = _case([100], [n], kv, 2, dim)
    width = 16384
    table = torch.full((1, width), -1, dtype=torch.int32, device=DEV)
    for p in {(L - n) // 64, (L - 1) // 64}:
        table[0, p] = p % c["pages"]
    c.update(seq=[L], table=table.cpu().numpy())
    c["batch"] = D.Batch(torch.tensor([L], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV), table, c["pages"])
    f = (1e6 ** (-2.0 * torch.arange(rope // 2).double() / rope) / 8.0).float()
    f[0] = 1.5
    before = _blocks(c["cache"], kv, dim)
    q_out = D.dsa_kv8_append(c["k"], c["v"], c["cache"], c["batch"], q=c["q"], rope_dims=rope,
                             rope_style=D.ROPE_HALVES if halves else D.ROPE_INTERLEAVED, inv_freq=f.to(DEV))
    _check(c, before, rope, halves, q_out, None, f.double().numpy())
    before = _blocks(c["cache"], kv, dim)
    q_out = D.dsa_kv8_append(c["k"], c["v"], c["cache"], c["batch"], q=c["q"], rope_dims=rope,
                             rope_style=D.ROPE_HALVES if halves else D.ROPE_INTERLEAVED, rope_base=500000.0)
    _check(c, before, rope, halves, q_out, None, None, 500000.0)


def test_append_padded_batch_and_skipped_positions():
    """Rows behind the last request, pages outside the cache, positions below zero and behind the table: skipped, recorded, rotated."""
    kv, dim = 2, 128
    c = _case([70, 3, 64, 200], [5, 6, 10, 12], kv, 2, dim, pad_rows=3)
    b = c["batch"]
    table = torch.tensor(c["table"][:, :3].copy(), device=DEV)           # three pages: request 3's new tokens lie behind them
    table[0, 1] = c["pages"]
    table[2, 0] = -1
    c["table"] = table.cpu().numpy()
    c["batch"] = D.Batch(b.seq_len, b.q_start, table, c["pages"], max_seq_len=192, max_q_len=12, total_q=c["T"] + 3)
    before = _blocks(c["cache"], kv, dim)
    st = D.new_device_status(DEV)
    q_out = torch.full((c["T"] + 3, c["heads"], dim), 7.0, dtype=torch.bfloat16, device=DEV)
    k_out = torch.full((c["T"] + 3, kv, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    D.dsa_kv8_append(c["k"], c["v"], c["cache"], c["batch"], q=c["q"], q_out=q_out, k_out=k_out, dev_status=st)
    _check(c, before, dim, True, q_out, k_out)
    assert torch.all(q_out[c["T"]:] == 7.0) and torch.all(k_out[c["T"]:] == 7.0)
    assert D.dsa_device_status_read(st)[0] == D.DEVERR_PAGE_RANGE | D.DEVERR_INDEX_RANGE


def test_append_takes_no_row_behind_total_q():
    """A total_q that ends inside a block of new tokens: what is behind it is neither read nor written."""
    kv, dim = 2, 64
    c = _case([70, 40], [5, 20], kv, 2, dim, seed=60)
    got, want = c["cache"].clone(), c["cache"].clone()
    short = D.Batch(c["batch"].seq_len, c["batch"].q_start, c["batch"].page_table, c["pages"], max_seq_len=128, max_q_len=20, total_q=15)
    exact = D.Batch(torch.tensor([70, 30], dtype=torch.int32, device=DEV), torch.tensor([0, 5, 15], dtype=torch.int32, device=DEV),
                    c["batch"].page_table, c["pages"], max_seq_len=128, max_q_len=10, total_q=15)
    c["k"][15:], c["v"][15:] = 1e30, float("inf")
    q_out = torch.full((25, c["heads"], dim), 7.0, dtype=torch.bfloat16, device=DEV)
    D.dsa_kv8_append(c["k"], c["v"], want, exact, q=c["q"])
    D.dsa_kv8_append(c["k"], c["v"], got, short, q=c["q"], q_out=q_out)
    assert torch.equal(got, want) and torch.all(q_out[15:] == 7.0)


def test_append_in_place_on_a_stream_and_in_a_graph():
    kv, dim, rope = 2, 64, 64
    c = _case([33, 90], [3, 40], kv, 3, dim)
    ref, before = c["cache"].clone(), c["cache"].clone()
    want_k = torch.empty(c["T"], kv, dim, dtype=torch.bfloat16, device=DEV)
    want_q = D.dsa_kv8_append(c["k"], c["v"], ref, c["batch"], q=c["q"], rope_dims=rope, k_out=want_k)
    q, k, v = (c[x].contiguous() for x in "qkv")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    D.dsa_kv8_append(k, v, c["cache"], c["batch"], q=q, rope_dims=rope, q_out=q, k_out=k, stream=side)
    side.synchronize()
    assert torch.equal(c["cache"], ref) and torch.equal(q, want_q) and torch.equal(k, want_k)
    cache, q_out = before.clone(), torch.empty_like(want_q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.dsa_kv8_append(c["k"], c["v"], cache, c["batch"], q=c["q"], rope_dims=rope, q_out=q_out)
    assert torch.equal(cache, before)
    for _ in range(2):                                     # the same tokens twice: the same cache
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cache, ref) and torch.equal(q_out, want_q)


def test_append_many_heads():
    """More jobs than warps, a group of 64, and 64 heads of their own."""
    for kv, group, dim in ((1, 64, 128), (64, 1, 64), (33, 2, 64)):
        c = _case([77, 18], [20, 18], kv, group, dim)
        before = _blocks(c["cache"], kv, dim)
        q_out = D.dsa_kv8_append(c["k"], c["v"], c["cache"], c["batch"], q=c["q"], rope_dims=32, rope_style=D.ROPE_INTERLEAVED)
        _check(c, before, 32, False, q_out)
