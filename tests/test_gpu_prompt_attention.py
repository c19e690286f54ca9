"""dsa_prompt_attention against the 64-bit oracle, at the bounds derived in tests/grouped.py (probabilities in bf16)."""

import numpy as np
import pytest
import torch

import dsa_sparse_attention_indexer_gb300 as D
from tests.grouped import DEV, bounds, check, f64

pytestmark = pytest.mark.gpu

P = 2.0 ** -8                                              # half a step of bf16


def _case(n, past, kv, group, dim, seed=0, pad=0, size=1.0):
    g = torch.Generator().manual_seed(99 + seed)
    past = [past] * len(n) if isinstance(past, int) else past
    L = [max(0, a + b) for a, b in zip(n, past)]
    T, K = sum(n), sum(L)
    q = (torch.randn(T + pad, kv * group, dim, generator=g) * size).to(torch.bfloat16)
    k, v = (torch.randn(K + pad, kv, dim, generator=g).to(torch.bfloat16) for _ in range(2))
    if pad:                                                # what lies behind the last sequence is no one's business
        k[K:], v[K:] = float("nan"), float("inf")
    qs, ks = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (n, L))
    longest = max(n + [-(-(T + pad) // len(n))]), max(L + [-(-(K + pad) // len(n))])
    batch = D.PromptBatch(torch.tensor(qs, device=DEV), torch.tensor(ks, device=DEV), max_q_len=longest[0], max_k_len=longest[1],
                          total_q=T + pad, total_k=K + pad)
    return dict(n=n, L=L, qs=qs, ks=ks, q=q.to(DEV), k=k.to(DEV), v=v.to(DEV), batch=batch, T=T, pad=pad, dim=dim, heads=kv * group)


def _expected(c, scale=None):
    scale = c["dim"] ** -0.5 if scale is None else scale
    got = []
    q, k, v = f64(c["q"]), f64(c["k"]), f64(c["v"])
    for r, (n, L) in enumerate(zip(c["n"], c["L"])):
        if n:
            a, b = c["qs"][r], c["ks"][r]
            got.append(bounds(q[a:a + n], k[b:b + L], v[b:b + L], L - n, scale, P))
    return [np.concatenate(x) for x in zip(*got)]


def _run(c, dtype=D.DTYPE_BF16, scale=None, ws=None, stream=None, **kw):
    T = c["T"] + c["pad"]
    out = torch.full((T, c["heads"], c["dim"]), 7.0, dtype=torch.float32 if dtype == D.DTYPE_F32 else torch.bfloat16, device=DEV)
    lse = torch.full((T, c["heads"]), 7.0, device=DEV)
    st = D.new_device_status(DEV)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    t = dict(q=c["q"], k=c["k"], v=c["v"], **{})
    t.update(kw)
    D.dsa_prompt_attention(t["q"], t["k"], t["v"], c["batch"], softmax_scale=scale, out=out, out_dtype=dtype, lse=lse, ws=ws, dev_status=st,
                           stream=stream)
    torch.cuda.synchronize()
    assert torch.all(out[c["T"]:] == 7.0) and torch.all(lse[c["T"]:] == 7.0)           # rows behind the last sequence
    return out, lse, D.dsa_device_status_read(st)[0]


SHAPES = [
    # q lengths, keys before them, kv_heads, group, dim
    ([1], 0, 1, 1, 64),
    ([1], 0, 1, 1, 128),
    ([1], 0, 1, 1, 256),
    ([128], 0, 1, 1, 128),
    ([129], 0, 2, 8, 128),
    ([300], 0, 1, 1, 64),
    ([257, 1, 64], 0, 2, 4, 64),
    ([17, 5, 100, 33], 0, 2, 7, 128),
    ([130, 128, 127], 0, 1, 2, 256),
    ([64, 65, 3], 0, 2, 5, 256),
    ([513], 0, 3, 1, 128),
    ([40, 0, 1, 90], [0, 5, 200, 131], 2, 4, 128),
    ([10, 70], [-4, -70], 1, 4, 64),                        # rows that see nothing, a sequence without keys
    ([3, 9], 0, 1, 128, 64),
    ([50], 0, 1, 64, 128),
    ([70, 3], 0, 4, 12, 64),
    ([1000], 0, 1, 1, 256),
    ([900], 0, 1, 3, 128),
    ([1] * 40 + [300] + [2] * 37, 0, 1, 8, 128),
]


@pytest.mark.parametrize("n,past,kv,group,dim", SHAPES)
def test_attention(n, past, kv, group, dim):
    c = _case(n, past, kv, group, dim, seed=len(n) + dim, pad=3)
    want = _expected(c)
    for dtype in (D.DTYPE_F32, D.DTYPE_BF16):
        out, lse, bits = _run(c, dtype)
        check(out, lse, want)
        assert bits == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_more_items_than_ctas(dim):
    """Every CTA takes several items, of long and short sequences, one after the other."""
    n = [700, 1, 33, 450, 129, 256, 5, 600, 0, 320] * 3
    c = _case(n, 0, 4, 2, dim, seed=dim)
    out, lse, bits = _run(c)
    check(out, lse, _expected(c))
    assert bits == 0


def test_large_scores():
    """References that grow from step to step: scores in the thousands, ascending keys."""
    c = _case([600, 300], 0, 1, 2, 128, seed=1, size=200.0)
    check(*_run(c, D.DTYPE_F32)[:2], _expected(c))
    c = _case([700], 0, 1, 1, 64, seed=2)
    c["k"] *= torch.linspace(0.1, 40, 700, device=DEV)[:, None, None].to(torch.bfloat16)
    c["q"].abs_()
    c["k"].abs_()
    check(*_run(c, D.DTYPE_F32)[:2], _expected(c))


@pytest.mark.parametrize("dim,group", [(64, 1), (128, 4), (256, 2)])
def test_values_that_are_not_finite_reach_the_rows_that_see_them(dim, group):
    c = _case([300, 140], [60, 0], 2, group, dim, seed=3)
    v = c["v"]
    v[5, 0, 3] = float("inf")                               # all rows but none see it
    v[200, 1, dim - 1] = float("nan")                       # rows from 140 on
    v[359, 0, 7] = -float("inf")                            # the last row alone
    v[358, 0, 7] = float("inf")
    v[360, 1, 0] = float("nan")                             # the second sequence's first key: all of its rows
    v[499, 1, 9] = float("inf")
    c["k"][300, 1, 2] = float("nan")                        # rows from 240 on: NaN scores
    out, lse, _ = _run(c, D.DTYPE_F32)
    want = _expected(c)
    # the oracle's sums hold infinities where the formula does; a NaN score makes its whole row NaN
    want[0][np.isnan(want[1])] = np.nan
    got, exact = f64(out), want[0]
    assert np.array_equal(np.isnan(got), np.isnan(exact)) and np.array_equal(np.isposinf(got), np.isposinf(exact))
    assert np.array_equal(np.isneginf(got), np.isneginf(exact)) and np.isinf(exact).any() and np.isnan(exact).any()
    f = np.isfinite(exact)
    assert np.all(np.abs(got[f] - exact[f]) <= (want[2] * 1.001 + 1e-6)[f])
    z = f64(lse)
    assert np.array_equal(np.isnan(z), np.isnan(want[1]))


@pytest.mark.parametrize("bound,dim", [(100_000, 64), (200_000, 64), (60_000, 128), (40_000, 256)])
def test_runs_of_heads_and_items_dealt_out(bound, dim):
    """A large bound on the keys lays the heads out in runs of one or two, the last one shorter, and has the items dealt out
    as the CTAs get there: the same from a workspace of any content, replayed from a graph, and without it."""
    c = _case([700, 300, 1, 90], [5, 400, 0, 0], 7, 2, dim, seed=dim, pad=2)
    want = _expected(c)
    plain, _, _ = _run(c)
    check(*_run(c)[:2], want)
    b = c["batch"]
    c["batch"] = D.PromptBatch(b.q_start, b.k_start, max_q_len=b.c.max_q_len, max_k_len=bound, total_q=b.total_q, total_k=b.total_k)
    ws = torch.full((max(256, D.dsa_prompt_attention_workspace_size(c["batch"], c["heads"], 7, dim)),), 0xff, dtype=torch.uint8, device=DEV)
    out, lse, bits = _run(c, ws=ws)
    check(out, lse, want)
    assert bits == 0 and torch.equal(out[:c["T"]], plain[:c["T"]])
    again = torch.zeros_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.dsa_prompt_attention(c["q"], c["k"], c["v"], c["batch"], out=again, ws=ws)
    for _ in range(3):
        again.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(again[:c["T"]], plain[:c["T"]])


def test_low_scores_behind_infinite_keys():
    """Keys whose scores are minus infinity set no reference: the first others may be far below 0."""
    c = _case([100], [300], 1, 4, 64, seed=42)
    c["k"].copy_(c["k"].abs() + 1)
    c["k"][:260, :, 0] = -float("inf")
    c["q"].copy_(-(c["q"].abs() + 1) * 8)
    c["q"][..., 0] = 1.0
    want = _expected(c)
    assert np.isfinite(want[0]).all() and want[1].max() < -104        # exp of it is below the smallest fp32
    out, lse, bits = _run(c, D.DTYPE_F32)
    check(out, lse, want)
    assert bits == 0


def test_strides_stream_graph_and_workspace():
    c = _case([200, 77], [0, 40], 2, 4, 128, seed=4)
    want = _expected(c)
    out, lse, _ = _run(c)
    check(out, lse, want)
    # parts of one projection's rows, and heads in front of the rows
    both = torch.cat([c["k"], c["v"], torch.randn_like(c["v"])], 1)
    wide = torch.cat([torch.randn_like(c["q"]), c["q"]], 1)
    front = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (c["q"], c["k"], c["v"])]
    for kw in (dict(k=both[:, :2], v=both[:, 2:4], q=wide[:, 8:]), dict(q=front[0], k=front[1], v=front[2])):
        o2, l2, _ = _run(c, **kw)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    nbytes = D.dsa_prompt_attention_workspace_size(c["batch"], 8, 2, 128)
    for fill in (0, 0xff):
        ws = torch.full((nbytes,), fill, dtype=torch.uint8, device=DEV)
        o2, l2, _ = _run(c, ws=ws, stream=torch.cuda.Stream())
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.dsa_prompt_attention(c["q"], c["k"], c["v"], c["batch"], out=o2, lse=l2, ws=ws)
    for _ in range(2):
        o2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    check(*_run(c, scale=0.5)[:2], _expected(c, 0.5))


def test_inputs_and_outputs_that_begin_at_16_bytes():
    c = _case([150, 20], 0, 2, 4, 64, seed=7)
    want, _, _ = _run(c)

    def moved(x):
        room = torch.zeros(x.numel() + 8, dtype=x.dtype, device=DEV)
        y = room[8:].view(x.shape)
        y.copy_(x)
        return y

    out = moved(want) * 0
    out = moved(out)
    D.dsa_prompt_attention(moved(c["q"]), moved(c["k"]), moved(c["v"]), c["batch"], out=out)
    assert torch.equal(out, want)


def test_without_keys():
    c = _case([5, 3], [-5, -3], 1, 2, 64, seed=5)
    out, lse, bits = _run(c)
    assert torch.all(out == 0) and torch.all(lse == -float("inf")) and bits == 0


def test_timeout_is_recorded_and_the_next_call_is_right():
    c = _case([1500, 200], 0, 2, 4, 128, seed=6)
    try:
        D.dsa_debug_set_wait_limit_ns(0)
        for _ in range(3):
            _, _, bits = _run(c)
            assert bits & D.DEVERR_TIMEOUT
    finally:
        D.dsa_debug_set_wait_limit_ns(2_000_000_000)
    out, lse, bits = _run(c)
    check(out, lse, _expected(c))
    assert bits == 0
