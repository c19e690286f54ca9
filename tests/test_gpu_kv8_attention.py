"""dsa_kv8_attention against the 64-bit oracle, at the bounds derived in tests/grouped.py."""

import numpy as np
import pytest
import torch

import dsa_sparse_attention_indexer_gb300 as D
from oracle import dsa_oracle as O
from tests.grouped import DEV, bounds, cache_case, check, expected, f64, place

pytestmark = pytest.mark.gpu


def _run(c, dtype=D.DTYPE_BF16, scale=None, ws=None, stream=None, q=None):
    T = c["T"] + c["pad"]
    out = torch.full((T, c["heads"], c["dim"]), 7.0, dtype=torch.float32 if dtype == D.DTYPE_F32 else torch.bfloat16, device=DEV)
    lse = torch.full((T, c["heads"]), 7.0, device=DEV)
    st = D.new_device_status(DEV)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    D.dsa_kv8_attention(c["q"] if q is None else q, c["dev_cache"], c["batch"], kv_heads=c["kv"], softmax_scale=scale, out=out, out_dtype=dtype, lse=lse,
                        ws=ws, dev_status=st, stream=stream)
    torch.cuda.synchronize()
    assert torch.all(out[c["T"]:] == 7.0) and torch.all(lse[c["T"]:] == 7.0)           # rows behind the last request
    return out, lse, D.dsa_device_status_read(st)[0]


SHAPES = [
    # seq_len, q_len, kv_heads, group, dim
    ([1], [1], 1, 1, 64),
    ([1, 15, 16, 17, 31], [1] * 5, 2, 8, 128),
    ([63, 64, 65, 127, 128, 129], [1] * 6, 2, 4, 64),
    ([100, 700, 3], [1] * 3, 1, 2, 256),
    ([1000, 33, 512], [1] * 3, 8, 8, 128),
    ([20000], [1], 1, 8, 128),
    ([5000, 7000], [1, 1], 1, 64, 128),
    ([300, 129, 64], [1] * 3, 2, 7, 128),
    ([300, 129, 64], [1] * 3, 2, 12, 64),
    ([300, 129], [1] * 2, 2, 16, 256),
    ([200, 64, 130, 77], [6, 1, 0, 3], 2, 4, 128),
    ([200, 64, 6], [6, 6, 6], 4, 4, 256),
    ([65, 66], [2, 2], 3, 5, 64),
    ([190, 100], [33, 100], 2, 3, 128),
    ([150], [70], 1, 5, 256),
    ([128, 127], [128, 3], 2, 1, 64),
    ([257], [140], 2, 8, 128),
    ([40], [3], 1, 128, 64),
    # 17 to 64 rows: two halves of columns
    ([100, 300], [5, 6], 2, 4, 256),
    ([1000, 65], [8, 4], 1, 4, 256),
    ([777, 200, 40], [6, 1, 5], 2, 8, 128),
    ([130, 3000], [60, 33], 2, 1, 64),
    ([90], [1], 1, 61, 128),
    # many rows a request, alone and beside few
    ([300], [300], 1, 1, 128),
    ([300], [129], 2, 1, 64),
    ([520, 77], [260, 77], 2, 2, 256),
    ([700, 1000, 64, 200], [200, 1, 64, 0], 2, 8, 128),
    ([500, 100], [90, 33], 2, 7, 64),
    ([1100], [700], 1, 5, 128),
    ([260, 129, 90], [17, 5, 40], 1, 64, 256),
]


@pytest.mark.parametrize("seq,n,kv,group,dim", SHAPES)
def test_attention(seq, n, kv, group, dim):
    c = cache_case(seq, n, kv, group, dim, seed=len(seq) + dim, pad_rows=2)
    want = expected(c)
    for dtype in (D.DTYPE_F32, D.DTYPE_BF16):
        out, lse, bits = _run(c, dtype)
        check(out, lse, want)
        assert bits == 0


def test_many_requests_of_all_lengths():
    """More requests than threads plan at once, lengths 1 .. 400; shares that begin and end anywhere."""
    seq = [1 + (37 * i) % 400 for i in range(500)]
    c = cache_case(seq, [1] * 500, 1, 4, 64, seed=5)
    out, lse, bits = _run(c)
    check(out, lse, expected(c))
    assert bits == 0


@pytest.mark.parametrize("dim,n", [(64, 1), (128, 1), (256, 1), (64, 20), (128, 17), (256, 9)])
def test_shares_of_many_pages(dim, n):
    """Shares of more pages than a CTA holds at once, several times over, of an odd number of pages each."""
    seq = [7000 + 333 * (i % 7) for i in range(40)]
    c = cache_case(seq, [n] * 40, 1, 2, dim, seed=dim)
    out, lse, bits = _run(c)
    check(out, lse, expected(c))
    assert bits == 0


def test_scales_far_apart():
    """Blocks' scales from 2^-24 to 2^24 side by side, in any order: each output to its own precision."""
    for seed in range(3):
        c = cache_case([600, 90], [3, 1], 2, 4, 128, seed=seed)
        s = D.kv8_views(c["cache"], 2, 128)[2]
        g = torch.Generator().manual_seed(seed)
        s[:, :, 1] = torch.exp2(torch.randint(-24, 25, s[:, :, 1].shape, generator=g).float())
        place(c)
        for scale in (None, 1.0):
            out, lse, _ = _run(c, D.DTYPE_F32, scale)
            check(out, lse, expected(c, scale))


def test_large_scores_and_a_dominating_token():
    c = cache_case([4000], [1], 1, 8, 128, seed=3, q_size=300.0)
    check(*_run(c, D.DTYPE_F32)[:2], expected(c))
    # one key far above the others, first, in the middle and last, then the sum of many small ones behind it
    for at in (0, 2000, 3999):
        c = cache_case([4000], [1], 1, 8, 128, seed=4, q_size=0.05)
        k = D.kv8_views(c["cache"], 1, 128)[0]
        pg, blk, tok = int(c["table"][0, at // 64]), at % 64 // 16, at % 16
        k[pg, 0, blk, tok] = (torch.sign(c["q"][0, 3].float().cpu()) * 448).to(torch.float8_e4m3fn)
        place(c)
        check(*_run(c, D.DTYPE_F32)[:2], expected(c))


def test_a_context_of_equal_scores():
    c = cache_case([9000], [1], 1, 8, 128, seed=6)
    c["q"].zero_()
    check(*_run(c, D.DTYPE_F32)[:2], expected(c))


def test_unseen_rows_may_hold_anything():
    """NaN codes and scales of any bits behind every request's end and in pages that no one holds."""
    c = cache_case([50, 17, 64, 130], [3, 1, 2, 5], 2, 4, 128, seed=8)
    want = expected(c)
    k, v, s = (x.view(torch.uint8) if x.dtype != torch.float32 else x for x in D.kv8_views(c["cache"], 2, 128))
    used = torch.zeros(c["pages"], dtype=torch.bool)
    for r, L in enumerate(c["seq"]):
        for p in range((L + 63) // 64):
            pg = int(c["table"][r, p])
            used[pg] = True
            for blk in range(4):
                left = min(16, max(0, L - p * 64 - blk * 16))
                k[pg, :, blk, left:] = 0x7f
                v[pg, :, blk, :, left:] = 0xff
                if left == 0:
                    s[pg, :, :, blk] = float("nan")
    c["cache"][~used] = 0xff
    place(c)
    out, lse, bits = _run(c)
    check(out, lse, want)
    assert bits == 0


def test_nan_reaches_the_rows_that_see_it():
    for dim, group, n in ((128, 4, 5), (64, 1, 40), (256, 2, 9), (128, 8, 70), (64, 2, 90), (256, 8, 80)):
        c = cache_case([100, 90], [n, 1], 2, group, dim, seed=9)
        k, v, _ = D.kv8_views(c["cache"], 2, dim)
        for p, what in ((98, v), (97, k), (20, None)):
            pg, blk, tok = int(c["table"][0, p // 64]), p % 64 // 16, p % 16
            if what is v:
                v.view(torch.uint8)[pg, 0, blk, 5, tok] = 0x7f
                v.view(torch.uint8)[pg, 1, blk, dim - 1, tok] = 0xff
            elif what is k:
                k.view(torch.uint8)[pg, 1, blk, tok, 3] = 0xff
        pg = int(c["table"][1, 0])
        v.view(torch.uint8)[pg, 0, 0, 7, 0] = 0x7f          # every row of request 1 sees this one
        place(c)
        out, lse, _ = _run(c, D.DTYPE_F32)
        want = expected(c)
        assert np.isnan(want[0]).any() and not np.isnan(want[0]).all()
        # a NaN score makes the whole row NaN
        bad = np.isnan(want[1])
        want[0][bad] = np.nan
        check(out, lse, want)


def test_pages_outside_the_cache_and_lengths_outside_the_table():
    c = cache_case([300, 200, 100, 5], [2, 1, 3, 9], 2, 3, 128, seed=10)
    c["table"][0, 2], c["table"][1, 0], c["table"][1, 3] = c["pages"], -1, -7
    place(c)
    out, lse, bits = _run(c)
    check(out, lse, expected(c))                            # request 3 has 9 new tokens and holds 5: its first rows see nothing
    assert bits == D.DEVERR_PAGE_RANGE | D.DEVERR_INDEX_RANGE
    c = cache_case([128, 64], [1, 1], 1, 2, 64, seed=11)
    c["seq"] = [500, 64]                                    # two pages of the table: positions from 128 on are not seen
    place(c)
    out, lse, bits = _run(c)
    want = expected(dict(c, seq=[128, 64]))
    check(out, lse, want)
    assert bits == D.DEVERR_INDEX_RANGE
    c["seq"] = [-3, 0]
    place(c)
    out, lse, bits = _run(c)
    assert torch.all(out == 0) and torch.all(lse == -float("inf")) and bits == D.DEVERR_INDEX_RANGE


def test_strides_scale_stream_graph_and_workspace():
    c = cache_case([400, 70, 1000], [2, 1, 4], 2, 4, 128, seed=12)
    want = expected(c)
    out, lse, _ = _run(c)
    check(out, lse, want)
    # q as a part of wider rows, and with its heads in front
    wide = torch.randn(c["T"], c["heads"] + 4, 128, device=DEV).to(torch.bfloat16)
    wide[:, 2:2 + c["heads"]] = c["q"]
    turned = c["q"].transpose(0, 1).contiguous().transpose(0, 1)
    for q in (wide[:, 2:2 + c["heads"]], turned):
        o2, l2, _ = _run(c, q=q)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    # the same bits with a dirty workspace, on another stream and from a graph
    nbytes = D.dsa_kv8_attention_workspace_size(c["batch"], c["heads"], c["kv"], 128)
    for fill in (0, 0xff, 0xab):
        ws = torch.full((nbytes,), fill, dtype=torch.uint8, device=DEV)
        o2, l2, _ = _run(c, ws=ws, stream=torch.cuda.Stream())
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        D.dsa_kv8_attention(c["q"], c["dev_cache"], c["batch"], kv_heads=2, out=o2, lse=l2, ws=ws)
    for _ in range(2):
        o2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    check(*_run(c, scale=0.7)[:2], expected(c, 0.7))


def test_extreme_queries():
    """Rows whose q is far above and below fp16's range, zero, and NaN."""
    c = cache_case([90, 90], [1, 2], 1, 8, 64, seed=13)
    c["q"][0, 0] *= 1e6
    c["q"][0, 1] *= 1e-20
    c["q"][0, 2] = 0
    c["q"][1, 3, 5] = float("nan")
    out, lse, _ = _run(c, D.DTYPE_F32)
    want = expected(c)
    want[0][np.isnan(want[1])] = np.nan
    check(out, lse, want)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_chunks_beside_decode_rows(dim):
    """Chunks whose items are more than the CTAs, a page that is not there, and rows behind the last request."""
    c = cache_case([900, 1500, 65, 700, 333], [300, 1, 65, 640, 2], 4, 4, dim, seed=dim, pad_rows=2)
    c["table"][0, 3] = -1
    c["table"][3, 10] = c["pages"] + 5
    place(c)
    out, lse, bits = _run(c)
    check(out, lse, expected(c))
    assert bits == D.DEVERR_PAGE_RANGE


def test_prefill_scales_far_apart_and_large_scores():
    for seed, size in ((0, 1.0), (1, 300.0)):
        c = cache_case([600], [150], 2, 4, 128, seed=seed, q_size=size)
        s = D.kv8_views(c["cache"], 2, 128)[2]
        g = torch.Generator().manual_seed(seed)
        s[:, :, 1] = torch.exp2(torch.randint(-24, 25, s[:, :, 1].shape, generator=g).float())
        place(c)
        check(*_run(c, D.DTYPE_F32)[:2], expected(c))


def test_prefill_unseen_rows_and_lengths():
    c = cache_case([150, 130], [100, 130], 2, 2, 128, seed=20)
    want = expected(c)
    k, v, s = (x.view(torch.uint8) if x.dtype != torch.float32 else x for x in D.kv8_views(c["cache"], 2, 128))
    for r, L in enumerate(c["seq"]):
        for blk in range(L // 16, 12):
            pg, at = int(c["table"][r, blk // 4]), blk % 4
            left = max(0, L - blk * 16)
            k[pg, :, at, left:] = 0x7f
            v[pg, :, at, :, left:] = 0xff
            if left == 0:
                s[pg, :, :, at] = float("nan")
    place(c)
    out, lse, bits = _run(c)
    check(out, lse, want)
    assert bits == 0
    # fewer tokens held than new ones: rows that see nothing; more than the table has: positions that no one sees
    for seq, n in (([60], [100]), ([500], [120])):
        c = cache_case([128], n, 1, 4, 64, seed=21)
        c["seq"] = seq
        place(c)
        out, lse, bits = _run(c)
        L = min(seq[0], 128)
        k, v, ok = O.kv8_read(c["cache"].numpy().reshape(-1), 1, 64, c["table"][0].numpy(), L, c["pages"])
        check(out, lse, bounds(f64(c["q"]), k, v, seq[0] - n[0], 64 ** -0.5, 2.0 ** -11, ok))
        assert bits == D.DEVERR_INDEX_RANGE


@pytest.mark.parametrize("seq,n,kv,group,dim", [
    ([5000], [100], 1, 8, 128),                    # few items of many steps
    ([5000], [70], 1, 1, 64),                      # one tile of two
    ([2047], [65], 1, 2, 256),
    ([2048], [65], 1, 2, 256),
    ([20000], [17], 1, 5, 64),
    ([3000], [800], 8, 8, 128),                    # one round of items and some
    ([4000, 300, 2500, 1024], [200, 130, 1, 90], 2, 4, 128),      # long and short ones, and some that are not cut
    ([3000, 2100], [1300, 90], 1, 16, 256),
    ([1500], [1500], 2, 4, 64),                    # pieces that some rows see nothing of
])
def test_items_cut_along_the_keys(seq, n, kv, group, dim):
    c = cache_case(seq, n, kv, group, dim, seed=dim + len(seq), pad_rows=3)
    want = expected(c)
    for dtype in (D.DTYPE_F32, D.DTYPE_BF16):
        out, lse, bits = _run(c, dtype)
        check(out, lse, want)
        assert bits == 0


@pytest.mark.parametrize("pages,dim", [(4000, 64), (2000, 128), (4096, 128), (1000, 256)])
def test_runs_of_heads_and_items_dealt_out(pages, dim):
    """A wide page table lays the heads out in runs, the last one shorter, and has the items dealt out as the CTAs get there."""
    c = cache_case([900, 2300, 100, 40], [700, 200, 90, 1], 7, 2, dim, seed=dim, pad_rows=2, max_pages=pages)
    want = expected(c)
    ws = torch.full((D.dsa_kv8_attention_workspace_size(c["batch"], c["heads"], 7, dim),), 0xff, dtype=torch.uint8, device=DEV)
    out, lse, bits = _run(c, ws=ws)
    check(out, lse, want)
    assert bits == 0
    again = torch.zeros_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.dsa_kv8_attention(c["q"], c["dev_cache"], c["batch"], kv_heads=7, out=again, ws=ws)
    for _ in range(3):
        again.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(again[:c["T"]], out[:c["T"]])


def test_cut_items_with_nan_and_pages_that_are_not_there():
    c = cache_case([4000], [100], 1, 4, 128, seed=40)
    k, v, _ = (x.view(torch.uint8) if x.dtype != torch.float32 else x for x in D.kv8_views(c["cache"], 1, 128))
    at = 3950                                              # rows from 50 on see it
    v[int(c["table"][0, at // 64]), 0, at % 64 // 16, 5, at % 16] = 0x7f
    v[int(c["table"][0, 10]), 0, 2, 77, 3] = 0xff           # all rows do
    c["table"][0, 20] = -1
    c["table"][0, 60] = c["pages"]
    place(c)
    out, lse, bits = _run(c)
    check(out, lse, expected(c))
    assert bits == D.DEVERR_PAGE_RANGE
    # whole pieces whose pages are not there, and whole requests
    for gone in (slice(0, 20), slice(16, 48), slice(0, 63)):
        c = cache_case([4000], [100], 1, 4, 128, seed=41)
        c["table"][0, gone] = -1
        place(c)
        out, lse, bits = _run(c)
        check(out, lse, expected(c))
        assert bits == D.DEVERR_PAGE_RANGE


@pytest.mark.parametrize("n", [3, 100])
def test_low_scores_behind_pages_that_are_not_there(n):
    """What a row has not seen sets no reference: the first scores that it sees may be far below 0."""
    c = cache_case([600], [n], 1, 4, 64, seed=42)
    k = D.kv8_views(c["cache"], 1, 64)[0]
    k.copy_(k.float().abs().clamp(min=16).to(torch.float8_e4m3fn))
    c["q"] = -(c["q"].abs() + 1) * 64
    c["table"][0, :3] = -1
    place(c)
    want = expected(c)
    assert want[1].max() < -104                           # exp of it is below the smallest fp32
    out, lse, bits = _run(c, D.DTYPE_F32)
    check(out, lse, want)
    assert bits == D.DEVERR_PAGE_RANGE
    # as far below as the scale can put them: one position has all of the weight, and its log-sum is finite; or, where
    # there are many rows, it is recorded that such scores' probabilities are not to be had
    out, lse, bits = _run(c, D.DTYPE_F32, 1e30)
    if bits & D.DEVERR_FP16_RANGE:
        assert n == 100
    else:
        check(out, lse, expected(c, 1e30))
        assert torch.isfinite(lse[:n]).all() and out[:n].abs().amax(2).min() > 0


def test_the_largest_scores_of_many_rows():
    """Scores up to 2^23 are right, and beyond 2^24 they are recorded: here of keys that differ from a row's best by 2^-4 and more of it."""
    c = cache_case([700], [100], 1, 2, 64, seed=44)
    k = D.kv8_views(c["cache"], 1, 64)[0]
    k.fill_(0)
    k[..., 0] = 1.0
    best = k[int(c["table"][0, 500 // 64]), 0, 500 % 64 // 16, 500 % 16]
    best[0] = 2.0
    D.kv8_views(c["cache"], 1, 64)[2][:, :, 0] = 1.0
    c["q"].zero_()
    c["q"][..., 0] = 1.0
    place(c)
    for scale, far in ((2.0 ** 22 - 1, False), (2.0 ** 26, True)):
        out, lse, bits = _run(c, D.DTYPE_F32, scale)
        assert bits == (D.DEVERR_FP16_RANGE if far else 0)
        if not far:
            _, v, _ = O.kv8_read(c["cache"].numpy().reshape(-1), 1, 64, c["table"][0].numpy(), 700, c["pages"])
            assert np.allclose(f64(out[:100]), v[500], rtol=2.0 ** -10, atol=0)              # P and a sum of one
            assert np.allclose(f64(lse[:100]), 2 * scale, rtol=2.0 ** -22)


def test_cut_items_from_a_graph_and_on_two_streams():
    """Calls that share a workspace one after the other, and calls with their own beside each other."""
    c = cache_case([5000, 900], [120, 90], 1, 8, 128, seed=43)
    want, _, _ = _run(c)
    size = D.dsa_kv8_attention_workspace_size(c["batch"], c["heads"], c["kv"], c["dim"])
    shared = torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(want) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    for g, out in zip(graphs, outs):
        with torch.cuda.graph(g):
            D.dsa_kv8_attention(c["q"], c["dev_cache"], c["batch"], kv_heads=1, out=out, ws=shared)
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    streams, own = [torch.cuda.Stream() for _ in range(2)], [torch.full((size,), 0xff, dtype=torch.uint8, device=DEV) for _ in range(2)]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o, w in zip(streams, outs, own):
            D.dsa_kv8_attention(c["q"], c["dev_cache"], c["batch"], kv_heads=1, out=o, ws=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_outputs_that_begin_at_16_bytes():
    """Outputs, their log-sums and the cache at the least alignment that the calls ask for."""
    for n in (3, 100):
        c = cache_case([300], [n], 2, 4, 64, seed=24)
        want, _, _ = _run(c)
        room = torch.zeros(n * 8 * 64 + 8, dtype=torch.bfloat16, device=DEV)
        out = room[8:].view(n, 8, 64)
        lse = torch.empty(n * 8 + 1, device=DEV)[1:].view(n, 8)
        cache = torch.empty(c["dev_cache"].numel() + 16, dtype=torch.uint8, device=DEV)[16:]
        cache.copy_(c["dev_cache"].flatten())
        D.dsa_kv8_attention(c["q"], cache, c["batch"], kv_heads=2, out=out, lse=lse)
        assert torch.equal(out, want)


def test_queries_that_a_tensor_map_does_not_take():
    """One row of q for all tokens: a stride of 0."""
    c = cache_case([300], [100], 2, 4, 64, seed=22)
    one = c["q"][:1]
    c["q"] = one.expand(100, 8, 64).contiguous()
    want = expected(c)
    out, lse, bits = _run(c, q=one.expand(100, 8, 64))
    check(out, lse, want)


def test_prefill_timeout_is_recorded_and_the_next_call_is_right():
    c = cache_case([3000], [500], 2, 4, 128, seed=23)
    try:
        D.dsa_debug_set_wait_limit_ns(0)
        for _ in range(3):
            _, _, bits = _run(c)
            assert bits & D.DEVERR_TIMEOUT
    finally:
        D.dsa_debug_set_wait_limit_ns(2_000_000_000)
    out, lse, bits = _run(c)
    check(out, lse, expected(c))
    assert bits == 0


def test_timeout_is_recorded_and_the_next_call_is_right():
    c = cache_case([3000, 800], [1, 2], 2, 8, 128, seed=14)
    long = cache_case([100000], [1], 2, 8, 128, seed=15)   # a dozen pages and more for every SM: they cannot all be there at once
    try:
        D.dsa_debug_set_wait_limit_ns(0)
        for _ in range(3):
            _, _, bits = _run(long)
            assert bits & D.DEVERR_TIMEOUT
    finally:
        D.dsa_debug_set_wait_limit_ns(2_000_000_000)
    out, lse, bits = _run(c)
    check(out, lse, expected(c))
    assert bits == 0
