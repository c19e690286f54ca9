"""GPU parity of dsa_window_mla and dsa_tree_mla with the fp64 oracle.

Cache rows that no row of their request sees hold NaN codes, infinite scales
and NaN RoPE dims, and pages without a visible position are -1, so a read in a
masked place shows.

Tolerances, per row and head (weights p_j, latents c_j, scores S_j):
* scores: 576 products summed in fp32 in steps of 16 (36 additions, each off by
  at most 2^-23 of the largest partial sum, which sum |q_d k_d| bounds) and one
  fp32 product with the scale: dS = 40 * 2^-23 * scale * max_j sum_d |q_d k_d|;
* lse: dS, the exponentials and their fp32 sums (2^-20), the logarithm and the
  final sum (2^-22 of the value);
* out: sum_j p_j |c_j| times the rounding of p_j to fp16 (2^-11), twice dS (in
  p_j and in the sum) and 2^-18 for exponentials, sums and the division; a p_j below
  fp16's smallest step is off by at most 2^-25 of the largest: 2^-25 sum_j |c_j|;
* bf16 outputs add half a step, 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

import dsa_sparse_attention_indexer_gb300 as D
from oracle import dsa_oracle as O
from tests.oracle_side import ATTN_REL_L2, bf16_bits, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
SENTINEL = -77.0


def make_case(seed, seq, q_len, sees, *, q_scale=1.0, pad_rows=0, spare_pages=3, full_table=False):
    """sees(r, t) -> positions that row t of request r sees.  Latent caches, batch
    descriptor and queries on the device; per row its positions and latent rows."""
    g = torch.Generator().manual_seed(seed)
    B = len(seq)
    width = max(1, max((L + 63) // 64 for L in seq))
    vis = [[np.asarray(sees(r, t), dtype=np.int64) for t in range(q_len[r])] for r in range(B)]
    need = np.zeros((B, width), bool)
    for r in range(B):
        for v in vis[r]:
            need[r, v // 64] = True
        if full_table:
            need[r, :(seq[r] + 63) // 64] = True
    pages = int(need.sum()) + spare_pages
    perm = torch.randperm(pages, generator=g).numpy()
    table = np.full((B, width), -1, np.int32)
    table[need] = perm[:need.sum()]
    cache = np.zeros((pages * 64, 656), np.uint8)
    cache[:, :512] = 0x7f                                            # E4M3 NaN
    cache[:, 512:528] = np.frombuffer(np.array([np.inf] * 4, np.float32).tobytes(), np.uint8)
    cache[:, 528:] = np.frombuffer(np.array([0x7fc0] * 64, np.uint16).tobytes(), np.uint8)
    cache = cache.reshape(pages, -1)
    rows = []
    for r in range(B):
        seen = np.unique(np.concatenate([np.zeros(0, np.int64)] + vis[r]))
        c = f64((torch.randn(len(seen), 512, generator=g) * torch.exp(torch.randn(len(seen), 1, generator=g))).to(torch.bfloat16))
        codes, scales = O.latent_quantize(c)
        rope = torch.randn(len(seen), 64, generator=g).to(torch.bfloat16)
        slots = table[r, seen // 64].astype(np.int64) * 64 + seen % 64
        if len(seen):
            O.latent_cache_write(cache, slots, codes, scales, bf16_bits(rope))
        for v in vis[r]:
            rows.append((v, O.latent_cache_read_rows(cache, table[r], v) if len(v) else np.zeros((0, 576))))
    T = len(rows)
    q = (torch.randn(T + pad_rows, 64, 576, generator=g) * q_scale).to(torch.bfloat16)
    start = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    batch = D.Batch(dev(np.array(seq, np.int32)), dev(start), dev(table), pages, max_seq_len=max(max(seq), 1),
                    max_q_len=max(max(q_len), -(-(T + pad_rows) // B)), total_q=T + pad_rows)
    return dict(T=T, rows=rows, q=q, dq=q.to(DEV), kv=dev(cache.reshape(-1)), batch=batch, pages=pages, table=table)


def reference(q, kv, scale=1.0 / 16):
    """(out, lse, bound of an fp32 output, bound of lse) of one row, in 64 bits."""
    if len(kv) == 0:
        return np.zeros((64, 512)), np.full(64, -np.inf), np.zeros((64, 512)), np.zeros(64)
    out, lse = O.sparse_mla(q, np.arange(len(kv)), kv, len(kv), scale)
    s = (q @ kv.T) * scale
    p = np.exp(s - lse[:, None])
    dS = 40 * 2.0 ** -23 * scale * (np.abs(q) @ np.abs(kv).T).max(1)
    c = np.abs(kv[:, :512])
    bound = (p @ c) * (2.0 ** -11 + 2 * dS[:, None] + 2.0 ** -18) + 2.0 ** -25 * p.max(1)[:, None] * c.sum(0)
    return out, lse, bound + 1e-30, dS + 2.0 ** -20 + 2.0 ** -22 * np.abs(lse)


def compare(c, out, lse, scale=1.0 / 16, kv_of=lambda i, kv: kv):
    out, lse = f64(out), f64(lse) if lse is not None else None
    bf16 = 2.0 ** -8
    for i, (_, kv) in enumerate(c["rows"]):
        ref, z, tol, ztol = reference(f64(c["q"][i]), kv_of(i, kv), scale)
        if c["bf16"]:
            tol = tol + bf16 * (np.abs(ref) + tol)
        err = np.abs(out[i] - ref)
        assert (err <= tol).all(), f"row {i}: {(err > tol).sum()} values off, worst {np.max(err / np.maximum(tol, 1e-30)):.2f} of the bound"
        if not c["bf16"] and len(kv):
            # the library's relative bar.  Its absolute one, 1e-2, is for latents ~N(0, 1): half an fp16 step of p
            # times |c| alone passes it from |c| = 20.5 on (2^-11 * 20.5 = 1e-2), and these reach 4 exp(3) = 80
            assert np.linalg.norm(out[i] - ref) <= ATTN_REL_L2 * np.linalg.norm(ref), f"row {i}"
        if lse is not None:
            assert np.array_equal(np.isinf(lse[i]), np.isinf(z)), f"row {i}"
            f = np.isfinite(z)
            assert (np.abs(lse[i][f] - z[f]) <= ztol[f]).all(), f"row {i}: lse off by {np.max(np.abs(lse[i][f] - z[f])):.2e}"


def run(c, call, f32=True, stream=None, ws=None, want_status=0, scale=1.0 / 16):
    n = c["batch"].total_q
    out = torch.full((n, 64, 512), SENTINEL, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    lse = torch.full((n, 64), SENTINEL, dtype=torch.float32, device=DEV)
    st = D.new_device_status(DEV)
    kw = dict(out=out, lse=lse, out_dtype=D.DTYPE_F32 if f32 else D.DTYPE_BF16, dev_status=st, stream=stream, ws=ws,
              softmax_scale=scale)
    call(c, kw)
    c["bf16"] = not f32
    got = D.dsa_device_status_read(st, stream)
    assert got[0] == want_status, got
    return out, lse


def window_call(window, sinks):
    return lambda c, kw: D.dsa_window_mla(c["dq"], c["kv"], c["batch"], window=window, sinks=sinks, **kw)


def tree_call(masks):
    m = torch.tensor([x - (1 << 64) if x >> 63 else x for x in masks], dtype=torch.int64).to(DEV)
    return lambda c, kw: D.dsa_tree_mla(c["dq"], m, c["kv"], c["batch"], **kw)


def window_case(seed, seq, q_len, window, sinks, **kw):
    return make_case(seed, seq, q_len, lambda r, t: O.window_positions(seq[r] - q_len[r] + t, window, sinks), **kw)


WINDOW = [
    # contexts and windows around the page and tile edges, one row each
    ([1], [1], 1, 0), ([1], [1], 64, 9), ([63, 64, 65, 128, 129], [1] * 5, 64, 0), ([63, 64, 65, 128, 129], [1] * 5, 65, 1),
    ([200, 257], [1, 1], 1, 0), ([200, 257], [1, 1], 1, 1), ([200, 257], [1, 1], 63, 64), ([500, 130], [1, 1], 70, 65),
    # the sinks reach into the window, or past the row
    ([300], [1], 100, 250), ([300, 40], [1, 1], 10, 1000), ([300], [1], 2 ** 31 - 1, 0), ([300], [1], 2 ** 31 - 1, 2 ** 31 - 1),
    # several rows a request, requests without rows, requests that are all new
    ([130, 64, 7, 0, 900], [5, 64, 7, 0, 3], 50, 3), ([700], [150], 129, 17), ([1, 0, 2], [1, 0, 2], 8, 8),
    # many tiles and a gap, ragged; more rows than SMs
    ([5000, 1717, 3001], [1, 2, 1], 2500, 100), ([90 + 3 * r for r in range(200)], [1] * 200, 40, 5),
]


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("seq,q_len,window,sinks", WINDOW)
def test_window(seq, q_len, window, sinks, f32):
    c = window_case(len(seq) * 1000 + window % 997, seq, q_len, window, sinks)
    compare(c, *run(c, window_call(window, sinks), f32))


def rand_tree(rng, n):
    masks = []
    for u in range(n):
        p = rng.integers(-1, u) if u else -1
        masks.append((masks[p] if p >= 0 else 0) | 1 << u)
    return masks


def tree_case(seed, seq, masks, **kw):
    q_len = [len(m) for m in masks]
    c = make_case(seed, seq, q_len, lambda r, t: O.tree_positions(seq[r] - q_len[r], masks[r][t], q_len[r]), **kw)
    return c, tree_call([x for m in masks for x in m])


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("seq,nodes", [([9], [8]), ([1], [1]), ([64, 65, 190], [1, 1, 64]), ([64], [64]), ([1000, 77, 300], [16, 7, 33]),
                                       ([2500, 2600], [64, 20]), ([40 + r for r in range(30)], [8] * 30)])
def test_tree(seq, nodes, f32):
    rng = np.random.default_rng(sum(seq))
    c, call = tree_case(sum(nodes), seq, [rand_tree(rng, n) for n in nodes])
    compare(c, *run(c, call, f32))


def test_tree_masks_that_are_no_tree():
    """Any pattern: rows that see nothing, only the prefix, later nodes, not themselves; bits beyond the request's tokens."""
    full = (1 << 64) - 1
    masks = [[0, 0, 1], [full, 0, full & ~7, 1 << 63], [full] * 64, [1 << 63 | 5] * 64]
    seq = [3, 100, 64, 130]
    c, call = tree_case(5, seq, masks)
    compare(c, *run(c, call))


def test_chain_of_drafts_is_causal_attention():
    """A tree that is a chain sees what causal rows see: the two calls agree."""
    seq, n = [300, 1000], [6, 6]
    c, call = tree_case(8, seq, [[(2 << u) - 1 for u in range(k)] for k in n])
    a, za = run(c, call)
    b, zb = run(c, window_call(1 << 20, 0))
    compare(c, a, za)
    assert torch.allclose(a, b, rtol=0, atol=0) and torch.equal(za, zb)


def test_rows_with_no_visible_position_and_a_padded_batch():
    """Rows behind q_start[B] keep what was there; a request shorter than its new tokens sees nothing."""
    c = window_case(11, [70, 130], [2, 1], 40, 2, pad_rows=5)
    out, lse = run(c, window_call(40, 2))
    compare(c, out, lse)
    assert (out[3:] == SENTINEL).all() and (lse[3:] == SENTINEL).all()
    c["batch"].seq_len[0] = 1                                        # q_len 2 > seq_len 1
    out, lse = run(c, window_call(40, 2))
    assert (out[:2] == 0).all() and torch.isinf(lse[:2]).all() and (lse[:2] < 0).all()


@pytest.mark.parametrize("scale,q_scale", [(1.0 / 16, 3e4), (1.0 / 16, 1e-6), (4.0, 1.0), (1e-3, 1e3), (1e-30, 1.0)])
def test_magnitudes(scale, q_scale):
    """Queries far outside fp16's range and sharp or flat softmaxes."""
    c = window_case(3, [400, 90], [1, 2], 300, 3, q_scale=q_scale)
    compare(c, *run(c, window_call(300, 3), scale=scale), scale=scale)


def test_bad_pages_are_recorded_and_not_seen():
    c = window_case(21, [400, 700], [1, 3], 250, 70, full_table=True)
    table = c["batch"].page_table
    for r, k, bad in ((0, 4, -1), (1, 0, c["pages"]), (1, 10, 2 ** 31 - 1)):
        table[r, k] = bad
    out, lse = run(c, window_call(250, 70), want_status=D.DEVERR_PAGE_RANGE)
    bad = {0: [4], 1: [0, 10]}

    def kept(i, kv):
        return kv[~np.isin(c["rows"][i][0] // 64, bad[0 if i == 0 else 1])]

    compare(c, out, lse, kv_of=kept)


def test_a_row_whose_only_page_is_bad_sees_nothing():
    c = window_case(22, [40, 40], [1, 1], 64, 0)
    c["batch"].page_table[1, 0] = -1
    out, lse = run(c, window_call(64, 0), want_status=D.DEVERR_PAGE_RANGE)
    compare(c, out, lse, kv_of=lambda i, kv: kv if i == 0 else kv[:0])


def test_contexts_longer_than_the_table_are_cut():
    c = window_case(23, [128, 100], [1, 1], 100, 0)
    c["batch"].seq_len[0] = 200                                      # the table holds 128 positions
    out, lse = run(c, window_call(172, 0), want_status=D.DEVERR_INDEX_RANGE)
    ok = window_case(23, [128, 100], [1, 1], 100, 0)
    good, z = run(ok, window_call(100, 0))
    assert torch.equal(out, good) and torch.equal(lse, z)


def test_cache_beyond_32_bits():
    """A pool of 4.6 GB with the pages of the call at its far end."""
    c = window_case(31, [500], [2], 400, 10)
    far, off = 110_000, 110_000 - c["pages"]
    kv = torch.empty(far * D.KV_PAGE_BYTES, dtype=torch.uint8, device=DEV)
    kv[off * D.KV_PAGE_BYTES:] = c["kv"]
    t = c["batch"].page_table
    t[t >= 0] += off
    b = c["batch"].c
    c["kv"], c["batch"] = kv, D.Batch(c["batch"].seq_len, c["batch"].q_start, t, far, max_seq_len=b.max_seq_len, max_q_len=2, total_q=2)
    compare(c, *run(c, window_call(400, 10)))


def test_latents_out_of_range_are_recorded():
    c = window_case(41, [100], [1], 100, 0)
    kv = c["kv"].view(-1, 64, 656)
    kv[int(c["table"][0, 1]), 3, 512:516] = torch.tensor([2.0 ** -20]).view(torch.uint8).to(DEV)
    run(c, window_call(100, 0), want_status=D.DEVERR_FP16_RANGE)
    c["dq"][0, 0, 0] = float("inf")
    kv[int(c["table"][0, 1]), 3, 512:516] = torch.tensor([1.0]).view(torch.uint8).to(DEV)
    run(c, window_call(100, 0), want_status=D.DEVERR_FP16_RANGE)


def test_other_streams_dirty_workspaces_and_graphs_that_share_one():
    a = window_case(51, [900, 333], [1, 1], 700, 9)
    b, call_b = tree_case(52, [2000, 100], [rand_tree(np.random.default_rng(1), 20), [1, 3]])
    call_a = window_call(700, 9)
    ws = torch.empty(max(D.dsa_dense_mla_workspace_size(x["batch"]) for x in (a, b)), dtype=torch.uint8, device=DEV)
    want_a, want_b = run(a, call_a), run(b, call_b)
    compare(a, *want_a)
    compare(b, *want_b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for fill in (0, 0xAB, 0xFF):
        with torch.cuda.stream(side):
            ws.fill_(fill)
        got = run(a, call_a, stream=side, ws=ws)
        assert torch.equal(got[0], want_a[0]) and torch.equal(got[1], want_a[1])
    # two captured graphs on one workspace, replayed in turn with the inputs changed in between
    side.synchronize()
    outs = {}
    graphs = {}
    for name, x, call in (("a", a, call_a), ("b", b, call_b)):
        n = x["batch"].total_q
        outs[name] = (torch.zeros(n, 64, 512, device=DEV), torch.zeros(n, 64, device=DEV))
        graphs[name] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[name]):
            call(x, dict(out=outs[name][0], lse=outs[name][1], out_dtype=D.DTYPE_F32, ws=ws))
    for name, want in (("a", want_a), ("b", want_b), ("b", want_b), ("a", want_a)):
        outs[name][0].zero_()
        graphs[name].replay()
        assert torch.equal(outs[name][0], want[0]) and torch.equal(outs[name][1], want[1])
    a["dq"].neg_()
    neg = run(a, call_a)
    graphs["a"].replay()
    assert torch.equal(outs["a"][0], neg[0]) and not torch.equal(neg[0], want_a[0])


def test_results_do_not_change_from_call_to_call():
    c = window_case(61, [3000, 50, 1200], [2, 1, 9], 1100, 30)
    first = run(c, window_call(1100, 30))
    for _ in range(5):
        again = run(c, window_call(1100, 30))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_binding_refuses_short_and_foreign_tensors():
    c = window_case(71, [100], [1], 100, 0)
    with pytest.raises(ValueError):
        D.dsa_window_mla(c["dq"], c["kv"][:-1], c["batch"], window=4)
    with pytest.raises(ValueError):
        D.dsa_window_mla(c["dq"].transpose(1, 2), c["kv"], c["batch"], window=4)
    with pytest.raises(TypeError):
        D.dsa_tree_mla(c["dq"], torch.zeros(1, dtype=torch.int32, device=DEV), c["kv"], c["batch"])
    with pytest.raises(ValueError):
        D.dsa_tree_mla(c["dq"], torch.zeros(0, dtype=torch.int64, device=DEV), c["kv"], c["batch"])
    with pytest.raises(D.DsaError):
        D.dsa_window_mla(c["dq"], c["kv"], c["batch"], window=0)


@pytest.mark.parametrize("seq,q_len,window", [([100], [1], 100), ([40000, 900], [1, 2], 39000), ([700, 0, 600], [300, 0, 64], 260)])
def test_a_wait_that_runs_out_is_recorded_and_nothing_else_is_touched(seq, q_len, window):
    """With no time to wait, the kernel winds down from its first tile on: it reads no tile that was not
    laid out, leaves rows behind the last request alone, and the next call is right."""
    c = window_case(81, seq, q_len, window, 0, pad_rows=3)
    n = c["T"]
    for _ in range(3):
        st = D.new_device_status(DEV)
        out = torch.full((n + 3, 64, 512), SENTINEL, device=DEV)
        lse = torch.full((n + 3, 64), SENTINEL, device=DEV)
        try:
            D.dsa_debug_set_wait_limit_ns(0)
            D.dsa_window_mla(c["dq"], c["kv"], c["batch"], window=window, out=out, out_dtype=D.DTYPE_F32, lse=lse, dev_status=st)
            torch.cuda.synchronize()
        finally:
            D.dsa_debug_set_wait_limit_ns(2_000_000_000)
        assert D.dsa_device_status_read(st)[0] == D.DEVERR_TIMEOUT
        assert (out[n:] == SENTINEL).all() and (lse[n:] == SENTINEL).all()
        compare(c, *run(c, window_call(window, 0)))


LARGE = [(1.0 / 16, 1e8), (1.0 / 16, 1e9), (1.0 / 16, 1e12), (1.0 / 16, 1e30), (1.0 / 16, 1e33), (1.0 / 16, 1e36), (3e38, 1e-36), (1e30, 1e-6)]


@pytest.mark.parametrize("scale,q_scale", LARGE)
def test_large_scores_of_one_position(scale, q_scale):
    """A row that sees one position gives its latent (P's fp16 rounding aside) and its score, however
    large and of either sign: |S| up to 1e37."""
    c = window_case(7, [90, 300], [1, 2], 1, 0, q_scale=q_scale)
    out, lse = (f64(x) for x in run(c, window_call(1, 0), scale=scale))
    for i, (_, kv) in enumerate(c["rows"]):
        q = f64(c["q"][i])
        s, mag = scale * (q @ kv[0]), scale * (np.abs(q) @ np.abs(kv[0]))
        assert (np.abs(out[i] - kv[:, :512]) <= (2.0 ** -11 + 2.0 ** -18) * np.abs(kv[:, :512])).all(), f"row {i}"
        assert (np.abs(lse[i] - s) <= 40 * 2.0 ** -23 * mag + 2.0 ** -22 * np.abs(s) + 2.0 ** -20).all(), f"row {i}"


@pytest.mark.parametrize("scale,q_scale", LARGE)
def test_large_scores_of_many_positions(scale, q_scale):
    """Where the largest score leads by more than the scores' own error, its latent is the output, in
    whole rows and in rows that several shares hold; no head is without a number."""
    c = window_case(9, [700, 40000], [2, 1], 20000, 3, q_scale=q_scale)
    out, lse = (f64(x) for x in run(c, window_call(20000, 3), scale=scale))
    sure = 0
    for i, (_, kv) in enumerate(c["rows"]):
        q = f64(c["q"][i])
        s = scale * (q @ kv.T)
        dS = 40 * 2.0 ** -23 * scale * (np.abs(q) @ np.abs(kv).T).max(1)
        top = np.sort(s, 1)[:, -2:]
        assert np.isfinite(out[i]).all() and (np.abs(lse[i] - top[:, 1]) <= dS + 2.0 ** -22 * np.abs(top[:, 1]) + 12).all(), f"row {i}"
        for h in np.nonzero(top[:, 1] - top[:, 0] > 2 * dS + 60)[0]:
            best = kv[s[h].argmax(), :512]
            assert (np.abs(out[i, h] - best) <= (2.0 ** -11 + 2.0 ** -18) * np.abs(best) + 2.0 ** -60).all(), f"row {i}, head {h}"
            sure += 1
    assert sure > 100


def test_a_long_tail_behind_a_dominating_sink():
    """One position of zero latent whose score leads by 8 to 22 nats and 131,072 others, in so many rows
    that a share holds whole ones: the output is the others'.  P of a position is off by 2^-11 of itself,
    or by half of fp16's smallest step, 2^-25, against a sum of P of at least 2^3 in a piece's first 32
    tiles of two pages and 2^9 behind them.  O is summed by the tensor core, 16 positions a step, each
    off by at most 2^-23 of a partial sum: every latent is positive, so of the value, n / 16 times."""
    g = torch.Generator(device=DEV).manual_seed(17)
    rows, n = 304, 131072 + 304
    lat = torch.randn(n, 512, generator=g, device=DEV).abs().to(torch.bfloat16)
    rope = (0.05 * torch.randn(n, 64, generator=g, device=DEV)).to(torch.bfloat16)
    lead = torch.where(torch.randn(64, generator=g, device=DEV) > 0, 1.0, -1.0)
    lat[0], rope[0] = 0, lead.to(torch.bfloat16)
    q = torch.zeros(rows, 64, 576, device=DEV)
    q[:, :, 512:] = lead * torch.linspace(2.0, 5.5, 64, device=DEV)[:, None]    # times 64 / 16: 8 .. 22
    q = q.to(torch.bfloat16)
    pages = (n + 63) // 64
    kv = torch.zeros(pages * D.KV_PAGE_BYTES, dtype=torch.uint8, device=DEV)
    D.dsa_latent_kv_store(lat, rope, torch.arange(n, device=DEV), kv)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    batch = D.Batch(ints(n), ints(0, rows), table, pages, max_seq_len=n, max_q_len=rows, total_q=rows)
    st = D.new_device_status(DEV)
    lse = torch.empty(rows, 64, device=DEV)
    out = D.dsa_window_mla(q, kv, batch, window=n, out_dtype=D.DTYPE_F32, lse=lse, dev_status=st).double()
    assert D.dsa_device_status_read(st)[0] == 0
    raw = kv.view(-1, 656)[:n]
    k = raw[:, :512].contiguous().view(torch.float8_e4m3fn).double()
    k = torch.cat([k * raw[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, 1), rope.double()], 1)
    for i in (0, 1, 151, 302, 303):
        kk = k[: n - rows + 1 + i]
        s = q[i].double() @ kk.T / 16
        z = torch.logsumexp(s, 1)
        p = torch.exp(s - z[:, None])
        want = p @ kk[:, :512]
        dS = 40 * 2.0 ** -23 * (q[i].double().abs() @ kk.abs().T).amax(1) / 16
        tol = want * (2.0 ** -11 + 2 * dS[:, None] + 2.0 ** -18 + n / 16 * 2.0 ** -23) + 2.0 ** -34 * kk[:, :512].sum(0) + 2.0 ** -28 * kk[:4096, :512].sum(0)
        err = (out[i] - want).abs()
        assert bool((err <= tol).all()), f"row {i}: worst {float((err / tol).max()):.1f} of the bound, {float((err / want).max()):.2%} of the value"
        assert bool(((lse[i].double() - z).abs() <= dS + 2.0 ** -20 + 2.0 ** -22 * z.abs()).all())


@pytest.mark.parametrize("what", ["latent", "rope"])
@pytest.mark.parametrize("seq,window", [([300, 130], 200), ([30000, 130], 29000)])
def test_a_nan_that_a_row_sees_shows(seq, window, what):
    """Its row is NaN, in one share or several, never the zeros of a row that sees nothing."""
    c = window_case(43, seq, [2, 1], window, 3)
    at = seq[0] - 2 - window + 1                                     # the first row's first position, which the second does not see
    kv = c["kv"].view(-1, 64, 656)
    page = int(c["table"][0, at // 64])
    if what == "latent":
        kv[page, at % 64, 77] = 0x7f
    else:
        kv[page, at % 64, 528:530] = torch.tensor([0x7fc0], dtype=torch.int16).view(torch.uint8).to(DEV)
    out, lse = run(c, window_call(window, 3), want_status=D.DEVERR_FP16_RANGE if what == "rope" else 0)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    for i in (1, 2):
        ref, z, tol, ztol = reference(f64(c["q"][i]), c["rows"][i][1])
        assert (np.abs(f64(out[i]) - ref) <= tol).all() and (np.abs(f64(lse[i]) - z) <= ztol).all()


def test_contexts_up_to_the_largest_length():
    """2^31 - 1 tokens, whose last page ends past what 32 bits hold, with all but the window's pages given back."""
    L, window = 2 ** 31 - 1, 100
    c = window_case(29, [200], [1], window, 0)                       # the positions 100 .. 199 of 200 become the last of L
    kv = c["kv"].view(-1, 64, 656)
    rows = torch.stack([kv[int(c["table"][0, j // 64]), j % 64] for j in range(100, 200)])
    far = torch.full((3 * 64, 656), 0x7f, dtype=torch.uint8, device=DEV)
    at = torch.arange(L - 100, L, device=DEV)
    table = torch.full((1, 2 ** 25), -1, dtype=torch.int32, device=DEV)
    table[0, 2 ** 25 - 2:] = torch.tensor([2, 0], dtype=torch.int32, device=DEV)
    far[table[0, at // 64].long() * 64 + at % 64] = rows
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    c["kv"], c["batch"] = far.view(-1), D.Batch(ints(L), ints(0, 1), table, 3, max_seq_len=L, max_q_len=1, total_q=1)
    compare(c, *run(c, window_call(window, 0)))


def test_what_a_call_allocates_is_memory_of_its_stream(monkeypatch):
    """Outputs and workspaces that the caller does not give are allocated on the call's stream: a workspace
    is free again when the call returns, and work of another stream must not get it before the kernels
    have run.  The results are those of a call on the current stream."""
    c = window_case(91, [3000, 70], [1, 1], 2500, 3)
    mask = torch.ones(2, dtype=torch.int64, device=DEV)
    topk = torch.full((2, D.TOPK), -1, dtype=torch.int32, device=DEV)
    topk[:, :70] = torch.arange(70, device=DEV)
    caches = D.CacheSet([], c["pages"])
    qi, w = torch.randn(2, 32, 128, device=DEV).to(torch.bfloat16), torch.rand(2, 32, device=DEV)
    idx = torch.zeros(c["pages"] * D.IDXK_PAGE_BYTES, dtype=torch.uint8, device=DEV)
    scores = torch.randn(2, 3000, device=DEV)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    full = window_case(92, [300, 70], [1, 1], 300, 0, full_table=True)
    b = full["batch"]
    calls = {
        "window": lambda s: D.dsa_window_mla(c["dq"], c["kv"], c["batch"], window=2500, sinks=3, stream=s),
        "tree": lambda s: D.dsa_tree_mla(full["dq"], mask, full["kv"], b, stream=s),
        "commit": lambda s: D.dsa_tree_commit(ints([0], [-1]), c["batch"], caches, stream=s),
        "sparse": lambda s: D.dsa_sparse_mla_decode(full["dq"], topk, full["kv"], b, stream=s),
        "topk": lambda s: D.dsa_indexer_topk(qi, w, idx, b, stream=s),
        "from_scores": lambda s: D.dsa_topk_from_scores(scores, ints(3000, 70), stream=s),
    }
    want = {name: call(None) for name, call in calls.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    seen, real = [], torch.empty

    def empty(*a, **k):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return real(*a, **k)

    for name, call in calls.items():
        del seen[:]
        monkeypatch.setattr(torch, "empty", empty)
        got = call(side)
        monkeypatch.setattr(torch, "empty", real)
        assert seen and all(x == side.cuda_stream for x in seen), name
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want[name]), name


def test_windows_and_sinks_beyond_32_bits_are_the_whole_context():
    c = window_case(95, [300, 129], [1, 2], 2 ** 40, 0)
    whole = run(c, window_call(2 ** 31 - 1, 0))
    compare(c, *whole)
    for window, sinks in ((2 ** 31, 0), (2 ** 32 + 5, 0), (2 ** 63, 0), (1, 2 ** 32), (1, 2 ** 32 + 3)):
        out, lse = run(c, window_call(window, sinks))
        assert torch.equal(out, whole[0]) and torch.equal(lse, whole[1]), (window, sinks)
    for window, sinks in ((0, 0), (-2 ** 32 + 5, 0), (5, -1), (5, -2 ** 32 + 1)):
        with pytest.raises(D.DsaError):
            D.dsa_window_mla(c["dq"], c["kv"], c["batch"], window=window, sinks=sinks)
