"""GPU parity of the token and page calls with the oracle's plain definitions:
everything here is whole numbers and has to be equal.  The last test runs the
calls together as a serving loop would."""

import numpy as np
import pytest
import torch

import dsa_sparse_attention_indexer_gb300 as D
from oracle import dsa_oracle as O
from tests.oracle_side import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BYTES = {D.CACHE_KV: D.KV_PAGE_BYTES, D.CACHE_IDXK: D.IDXK_PAGE_BYTES, D.CACHE_IDXK_MXFP4: D.IDXK_MXFP4_PAGE_BYTES}


def dev(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype))).to(DEV)


def token_rows(page_bytes, kind):
    """[64, row bytes] view of each token's bytes in a page (payload, then scale word)."""
    if kind == D.CACHE_KV:
        return page_bytes.reshape(-1, 64, 656)
    payload = 128 if kind == D.CACHE_IDXK else 64
    p = page_bytes[:, :64 * payload].reshape(-1, 64, payload)
    return np.concatenate([p, page_bytes[:, 64 * payload:].reshape(-1, 64, 4)], 2)


def raw_caches(rng, pages, kinds):
    return [rng.integers(0, 256, (pages, BYTES[k]), dtype=np.uint8) for k in kinds]


def device_caches(host, kinds, pages):
    t = [torch.from_numpy(h.copy()).to(DEV) for h in host]
    return t, D.CacheSet(list(zip(t, kinds)), pages)


ALL = [D.CACHE_KV, D.CACHE_IDXK, D.CACHE_IDXK_MXFP4, D.CACHE_KV]


@pytest.mark.parametrize("kinds", [[D.CACHE_KV], ALL, [D.CACHE_IDXK_MXFP4] * 130, [D.CACHE_IDXK] * 128, []])
@pytest.mark.parametrize("prefix,q_len,accept", [
    ([0], [1], [[0]]), ([60], [8], [[0, 3, 7, -1]]), ([63, 64, 100], [64, 1, 9], [[5, 4, 63, 0], [0, -1, -1, -1], [-1, 3, 3, 3]]),
    ([10], [64], [list(range(63, -1, -1))]), ([200, 7], [40, 40], [[2] * 5, [39, 38, 0, 40, 1]]), ([130], [33], [[1 + 2 * k for k in range(16)]])])
def test_tree_commit(prefix, q_len, accept, kinds):
    rng = np.random.default_rng(sum(prefix) + len(kinds))
    B, seq = len(prefix), [p + n for p, n in zip(prefix, q_len)]
    width = max((s + 63) // 64 for s in seq)
    pages = B * width + 2
    table = rng.permutation(pages)[: B * width].reshape(B, width).astype(np.int32)
    host = raw_caches(rng, pages, kinds)
    t, caches = device_caches(host, kinds, pages)
    start = np.concatenate([[0], np.cumsum(q_len)])
    batch = D.Batch(dev(seq), dev(start), dev(table), pages, max_seq_len=max(seq), max_q_len=max(q_len), total_q=int(start[-1]))
    st = D.new_device_status(DEV)
    got = D.dsa_tree_commit(dev(accept), batch, caches, dev_status=st)
    bad = any(any(0 <= a for a in row[:1]) and any(a >= q_len[r] for a in row) for r, row in enumerate(accept))
    assert D.dsa_device_status_read(st)[0] == (D.DEVERR_INDEX_RANGE if bad else 0)
    for i, kind in enumerate(kinds):
        want = token_rows(host[i], kind)
        for r in range(B):
            at = np.arange(seq[r])
            slots = (table[r, at // 64], at % 64)
            rows, _ = O.tree_commit(want[slots], prefix[r], q_len[r], accept[r])
            want[slots] = rows
        assert np.array_equal(token_rows(t[i].cpu().numpy(), kind), want), f"cache {i}"
    assert got.cpu().tolist() == [prefix[r] + O.tree_commit(np.zeros(seq[r]), prefix[r], q_len[r], accept[r])[1] for r in range(B)]


def test_commit_records_bad_pages_and_lengths():
    pages, table = 4, np.array([[0, -1], [2, 9], [3, 3]], np.int32)
    host = raw_caches(np.random.default_rng(1), pages, [D.CACHE_KV])
    t, caches = device_caches(host, [D.CACHE_KV], pages)
    batch = D.Batch(dev([70, 70, 3]), dev([0, 8, 16, 20]), dev(table), pages, max_seq_len=128, max_q_len=8, total_q=20)
    st = D.new_device_status(DEV)
    got = D.dsa_tree_commit(dev([[4], [4], [2]]), batch, caches, dev_status=st)
    assert D.dsa_device_status_read(st)[0] == D.DEVERR_PAGE_RANGE | D.DEVERR_INDEX_RANGE
    assert np.array_equal(t[0].cpu().numpy(), host[0])
    assert got.cpu().tolist()[:2] == [63, 63]


def pool_state(rng, pages, rows, width, held):
    ref, table = np.zeros(pages, np.int32), np.full((rows, width), -1, np.int32)
    perm = rng.permutation(pages)
    at = 0
    for r, n in enumerate(held):
        table[r, :n] = perm[at: at + n]
        at += n
    ref[perm[:at]] = 1
    ref[perm[at: at + (pages - at) // 3]] = 2                        # set aside by others
    return ref, table


@pytest.mark.parametrize("pages,width,n", [(1, 1, 1), (7, 3, 2), (100, 9, 5), (16384, 40, 64), (16385, 17, 300), (70001, 20, 1000)])
def test_reserve_and_release(pages, width, n):
    rng = np.random.default_rng(pages)
    rows = n + 3
    held = [int(rng.integers(0, min(width, max(1, pages // (2 * rows))) + 1)) if pages >= 2 * rows else 0 for _ in range(rows)]
    ref, table = pool_state(rng, pages, rows, width, held)
    dref, dtable = dev(ref), dev(table)
    for step in range(3):
        st = D.new_device_status(DEV)
        row = rng.permutation(rows)[:n]
        have = [int(held[r]) * 64 - int(rng.integers(0, 64)) if held[r] else 0 for r in row]
        want = [int(rng.integers(0, width * 64 + 1)) for _ in row]
        errors = O.pages_reserve(ref, table, row.tolist(), have, want)
        D.dsa_pages_reserve(dref, dtable, dev(row), dev(have), dev(want), dev_status=st)
        s = D.dsa_device_status_read(st)
        assert (s[0], s[1]) == (D.DEVERR_PAGE_POOL if errors else 0, errors)
        assert np.array_equal(dtable.cpu().numpy(), table) and np.array_equal(dref.cpu().numpy(), ref)
        row = rng.integers(0, rows, n)                               # rows may be named twice
        first = rng.integers(-2, width + 2, n)
        end = first + rng.integers(-1, width + 2, n)
        st = D.new_device_status(DEV)
        errors = O.pages_release(ref, table, row.tolist(), first.tolist(), end.tolist())
        D.dsa_pages_release(dref, dtable, dev(row), dev(first), dev(end), dev_status=st)
        assert D.dsa_device_status_read(st)[1] == errors == 0
        assert np.array_equal(dtable.cpu().numpy(), table) and np.array_equal(dref.cpu().numpy(), ref)
        held = rng.integers(0, width + 1, rows).tolist()


def test_reserve_refuses_rows_and_lengths():
    ref, table = np.zeros(40, np.int32), np.full((4, 6), -1, np.int32)
    table[2, 1] = 7
    ref[7] = 1
    dref, dtable = dev(ref), dev(table)
    row, have, want = [1, 9, 1, -1, 2, 3, 0], [0, 0, 0, 0, 0, -5, 2 ** 31 - 1], [65, 64, 640, 1, 130, 2 ** 31 - 1, 2 ** 31 - 1]
    st = D.new_device_status(DEV)
    D.dsa_pages_reserve(dref, dtable, dev(row), dev(have), dev(want), dev_status=st)
    errors = O.pages_reserve(ref, table, row, have, want)
    s = D.dsa_device_status_read(st)
    assert s[0] == D.DEVERR_INDEX_RANGE and s[1] == errors == 5
    assert np.array_equal(dtable.cpu().numpy(), table) and np.array_equal(dref.cpu().numpy(), ref)
    assert table[2].tolist()[1] == 7                                 # an entry that holds a page keeps it


def test_release_records_bad_counts_and_pages():
    ref, table = np.array([0, 1, -3, 2], np.int32), np.array([[0, 1, 2, 3], [3, 3, 4, -1]], np.int32)
    dref, dtable = dev(ref), dev(table)
    st = D.new_device_status(DEV)
    D.dsa_pages_release(dref, dtable, dev([0, 1, 5, 0]), dev([0] * 4), dev([4, 2, 1, 4]), dev_status=st)
    errors = O.pages_release(ref, table, [0, 1, 5, 0], [0] * 4, [4, 2, 1, 4])
    s = D.dsa_device_status_read(st)
    assert s[0] == D.DEVERR_PAGE_COUNT | D.DEVERR_INDEX_RANGE and s[1] == errors
    assert np.array_equal(dtable.cpu().numpy(), table) and np.array_equal(dref.cpu().numpy(), ref)
    st = D.new_device_status(DEV)
    D.dsa_pages_release(dref, dtable, dev([1]), dev([2]), dev([3]), dev_status=st)
    assert D.dsa_device_status_read(st)[0] == D.DEVERR_PAGE_RANGE


@pytest.mark.parametrize("kinds", [[D.CACHE_KV], ALL, [D.CACHE_IDXK_MXFP4] * 129, []])
@pytest.mark.parametrize("width,src,dst,length", [
    (1, [0], [1], [1]), (3, [0, 0, 0], [1, 2, 3], [64, 65, 63]), (3, [0, 4], [1, 2], [0, 150]), (2, [0], [3], [128]),
    (4, [0, 1, 4, 4], [2, 3, 5, 6], [191, 192, 193, 256]), (40, [0] * 6, [1, 2, 3, 4, 5, 6], [2500, 1, 640, 641, 700, 2560])])
def test_fork(width, src, dst, length, kinds):
    rng = np.random.default_rng(width * 10 + len(kinds))
    rows = 7
    held = [width if r in src else 0 for r in range(rows)]
    pages = sum(held) + 9
    ref, table = pool_state(rng, pages, rows, width, held)
    if width > 3:
        table[src[0], 1] = -1                                        # a page that a window left behind
    host = raw_caches(rng, pages, kinds)
    t, caches = device_caches(host, kinds, pages)
    dref, dtable = dev(ref), dev(table)
    st = D.new_device_status(DEV)
    D.dsa_pages_fork(dref, dtable, dev(src), dev(dst), dev(length), caches, dev_status=st)
    errors, copies = O.pages_fork(ref, table, src, dst, length)
    s = D.dsa_device_status_read(st)
    assert s[1] == errors and (errors == 0) == (s[0] == 0)
    assert np.array_equal(dtable.cpu().numpy(), table) and np.array_equal(dref.cpu().numpy(), ref)
    for i, kind in enumerate(kinds):
        want = token_rows(host[i], kind)
        for a, b, n in copies:
            want[b, :n] = want[a, :n]
        assert np.array_equal(token_rows(t[i].cpu().numpy(), kind), want), f"cache {i}"


def test_fork_refusals_and_an_empty_pool():
    ref, table = np.ones(20, np.int32), np.full((6, 4), -1, np.int32)
    table[0], table[1] = [0, 1, 2, 3], [4, 5, 25, 7]
    ref[[9, 13]] = 0
    dref, dtable = dev(ref), dev(table)
    src, dst, length = [0, 0, 1, 0, 7, 1, 1], [2, 2, 0, 3, 4, 4, 5], [70, 70, 10, 300, 5, 150, 200]
    st = D.new_device_status(DEV)
    D.dsa_pages_fork(dref, dtable, dev(src), dev(dst), dev(length), D.CacheSet([], 20), dev_status=st)
    errors, _ = O.pages_fork(ref, table, src, dst, length)
    s = D.dsa_device_status_read(st)
    assert s[0] == D.DEVERR_INDEX_RANGE | D.DEVERR_PAGE_RANGE and s[1] == errors
    assert np.array_equal(dtable.cpu().numpy(), table) and np.array_equal(dref.cpu().numpy(), ref)
    ref[:] = 1                                                       # no page left: the child lacks its last page
    table[2:] = -1
    dref, dtable = dev(ref), dev(table)
    st = D.new_device_status(DEV)
    D.dsa_pages_fork(dref, dtable, dev([0]), dev([2]), dev([70]), D.CacheSet([], 20), dev_status=st)
    assert D.dsa_device_status_read(st)[0] == D.DEVERR_PAGE_POOL
    O.pages_fork(ref, table, [0], [2], [70])
    assert np.array_equal(dtable.cpu().numpy(), table) and np.array_equal(dref.cpu().numpy(), ref)


def test_reserve_of_many_rows_in_a_large_pool():
    """As many requests as one call takes, rows named again among them, and so few free
    pages up front that the walk goes round several times."""
    rng = np.random.default_rng(77)
    pages, rows, width, n = 400001, 4500, 6, 4096
    ref = rng.integers(1, 4, pages).astype(np.int32)
    ref[rng.permutation(pages)[:7000]] = 0
    ref[-3:] = 0
    table = np.full((rows, width), -1, np.int32)
    table[::7, 1] = 5                                                # entries that hold a page keep it
    row = rng.permutation(rows)[:n]
    row[rng.permutation(n)[:200]] = row[rng.permutation(n)[:200]]
    row[[3, 4000]] = [rows, -7]
    have = rng.integers(0, 2 * 64, n)
    want = np.minimum(have + rng.integers(-64, 5 * 64, n), width * 64)
    dref, dtable = dev(ref), dev(table)
    st = D.new_device_status(DEV)
    D.dsa_pages_reserve(dref, dtable, dev(row), dev(have), dev(want), dev_status=st)
    errors = O.pages_reserve(ref, table, row.tolist(), have.tolist(), want.tolist())
    s = D.dsa_device_status_read(st)
    assert s[1] == errors and s[0] == D.DEVERR_INDEX_RANGE | D.DEVERR_PAGE_POOL
    assert np.array_equal(dtable.cpu().numpy(), table) and np.array_equal(dref.cpu().numpy(), ref)


def test_fork_of_many_rows():
    """Children named again, and named as sources, in a call of as many as there may be."""
    rng = np.random.default_rng(78)
    rows, width, n = 4300, 3, 4096
    ref, table = pool_state(rng, 20000, rows, width, [width if r < 100 else 0 for r in range(rows)])
    src = rng.integers(0, 100, n)
    dst = 100 + rng.permutation(rows - 100)[:n]
    dst[rng.permutation(n)[:50]] = dst[rng.permutation(n)[:50]]
    dst[[7, 9, 4095]] = [src[0], -1, rows]
    length = rng.integers(0, width * 64 + 1, n)
    host = raw_caches(rng, 20000, [D.CACHE_IDXK_MXFP4])
    t, caches = device_caches(host, [D.CACHE_IDXK_MXFP4], 20000)
    dref, dtable = dev(ref), dev(table)
    st = D.new_device_status(DEV)
    D.dsa_pages_fork(dref, dtable, dev(src), dev(dst), dev(length), caches, dev_status=st)
    errors, copies = O.pages_fork(ref, table, src.tolist(), dst.tolist(), length.tolist())
    s = D.dsa_device_status_read(st)
    assert (s[0], s[1]) == (D.DEVERR_INDEX_RANGE, errors)
    assert np.array_equal(dtable.cpu().numpy(), table) and np.array_equal(dref.cpu().numpy(), ref)
    want = token_rows(host[0], D.CACHE_IDXK_MXFP4)
    for a, b, m in copies:
        want[b, :m] = want[a, :m]
    assert np.array_equal(token_rows(t[0].cpu().numpy(), D.CACHE_IDXK_MXFP4), want)


def test_commit_of_whole_lists_in_many_caches():
    """63 moves a request: the rows of two caches at most fit one round."""
    rng = np.random.default_rng(79)
    kinds = [D.CACHE_KV, D.CACHE_IDXK, D.CACHE_IDXK_MXFP4] * 3
    B, pages = 3, 12
    host = raw_caches(rng, pages, kinds)
    t, caches = device_caches(host, kinds, pages)
    table = rng.permutation(pages).reshape(B, 4).astype(np.int32)
    seq, accept = [200, 64, 130], np.stack([rng.permutation(64) for _ in range(B)]).astype(np.int32)
    batch = D.Batch(dev(seq), dev([0, 64, 128, 192]), dev(table), pages, max_seq_len=256, max_q_len=64, total_q=192)
    st = D.new_device_status(DEV)
    got = D.dsa_tree_commit(dev(accept), batch, caches, dev_status=st)
    assert D.dsa_device_status_read(st)[0] == 0 and got.cpu().tolist() == seq
    for i, kind in enumerate(kinds):
        before, want = token_rows(host[i], kind), token_rows(host[i], kind).copy()
        for r in range(B):
            for k, u in enumerate(accept[r]):
                a, b = seq[r] - 64 + u, seq[r] - 64 + k
                want[table[r, b // 64], b % 64] = before[table[r, a // 64], a % 64]
        assert np.array_equal(token_rows(t[i].cpu().numpy(), kind), want), f"cache {i}"


def test_a_cache_is_named_once():
    t = torch.zeros(2 * D.KV_PAGE_BYTES, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        D.CacheSet([(t, D.CACHE_KV), (t[:D.KV_PAGE_BYTES], D.CACHE_KV)], 1)
    D.CacheSet([(t[:D.KV_PAGE_BYTES], D.CACHE_KV), (t[D.KV_PAGE_BYTES:], D.CACHE_KV)], 1)


def test_commit_does_not_take_the_lengths_it_reads():
    seq = dev([8])
    batch = D.Batch(seq, dev([0, 4]), dev([[0]]), 1, max_seq_len=64, max_q_len=4, total_q=4)
    with pytest.raises(D.DsaError):
        D.dsa_tree_commit(dev([[0, 2]]), batch, D.CacheSet([], 1), new_seq_len=seq)
    assert D.dsa_tree_commit(dev([[0, 2]]), batch, D.CacheSet([], 1)).tolist() == [6]


def test_binding_refuses_mixed_lists():
    ref, table, one = dev([0] * 8), dev([[-1] * 4]), dev([0])
    with pytest.raises(ValueError):
        D.dsa_pages_reserve(ref, table, one, one, dev([0, 1]))
    with pytest.raises(ValueError):
        D.dsa_pages_fork(ref, table, one, one, one, D.CacheSet([(torch.zeros(41984, dtype=torch.uint8, device=DEV), D.CACHE_KV)], 1))
    with pytest.raises(ValueError):
        D.dsa_pages_release(ref, table.view(-1), one, one, one)
    D.dsa_pages_release(ref, table, one[:0], one[:0], one[:0])       # no requests: nothing to do


def store(caches, c, rope, k, pos, slot):
    D.dsa_latent_kv_store(c, rope, slot, caches[0])
    D.dsa_index_k_store(k, pos, slot, caches[1])


def slots_of(table, r, pos):
    return table[r, pos // 64].to(torch.int64) * 64 + pos % 64


def test_a_serving_loop():
    """Prompt -> fork into samples -> each verifies a tree -> commit -> the next
    tree; at the end everything is given back.  The committed caches give the same
    attention as caches written token by token with the accepted path alone, and
    the whole step (tree attention, commit) replays from one captured graph."""
    g = torch.Generator().manual_seed(9)
    B, prompt, steps, n = 3, 150, 4, 10
    width, pages, rows = 8, 60, B + 1
    kv = torch.zeros(pages * D.KV_PAGE_BYTES, dtype=torch.uint8, device=DEV)
    idx = torch.zeros(pages * D.IDXK_PAGE_BYTES, dtype=torch.uint8, device=DEV)
    ref, table = torch.zeros(pages, dtype=torch.int32, device=DEV), torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    caches = D.CacheSet([(kv, D.CACHE_KV), (idx, D.CACHE_IDXK)], pages)
    st = D.new_device_status(DEV)
    draw = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(DEV)  # noqa: E731
    D.dsa_pages_reserve(ref, table, dev([0]), dev([0]), dev([prompt]), dev_status=st)
    pos = torch.arange(prompt, dtype=torch.int32, device=DEV)
    first = (draw(prompt, 512), draw(prompt, 64), draw(prompt, 128))
    store((kv, idx), first[0], first[1], first[2], pos, slots_of(table, 0, pos.long()))
    D.dsa_pages_fork(ref, table, dev([0] * B), dev([1, 2, 3]), dev([prompt] * B), caches, dev_status=st)
    D.dsa_pages_release(ref, table, dev([0]), dev([0]), dev([width]), dev_status=st)
    assert int((ref == B).sum()) == prompt // 64 and int((ref == 1).sum()) == B
    seq = torch.full((B,), prompt, dtype=torch.int32, device=DEV)
    held = [[first] for _ in range(B)]                               # each sample's accepted tokens
    batch = D.Batch(torch.full((B,), prompt + n, dtype=torch.int32, device=DEV), dev(np.arange(B + 1) * n), table[1:].contiguous(),
                    pages, max_seq_len=width * 64, max_q_len=n, total_q=B * n)
    mask = torch.zeros(B * n, dtype=torch.int64, device=DEV)
    accept = torch.full((B, n), -1, dtype=torch.int32, device=DEV)
    q, out, lse = draw(B * n, 64, 576), torch.empty(B * n, 64, 512, device=DEV), torch.empty(B * n, 64, device=DEV)
    ws = D.workspace(D.dsa_dense_mla_workspace_size(batch), DEV)
    graph = torch.cuda.CUDAGraph()
    rng = np.random.default_rng(4)
    for step in range(steps):
        D.dsa_pages_reserve(ref, table, dev([1, 2, 3]), seq, seq + n, dev_status=st)
        batch.page_table.copy_(table[1:])
        batch.seq_len.copy_(seq + n)
        parents = [[-1] + [int(rng.integers(-1, u)) for u in range(1, n)] for _ in range(B)]
        masks, paths, depth = [], [], []
        for p in parents:
            m, at = [], {-1: []}
            for u in range(n):
                m.append((m[p[u]] if p[u] >= 0 else 0) | 1 << u)
                at[u] = at[p[u]] + [u]
            masks += m
            depth.append([len(at[u]) - 1 for u in range(n)])
            paths.append(at[int(rng.integers(0, n))])
        mask.copy_(torch.tensor(masks, dtype=torch.int64))
        accept.fill_(-1)
        for r, p in enumerate(paths):
            accept[r, : len(p)] = torch.tensor(p, dtype=torch.int32)
        q.copy_(draw(B * n, 64, 576))
        new = [(draw(n, 512), draw(n, 64), draw(n, 128)) for _ in range(B)]
        lens = seq.cpu().tolist()
        for r in range(B):
            at = torch.arange(n, device=DEV) + lens[r]               # the node's slot; its position is its depth's
            store((kv, idx), *new[r], dev(depth[r]) + lens[r], slots_of(table, 1 + r, at))

        def one():
            D.dsa_tree_mla(q, mask, kv, batch, out=out, lse=lse, out_dtype=D.DTYPE_F32, ws=ws, dev_status=st)
            D.dsa_tree_commit(accept, batch, caches, new_seq_len=seq, dev_status=st)

        if step == 0:
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                one()
        graph.replay()
        for r in range(B):
            held[r].append(tuple(x[torch.tensor(paths[r], device=DEV)] for x in new[r]))
        assert seq.cpu().tolist() == [a + len(p) for a, p in zip(lens, paths)]
    assert D.dsa_device_status_read(st)[0] == 0
    # caches written with the accepted tokens alone give the same attention
    lens = seq.cpu().tolist()
    t2 = torch.arange(B * width, dtype=torch.int32, device=DEV).view(B, width)
    kv2 = torch.zeros(B * width * D.KV_PAGE_BYTES, dtype=torch.uint8, device=DEV)
    idx2 = torch.zeros(B * width * D.IDXK_PAGE_BYTES, dtype=torch.uint8, device=DEV)
    for r in range(B):
        c, rope, k = (torch.cat([h[i] for h in held[r]]) for i in range(3))
        assert c.shape[0] == lens[r]
        pos = torch.arange(lens[r], dtype=torch.int32, device=DEV)
        store((kv2, idx2), c, rope, k, pos, slots_of(t2, r, pos.long()))
    qd = draw(B, 64, 576)
    one_row = dev(np.arange(B + 1))
    got = [D.dsa_window_mla(qd, cache, D.Batch(seq, one_row, t, np_, max_seq_len=width * 64, max_q_len=1, total_q=B), window=1 << 20,
                            out_dtype=D.DTYPE_F32)
           for cache, t, np_ in ((kv, table[1:].contiguous(), pages), (kv2, t2, B * width))]
    assert torch.equal(got[0], got[1])
    # the oracle's attention over the committed cache
    host = kv.cpu().numpy().reshape(pages, -1)
    for r in range(B):
        rows_ = O.latent_cache_read_rows(host, table[1 + r].cpu().numpy(), np.arange(lens[r]))
        want, _ = O.sparse_mla(f64(qd[r]), np.arange(lens[r]), rows_, lens[r])
        assert np.linalg.norm(f64(got[0][r]) - want) <= 1e-3 * np.linalg.norm(want)
    # the committed index keys are those of the accepted tokens at their positions
    mine, plain = (token_rows(x.cpu().numpy().reshape(-1, D.IDXK_PAGE_BYTES), D.CACHE_IDXK) for x in (idx, idx2))
    for r in range(B):
        j = np.arange(lens[r])
        assert np.array_equal(mine[table[1 + r].cpu().numpy()[j // 64], j % 64], plain[t2[r].cpu().numpy()[j // 64], j % 64])
    D.dsa_pages_release(ref, table, dev([1, 2, 3]), dev([0] * 3), dev([width] * 3), dev_status=st)
    assert D.dsa_device_status_read(st)[0] == 0
    assert (ref == 0).all() and (table == -1).all()


def test_reserve_takes_every_free_page_before_it_gives_up():
    """Entries that hold a page take none: the pages they passed over go to the entries that lack one."""
    ref, table = np.ones(40, np.int32), np.full((3, 12), -1, np.int32)
    table[1, :8] = range(8)
    ref[[9, 13, 20, 21, 39]] = 0
    for want in (10, 12):                                            # 2 and 4 missing entries behind 8 held ones, 5 free pages
        r, t = ref.copy(), table.copy()
        dref, dtable = dev(r), dev(t)
        st = D.new_device_status(DEV)
        D.dsa_pages_reserve(dref, dtable, dev([1]), dev([0]), dev([want * 64]), dev_status=st)
        assert D.dsa_device_status_read(st)[0] == 0
        assert O.pages_reserve(r, t, [1], [0], [want * 64]) == 0
        assert np.array_equal(dtable.cpu().numpy(), t) and np.array_equal(dref.cpu().numpy(), r)
        assert (t[1, :want] >= 0).all() and (r == 0).sum() == 5 - (want - 8)


@pytest.mark.parametrize("pages,free", [(30, 6), (5000, 700), (40000, 20000), (300001, 3000), (300001, 12000)])
def test_reserve_with_held_entries_in_a_short_pool(pages, free):
    """Held entries anywhere among the call's, and fewer, as many and more free pages than missing entries."""
    rng = np.random.default_rng(pages + free)
    width = 9
    rows = max(3, min(4000, 2 * free // width))
    for missing in (free // 2, free, free + 5):
        ref, table = np.ones(pages, np.int32), np.full((rows, width), -1, np.int32)
        flat = rng.permutation(rows * width)
        table.reshape(-1)[flat[min(missing, rows * width):]] = rng.integers(0, pages, max(0, rows * width - missing))
        ref[rng.permutation(pages)[:free]] = 0
        row = rng.permutation(rows)
        dref, dtable = dev(ref), dev(table)
        st = D.new_device_status(DEV)
        D.dsa_pages_reserve(dref, dtable, dev(row), dev([0] * rows), dev([width * 64] * rows), dev_status=st)
        errors = O.pages_reserve(ref, table, row.tolist(), [0] * rows, [width * 64] * rows)
        s = D.dsa_device_status_read(st)
        assert errors == max(0, min(missing, rows * width) - free)
        assert (s[0], s[1]) == (D.DEVERR_PAGE_POOL if errors else 0, errors)
        assert np.array_equal(dtable.cpu().numpy(), table) and np.array_equal(dref.cpu().numpy(), ref)


def test_commit_of_a_request_shorter_than_its_new_tokens():
    """Nothing moves, its length stays and it is recorded, whether anything was accepted or not."""
    host = raw_caches(np.random.default_rng(2), 3, [D.CACHE_KV])
    t, caches = device_caches(host, [D.CACHE_KV], 3)
    batch = D.Batch(dev([3, 0, 70]), dev([0, 4, 7, 10]), dev([[0, -1], [1, -1], [2, -1]]), 3, max_seq_len=128, max_q_len=4, total_q=10)
    for accept in ([[2], [1], [-1]], [[-1], [-1], [-1]]):
        st = D.new_device_status(DEV)
        got = D.dsa_tree_commit(dev(accept), batch, caches, dev_status=st)
        s = D.dsa_device_status_read(st)
        assert (s[0], s[1]) == (D.DEVERR_INDEX_RANGE, 2)
        assert got.cpu().tolist() == [3, 0, 67]
        assert np.array_equal(t[0].cpu().numpy(), host[0])


def test_reserve_records_a_held_length_beyond_the_table():
    ref, table = np.zeros(40, np.int32), np.full((3, 6), -1, np.int32)
    dref, dtable = dev(ref), dev(table)
    row, have, want = [0, 1, 2], [6 * 64 + 1, 6 * 64, 2 ** 31 - 1], [64, 64, 6 * 64]
    st = D.new_device_status(DEV)
    D.dsa_pages_reserve(dref, dtable, dev(row), dev(have), dev(want), dev_status=st)
    errors = O.pages_reserve(ref, table, row, have, want)
    s = D.dsa_device_status_read(st)
    assert (s[0], s[1]) == (D.DEVERR_INDEX_RANGE, 2) and errors == 2
    assert np.array_equal(dtable.cpu().numpy(), table) and np.array_equal(dref.cpu().numpy(), ref)


def test_caches_that_overlap_are_refused():
    n = 3
    t = torch.zeros(2 * n * D.KV_PAGE_BYTES + 64, dtype=torch.uint8, device=DEV)
    for at in (16, D.KV_PAGE_BYTES, n * D.KV_PAGE_BYTES - 16):
        with pytest.raises(ValueError):
            D.CacheSet([(t, D.CACHE_KV), (t[at:], D.CACHE_KV)], n)
        with pytest.raises(ValueError):
            D.CacheSet([(t[at:], D.CACHE_IDXK), (t, D.CACHE_KV)], n)
    D.CacheSet([(t[n * D.KV_PAGE_BYTES:], D.CACHE_IDXK), (t, D.CACHE_KV)], n)


def test_reserve_of_nearly_2_to_31_entries_without_a_free_page():
    """The last entries of the largest table are looked at, and nothing past them: 64 rows of 2^25 - 1 pages, all
    of which hold page 0 but three."""
    rows, width = 64, 2 ** 25 - 1
    ref, table = dev([3] * 20), torch.zeros(rows, width, dtype=torch.int32, device=DEV)
    table[0, 5] = table[rows - 1, width - 1] = table[rows - 1, width - 700] = -1
    st = D.new_device_status(DEV)
    D.dsa_pages_reserve(ref, table, dev(range(rows)), dev([0] * rows), dev([width * 64] * rows), dev_status=st)
    s = D.dsa_device_status_read(st)
    assert (s[0], s[1]) == (D.DEVERR_PAGE_POOL, 3)
    assert int(torch.count_nonzero(table)) == 3 and (ref == 3).all()
    ref[7], ref[12] = 0, 0                                           # two of the three can be served
    st = D.new_device_status(DEV)
    D.dsa_pages_reserve(ref, table[rows - 1:], dev([0]), dev([(width - 1000) * 64]), dev([width * 64]), dev_status=st)
    assert D.dsa_device_status_read(st)[0] == 0
    assert table[rows - 1, [width - 700, width - 1]].tolist() == [7, 12] and ref.tolist() == [3] * 7 + [1] + [3] * 4 + [1] + [3] * 7
