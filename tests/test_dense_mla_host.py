"""Host-side checks of the windowed / tree MLA calls and of the token and page
calls: what they refuse, on the CPU, before anything is launched.  Fake device
addresses are never dereferenced on these paths."""

import ctypes
import os

import numpy as np
import pytest
import torch

import dsa_sparse_attention_indexer_gb300 as D
from oracle import dsa_oracle as O

OK, INVALID, ALIGN, UNSUPPORTED, WS = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(D.LIB_PATH):
        from dsa_sparse_attention_indexer_gb300 import build
        build.build()
    return D.lib()


FK, ODD, WSP = ctypes.c_void_p(0x30000000), ctypes.c_void_p(0x30000004), ctypes.c_void_p(0x40000000)
N = None


def _batch(B=2, T=2, max_seq=4096, max_q=1, pages=128, **kw):
    b = D.DsaBatch(B, (max_seq + 63) // 64, max_seq, max_q, T, pages, 0x10000000, 0x10000100, 0x10000200)
    for k, v in kw.items():
        setattr(b, k, v)
    return ctypes.byref(b)


def _window(L, q=FK, kv=FK, b=None, window=64, sinks=4, scale=0.0625, out=FK, dtype=0, ws=WSP, n=1 << 40):
    return L.dsa_window_mla(q, kv, b or _batch(), window, sinks, scale, out, dtype, N, ws, n, N, N)


def _tree(L, q=FK, mask=FK, kv=FK, b=None, scale=0.0625, out=FK, dtype=0, ws=WSP, n=1 << 40):
    return L.dsa_tree_mla(q, mask, kv, b or _batch(), scale, out, dtype, N, ws, n, N, N)


def test_dense_mla_workspace_size(L):
    n = ctypes.c_size_t(0)
    assert L.dsa_dense_mla_workspace_size(_batch(), ctypes.byref(n)) == OK and n.value > 0
    assert L.dsa_dense_mla_workspace_size(_batch(), N) == INVALID
    assert L.dsa_dense_mla_workspace_size(N, ctypes.byref(n)) == INVALID
    assert L.dsa_dense_mla_workspace_size(_batch(max_pages=1), ctypes.byref(n)) == INVALID


@pytest.mark.parametrize("call", [_window, _tree])
def test_dense_mla_argument_errors(L, call):
    assert call(L, q=N) == INVALID
    assert call(L, kv=N) == INVALID
    assert call(L, out=N) == INVALID
    assert call(L, ws=N) == INVALID
    assert call(L, dtype=2) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(L, scale=scale) == INVALID
    assert call(L, q=ODD) == ALIGN
    assert call(L, kv=ODD) == ALIGN
    assert call(L, out=ODD) == ALIGN
    assert call(L, ws=ODD) == ALIGN
    assert call(L, n=1024) == WS
    assert call(L, b=_batch(max_pages=1)) == INVALID
    assert call(L, b=_batch(num_pages=1 << 26)) == UNSUPPORTED        # slots beyond 32 bits
    assert call(L, q=N, kv=N, out=N, ws=N, n=0, b=_batch(T=0)) == OK  # no rows: nothing to do


def test_window_and_tree_bounds(L):
    assert _window(L, window=0) == INVALID
    assert _window(L, window=-5) == INVALID
    assert _window(L, sinks=-1) == INVALID
    assert _tree(L, mask=N) == INVALID
    assert _tree(L, mask=ODD) == ALIGN
    assert _tree(L, b=_batch(T=100, max_q=65)) == UNSUPPORTED
    assert _tree(L, q=N, mask=N, kv=N, out=N, ws=N, n=0, b=_batch(T=0, max_q=64)) == OK


def _list(*entries):
    return (D.DsaCache * max(1, len(entries)))(*[D.DsaCache(p, k, 0) for p, k in entries])


def test_commit_argument_errors(L):
    one = _list((0x50000000, 0))

    def commit(accept=FK, width=4, b=None, caches=one, n=1):
        return L.dsa_tree_commit(accept, width, b or _batch(), caches, n, FK, N, N)

    assert commit(accept=N) == INVALID
    assert commit(width=-1) == INVALID
    assert commit(width=65) == UNSUPPORTED
    assert commit(n=-1) == INVALID
    assert commit(caches=N, n=1) == INVALID
    assert commit(caches=_list((None, 0))) == INVALID
    assert commit(caches=_list((0x50000000, 3))) == INVALID
    assert commit(caches=_list((0x50000000, -1))) == INVALID
    assert commit(caches=_list((0x50000008, 0))) == ALIGN
    assert commit(b=_batch(num_pages=0)) == INVALID
    assert L.dsa_tree_commit(N, 0, _batch(), N, 0, N, N, N) == OK     # nothing to move, no lengths asked for


def test_commit_refuses_to_write_the_lengths_it_reads(L):
    one = _list((0x50000000, 0))
    for at in (0x10000000, 0x10000004):                               # the batch's seq_len, two requests
        assert L.dsa_tree_commit(FK, 4, _batch(), one, 1, ctypes.c_void_p(at), N, N) == INVALID
    assert L.dsa_tree_commit(FK, 4, _batch(), N, 0, ctypes.c_void_p(0x10000000), N, N) == INVALID


def test_pool_argument_errors(L):
    one = _list((0x50000000, 1))

    def reserve(ref=FK, pages=128, table=FK, rows=8, width=64, row=FK, a=FK, b=FK, n=2):
        return L.dsa_pages_reserve(ref, pages, table, rows, width, row, a, b, n, N, N)

    def release(ref=FK, pages=128, table=FK, rows=8, width=64, row=FK, a=FK, b=FK, n=2):
        return L.dsa_pages_release(ref, pages, table, rows, width, row, a, b, n, N, N)

    def fork(ref=FK, pages=128, table=FK, rows=8, width=64, row=FK, a=FK, b=FK, n=2):
        return L.dsa_pages_fork(ref, pages, table, rows, width, row, a, b, n, one, 1, N, N)

    for call in (reserve, release, fork):
        for kw in (dict(ref=N), dict(table=N), dict(row=N), dict(a=N), dict(b=N), dict(n=-1), dict(pages=0), dict(rows=0),
                   dict(width=0)):
            assert call(**kw) == INVALID, (call.__name__, kw)
        assert call(ref=ODD) == ALIGN
        assert call(pages=1 << 25) == UNSUPPORTED
        assert call(ref=N, table=N, row=N, a=N, b=N, n=0) == OK
        assert call(rows=1 << 20, width=1 << 11) == UNSUPPORTED       # 2^31 table entries
    assert reserve(n=4097) == UNSUPPORTED
    assert fork(n=4097) == UNSUPPORTED
    assert L.dsa_pages_fork(FK, 128, FK, 8, 64, FK, FK, FK, 2, _list((0x50000004, 1)), 1, N, N) == ALIGN
    assert L.dsa_pages_fork(FK, 128, FK, 8, 64, FK, FK, FK, 2, N, 1, N, N) == INVALID


def test_binding_refuses_what_the_library_cannot_check():
    host = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        D.dsa_pages_reserve(host[0], host, host[0], host[0], host[0])     # host tensors
    with pytest.raises(ValueError):
        D.CacheSet([(torch.zeros(64, dtype=torch.uint8), 9)], 1)          # unknown kind
    with pytest.raises(ValueError):
        D.CacheSet([(torch.zeros(41984, dtype=torch.uint8), D.CACHE_KV)], 1)
    with pytest.raises(TypeError):
        D.dsa_tree_commit(host.float(), None, None)


def test_oracle_positions_and_pool():
    assert O.window_positions(5, 2, 1).tolist() == [0, 4, 5]
    assert O.window_positions(5, 100, 0).tolist() == list(range(6))
    assert O.window_positions(0, 1, 9).tolist() == [0]
    assert O.window_positions(-1, 4, 4).tolist() == []
    assert O.tree_positions(3, 0b1010, 3).tolist() == [0, 1, 2, 4]
    rows, kept = O.tree_commit(np.arange(8), 3, 5, [0, 2, 4, -1])
    assert rows.tolist() == [0, 1, 2, 3, 5, 7, 6, 7] and kept == 3
    ref, table = np.array([1, 0, 0, 1, 0]), np.full((3, 3), -1)
    table[0, 0], table[1, 0] = 0, 3
    assert O.pages_reserve(ref, table, [1, 0], [64, 1], [129, 70]) == 0
    assert table.tolist() == [[0, 4, -1], [3, 1, 2], [-1, -1, -1]] and ref.tolist() == [1, 1, 1, 1, 1]
    assert O.pages_release(ref, table, [1, 1], [1, 0], [9, 2]) == 0
    assert table[1].tolist() == [-1] * 3 and ref.tolist() == [1, 0, 0, 0, 1]
    errors, copies = O.pages_fork(ref, table, [0, 0], [1, 1], [70, 70])
    assert errors == 1 and copies == [(4, 1, 6)] and table[1].tolist() == [0, 1, -1] and ref.tolist() == [2, 1, 0, 0, 1]


def test_oracle_reserve_uses_the_pages_that_held_entries_pass_over():
    ref, table = np.array([1, 0, 1, 0, 0]), np.array([[0, 2, -1, -1, -1]])
    assert O.pages_reserve(ref, table, [0], [0], [5 * 64]) == 0
    assert table.tolist() == [[0, 2, 4, 1, 3]] and ref.tolist() == [1] * 5
    ref, table = np.array([1, 0, 1, 0, 1]), np.array([[0, 2, -1, -1, -1]])
    assert O.pages_reserve(ref, table, [0], [0], [5 * 64]) == 1
    assert table.tolist() == [[0, 2, 1, 3, -1]] and ref.tolist() == [1] * 5
