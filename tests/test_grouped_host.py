"""Host-side checks of the calls on grouped heads: what they refuse, on the CPU, before anything is launched.
Fake device addresses are never dereferenced on these paths."""

import ctypes
import os

import numpy as np
import pytest
import torch

import dsa_sparse_attention_indexer_gb300 as D
from oracle import dsa_oracle as O

OK, INVALID, ALIGN, UNSUPPORTED, WS = 0, 1, 2, 3, 4
N = None
FK, ODD, WSP = ctypes.c_void_p(0x30000000), ctypes.c_void_p(0x30000004), ctypes.c_void_p(0x40000000)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(D.LIB_PATH):
        from dsa_sparse_attention_indexer_gb300 import build
        build.build()
    return D.lib()


def _batch(B=2, T=2, max_seq=4096, max_q=1, pages=128, **kw):
    b = D.DsaBatch(B, (max_seq + 63) // 64, max_seq, max_q, T, pages, 0x10000000, 0x10000100, 0x10000200)
    for k, v in kw.items():
        setattr(b, k, v)
    return ctypes.byref(b)


def _h(data=0x30000000, tok=1024, head=128):
    return ctypes.byref(D.DsaHeads(data, tok, head))


def _append(L, k=_h(), v=_h(), q=_h(), b=None, heads=16, kv=4, dim=128, rope=128, style=1, base=10000.0, freq=N, cache=FK, q_out=FK,
            k_out=N):
    return L.dsa_kv8_append(k, v, q, b or _batch(), heads, kv, dim, rope, style, base, freq, cache, q_out, k_out, N, N)


def _shapes(L, call):
    for heads, kv in ((0, 1), (1, 0), (-4, 1), (4, -1)):
        assert call(L, heads=heads, kv=kv) == INVALID
    for heads, kv in ((5, 2), (129, 1), (258, 2), (65536, 65536)):
        assert call(L, heads=heads, kv=kv) == UNSUPPORTED
    for dim in (0, -64, 32, 96, 192, 512):
        assert call(L, dim=dim) == UNSUPPORTED


def test_append_refusals(L):
    _shapes(L, _append)
    for name in ("k", "v", "cache"):
        assert _append(L, **{name: N}) == INVALID
    assert _append(L, q=N) == INVALID and _append(L, q_out=N) == INVALID            # both or neither
    for name in ("k", "v", "q"):
        assert _append(L, **{name: _h(data=None)}) == INVALID
        assert _append(L, **{name: _h(data=0x30000002)}) == ALIGN
        assert _append(L, **{name: _h(tok=-8)}) == INVALID and _append(L, **{name: _h(head=-8)}) == INVALID
        assert _append(L, **{name: _h(tok=1028)}) == ALIGN and _append(L, **{name: _h(head=4)}) == ALIGN
    for name in ("cache", "q_out", "k_out"):
        assert _append(L, **{name: ODD}) == ALIGN
    assert _append(L, style=2) == INVALID and _append(L, style=-1) == INVALID
    assert _append(L, rope=-16) == INVALID and _append(L, rope=144) == INVALID and _append(L, rope=8) == UNSUPPORTED
    for base in (0.0, -1.0, float("nan"), float("inf")):
        assert _append(L, base=base) == INVALID
    assert _append(L, b=_batch(max_pages=1)) == INVALID
    assert _append(L, b=_batch(T=0), k=N, v=N, q=N, cache=N, q_out=N) == OK          # nothing to do


def _attention(L, q=_h(), cache=FK, b=None, heads=16, kv=4, dim=128, scale=0.0625, out=FK, dtype=0, ws=WSP, n=1 << 40):
    return L.dsa_kv8_attention(q, cache, b or _batch(), heads, kv, dim, scale, out, dtype, N, ws, n, N, N)


def _attention_errors(L, call):
    _shapes(L, call)
    for name in ("q", "out", "ws"):
        assert call(L, **{name: N}) == INVALID
    assert call(L, q=_h(data=None)) == INVALID and call(L, q=_h(data=0x30000008)) == ALIGN
    assert call(L, q=_h(tok=-8)) == INVALID and call(L, q=_h(head=-8)) == INVALID
    assert call(L, q=_h(tok=1020)) == ALIGN and call(L, q=_h(head=12)) == ALIGN
    for name in ("out", "ws"):
        assert call(L, **{name: ODD}) == ALIGN
    assert call(L, dtype=2) == INVALID and call(L, dtype=-1) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(L, scale=scale) == INVALID
    assert call(L, n=1024) == WS


def test_kv8_attention_refusals(L):
    _attention_errors(L, _attention)
    assert _attention(L, cache=N) == INVALID and _attention(L, cache=ODD) == ALIGN
    assert _attention(L, b=_batch(max_pages=1)) == INVALID
    assert _attention(L, b=_batch(T=0), q=N, cache=N, out=N, ws=N) == OK
    assert _attention(L, b=_batch(T=1 << 28, max_q=1 << 27), heads=128, kv=1) == UNSUPPORTED
    # refused before either of its kernels runs
    assert _attention(L, b=_batch(B=2, T=1 << 27, max_q=1 << 26, max_seq=0x7fffff00, max_pages=1 << 25)) == UNSUPPORTED
    n = ctypes.c_size_t(0)
    assert L.dsa_kv8_attention_workspace_size(_batch(), 16, 4, 128, ctypes.byref(n)) == OK and n.value > 0
    assert L.dsa_kv8_attention_workspace_size(_batch(), 16, 4, 128, N) == INVALID
    assert L.dsa_kv8_attention_workspace_size(N, 16, 4, 128, ctypes.byref(n)) == INVALID
    assert L.dsa_kv8_attention_workspace_size(_batch(), 16, 5, 128, ctypes.byref(n)) == UNSUPPORTED


def _prompt_batch(B=2, max_q=64, max_k=64, T=100, K=100, qs=0x10000000, ks=0x10000100, reserved=0):
    return ctypes.byref(D.DsaPrompt(B, max_q, max_k, reserved, T, K, qs, ks))


def _prompt(L, q=_h(), k=_h(), v=_h(), b=None, heads=16, kv=4, dim=128, scale=0.0625, out=FK, dtype=0, ws=WSP, n=1 << 40):
    return L.dsa_prompt_attention(q, k, v, b or _prompt_batch(), heads, kv, dim, scale, out, dtype, N, ws, n, N, N)


def test_prompt_attention_refusals(L):
    _attention_errors(L, lambda L, n=1 << 40, **kw: _prompt(L, n=min(n, 255) if n < 1 << 40 else n, **kw))
    for name in ("k", "v"):
        assert _prompt(L, **{name: N}) == INVALID
        assert _prompt(L, **{name: _h(data=0x30000002)}) == ALIGN and _prompt(L, **{name: _h(tok=-8)}) == INVALID
    for name in ("q", "k", "v"):
        assert _prompt(L, **{name: _h(tok=0)}) == UNSUPPORTED and _prompt(L, **{name: _h(head=0)}) == UNSUPPORTED
        assert _prompt(L, **{name: _h(tok=1 << 38)}) == UNSUPPORTED
    for kw in (dict(B=0), dict(max_q=-1), dict(max_k=-1), dict(T=-1), dict(K=-1), dict(qs=None), dict(ks=None), dict(reserved=1), dict(T=129), dict(K=129)):
        assert _prompt(L, b=_prompt_batch(**kw)) == INVALID
    assert _prompt(L, b=_prompt_batch(B=65536)) == UNSUPPORTED
    assert _prompt(L, b=_prompt_batch(max_q=1 << 30, T=(1 << 31) - 1)) == UNSUPPORTED
    assert _prompt(L, b=_prompt_batch(T=0), q=N, k=N, v=N, out=N, ws=N) == OK
    n = ctypes.c_size_t(0)
    assert L.dsa_prompt_attention_workspace_size(_prompt_batch(), 16, 4, 128, ctypes.byref(n)) == OK and n.value > 0
    assert L.dsa_prompt_attention_workspace_size(_prompt_batch(), 16, 4, 128, N) == INVALID
    assert L.dsa_prompt_attention_workspace_size(N, 16, 4, 128, ctypes.byref(n)) == INVALID
    assert L.dsa_prompt_attention_workspace_size(_prompt_batch(), 16, 4, 192, ctypes.byref(n)) == UNSUPPORTED


def test_kv8_page_bytes_and_views():
    kv, dim = 3, 64
    page = D.kv8_page_bytes(kv, dim)
    assert page == kv * (128 * dim + 32) and page % 16 == 0
    cache = torch.arange(2 * page, dtype=torch.int64).to(torch.uint8)
    k, v, s = D.kv8_views(cache, kv, dim)
    assert k.shape == (2, kv, 4, 16, dim) and v.shape == (2, kv, 4, dim, 16) and s.shape == (2, kv, 2, 4)
    flat = cache.numpy()
    at = page + 2 * (128 * dim + 32)                        # page 1, head 2
    assert k.view(torch.uint8)[1, 2, 3, 5, 7] == flat[at + (3 * 16 + 5) * dim + 7]
    assert v.view(torch.uint8)[1, 2, 3, 5, 7] == flat[at + 64 * dim + 3 * 16 * dim + 5 * 16 + 7]
    assert s.view(torch.uint8)[1, 2, 1].flatten()[9] == flat[at + 128 * dim + 16 + 9]


def test_oracle_rotation_and_blocks():
    """The oracle against complex rotation, and a block that grows token by token against one that is appended at once."""
    rng = np.random.default_rng(3)
    x, pos = rng.standard_normal((5, 2, 64)), np.array([0, 1, 77, 1000003, 12])
    for halves in (True, False):
        y = O.rope_pairs(x, pos, 32, halves, base=500.0)
        f = 500.0 ** (-np.arange(16) / 16)
        turn = np.exp(1j * pos[:, None, None] * f)
        z = (x[..., :16] + 1j * x[..., 16:32] if halves else x[..., 0:32:2] + 1j * x[..., 1:32:2]) * turn
        got = y[..., :16] + 1j * y[..., 16:32] if halves else y[..., 0:32:2] + 1j * y[..., 1:32:2]
        assert np.allclose(got, z, atol=1e-9) and np.array_equal(y[..., 32:], x[..., 32:])
    new = rng.standard_normal((16, 64)) * 2.0 ** np.arange(16)[:, None]
    codes, e = np.zeros((16, 64), np.uint8), 0
    for t in range(16):
        codes, e = O.kv8_block_append(codes, e, t, new[t:t + 1])
        top = np.abs(new[:t + 1]).max()
        assert top <= 448 * 2.0 ** e and top > 224 * 2.0 ** e
        off = np.abs(O.e4m3_decode(codes[:t + 1]) * 2.0 ** e - new[:t + 1])
        # half a step of a normal code, 2^-4 of it, and less than a whole subnormal step however often it grew
        assert np.all(off <= 2.0 ** -4 * np.abs(new[:t + 1]) + 2.0 ** (e - 9))
    once, e1 = O.kv8_block_append(np.zeros((16, 64), np.uint8), 0, 0, new)
    assert e1 == e and np.array_equal(once[15], codes[15])
    assert O.kv8_block_append(np.zeros((16, 4), np.uint8), 5, 0, np.zeros((3, 4)))[1] == -24


def test_oracle_grouped_attention():
    """The oracle against torch's definition of softmax over a dense mask."""
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((6, 6, 16), (9, 2, 16), (9, 2, 16)))
    out, lse, size = O.grouped_attention(q.numpy(), k.numpy(), v.numpy(), -2, 0.3)
    kk, vv = k.repeat_interleave(3, 1), v.repeat_interleave(3, 1)
    s = 0.3 * torch.einsum("nhd,lhd->nhl", q, kk)
    s = s.masked_fill(torch.arange(9) > torch.arange(6)[:, None, None] - 2, -float("inf"))
    assert np.all(out[:2] == 0) and np.all(lse[:2] == -np.inf)
    want = torch.einsum("nhl,lhd->nhd", torch.softmax(s[2:], -1), vv)
    assert np.allclose(size[2:], torch.einsum("nhl,lhd->nhd", torch.softmax(s[2:], -1), vv.abs()).numpy())
    assert np.allclose(out[2:], want.numpy()) and np.allclose(lse[2:], torch.logsumexp(s[2:], -1).numpy())
