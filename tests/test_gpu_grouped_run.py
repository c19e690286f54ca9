"""The grouped-head calls together, as a layer of ordinary heads uses them on the pool of pages: prompts on their fresh keys
while the cache takes them, a second chunk over the cache, decoding from one captured graph, a verify step that is partly
taken back, and a request that begins with another one's full pages.

Every attention is held against the 64-bit oracle on what it was given: the rotated rows and the cache's codes, at the bounds
of tests/grouped.py.  The cache is held against the exact keys and values: a code is off by half a step, 2^-4 of itself or, where
it is subnormal, 2^-10 of its scale; growing scales round subnormal codes again, by 2^-10 of each scale on the way, together at
most 2 * 2^-10 of the last one; the rotation in fp32 by (products and sine, a few 2^-24) less than 2^-21 of the pair's size.
"""

import numpy as np
import pytest
import torch

import dsa_sparse_attention_indexer_gb300 as D
from oracle import dsa_oracle as O
from tests.grouped import DEV, bounds, check, f64

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32), device=DEV)


class Layer:
    """One layer's cache, page table and pool, and on the host the exact keys and values that each request has taken."""

    def __init__(self, rows, kv, group, dim, width=8, pages=40, seed=0):
        self.kv, self.group, self.dim, self.width, self.pages = kv, group, dim, width, pages
        self.g = torch.Generator().manual_seed(seed)
        self.cache = torch.full((pages * D.kv8_page_bytes(kv, dim),), 0x7f, dtype=torch.uint8, device=DEV)   # NaN wherever nothing was written
        self.ref = torch.zeros(pages, dtype=torch.int32, device=DEV)
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
        self.st = D.new_device_status(DEV)
        self.k, self.v = [np.zeros((0, kv, dim)) for _ in range(rows)], [np.zeros((0, kv, dim)) for _ in range(rows)]
        self.caches = D.CacheSet([], pages)

    def reserve(self, rows, have, want):
        D.dsa_pages_reserve(self.ref, self.table, dev(rows), dev(have), dev(want), dev_status=self.st)

    def fresh(self, n):
        """One projection's output, of which q, k and v are parts."""
        heads = self.kv * (self.group + 2)
        x = torch.randn(n, heads, self.dim, generator=self.g).to(torch.bfloat16).to(DEV)
        return x, *x.split([self.kv * self.group, self.kv, self.kv], 1)

    def batch(self, rows, n, seq):
        start = np.concatenate([[0], np.cumsum(n)])
        return D.Batch(dev(seq), dev(start), self.table[rows].contiguous(), self.pages, max_seq_len=self.width * 64,
                       max_q_len=max(n), total_q=int(start[-1]))

    def took(self, rows, n, k, v):
        at = 0
        for r, m in zip(rows, n):
            pos = len(self.k[r]) + np.arange(m)
            self.k[r] = np.concatenate([self.k[r], O.rope_pairs(f64(k[at:at + m]), pos, self.dim, True)])
            self.v[r] = np.concatenate([self.v[r], f64(v[at:at + m])])
            at += m

    def read(self, r, length):
        k, v, ok = O.kv8_read(self.cache.cpu().numpy(), self.kv, self.dim, self.table[r].cpu().numpy(), length, self.pages)
        assert ok.all()
        return k, v

    def check_cache(self, r):
        L = len(self.k[r])
        k, v = self.read(r, L)
        scales = f64(D.kv8_views(self.cache, self.kv, self.dim)[2])[self.table[r].cpu().numpy()[:-(-L // 64)]]
        each = np.repeat(scales.transpose(0, 3, 1, 2).reshape(-1, self.kv, 2), 16, 0)[:L]     # [L, kv, keys / values]
        h = self.dim // 2
        pair = np.hypot(self.k[r][..., :h], self.k[r][..., h:])
        pair = np.concatenate([pair, pair], -1)
        assert np.all(np.abs(k - self.k[r]) <= 2.0 ** -4 * np.abs(self.k[r]) + 2.0 ** -9 * each[..., :1] + 2.0 ** -20 * pair)
        assert np.all(np.abs(v - self.v[r]) <= 2.0 ** -4 * np.abs(self.v[r]) + 2.0 ** -9 * each[..., 1:])

    def check_attention(self, rows, n, seq, q, out, lse):
        want = []
        at = 0
        for r, m, L in zip(rows, n, seq):
            k, v = self.read(r, L)
            want.append(bounds(f64(q[at:at + m]), k, v, L - m, self.dim ** -0.5, 2.0 ** -11))
            at += m
        check(out, lse, [np.concatenate(x) for x in zip(*want)], f"{n} of {seq}")


@pytest.mark.parametrize("kv,group,dim", [(2, 4, 128), (1, 7, 64), (2, 3, 256)])
def test_a_serving_loop(kv, group, dim):
    l = Layer(5, kv, group, dim, seed=dim)
    heads, rows = kv * group, [0, 1, 2]
    prompt, chunk = [70, 1, 129], [100, 0, 33]
    # prompts: into the cache, and attention on the rotated rows themselves
    l.reserve(rows, [0] * 3, prompt)
    x, q, k, v = l.fresh(sum(prompt))
    b = l.batch(rows, prompt, prompt)
    kr = torch.empty(sum(prompt), kv, dim, dtype=torch.bfloat16, device=DEV)
    qr = D.dsa_kv8_append(k, v, l.cache, b, q=q, k_out=kr, dev_status=l.st)
    pb = D.PromptBatch(b.q_start, max_q_len=max(prompt), total_q=sum(prompt))
    lse = torch.empty(sum(prompt), heads, device=DEV)
    out = D.dsa_prompt_attention(qr, kr, v, pb, lse=lse, dev_status=l.st)
    l.took(rows, prompt, k, v)
    at, want = 0, []
    for n in prompt:
        want.append(bounds(*(f64(t[at:at + n]) for t in (qr, kr, v)), 0, dim ** -0.5, 2.0 ** -8))
        at += n
    check(out, lse, [np.concatenate(w) for w in zip(*want)], "prompts")
    # a second chunk of two of them, over the cache
    seq = [a + c for a, c in zip(prompt, chunk)]
    l.reserve(rows, prompt, seq)
    x, q, k, v = l.fresh(sum(chunk))
    b = l.batch(rows, chunk, seq)
    qr = D.dsa_kv8_append(k, v, l.cache, b, q=q, dev_status=l.st)
    lse = torch.empty(sum(chunk), heads, device=DEV)
    out = D.dsa_kv8_attention(qr, l.cache, b, kv_heads=kv, lse=lse, dev_status=l.st)
    l.took(rows, chunk, k, v)
    l.check_attention(rows, chunk, seq, qr, out, lse)
    # decoding, pages and all from one graph
    x, q, k, v = l.fresh(3)
    b = l.batch(rows, [1] * 3, seq)
    b_table, have = b.page_table, torch.tensor(seq, dtype=torch.int32, device=DEV)
    row = dev(rows)
    qr, out, lse = torch.empty(3, heads, dim, dtype=torch.bfloat16, device=DEV), torch.empty(3, heads, dim, device=DEV), torch.empty(3, heads, device=DEV)
    ws = D.workspace(D.dsa_kv8_attention_workspace_size(b, heads, kv, dim), DEV)

    def step():
        b.seq_len.copy_(have + 1)
        D.dsa_pages_reserve(l.ref, l.table, row, have, b.seq_len, dev_status=l.st)
        b_table.copy_(l.table[:3])
        D.dsa_kv8_append(k, v, l.cache, b, q=q, q_out=qr, dev_status=l.st)
        D.dsa_kv8_attention(qr, l.cache, b, kv_heads=kv, out=out, out_dtype=D.DTYPE_F32, lse=lse, ws=ws, dev_status=l.st)
        have.copy_(b.seq_len)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(40):                                              # over ends of blocks and of pages
        x.copy_(l.fresh(3)[0])
        graph.replay()
        seq = [s + 1 for s in seq]
        l.took(rows, [1] * 3, k, v)
        if i in (0, 15, 39):
            l.check_attention(rows, [1] * 3, seq, qr, out, lse)
    assert have.cpu().tolist() == seq
    # six tokens verified, two of them kept, the pages of the others given back
    n = [6] * 3
    l.reserve(rows, seq, [s + 6 for s in seq])
    x, q, k, v = l.fresh(18)
    k[2::6] *= 64.0                                                  # a rejected token may have raised a scale
    b = l.batch(rows, n, [s + 6 for s in seq])
    qr = D.dsa_kv8_append(k, v, l.cache, b, q=q, dev_status=l.st)
    lse = torch.empty(18, heads, device=DEV)
    out = D.dsa_kv8_attention(qr, l.cache, b, kv_heads=kv, lse=lse, dev_status=l.st)
    l.check_attention(rows, n, [s + 6 for s in seq], qr, out, lse)
    keep = torch.tensor([0, 1, 6, 7, 12, 13], device=DEV)
    l.took(rows, [2] * 3, k[keep], v[keep])
    seq = [s + 2 for s in seq]
    D.dsa_pages_release(l.ref, l.table, row, dev([-(-s // 64) for s in seq]), dev([l.width] * 3), dev_status=l.st)
    # a request that begins with the third one's first two pages, and one decode step of all four
    D.dsa_pages_fork(l.ref, l.table, dev([2]), dev([3]), dev([128]), l.caches, dev_status=l.st)
    l.k[3], l.v[3] = l.k[2][:128], l.v[2][:128]
    rows, seq = rows + [3], seq + [128]
    l.reserve(rows, seq, [s + 1 for s in seq])
    seq = [s + 1 for s in seq]
    x, q, k, v = l.fresh(4)
    b = l.batch(rows, [1] * 4, seq)
    qr = D.dsa_kv8_append(k, v, l.cache, b, q=q, dev_status=l.st)
    lse = torch.empty(4, heads, device=DEV)
    out = D.dsa_kv8_attention(qr, l.cache, b, kv_heads=kv, lse=lse, dev_status=l.st)
    l.took(rows, [1] * 4, k, v)
    l.check_attention(rows, [1] * 4, seq, qr, out, lse)
    for r in rows:
        l.check_cache(r)
    assert D.dsa_device_status_read(l.st)[0] == 0
    D.dsa_pages_release(l.ref, l.table, dev(rows), dev([0] * 4), dev([l.width] * 4), dev_status=l.st)
    assert int(l.ref.abs().sum()) == 0 and D.dsa_device_status_read(l.st)[0] == 0
