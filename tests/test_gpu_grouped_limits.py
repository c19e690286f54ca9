"""The calls on grouped heads at the ends of what they take.  Bounds are those of tests/grouped.py; where a test needs
another it is derived beside it."""

from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import dsa_sparse_attention_indexer_gb300 as D
from oracle import dsa_oracle as O
from tests.grouped import DEV, bounds, cache_case, check, expected, f64, place

pytestmark = pytest.mark.gpu


def _attention(c, dtype=D.DTYPE_F32, scale=None):
    T = c["T"] + c["pad"]
    out = torch.full((T, c["heads"], c["dim"]), 7.0, dtype=torch.float32 if dtype == D.DTYPE_F32 else torch.bfloat16, device=DEV)
    lse = torch.full((T, c["heads"]), 7.0, device=DEV)
    st = D.new_device_status(DEV)
    D.dsa_kv8_attention(c["q"], c["dev_cache"], c["batch"], kv_heads=c["kv"], softmax_scale=scale, out=out, out_dtype=dtype, lse=lse, dev_status=st)
    torch.cuda.synchronize()
    return out, lse, D.dsa_device_status_read(st)[0]


@pytest.mark.parametrize("n", [1, 3, 100])
@pytest.mark.parametrize("size", [118, 125, -105, -120])
def test_queries_of_any_finite_size(n, size):
    """q of 2^118 and more and of 2^-120, with a scale that makes ordinary scores of them: the same bounds as ever."""
    c = cache_case([300], [n], 1, 4, 64, seed=50 + n)
    q = c["q"].float().clamp(-7.5, 7.5)
    c["q"] = (q * 2.0 ** (size // 2) * 2.0 ** (size - size // 2)).to(torch.bfloat16)
    assert torch.isfinite(c["q"]).all()
    scale = 2.0 ** (-3 - size)
    out, lse, bits = _attention(c, scale=scale)
    check(out, lse, expected(c, scale))
    assert bits == 0


@pytest.mark.parametrize("n", [2, 100])
def test_scores_that_vanish(n):
    """Units of a score below fp32's smallest number: every position counts the same."""
    c = cache_case([300], [n], 1, 4, 64, seed=60)
    c["q"] = (c["q"].float() * 2.0 ** -60).to(torch.bfloat16)
    out, lse, bits = _attention(c, scale=1e-30)
    check(out, lse, expected(c, 1e-30))
    assert bits == 0


def test_scores_beyond_all_range():
    """Units of a score above fp32's largest number: a row's best position has all of the weight, or, of many rows, it is recorded."""
    for n in (2, 100):
        c = cache_case([300], [n], 1, 4, 64, seed=61)
        c["q"] = (c["q"].float() * 2.0 ** 100).to(torch.bfloat16)
        out, lse, bits = _attention(c, scale=1e30)
        if n == 100:
            assert bits == D.DEVERR_FP16_RANGE
            continue
        assert bits == 0
        want = expected(c, 1e30)
        err = np.abs(f64(out) - want[0])
        assert np.all(err <= 2.0 ** -11 * np.abs(want[0]) + 2.0 ** -22 * np.abs(want[0]))


def _long_context(L, n, group, dim, seed):
    """A context of L tokens: its last two pages are their own, all others are one page whose scores lie so far below (by 250
    of a logarithm and more) that their probabilities, 2^31 of them together, are below 2^-300 of the others'.  Places of the
    last page behind the context hold keys that outdo all others."""
    width = (L + 63) // 64
    c = cache_case([192], [n], 1, group, dim, seed=seed)
    c["q"][..., 0] = 8.0
    k, v, s = D.kv8_views(c["cache"], 1, dim)
    first, own = int(c["table"][0, 0]), [int(x) for x in c["table"][0, 1:3]]
    k[first] = 0
    k[first, ..., 0] = -256.0
    s[first, :, 0] = dim ** 0.5 / 8                        # a score of -256 / sqrt(dim) * sqrt(dim)
    for pg in own:
        k[pg, ..., 0] = 0
    left = L - (width - 1) * 64
    for t in range(left, 64):
        k[own[1], 0, t // 16, t % 16] = 0
        k[own[1], 0, t // 16, t % 16, 0] = 448.0
        v[own[1], 0, t // 16, :, t % 16] = 448.0
    c["dev_cache"] = c["cache"].to(DEV)
    table = torch.full((1, width), first, dtype=torch.int32, device=DEV)
    table[0, -2:] = torch.tensor(own, dtype=torch.int32, device=DEV)
    c["batch"] = D.Batch(torch.tensor([L], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV), table, c["pages"],
                         max_seq_len=L, max_q_len=n, total_q=n)
    behind = 64 + left                                     # tokens of the two pages
    kk, vv, ok = O.kv8_read(c["cache"].numpy().reshape(-1), 1, dim, np.array(own), behind, c["pages"])
    return c, bounds(f64(c["q"]), kk, vv, behind - n, dim ** -0.5, 2.0 ** -11, ok)


@pytest.mark.parametrize("L", [2 ** 31 - 1, 2 ** 31 - 127])
def test_many_rows_of_the_longest_contexts(L):
    c, want = _long_context(L, 9, 8, 64, 1)
    out, lse, bits = _attention(c)
    check(out, lse, want)
    assert bits == 0


@pytest.mark.parametrize("L,n", [(2 ** 31 - 1, 1), (2 ** 31 - 10, 1), (2 ** 31 - 3, 6)])
def test_few_rows_of_the_longest_contexts(L, n):
    c, want = _long_context(L, n, 8, 64, 2)
    out, lse, bits = _attention(c)
    check(out, lse, want)
    assert bits == 0


def test_a_page_id_of_the_lowest_number_is_recorded():
    for n in (1, 100):
        c = cache_case([300], [n], 1, 4, 64, seed=62)
        c["table"][0, 1] = -2 ** 31
        place(c)
        out, lse, bits = _attention(c)
        check(out, lse, expected(c))
        assert bits == D.DEVERR_PAGE_RANGE


def _prompt(n, kv, group, dim, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(n, kv * group, dim, generator=g).to(torch.bfloat16)
    k, v = (torch.randn(n, kv, dim, generator=g).to(torch.bfloat16) for _ in range(2))
    q[..., 0] = 16.0
    batch = D.PromptBatch(torch.tensor([0, n], dtype=torch.int32, device=DEV))

    def call(k, v):
        out, lse = torch.empty(n, kv * group, dim, device=DEV), torch.empty(n, kv * group, device=DEV)
        D.dsa_prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), batch, out=out, out_dtype=D.DTYPE_F32, lse=lse)
        torch.cuda.synchronize()
        return out, lse

    return q, k, v, call


@pytest.mark.parametrize("n,kv,group,dim", [(256, 2, 1, 64), (256, 1, 1, 128), (64, 2, 4, 128), (128, 1, 1, 256), (40, 1, 8, 64)])
def test_infinite_values_behind_probabilities_of_zero(n, kv, group, dim):
    """Keys whose scores are so far below a row's best that their P is 0, with values that are not finite: rows of an item (two
    tiles of 128 rows, one at 256 dims) get them whole where some row of it does not see the key, whichever tile each is in;
    rows of items behind it, all of which see it, get them or a NaN."""
    q, k, v, call = _prompt(n, kv, group, dim, 90 + dim)
    k[5, :, 0], k[n // 2, :, 0] = -150.0, -150.0
    v[5, 0, 3], v[n // 2, 0, dim - 1], v[5, kv - 1, 9], v[n // 2, kv - 1, 11] = float("inf"), -float("inf"), float("nan"), float("inf")
    want = bounds(f64(q), f64(k), f64(v), 0, dim ** -0.5, 2.0 ** -8)
    first, lse = call(k, v)
    got, exact = f64(first), want[0].copy()
    rest = slice(128 // group * (2 if dim <= 128 else 1), n)
    exact[rest][np.isnan(got[rest]) & np.isinf(exact[rest])] = np.nan
    for kind in (np.isnan, np.isposinf, np.isneginf):
        assert np.array_equal(kind(got), kind(exact)) and kind(exact).any()
    f = np.isfinite(exact)
    assert np.all(np.abs(got[f] - exact[f]) <= (want[2] * (1 + 2.0 ** -24) + 2.0 ** -24 * np.abs(exact))[f])
    assert np.all(np.abs(f64(lse) - want[1]) <= want[3])
    for _ in range(10):
        assert torch.equal(call(k, v)[0].view(torch.int32), first.view(torch.int32))


def test_infinite_values_behind_probabilities_of_zero_in_long_prompts():
    """Where rows see all of a step's keys: infinite or NaN, the same in every call, and nothing else changes."""
    n, kv, group, dim = 1000, 2, 2, 64
    q, k, v, call = _prompt(n, kv, group, dim, 95)
    k[100, :, 0] = -150.0
    plain, _ = call(k, v)
    v[100, :, 7] = float("inf")
    first, _ = call(k, v)
    assert torch.equal(first[:100], plain[:100]) and not torch.isfinite(first[100:, :, 7]).any() and not torch.isneginf(first[100:, :, 7]).any()
    first[100:, :, 7] = plain[100:, :, 7]
    assert torch.equal(first, plain)
    v[100, :, 7] = float("inf")
    again = [call(k, v)[0].view(torch.int32) for _ in range(10)]
    assert all(torch.equal(x, again[0]) for x in again)


@pytest.mark.parametrize("n,past,heads,dim", [
    ([96, 1, 7], [5, 1205, 984], 64, 256),                  # one tile of rows: a step's values come behind the next one's keys
    ([1] * 30, [0, 253, 0, 161, 282, 316, 140, 186, 859, 357] * 3, 64, 256),
    ([200, 100, 130, 40, 300], [1000, 0, 700, 30, 5], 32, 256),
    ([300, 60, 129, 257, 40] * 6, [700, 0, 5, 300, 0] * 6, 8, 128),            # second tiles without rows between others
    ([300, 130, 129, 257, 140] * 6, [900, -130, 500, -120, -10] * 6, 16, 64),  # and first tiles that see nothing
])
def test_what_lies_behind_a_sequence_reaches_none_of_its_rows(n, past, heads, dim):
    """Every other sequence, and the rows behind the last one, of NaN keys and infinite or NaN values: the rows of the sequences
    between them get the same bits as with finite ones there, call after call."""
    g = torch.Generator().manual_seed(97)
    L = [max(0, a + b) for a, b in zip(n, past)]
    T, K = sum(n), sum(L)
    q, k, v = (torch.randn(rows, heads, dim, generator=g).to(torch.bfloat16).to(DEV) for rows in (T, K + 5, K + 5))
    starts, ends = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (n, L))
    batch = D.PromptBatch(torch.tensor(starts, device=DEV), torch.tensor(ends, device=DEV), max_q_len=max(n), max_k_len=max(L) + 5, total_q=T,
                          total_k=K + 5)
    row, key = (torch.repeat_interleave(torch.arange(len(n)), torch.tensor(x)).to(DEV) for x in (n, L))
    behind = torch.full((5,), len(n), device=DEV)
    key = torch.cat([key, behind])
    plain = D.dsa_prompt_attention(q, k, v, batch, out_dtype=D.DTYPE_F32)
    assert torch.isfinite(plain).all()
    for odd in (0, 1):
        bad = (key % 2 == odd) | (key == len(n))
        for fill in (float("inf"), float("nan")):
            kk, vv = k.masked_fill(bad[:, None, None], float("nan")), v.masked_fill(bad[:, None, None], fill)
            for _ in range(25):
                out = D.dsa_prompt_attention(q, kk, vv, batch, out_dtype=D.DTYPE_F32)
                assert torch.equal(out[row % 2 != odd], plain[row % 2 != odd])


PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def _turned(x, positions, freqs, halves):
    """x [rows, heads, dim] with the pairs of its first 2 len(freqs) dims turned by position * freq, angles from 70 digits."""
    getcontext().prec = 70
    ang = np.array([[float(Decimal(int(p)) * f / (2 * PI) % 1 * 2 * PI) for f in freqs] for p in positions])[:, None]
    n = len(freqs)
    i = np.arange(n)
    a, b = (i, i + n) if halves else (2 * i, 2 * i + 1)
    y, size = x.copy(), np.abs(x)
    y[..., a], y[..., b] = x[..., a] * np.cos(ang) - x[..., b] * np.sin(ang), x[..., a] * np.sin(ang) + x[..., b] * np.cos(ang)
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size


@pytest.mark.parametrize("given,halves", [(True, True), (True, False), (False, True)])
def test_angles_at_the_farthest_positions(given, halves):
    """Positions up to 2^31 - 2, frequencies far above 1 (given, or of a base below 1).  The bound is that of the tests of the
    append: 2^-21 of a pair's size and half a step of bf16; an angle's turn is known to 2^-32."""
    kv, dim, rope, n, L = 1, 64, 32, 5, 2 ** 31 - 1
    g = torch.Generator().manual_seed(80)
    q, k, v = (torch.randn(n, h, dim, generator=g).to(torch.bfloat16).to(DEV) for h in (2, kv, kv))
    table = torch.zeros(1, 2 ** 25, dtype=torch.int32, device=DEV)
    batch = D.Batch(torch.tensor([L], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV), table, 1,
                    max_seq_len=L, max_q_len=n, total_q=n)
    cache = torch.zeros(D.kv8_page_bytes(kv, dim), dtype=torch.uint8, device=DEV)
    if given:
        f = torch.tensor([1000.0, 1e6, 37654321.0, 4e9, 1.5, -2.5e5, 1e-3, 0.0] * 2, dtype=torch.float32)
        freqs, kw = [Decimal(float(x)) for x in f], dict(inv_freq=f.to(DEV))
    else:
        base = float(np.float32(2.0 ** -31 * 1.37))
        freqs, kw = [Decimal(base) ** (Decimal(-2 * i) / rope) for i in range(rope // 2)], dict(rope_base=base)
    k_out = torch.empty_like(k)
    q_out = D.dsa_kv8_append(k, v, cache, batch, q=q, rope_dims=rope, rope_style=D.ROPE_HALVES if halves else D.ROPE_INTERLEAVED, k_out=k_out, **kw)
    for got, x in ((q_out, q), (k_out, k)):
        want, size = _turned(f64(x), range(L - n, L), freqs, halves)
        off = 2.0 ** -21 * size
        off[..., rope:] = 0
        assert np.all(np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + off * (1 + 2.0 ** -8))


def _bounds_by_scale(c, scale=None):
    """Outputs and bounds per dim for blocks whose scales 2^e are far apart.  A probability is rounded to fp16 times its block's
    2^e, against a reference among the row's largest of these products, which stands at 2^6.5 or more (2^7, or a whole number
    next to it); fp16 rounds a number by 2^-11 of itself, or, below its normal range, by 2^-25: with M the largest p_j 2^e_j,
    p_j 2^e_j is off by max(2^-11 of itself, 2^-31.5 M), and an output by the sum of that times its dim's codes."""
    scale = c["dim"] ** -0.5 if scale is None else scale
    L, n, G = c["seq"][0], c["n"][0], c["group"]
    k, v, ok = O.kv8_read(c["cache"].numpy().reshape(-1), c["kv"], c["dim"], c["table"][0].numpy(), L, c["pages"])
    q = f64(c["q"])
    out, lse, W = O.grouped_attention(q, k, v, L - n, scale, ok)
    s = D.kv8_views(c["cache"], c["kv"], c["dim"])[2].double().numpy()
    e = np.stack([s[c["table"][0, j // 64], :, 1, j % 64 // 16] for j in range(L)])          # [L, kv]
    tol, lse_tol = np.zeros_like(out), np.zeros_like(lse)
    for h in range(c["heads"]):
        g = h // G
        a = scale * q[:, h] @ k[:, g].T
        a[np.arange(L)[None] > (L - n + np.arange(n))[:, None]] = -np.inf
        pe = np.exp(a - lse[:, h:h + 1]) * e[:, g]
        rounding = np.where(pe > 0, np.maximum(2.0 ** -11 * pe, 2.0 ** -31.5 * pe.max(1, keepdims=True)), 0.0)
        off = (2 * c["dim"] * 2.0 ** -24 + 2.0 ** -21) * scale * (np.abs(q[:, h]) @ np.abs(k[:, g]).T).max(1)
        tol[:, h] = rounding @ np.abs(v[:, g] / e[:, g, None]) + W[:, h] * (2 * off + (L + 64) * 2.0 ** -23)[:, None]
        lse_tol[:, h] = 2 * off + (L + 64) * 2.0 ** -23 + 2.0 ** -21 * (1 + np.abs(lse[:, h]))
    return out, lse, tol, lse_tol


@pytest.mark.parametrize("n", [3, 100])
@pytest.mark.parametrize("low", [-6, -12, -20, -24])
def test_dims_that_only_blocks_of_small_scales_hold(n, low):
    """Half of the dims are zero in every block of a large scale: what they get comes from the blocks of small ones."""
    c = cache_case([500], [n], 2, 4, 128, seed=70)
    k, v, s = D.kv8_views(c["cache"], 2, 128)
    v[:, :, ::2, ::2] = 0
    s[:, :, 1, ::2], s[:, :, 1, 1::2] = 1.0, 2.0 ** low
    place(c)
    out, lse, bits = _attention(c)
    want = _bounds_by_scale(c)
    assert np.abs(want[0][..., ::2]).min() > 0
    check(out, lse, want)
    assert bits == 0


@pytest.mark.parametrize("n", [1, 100])
def test_a_scale_that_a_token_taken_back_has_left(n):
    """A block whose scale is 2^14 times what its values need, its codes far below the largest."""
    c = cache_case([400], [n], 1, 4, 64, seed=71)
    k, v, s = D.kv8_views(c["cache"], 1, 64)
    pg = int(c["table"][0, 2])
    x = v[pg, 0, 1].float()
    v[pg, 0, 1] = (x * 2.0 ** -14).to(torch.float8_e4m3fn)
    s[pg, 0, 1, 1] *= 2.0 ** 14
    place(c)
    out, lse, bits = _attention(c)
    check(out, lse, _bounds_by_scale(c))
    assert bits == 0
