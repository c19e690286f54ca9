"""The calls on grouped heads at the ends of what they take.  Bounds are those of tests/grouped.py; where a test needs
another it is derived beside it."""

import numpy as np
import pytest
import torch

import dsa_sparse_attention_indexer_gb300 as D
from tests.grouped import DEV, cache_case, check, expected, f64

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
