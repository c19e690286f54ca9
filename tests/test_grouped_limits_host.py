"""Host-side checks of the ends of what the attention calls on grouped heads take; no address here is ever dereferenced."""

import ctypes
import os

import pytest

import dsa_sparse_attention_indexer_gb300 as D

INVALID = 1
AT, WS = ctypes.c_void_p(0x30000000), ctypes.c_void_p(0x40000000)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(D.LIB_PATH):
        from dsa_sparse_attention_indexer_gb300 import build
        build.build()
    return D.lib()


@pytest.mark.parametrize("scale", [2.1e38, 2.5e38, 3.0e38, 3.4e38])
def test_softmax_scales_whose_log2_units_fp32_does_not_hold(L, scale):
    h = ctypes.byref(D.DsaHeads(0x30000000, 1024, 128))
    b = D.DsaBatch(2, 64, 4096, 1, 2, 128, 0x10000000, 0x10000100, 0x10000200)
    assert L.dsa_kv8_attention(h, AT, ctypes.byref(b), 16, 4, 128, scale, AT, 0, None, WS, 1 << 40, None, None) == INVALID
    p = D.DsaPrompt(2, 64, 64, 0, 100, 100, 0x10000000, 0x10000100)
    assert L.dsa_prompt_attention(h, h, h, ctypes.byref(p), 16, 4, 128, scale, AT, 0, None, WS, 1 << 40, None, None) == INVALID
