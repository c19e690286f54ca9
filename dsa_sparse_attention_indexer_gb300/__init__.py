"""Python binding of libdsa, the GB300 DSA attention-step library.

Argument marshalling only: every step runs in the library's CUDA kernels.
PyTorch supplies device memory, streams and the output buffers.  If the shared
library has not been built, every call raises ``DsaLibraryMissing`` - there is
no fallback.

The function names follow the C ABI in ``include/dsa.h``.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from ctypes import POINTER, c_char_p, c_float, c_int32, c_int64, c_size_t, c_uint8, c_uint64, c_void_p

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libdsa.so")

PAGE_TOKENS = 64
INDEX_HEADS = 32
INDEX_HEAD_DIM = 128
IDXK_TOKEN_BYTES = 132
IDXK_PAGE_BYTES = 8448
IDXK_MXFP4_TOKEN_BYTES = 68
IDXK_MXFP4_PAGE_BYTES = 4352
MLA_HEADS = 64
LATENT_DIM = 512
ROPE_DIM = 64
QK_DIM = 576
KV_TOKEN_BYTES = 656
KV_PAGE_BYTES = 41984
TOPK = 2048
DTYPE_BF16 = 0
DTYPE_F32 = 1

DEVERR_SLOT_RANGE = 1
DEVERR_PAGE_RANGE = 2
DEVERR_INDEX_RANGE = 4
DEVERR_TIMEOUT = 8
DEVERR_FP16_RANGE = 16
DEVERR_PAGE_POOL = 32
DEVERR_PAGE_COUNT = 64

KV8_BLOCK = 16
KV8_MAX_EXP = 24
ROPE_INTERLEAVED = 0
ROPE_HALVES = 1

CACHE_KV = 0
CACHE_IDXK = 1
CACHE_IDXK_MXFP4 = 2
_CACHE_PAGE_BYTES = {CACHE_KV: KV_PAGE_BYTES, CACHE_IDXK: IDXK_PAGE_BYTES, CACHE_IDXK_MXFP4: IDXK_MXFP4_PAGE_BYTES}

ERR = {0: "DSA_OK", 1: "DSA_ERR_INVALID_ARGUMENT", 2: "DSA_ERR_ALIGNMENT", 3: "DSA_ERR_UNSUPPORTED",
       4: "DSA_ERR_WORKSPACE_TOO_SMALL", 5: "DSA_ERR_NO_TOPK_SOURCE", 6: "DSA_ERR_CUDA", 7: "DSA_ERR_DEVICE",
       8: "DSA_ERR_SCRATCH_LIMIT"}
NOALLOC_SCRATCH_BYTES = 16 << 20


class DsaLibraryMissing(ImportError):
    pass


class DsaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        self.name = ERR.get(code, str(code))
        super().__init__(f"{fn} -> {self.name} ({status_string(code)})")


class DsaScheduleConfig(ctypes.Structure):
    _fields_ = [("indexer_types", POINTER(c_char_p)), ("n_types", c_int32), ("cli_factor", c_int32),
                ("index_topk_pattern", c_char_p), ("index_topk_freq", c_int32), ("index_skip_topk_offset", c_int32)]


class DsaBatch(ctypes.Structure):
    _fields_ = [("batch", c_int32), ("max_pages", c_int32), ("max_seq_len", c_int32),
                ("max_q_len", c_int32), ("total_q", c_int64), ("num_pages", c_int64),
                ("seq_len", c_void_p), ("q_start", c_void_p), ("page_table", c_void_p)]


class DsaCache(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("kind", c_int32), ("reserved", c_int32)]


class DsaHeads(ctypes.Structure):
    _fields_ = [("data", c_void_p), ("token_stride", c_int64), ("head_stride", c_int64)]


class DsaPrompt(ctypes.Structure):
    _fields_ = [("batch", c_int32), ("max_q_len", c_int32), ("max_k_len", c_int32), ("reserved", c_int32),
                ("total_q", c_int64), ("total_k", c_int64), ("q_start", c_void_p), ("k_start", c_void_p)]


_lib = None

_SIGS = {
    "dsa_abi_version": (c_int32, []),
    "dsa_status_string": (c_char_p, [c_int32]),
    "dsa_device_status_reset": (c_int32, [c_void_p, c_void_p]),
    "dsa_device_status_read": (c_int32, [c_void_p, c_void_p, POINTER(c_int32)]),
    "dsa_debug_set_wait_limit_ns": (c_int32, [c_uint64]),
    "dsa_index_k_store": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_float,
                                    c_float, c_void_p, c_int64, c_void_p, c_void_p]),
    "dsa_index_k_store_mxfp4": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p, c_float,
                                          c_float, c_void_p, c_int64, c_void_p, c_void_p]),
    "dsa_indexer_topk_mxfp4": (c_int32, [c_void_p, c_void_p, c_void_p, POINTER(DsaBatch), c_void_p, c_void_p,
                                         c_void_p, c_int32, c_void_p, c_size_t, c_void_p, c_void_p]),
    "dsa_latent_kv_store_fused": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_float,
                                            c_float, c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_float,
                                            c_void_p, c_int64, c_void_p, c_void_p]),
    "dsa_latent_kv_store": (c_int32, [c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p,
                                      c_void_p]),
    "dsa_indexer_topk_workspace_size": (c_int32, [POINTER(DsaBatch), POINTER(c_size_t)]),
    "dsa_indexer_topk": (c_int32, [c_void_p, c_void_p, c_void_p, POINTER(DsaBatch), c_void_p, c_void_p,
                                   c_void_p, c_int32, c_void_p, c_size_t, c_void_p, c_void_p]),
    "dsa_indexer_topk_noalloc": (c_int32, [c_void_p, c_void_p, c_void_p, POINTER(DsaBatch), c_void_p, c_void_p,
                                           c_void_p, c_int32, c_void_p, c_void_p]),
    "dsa_indexer_scores_workspace_size": (c_int32, [POINTER(DsaBatch), POINTER(c_size_t)]),
    "dsa_indexer_scores": (c_int32, [c_void_p, c_void_p, c_void_p, POINTER(DsaBatch), c_void_p, c_int64,
                                     c_void_p, c_size_t, c_void_p, c_void_p]),
    "dsa_indexer_scores_cuda_core": (c_int32, [c_void_p, c_void_p, c_void_p, POINTER(DsaBatch), c_void_p, c_int64,
                                     c_void_p, c_size_t, c_void_p, c_void_p]),
    "dsa_topk_from_scores_workspace_size": (c_int32, [c_int32, c_int64, POINTER(c_size_t)]),
    "dsa_topk_from_scores": (c_int32, [c_void_p, c_int64, c_void_p, c_int32, c_int64, c_void_p, c_void_p,
                                       c_size_t, c_void_p]),
    "dsa_sparse_mla_workspace_size": (c_int32, [POINTER(DsaBatch), POINTER(c_size_t)]),
    "dsa_sparse_mla_decode": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, POINTER(DsaBatch), c_float,
                                        c_void_p, c_int32, c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "dsa_sparse_mla_prefill": (c_int32, [c_void_p, c_void_p, c_void_p, c_void_p, POINTER(DsaBatch), c_float,
                                         c_void_p, c_int32, c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "dsa_parse_indexer_types": (c_int32, [POINTER(c_char_p), c_int32, POINTER(c_uint8)]),
    "dsa_schedule_from_freq": (c_int32, [c_int32, c_int32, c_int32, POINTER(c_uint8)]),
    "dsa_schedule_resolve": (c_int32, [POINTER(DsaScheduleConfig), c_int32, POINTER(c_uint8)]),
    "dsa_topk_share_create": (c_int32, [POINTER(c_void_p)]),
    "dsa_topk_share_destroy": (c_int32, [c_void_p]),
    "dsa_topk_share_reset": (c_int32, [c_void_p]),
    "dsa_topk_share_publish": (c_int32, [c_void_p, c_int32, c_void_p, c_int64]),
    "dsa_topk_share_get": (c_int32, [c_void_p, POINTER(c_void_p), POINTER(c_int64), POINTER(c_int32)]),
    "dsa_mtp_topk_width": (c_int32, [c_int32, c_int32, POINTER(c_int32)]),
    "dsa_mtp_seed_write": (c_int32, [c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int32, c_void_p, c_void_p]),
    "dsa_topk_share_mtp_begin": (c_int32, [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_int64, c_int32,
                                           POINTER(c_int32)]),
    "dsa_topk_share_needs_scoring": (c_int32, [c_void_p, POINTER(c_int32)]),
    "dsa_topk_share_mtp_end": (c_int32, [c_void_p]),
    "dsa_dense_mla_workspace_size": (c_int32, [POINTER(DsaBatch), POINTER(c_size_t)]),
    "dsa_window_mla": (c_int32, [c_void_p, c_void_p, POINTER(DsaBatch), c_int32, c_int32, c_float, c_void_p, c_int32,
                                 c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "dsa_tree_mla": (c_int32, [c_void_p, c_void_p, c_void_p, POINTER(DsaBatch), c_float, c_void_p, c_int32, c_void_p,
                               c_void_p, c_size_t, c_void_p, c_void_p]),
    "dsa_tree_commit": (c_int32, [c_void_p, c_int32, POINTER(DsaBatch), POINTER(DsaCache), c_int32, c_void_p, c_void_p,
                                  c_void_p]),
    "dsa_pages_reserve": (c_int32, [c_void_p, c_int64, c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_int32,
                                    c_void_p, c_void_p]),
    "dsa_pages_release": (c_int32, [c_void_p, c_int64, c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_int32,
                                    c_void_p, c_void_p]),
    "dsa_pages_fork": (c_int32, [c_void_p, c_int64, c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_int32,
                                 POINTER(DsaCache), c_int32, c_void_p, c_void_p]),
    "dsa_kv8_append": (c_int32, [POINTER(DsaHeads), POINTER(DsaHeads), POINTER(DsaHeads), POINTER(DsaBatch), c_int32, c_int32,
                                 c_int32, c_int32, c_int32, c_float, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                                 c_void_p]),
    "dsa_kv8_attention_workspace_size": (c_int32, [POINTER(DsaBatch), c_int32, c_int32, c_int32, POINTER(c_size_t)]),
    "dsa_kv8_attention": (c_int32, [POINTER(DsaHeads), c_void_p, POINTER(DsaBatch), c_int32, c_int32, c_int32, c_float, c_void_p,
                                    c_int32, c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "dsa_prompt_attention_workspace_size": (c_int32, [POINTER(DsaPrompt), c_int32, c_int32, c_int32, POINTER(c_size_t)]),
    "dsa_prompt_attention": (c_int32, [POINTER(DsaHeads), POINTER(DsaHeads), POINTER(DsaHeads), POINTER(DsaPrompt), c_int32, c_int32,
                                       c_int32, c_float, c_void_p, c_int32, c_void_p, c_void_p, c_size_t, c_void_p, c_void_p]),
    "dsa_cp_topk_merge": (c_int32, [c_void_p, c_void_p, c_void_p, c_int32, c_int64, c_void_p, c_void_p, c_void_p,
                                    c_void_p]),
    "dsa_cp_topk_localize": (c_int32, [c_void_p, c_int64, c_void_p, c_void_p, c_void_p, c_void_p]),
    "dsa_cp_attention_merge": (c_int32, [c_void_p, c_void_p, c_int32, c_int64, c_void_p, c_int32, c_void_p,
                                         c_void_p]),
}


def lib():
    """The loaded libdsa (ctypes.CDLL); raises DsaLibraryMissing if not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise DsaLibraryMissing(
                f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        _lib = h
    return _lib


def status_string(code: int) -> str:
    return lib().dsa_status_string(code).decode()


def _check(fn: str, code: int):
    if code != 0:
        raise DsaError(fn, code)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, device=None):
    """The raw cudaStream_t of `stream` (default: the current stream of
    `device`).  A stream on another device than the call's tensors is refused:
    the kernels would run there with this device's pointers."""
    if stream is None:
        stream = torch.cuda.current_stream(None if device is None else device.index)
    elif device is not None and stream.device != torch.device(device):
        raise ValueError(f"stream is on {stream.device}, the call's tensors on {device}")
    return stream.cuda_stream


def _call(fn: str, device, *args):
    """Run C entry point `fn` with `device` current, so that the library's
    per-device set-up, its device queries and a default stream all refer to the
    device that holds the call's tensors."""
    f = getattr(lib(), fn)
    if torch.cuda.current_device() == device.index:        # switching costs more than a small call's launch
        code = f(*args)
    else:
        with torch.cuda.device(device):
            code = f(*args)
    _check(fn, code)


def _need(t: torch.Tensor, dtype, name: str, device=None, numel=None):
    """A device argument of the C ABI: a contiguous CUDA tensor of `dtype`, on
    `device` when given, with at least `numel` elements when given.  The
    library reads and writes through raw pointers, so a host tensor, a tensor on
    another GPU or a short buffer is rejected here, before any launch."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got one on {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, the call needs {numel}")
    return t


def _opt(t, dtype, name: str, device=None, numel=None):
    return None if t is None else _need(t, dtype, name, device, numel)


# ---------------------------------------------------------------------------
class Batch:
    """Owns the device tensors of one batch and the dsa_batch struct over them.

    seq_len int32 [B] and q_start int32 [B+1] (device), page_table int32
    [B, max_pages] (device).  Host bounds default to the tensors' values
    (read once, with a device sync).
    """

    def __init__(self, seq_len, q_start, page_table, num_pages: int, *, max_seq_len=None,
                 max_q_len=None, total_q=None):
        self.seq_len = _need(seq_len, torch.int32, "seq_len")
        self.q_start = _need(q_start, torch.int32, "q_start")
        self.page_table = _need(page_table, torch.int32, "page_table")
        B = seq_len.numel()
        if max_seq_len is None or max_q_len is None or total_q is None:
            sl = seq_len.cpu()
            qs = q_start.cpu()
            max_seq_len = int(sl.max()) if max_seq_len is None else max_seq_len
            max_q_len = int((qs[1:] - qs[:-1]).max()) if max_q_len is None else max_q_len
            total_q = int(qs[-1]) if total_q is None else total_q
        self.c = DsaBatch(B, page_table.shape[1], int(max_seq_len), int(max_q_len), int(total_q),
                          int(num_pages), seq_len.data_ptr(), q_start.data_ptr(), page_table.data_ptr())

    @property
    def total_q(self) -> int:
        return self.c.total_q

    def ref(self):
        return ctypes.byref(self.c)


def _ws_size(fn_name: str, batch: Batch) -> int:
    n = c_size_t(0)
    _check(fn_name, getattr(lib(), fn_name)(batch.ref(), ctypes.byref(n)))
    return n.value


def workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def _empty(shape, dtype, device, stream):
    """A tensor for a call on `stream` (None: the current one) that the call's caller did not give.
    It comes from that stream's memory, so that nothing enqueued elsewhere still uses it, and goes
    back only when the work that the current stream does on it until then has ended."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def new_device_status(device) -> torch.Tensor:
    return torch.zeros(4, dtype=torch.int32, device=device)


def dsa_device_status_read(dev_status: torch.Tensor, stream=None):
    _need(dev_status, torch.int32, "dev_status", numel=4)
    out = (c_int32 * 4)()
    with torch.cuda.device(dev_status.device):
        code = lib().dsa_device_status_read(_ptr(dev_status), _stream(stream, dev_status.device), out)
    if code not in (0, 7):
        _check("dsa_device_status_read", code)
    return list(out)



def dsa_debug_set_wait_limit_ns(ns: int) -> None:
    """Testing hook: limit (ns) of the pipeline waits of the decode score, the dense MLA and
    the grouped-head attention kernels for later launches, process-wide (2e9 by default; 0 = give up at once)."""
    _check("dsa_debug_set_wait_limit_ns", lib().dsa_debug_set_wait_limit_ns(int(ns)))

def dsa_device_status_reset(dev_status: torch.Tensor, stream=None):
    _need(dev_status, torch.int32, "dev_status", numel=4)
    _call("dsa_device_status_reset", dev_status.device, _ptr(dev_status), _stream(stream, dev_status.device))


# ---------------------------------------------------------------------------
def _store_args(k, pos, slot, idxk_cache, gamma, beta, dev_status):
    _need(k, torch.bfloat16, "k")
    dev, n = k.device, k.shape[0]
    _need(k, torch.bfloat16, "k", dev, n * INDEX_HEAD_DIM)
    _need(pos, torch.int32, "pos", dev, n)
    _need(slot, torch.int64, "slot", dev, n)
    _need(idxk_cache, torch.uint8, "idxk_cache", dev)
    _opt(gamma, torch.float32, "gamma", dev, INDEX_HEAD_DIM)
    _opt(beta, torch.float32, "beta", dev, INDEX_HEAD_DIM)
    _opt(dev_status, torch.int32, "dev_status", dev, 4)
    return n


def dsa_index_k_store(k, pos, slot, idxk_cache, *, gamma=None, beta=None, ln_eps=1e-6,
                      rope_base=10000.0, num_pages=None, dev_status=None, stream=None):
    n = _store_args(k, pos, slot, idxk_cache, gamma, beta, dev_status)
    if num_pages is None:
        num_pages = idxk_cache.numel() // IDXK_PAGE_BYTES
    _call("dsa_index_k_store", k.device,
        _ptr(k), _ptr(pos), _ptr(slot), n, _ptr(gamma), _ptr(beta), ln_eps, rope_base,
        _ptr(idxk_cache), num_pages, _ptr(dev_status), _stream(stream, k.device))


def dsa_index_k_store_mxfp4(k, pos, slot, idxk_cache, *, gamma=None, beta=None, ln_eps=1e-6,
                            rope_base=10000.0, num_pages=None, dev_status=None, stream=None):
    """dsa_index_k_store into an MXFP4 index-K cache (4352-byte pages, 32-byte aligned)."""
    _store_args(k, pos, slot, idxk_cache, gamma, beta, dev_status)
    if num_pages is None:
        num_pages = idxk_cache.numel() // IDXK_MXFP4_PAGE_BYTES
    _call("dsa_index_k_store_mxfp4", k.device,
        _ptr(k), _ptr(pos), _ptr(slot), k.shape[0], _ptr(gamma), _ptr(beta), ln_eps, rope_base,
        _ptr(idxk_cache), num_pages, _ptr(dev_status), _stream(stream, k.device))


def dsa_latent_kv_store_fused(kv_c, k_pe, pos, slot, kv_cache, *, kv_gamma=None, rms_eps=1e-6, rope_base=10000.0,
                              idx_k=None, idxk_cache=None, idx_gamma=None, idx_beta=None, ln_eps=1e-6,
                              num_pages=None, idx_num_pages=None, dev_status=None, stream=None):
    """Latent rows from raw kv_c / k_pe (RMSNorm, RoPE) and, with idx_k, the index keys too."""
    _need(kv_c, torch.bfloat16, "kv_c")
    dev, n = kv_c.device, kv_c.shape[0]
    _need(kv_c, torch.bfloat16, "kv_c", dev, n * LATENT_DIM)
    _need(k_pe, torch.bfloat16, "k_pe", dev, n * ROPE_DIM)
    _need(pos, torch.int32, "pos", dev, n)
    _need(slot, torch.int64, "slot", dev, n)
    _need(kv_cache, torch.uint8, "kv_cache", dev)
    _opt(kv_gamma, torch.float32, "kv_gamma", dev, LATENT_DIM)
    _opt(dev_status, torch.int32, "dev_status", dev, 4)
    if idx_k is not None:
        _need(idx_k, torch.bfloat16, "idx_k", dev, n * INDEX_HEAD_DIM)
        _need(idxk_cache, torch.uint8, "idxk_cache", dev)
        _opt(idx_gamma, torch.float32, "idx_gamma", dev, INDEX_HEAD_DIM)
        _opt(idx_beta, torch.float32, "idx_beta", dev, INDEX_HEAD_DIM)
    if num_pages is None:
        num_pages = kv_cache.numel() // KV_PAGE_BYTES
    if idx_num_pages is None:
        idx_num_pages = 0 if idxk_cache is None else idxk_cache.numel() // IDXK_PAGE_BYTES
    _call("dsa_latent_kv_store_fused", kv_c.device,
        _ptr(kv_c), _ptr(k_pe), _ptr(pos), _ptr(slot), kv_c.shape[0], _ptr(kv_gamma), rms_eps, rope_base,
        _ptr(kv_cache), num_pages, _ptr(idx_k), _ptr(idx_gamma), _ptr(idx_beta), ln_eps, _ptr(idxk_cache),
        idx_num_pages, _ptr(dev_status), _stream(stream, kv_c.device))


def dsa_latent_kv_store(c, rope, slot, kv_cache, *, num_pages=None, dev_status=None, stream=None):
    _need(c, torch.bfloat16, "c")
    dev, n = c.device, c.shape[0]
    _need(c, torch.bfloat16, "c", dev, n * LATENT_DIM)
    _need(rope, torch.bfloat16, "rope", dev, n * ROPE_DIM)
    _need(slot, torch.int64, "slot", dev, n)
    _need(kv_cache, torch.uint8, "kv_cache", dev)
    _opt(dev_status, torch.int32, "dev_status", dev, 4)
    if num_pages is None:
        num_pages = kv_cache.numel() // KV_PAGE_BYTES
    _call("dsa_latent_kv_store", c.device,
        _ptr(c), _ptr(rope), _ptr(slot), c.shape[0], _ptr(kv_cache), num_pages, _ptr(dev_status),
        _stream(stream, c.device))


def _indexer_args(q, w, idxk_cache, batch: Batch) -> int:
    """Checks the indexer's inputs against the batch; returns its query rows T."""
    _need(q, torch.bfloat16, "q")
    T = batch.total_q
    _need(q, torch.bfloat16, "q", q.device, T * INDEX_HEADS * INDEX_HEAD_DIM)
    _need(w, torch.float32, "w", q.device, T * INDEX_HEADS)
    _need(idxk_cache, torch.uint8, "idxk_cache", q.device)
    _need(batch.seq_len, torch.int32, "batch.seq_len", q.device)
    return T


def _ws(ws, nbytes, device, stream):
    """The call's workspace: allocated when not given, else a uint8 CUDA buffer.  An
    allocated one is freed when the call returns, so it is memory of the call's stream:
    only work that comes behind the call there may get it next."""
    if ws is not None:
        return _need(ws, torch.uint8, "ws", device)
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
        return workspace(nbytes, device)


def dsa_indexer_topk_workspace_size(batch: Batch) -> int:
    return _ws_size("dsa_indexer_topk_workspace_size", batch)


def dsa_indexer_topk(q, w, idxk_cache, batch: Batch, *, topk=None, topk_scores=None, share=None,
                     layer_id: int = 0, ws=None, dev_status=None, stream=None):
    """Indexer + top-2048.  Returns topk int32 [T, 2048] (allocated if not given)."""
    T = _indexer_args(q, w, idxk_cache, batch)
    if topk is None:
        topk = _empty((T, TOPK), torch.int32, q.device, stream)
    _need(topk, torch.int32, "topk", q.device, T * TOPK)
    _opt(topk_scores, torch.float32, "topk_scores", q.device, T * TOPK)
    _opt(dev_status, torch.int32, "dev_status", q.device, 4)
    ws = _ws(ws, dsa_indexer_topk_workspace_size(batch) if ws is None else 0, q.device, stream)
    _call("dsa_indexer_topk", q.device,
        _ptr(q), _ptr(w), _ptr(idxk_cache), batch.ref(), _ptr(topk), _ptr(topk_scores),
        None if share is None else share.handle, layer_id, _ptr(ws), ws.numel(), _ptr(dev_status),
        _stream(stream, q.device))
    return topk


def dsa_indexer_topk_mxfp4(q, w, idxk_cache, batch: Batch, *, topk=None, topk_scores=None, share=None,
                           layer_id: int = 0, ws=None, dev_status=None, stream=None):
    """dsa_indexer_topk over an MXFP4 index-K cache (at most 65535 query rows)."""
    T = _indexer_args(q, w, idxk_cache, batch)
    if topk is None:
        topk = _empty((T, TOPK), torch.int32, q.device, stream)
    _need(topk, torch.int32, "topk", q.device, T * TOPK)
    _opt(topk_scores, torch.float32, "topk_scores", q.device, T * TOPK)
    _opt(dev_status, torch.int32, "dev_status", q.device, 4)
    ws = _ws(ws, dsa_indexer_topk_workspace_size(batch) if ws is None else 0, q.device, stream)
    _call("dsa_indexer_topk_mxfp4", q.device,
        _ptr(q), _ptr(w), _ptr(idxk_cache), batch.ref(), _ptr(topk), _ptr(topk_scores),
        None if share is None else share.handle, layer_id, _ptr(ws), ws.numel(), _ptr(dev_status),
        _stream(stream, q.device))
    return topk


def dsa_indexer_topk_noalloc(q, w, idxk_cache, batch: Batch, *, topk=None, topk_scores=None, share=None,
                             layer_id: int = 0, dev_status=None, stream=None):
    """dsa_indexer_topk for decode batches on the library's fixed scratch (no workspace)."""
    T = _indexer_args(q, w, idxk_cache, batch)
    if topk is None:
        topk = _empty((T, TOPK), torch.int32, q.device, stream)
    _need(topk, torch.int32, "topk", q.device, T * TOPK)
    _opt(topk_scores, torch.float32, "topk_scores", q.device, T * TOPK)
    _opt(dev_status, torch.int32, "dev_status", q.device, 4)
    _call("dsa_indexer_topk_noalloc", q.device,
        _ptr(q), _ptr(w), _ptr(idxk_cache), batch.ref(), _ptr(topk), _ptr(topk_scores),
        None if share is None else share.handle, layer_id, _ptr(dev_status), _stream(stream, q.device))
    return topk


def dsa_indexer_scores(q, w, idxk_cache, batch: Batch, *, ld=None, scores=None, ws=None,
                       dev_status=None, stream=None):
    """Full fp32 score rows [T, ld] (debug / parity hook)."""
    T = _indexer_args(q, w, idxk_cache, batch)
    ld = batch.c.max_seq_len if ld is None else ld
    if scores is None:
        scores = _empty((T, ld), torch.float32, q.device, stream)
    _need(scores, torch.float32, "scores", q.device, T * ld)
    _opt(dev_status, torch.int32, "dev_status", q.device, 4)
    ws = _ws(ws, _ws_size("dsa_indexer_scores_workspace_size", batch) if ws is None else 0, q.device, stream)
    _call("dsa_indexer_scores", q.device,
        _ptr(q), _ptr(w), _ptr(idxk_cache), batch.ref(), _ptr(scores), ld, _ptr(ws), ws.numel(),
        _ptr(dev_status), _stream(stream, q.device))
    return scores


def dsa_indexer_scores_cuda_core(q, w, idxk_cache, batch: Batch, *, ld=None, scores=None, ws=None,
                                 dev_status=None, stream=None):
    """dsa_indexer_scores from the CUDA-core kernel (decode batches; comparison only)."""
    T = _indexer_args(q, w, idxk_cache, batch)
    ld = batch.c.max_seq_len if ld is None else ld
    if scores is None:
        scores = _empty((T, ld), torch.float32, q.device, stream)
    _need(scores, torch.float32, "scores", q.device, T * ld)
    _opt(dev_status, torch.int32, "dev_status", q.device, 4)
    ws = _ws(ws, T * (4096 + 128) if ws is None else 0, q.device, stream)
    _call("dsa_indexer_scores_cuda_core", q.device,
        _ptr(q), _ptr(w), _ptr(idxk_cache), batch.ref(), _ptr(scores), ld, _ptr(ws), ws.numel(),
        _ptr(dev_status), _stream(stream, q.device))
    return scores


def dsa_topk_from_scores(scores, valid_len, *, max_len=None, topk=None, stream=None):
    _need(scores, torch.float32, "scores")
    if scores.dim() != 2:
        raise ValueError(f"scores must be [rows, ld], got shape {tuple(scores.shape)}")
    rows, ld = scores.shape
    _need(valid_len, torch.int32, "valid_len", scores.device, rows)
    max_len = ld if max_len is None else max_len
    if topk is None:
        topk = _empty((rows, TOPK), torch.int32, scores.device, stream)
    _need(topk, torch.int32, "topk", scores.device, rows * TOPK)
    n = c_size_t(0)
    _check("dsa_topk_from_scores_workspace_size",
           lib().dsa_topk_from_scores_workspace_size(rows, max_len, ctypes.byref(n)))
    ws = _ws(None, n.value, scores.device, stream)
    _call("dsa_topk_from_scores", scores.device,
        _ptr(scores), ld, _ptr(valid_len), rows, max_len, _ptr(topk), _ptr(ws), ws.numel(), _stream(stream, scores.device))
    return topk


def dsa_sparse_mla_workspace_size(batch: Batch) -> int:
    return _ws_size("dsa_sparse_mla_workspace_size", batch)


def _mla(fn, q, topk, kv_cache, batch, softmax_scale, out, out_dtype, lse, share, ws, dev_status, stream):
    _need(q, torch.bfloat16, "q")
    T = batch.total_q
    dev = q.device
    _need(q, torch.bfloat16, "q", dev, T * MLA_HEADS * QK_DIM)
    _need(kv_cache, torch.uint8, "kv_cache", dev)
    _need(batch.seq_len, torch.int32, "batch.seq_len", dev)
    _opt(topk, torch.int32, "topk", dev, T * TOPK)
    out_t = torch.float32 if out_dtype == DTYPE_F32 else torch.bfloat16
    if out is None:
        out = _empty((T, MLA_HEADS, LATENT_DIM), out_t, dev, stream)
    _need(out, out_t, "out", dev, T * MLA_HEADS * LATENT_DIM)
    _opt(lse, torch.float32, "lse", dev, T * MLA_HEADS)
    _opt(dev_status, torch.int32, "dev_status", dev, 4)
    ws = _ws(ws, dsa_sparse_mla_workspace_size(batch) if ws is None else 0, dev, stream)
    _call(fn, dev,
          _ptr(q), _ptr(topk), None if share is None else share.handle, _ptr(kv_cache), batch.ref(),
          softmax_scale, _ptr(out), out_dtype, _ptr(lse), _ptr(ws), ws.numel(), _ptr(dev_status),
          _stream(stream, dev))
    return out


def dsa_sparse_mla_decode(q, topk, kv_cache, batch: Batch, *, softmax_scale=1.0 / 16, out=None,
                          out_dtype=DTYPE_BF16, lse=None, share=None, ws=None, dev_status=None, stream=None):
    return _mla("dsa_sparse_mla_decode", q, topk, kv_cache, batch, softmax_scale, out, out_dtype, lse,
                share, ws, dev_status, stream)


def dsa_sparse_mla_prefill(q, topk, kv_cache, batch: Batch, *, softmax_scale=1.0 / 16, out=None,
                           out_dtype=DTYPE_BF16, lse=None, share=None, ws=None, dev_status=None, stream=None):
    return _mla("dsa_sparse_mla_prefill", q, topk, kv_cache, batch, softmax_scale, out, out_dtype, lse,
                share, ws, dev_status, stream)


# ---------------------------------------------------------------------------
# MLA over a whole context: sliding window with sinks, draft trees.
def dsa_dense_mla_workspace_size(batch: Batch) -> int:
    return _ws_size("dsa_dense_mla_workspace_size", batch)


def _dense_mla_args(q, kv_cache, batch, out, out_dtype, lse, ws, dev_status, stream):
    _need(q, torch.bfloat16, "q")
    T, dev = batch.total_q, q.device
    _need(q, torch.bfloat16, "q", dev, T * MLA_HEADS * QK_DIM)
    _need(kv_cache, torch.uint8, "kv_cache", dev, batch.c.num_pages * KV_PAGE_BYTES)
    _need(batch.seq_len, torch.int32, "batch.seq_len", dev)
    out_t = torch.float32 if out_dtype == DTYPE_F32 else torch.bfloat16
    if out is None:
        out = _empty((T, MLA_HEADS, LATENT_DIM), out_t, dev, stream)
    _need(out, out_t, "out", dev, T * MLA_HEADS * LATENT_DIM)
    _opt(lse, torch.float32, "lse", dev, T * MLA_HEADS)
    _opt(dev_status, torch.int32, "dev_status", dev, 4)
    nbytes = 0
    if ws is None:
        with torch.cuda.device(dev):
            nbytes = dsa_dense_mla_workspace_size(batch)
    return out, _ws(ws, nbytes, dev, stream)


def dsa_window_mla(q, kv_cache, batch: Batch, *, window: int, sinks: int = 0, softmax_scale=1.0 / 16, out=None,
                   out_dtype=DTYPE_BF16, lse=None, ws=None, dev_status=None, stream=None):
    """Attention of every row over the last `window` positions up to its own and
    the context's first `sinks`; of either, 2^31 - 1 or more is the whole context.
    Returns out [T, 64, 512] (allocated if not given)."""
    window, sinks = (max(-1, min(int(n), 2 ** 31 - 1)) for n in (window, sinks))   # the library takes int32
    out, ws = _dense_mla_args(q, kv_cache, batch, out, out_dtype, lse, ws, dev_status, stream)
    _call("dsa_window_mla", q.device,
          _ptr(q), _ptr(kv_cache), batch.ref(), window, sinks, softmax_scale, _ptr(out), out_dtype, _ptr(lse), _ptr(ws),
          ws.numel(), _ptr(dev_status), _stream(stream, q.device))
    return out


def dsa_tree_mla(q, tree_mask, kv_cache, batch: Batch, *, softmax_scale=1.0 / 16, out=None, out_dtype=DTYPE_BF16,
                 lse=None, ws=None, dev_status=None, stream=None):
    """Attention of a draft tree's rows: the cached prefix and the new tokens whose
    bit is set in the row's mask (int64 [T], taken as 64 bits)."""
    out, ws = _dense_mla_args(q, kv_cache, batch, out, out_dtype, lse, ws, dev_status, stream)
    _need(tree_mask, torch.int64, "tree_mask", q.device, batch.total_q)
    _call("dsa_tree_mla", q.device,
          _ptr(q), _ptr(tree_mask), _ptr(kv_cache), batch.ref(), softmax_scale, _ptr(out), out_dtype, _ptr(lse), _ptr(ws),
          ws.numel(), _ptr(dev_status), _stream(stream, q.device))
    return out


# ---------------------------------------------------------------------------
# Tokens and pages of the caches.
class CacheSet:
    """Every layer's caches that one page table of `num_pages` pages serves:
    (uint8 tensor, CACHE_* kind) pairs, kept alive and checked here."""

    def __init__(self, caches, num_pages: int):
        self.num_pages = int(num_pages)
        self.tensors = [t for t, _ in caches]
        self.device = self.tensors[0].device if self.tensors else None
        self.c = (DsaCache * max(len(caches), 1))()
        for i, (t, kind) in enumerate(caches):
            if kind not in _CACHE_PAGE_BYTES:
                raise ValueError(f"cache {i} has unknown kind {kind}")
            _need(t, torch.uint8, f"cache {i}", self.device, self.num_pages * _CACHE_PAGE_BYTES[kind])
            self.c[i] = DsaCache(t.data_ptr(), kind, 0)
        spans = sorted((t.data_ptr(), t.data_ptr() + self.num_pages * _CACHE_PAGE_BYTES[kind]) for t, kind in caches)
        if any(end > begin for (_, end), (begin, _) in zip(spans, spans[1:])):
            raise ValueError("two of the caches share memory")

    def __len__(self) -> int:
        return len(self.tensors)


def _caches(caches: CacheSet, num_pages: int, dev):
    if len(caches) and (caches.device != dev or caches.num_pages < num_pages):
        raise ValueError(f"the caches hold {caches.num_pages} pages on {caches.device}, the call needs {num_pages} on {dev}")
    return caches.c, len(caches)


def dsa_tree_commit(accept, batch: Batch, caches: CacheSet, *, new_seq_len=None, dev_status=None, stream=None):
    """Move the accepted path's tokens (accept int32 [B, width], -1 ends a row) to the
    front of each request's new tokens in every cache.  Returns new_seq_len int32 [B]."""
    _need(accept, torch.int32, "accept")
    dev, B = accept.device, batch.c.batch
    if accept.dim() != 2 or accept.shape[0] != B:
        raise ValueError(f"accept must be [{B}, width], got {tuple(accept.shape)}")
    _need(batch.seq_len, torch.int32, "batch.seq_len", dev)
    c, n = _caches(caches, batch.c.num_pages, dev)
    if new_seq_len is None:
        new_seq_len = _empty(B, torch.int32, dev, stream)
    _need(new_seq_len, torch.int32, "new_seq_len", dev, B)
    _opt(dev_status, torch.int32, "dev_status", dev, 4)
    _call("dsa_tree_commit", dev, _ptr(accept), accept.shape[1], batch.ref(), c, n, _ptr(new_seq_len), _ptr(dev_status),
          _stream(stream, dev))
    return new_seq_len


def _pool_args(page_ref, page_table, lists, dev_status):
    """Checks a pool call's tensors; returns (device, rows, max_pages, n)."""
    _need(page_ref, torch.int32, "page_ref")
    dev = page_ref.device
    _need(page_table, torch.int32, "page_table", dev)
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be [rows, max_pages], got {tuple(page_table.shape)}")
    n = None
    for name, t in lists:
        _need(t, torch.int32, name, dev)
        if n is not None and t.numel() != n:
            raise ValueError(f"{name} holds {t.numel()} entries, the call's other lists {n}")
        n = t.numel()
    _opt(dev_status, torch.int32, "dev_status", dev, 4)
    return dev, page_table.shape[0], page_table.shape[1], n


def dsa_pages_reserve(page_ref, page_table, row, have_len, want_len, *, dev_status=None, stream=None):
    """Free pages, lowest first, for request row[i] to hold want_len[i] tokens where it holds have_len[i]."""
    dev, rows, max_pages, n = _pool_args(page_ref, page_table, (("row", row), ("have_len", have_len), ("want_len", want_len)),
                                         dev_status)
    _call("dsa_pages_reserve", dev, _ptr(page_ref), page_ref.numel(), _ptr(page_table), rows, max_pages, _ptr(row),
          _ptr(have_len), _ptr(want_len), n, _ptr(dev_status), _stream(stream, dev))


def dsa_pages_release(page_ref, page_table, row, first_page, end_page, *, dev_status=None, stream=None):
    """Entries [first_page[i], end_page[i]) of request row[i] give their pages back."""
    dev, rows, max_pages, n = _pool_args(page_ref, page_table,
                                         (("row", row), ("first_page", first_page), ("end_page", end_page)), dev_status)
    _call("dsa_pages_release", dev, _ptr(page_ref), page_ref.numel(), _ptr(page_table), rows, max_pages, _ptr(row),
          _ptr(first_page), _ptr(end_page), n, _ptr(dev_status), _stream(stream, dev))


def dsa_pages_fork(page_ref, page_table, src_row, dst_row, length, caches: CacheSet, *, dev_status=None, stream=None):
    """Request dst_row[i] becomes a copy of the first length[i] tokens of src_row[i]: full
    pages shared, the last partial one copied in every cache."""
    dev, rows, max_pages, n = _pool_args(page_ref, page_table,
                                         (("src_row", src_row), ("dst_row", dst_row), ("length", length)), dev_status)
    c, n_caches = _caches(caches, page_ref.numel(), dev)
    _call("dsa_pages_fork", dev, _ptr(page_ref), page_ref.numel(), _ptr(page_table), rows, max_pages, _ptr(src_row),
          _ptr(dst_row), _ptr(length), n, c, n_caches, _ptr(dev_status), _stream(stream, dev))


# ---------------------------------------------------------------------------
# Grouped heads beside the latent ones: the KV8 cache and attention.
def kv8_page_bytes(kv_heads: int, head_dim: int) -> int:
    """Bytes of a KV8 cache's page: 64 tokens of every head."""
    return kv_heads * (2 * PAGE_TOKENS * head_dim + 32)


def kv8_views(cache: torch.Tensor, kv_heads: int, head_dim: int):
    """Views of a KV8 cache: key codes [pages, kv_heads, 4, 16, head_dim] and value codes
    [pages, kv_heads, 4, head_dim, 16] (float8_e4m3fn), scales fp32 [pages, kv_heads, 2, 4]
    (keys', then values')."""
    part = PAGE_TOKENS * head_dim
    heads = cache.view(-1, kv_heads, 2 * part + 32)
    blocks = PAGE_TOKENS // KV8_BLOCK
    return (heads[..., :part].unflatten(-1, (blocks, KV8_BLOCK, head_dim)).view(torch.float8_e4m3fn),
            heads[..., part:2 * part].unflatten(-1, (blocks, head_dim, KV8_BLOCK)).view(torch.float8_e4m3fn),
            heads[..., 2 * part:].view(torch.float32).unflatten(-1, (2, blocks)))


def _heads(t: torch.Tensor, name: str, device=None, rows=None):
    """A dsa_heads of a bf16 [rows, heads, head_dim] CUDA tensor whose dims are neighbours."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3:
        raise ValueError(f"{name} must be [rows, heads, head_dim], got {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got one on {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")
    if stride[2] != 1 and t.numel():
        raise ValueError(f"{name}'s head_dim must be contiguous, its stride is {stride[2]}")
    if rows is not None and shape[0] < rows:
        raise ValueError(f"{name} holds {shape[0]} rows, the call needs {rows}")
    # the stride of an axis of one entry says nothing
    return DsaHeads(t.data_ptr(), stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0)


def dsa_kv8_append(k, v, cache, batch: Batch, *, q=None, rope_dims=None, rope_style: int = ROPE_HALVES, rope_base=10000.0,
                   inv_freq=None, q_out=None, k_out=None, dev_status=None, stream=None):
    """The batch's new keys and values (bf16 [total_q, kv_heads, head_dim], any strides of rows and
    heads) enter the KV8 cache, keys rotated by their positions in dims [0, rope_dims) (None: all).
    q (bf16 [total_q, heads, head_dim]) is rotated likewise into q_out, which is returned (allocated
    if not given; None without q); k_out receives the rotated keys if given."""
    dev, T = getattr(k, "device", None), batch.total_q
    ck = _heads(k, "k", None, T)
    kv_heads, dim = k.shape[1], k.shape[2]
    cv = _heads(v, "v", dev, T)
    if tuple(v.shape[1:]) != (kv_heads, dim):
        raise ValueError(f"v must be [rows, {kv_heads}, {dim}], got {tuple(v.shape)}")
    heads, cq = kv_heads, None
    if q is not None:
        cq = _heads(q, "q", dev, T)
        heads = q.shape[1]
        if q.shape[2] != dim:
            raise ValueError(f"q must be [rows, heads, {dim}], got {tuple(q.shape)}")
        if q_out is None:
            q_out = _empty((T, heads, dim), torch.bfloat16, dev, stream)
        _need(q_out, torch.bfloat16, "q_out", dev, T * heads * dim)
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    _opt(k_out, torch.bfloat16, "k_out", dev, T * kv_heads * dim)
    _need(cache, torch.uint8, "cache", dev, batch.c.num_pages * kv8_page_bytes(kv_heads, dim))
    _need(batch.seq_len, torch.int32, "batch.seq_len", dev)
    rope_dims = dim if rope_dims is None else rope_dims
    _opt(inv_freq, torch.float32, "inv_freq", dev, max(rope_dims, 0) // 2)
    _opt(dev_status, torch.int32, "dev_status", dev, 4)
    _call("dsa_kv8_append", dev, ctypes.byref(ck), ctypes.byref(cv), None if cq is None else ctypes.byref(cq), batch.ref(), heads,
          kv_heads, dim, rope_dims, rope_style, rope_base, _ptr(inv_freq), _ptr(cache), _ptr(q_out), _ptr(k_out),
          _ptr(dev_status), _stream(stream, dev))
    return q_out


def dsa_kv8_attention_workspace_size(batch: Batch, heads: int, kv_heads: int, head_dim: int) -> int:
    n = c_size_t(0)
    _check("dsa_kv8_attention_workspace_size",
           lib().dsa_kv8_attention_workspace_size(batch.ref(), heads, kv_heads, head_dim, ctypes.byref(n)))
    return n.value


def _attention_args(q, T, heads, dim, softmax_scale, out, out_dtype, lse, dev_status, stream):
    """Checks what the attention calls on grouped heads share; returns (softmax scale, out)."""
    dev = q.device
    out_t = torch.float32 if out_dtype == DTYPE_F32 else torch.bfloat16
    if out is None:
        out = _empty((T, heads, dim), out_t, dev, stream)
    _need(out, out_t, "out", dev, T * heads * dim)
    _opt(lse, torch.float32, "lse", dev, T * heads)
    _opt(dev_status, torch.int32, "dev_status", dev, 4)
    return dim ** -0.5 if softmax_scale is None else softmax_scale, out


def dsa_kv8_attention(q, cache, batch: Batch, *, kv_heads: int, softmax_scale=None, out=None, out_dtype=DTYPE_BF16, lse=None,
                      ws=None, dev_status=None, stream=None):
    """Causal attention of the batch's new tokens (q bf16 [total_q, heads, head_dim], any strides of
    rows and heads) over a KV8 cache.  softmax_scale defaults to head_dim ** -0.5.
    Returns out [total_q, heads, head_dim] (allocated if not given)."""
    T = batch.total_q
    cq = _heads(q, "q", None, T)
    dev, heads, dim = q.device, q.shape[1], q.shape[2]
    _need(cache, torch.uint8, "cache", dev, batch.c.num_pages * kv8_page_bytes(kv_heads, dim))
    _need(batch.seq_len, torch.int32, "batch.seq_len", dev)
    softmax_scale, out = _attention_args(q, T, heads, dim, softmax_scale, out, out_dtype, lse, dev_status, stream)
    nbytes = 0
    if ws is None:
        with torch.cuda.device(dev):
            nbytes = dsa_kv8_attention_workspace_size(batch, heads, kv_heads, dim)
    ws = _ws(ws, nbytes, dev, stream)
    _call("dsa_kv8_attention", dev, ctypes.byref(cq), _ptr(cache), batch.ref(), heads, kv_heads, dim, softmax_scale, _ptr(out),
          out_dtype, _ptr(lse), _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream, dev))
    return out


class PromptBatch:
    """Owns the device tensors of a batch of packed sequences and the dsa_prompt struct over them.

    q_start int32 [B+1] and k_start int32 [B+1] (device; None: q_start).  Host bounds default to
    the tensors' values (read once, with a device sync).
    """

    def __init__(self, q_start, k_start=None, *, max_q_len=None, max_k_len=None, total_q=None, total_k=None):
        self.q_start = _need(q_start, torch.int32, "q_start")
        self.k_start = self.q_start if k_start is None else _need(k_start, torch.int32, "k_start", q_start.device, q_start.numel())
        if q_start.numel() < 2:
            raise ValueError(f"q_start must hold at least 2 entries, got {q_start.numel()}")
        known = {}
        for name, t, longest, total in (("q", self.q_start, max_q_len, total_q), ("k", self.k_start, max_k_len, total_k)):
            if longest is None or total is None:
                s = t.cpu()
                longest = int((s[1:] - s[:-1]).max()) if longest is None else longest
                total = int(s[-1]) if total is None else total
            known[name] = int(longest), int(total)
        (max_q, n_q), (max_k, n_k) = known["q"], known["k"]
        self.c = DsaPrompt(q_start.numel() - 1, max_q, max_k, 0, n_q, n_k, self.q_start.data_ptr(), self.k_start.data_ptr())

    @property
    def total_q(self) -> int:
        return self.c.total_q

    @property
    def total_k(self) -> int:
        return self.c.total_k

    def ref(self):
        return ctypes.byref(self.c)


def dsa_prompt_attention_workspace_size(batch: PromptBatch, heads: int, kv_heads: int, head_dim: int) -> int:
    n = c_size_t(0)
    _check("dsa_prompt_attention_workspace_size",
           lib().dsa_prompt_attention_workspace_size(batch.ref(), heads, kv_heads, head_dim, ctypes.byref(n)))
    return n.value


def dsa_prompt_attention(q, k, v, batch: PromptBatch, *, softmax_scale=None, out=None, out_dtype=DTYPE_BF16, lse=None, ws=None,
                         dev_status=None, stream=None):
    """Causal attention of packed sequences: q bf16 [total_q, heads, head_dim], k and v bf16 [total_k,
    kv_heads, head_dim], any strides of rows and heads; a sequence's queries are its last tokens.
    softmax_scale defaults to head_dim ** -0.5.  Returns out [total_q, heads, head_dim]
    (allocated if not given)."""
    T = batch.total_q
    cq = _heads(q, "q", None, T)
    dev, heads, dim = q.device, q.shape[1], q.shape[2]
    ck, cv = _heads(k, "k", dev, batch.total_k), _heads(v, "v", dev, batch.total_k)
    kv_heads = k.shape[1]
    for name, t in (("k", k), ("v", v)):
        if tuple(t.shape[1:]) != (kv_heads, dim):
            raise ValueError(f"{name} must be [rows, {kv_heads}, {dim}], got {tuple(t.shape)}")
    _need(batch.q_start, torch.int32, "batch.q_start", dev)
    softmax_scale, out = _attention_args(q, T, heads, dim, softmax_scale, out, out_dtype, lse, dev_status, stream)
    nbytes = 0
    if ws is None:
        with torch.cuda.device(dev):
            nbytes = dsa_prompt_attention_workspace_size(batch, heads, kv_heads, dim)
    ws = _ws(ws, nbytes, dev, stream)
    _call("dsa_prompt_attention", dev, ctypes.byref(cq), ctypes.byref(ck), ctypes.byref(cv), batch.ref(), heads, kv_heads, dim,
          softmax_scale, _ptr(out), out_dtype, _ptr(lse), _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream, dev))
    return out


# ---------------------------------------------------------------------------
def dsa_parse_indexer_types(types) -> list:
    arr = (c_char_p * len(types))(*[t.encode() for t in types])
    out = (c_uint8 * len(types))()
    _check("dsa_parse_indexer_types", lib().dsa_parse_indexer_types(arr, len(types), out))
    return [bool(v) for v in out]


def dsa_schedule_from_freq(n_layers: int, freq: int, offset: int) -> list:
    out = (c_uint8 * n_layers)()
    _check("dsa_schedule_from_freq", lib().dsa_schedule_from_freq(n_layers, freq, offset, out))
    return [bool(v) for v in out]


def dsa_schedule_resolve(n_layers: int, *, indexer_types=None, cli_factor: int = 1, index_topk_pattern=None,
                         index_topk_freq: int = 1, index_skip_topk_offset=None) -> list:
    """Full (True) / shared (False) per layer from whichever schedule fields a config carries."""
    cfg = DsaScheduleConfig()
    keep = None
    if indexer_types is not None:
        keep = (c_char_p * len(indexer_types))(*[t.encode() for t in indexer_types])
        cfg.indexer_types = ctypes.cast(keep, POINTER(c_char_p))
        cfg.n_types = len(indexer_types)
    cfg.cli_factor = cli_factor
    cfg.index_topk_pattern = None if index_topk_pattern is None else index_topk_pattern.encode()
    cfg.index_topk_freq = index_topk_freq
    cfg.index_skip_topk_offset = -1 if index_skip_topk_offset is None else index_skip_topk_offset
    out = (c_uint8 * n_layers)()
    _check("dsa_schedule_resolve", lib().dsa_schedule_resolve(ctypes.byref(cfg), n_layers, out))
    del keep
    return [bool(v) for v in out]


class TopkShare:
    """The share handle: the last full layer's indices, read by shared layers."""

    def __init__(self):
        h = c_void_p()
        _check("dsa_topk_share_create", lib().dsa_topk_share_create(ctypes.byref(h)))
        self.handle = h

    def __del__(self):
        if getattr(self, "handle", None) is not None and _lib is not None:
            _lib.dsa_topk_share_destroy(self.handle)
            self.handle = None

    def reset(self):
        _check("dsa_topk_share_reset", lib().dsa_topk_share_reset(self.handle))

    def publish(self, layer_id: int, topk: torch.Tensor):
        _need(topk, torch.int32, "topk", numel=topk.shape[0] * TOPK)
        _check("dsa_topk_share_publish",
               lib().dsa_topk_share_publish(self.handle, layer_id, _ptr(topk), topk.shape[0]))

    def get(self):
        """(device pointer, rows, layer_id); raises DsaError(DSA_ERR_NO_TOPK_SOURCE) if empty."""
        p, rows, lid = c_void_p(), c_int64(), c_int32()
        _check("dsa_topk_share_get", lib().dsa_topk_share_get(self.handle, ctypes.byref(p),
                                                               ctypes.byref(rows), ctypes.byref(lid)))
        return p.value, rows.value, lid.value

    # ---- top-k reuse across the draft steps of one MTP iteration
    def mtp_begin(self, enabled: bool = True, eagle_topk: int = 1, keep_carry_seed: bool = False,
                  seed: torch.Tensor = None) -> bool:
        """Start an MTP iteration; returns whether the draft steps reuse top-k.
        seed: optional carried device int32 [rows, 2048] (kept alive by the caller)."""
        if seed is not None:
            _need(seed, torch.int32, "seed")
        on = c_int32()
        rows = 0 if seed is None else seed.shape[0]
        width = 0 if seed is None else seed.shape[1]
        _check("dsa_topk_share_mtp_begin", lib().dsa_topk_share_mtp_begin(
            self.handle, int(bool(enabled)), eagle_topk, int(bool(keep_carry_seed)), _ptr(seed), rows, width,
            ctypes.byref(on)))
        return bool(on.value)

    def needs_scoring(self) -> bool:
        """False while the iteration reuses published indices (skip the indexer)."""
        v = c_int32()
        _check("dsa_topk_share_needs_scoring", lib().dsa_topk_share_needs_scoring(self.handle, ctypes.byref(v)))
        return bool(v.value)

    def mtp_end(self):
        _check("dsa_topk_share_mtp_end", lib().dsa_topk_share_mtp_end(self.handle))

    @contextlib.contextmanager
    def mtp_iteration(self, enabled: bool = True, eagle_topk: int = 1, keep_carry_seed: bool = False,
                      seed: torch.Tensor = None):
        """`with share.mtp_iteration(...) as reuse:` - begin / end around the draft steps."""
        reuse = self.mtp_begin(enabled, eagle_topk, keep_carry_seed, seed)
        try:
            yield reuse
        finally:
            self.mtp_end()


def dsa_mtp_topk_width(index_topk: int = 2048, index_kpool: int = 1) -> int:
    v = c_int32()
    _check("dsa_mtp_topk_width", lib().dsa_mtp_topk_width(index_topk, index_kpool, ctypes.byref(v)))
    return v.value


def dsa_mtp_seed_write(topk, *, src_row=None, n=None, seed=None, width=None, dev_status=None, stream=None):
    """seed[r] = topk[src_row[r]] (2048 int32) followed by -1 tail slots."""
    _need(topk, torch.int32, "topk", numel=topk.shape[0] * TOPK)
    if src_row is not None:
        _need(src_row, torch.int32, "src_row", topk.device)
    if n is None:
        n = topk.shape[0] if src_row is None else src_row.shape[0]
    if width is None:
        width = dsa_mtp_topk_width() if seed is None else seed.shape[1]
    if seed is None:
        seed = _empty((n, width), torch.int32, topk.device, stream)
    _need(seed, torch.int32, "seed", topk.device, n * width)
    _opt(dev_status, torch.int32, "dev_status", topk.device, 4)
    _call("dsa_mtp_seed_write", topk.device,
        _ptr(topk), topk.shape[0], _ptr(src_row), n, _ptr(seed), width, _ptr(dev_status), _stream(stream, topk.device))
    return seed


def index_cache_scale_view(idxk_cache: torch.Tensor) -> torch.Tensor:
    """fp32 [num_pages, 64] view of the per-token scales inside an index-K cache."""
    pages = idxk_cache.view(-1, IDXK_PAGE_BYTES)
    return pages[:, PAGE_TOKENS * INDEX_HEAD_DIM:].view(torch.float32)


# ---------------------------------------------------------------------------
# Context-parallel split of long requests over the ranks of a process group
# ("GLM-5.3 推理全链路(十一)", 两个框架的对照; "Accelerating GLM-5.3-Flash on H200",
# prefill 的重点是少搬一次、少等一次).  See dsa.h for the steps.
CP_MAX_RANKS = 8


def dsa_cp_topk_merge(cand_pos, cand_scores, pos_offset, *, topk=None, topk_scores=None, dev_status=None,
                      stream=None):
    """Global top-2048 from every rank's list: cand_pos / cand_scores [G, rows, 2048],
    pos_offset int64 [G, rows].  Returns topk int32 [rows, 2048]."""
    _need(cand_pos, torch.int32, "cand_pos")
    if cand_pos.dim() != 3 or cand_pos.shape[2] != TOPK:
        raise ValueError(f"cand_pos must be [G, rows, {TOPK}], got {tuple(cand_pos.shape)}")
    G, rows = cand_pos.shape[0], cand_pos.shape[1]
    dev = cand_pos.device
    _need(cand_scores, torch.float32, "cand_scores", dev, G * rows * TOPK)
    _need(pos_offset, torch.int64, "pos_offset", dev, G * rows)
    if topk is None:
        topk = _empty((rows, TOPK), torch.int32, dev, stream)
    _need(topk, torch.int32, "topk", dev, rows * TOPK)
    _opt(topk_scores, torch.float32, "topk_scores", dev, rows * TOPK)
    _opt(dev_status, torch.int32, "dev_status", dev, 4)
    _call("dsa_cp_topk_merge", dev, _ptr(cand_pos), _ptr(cand_scores), _ptr(pos_offset), G, rows, _ptr(topk),
          _ptr(topk_scores), _ptr(dev_status), _stream(stream, dev))
    return topk


def dsa_cp_topk_localize(topk, slice_start, slice_len, *, local_topk=None, stream=None):
    """This rank's share of a global top-k list, in local positions, compacted."""
    _need(topk, torch.int32, "topk")
    rows, dev = topk.shape[0], topk.device
    _need(topk, torch.int32, "topk", dev, rows * TOPK)
    _need(slice_start, torch.int64, "slice_start", dev, rows)
    _need(slice_len, torch.int64, "slice_len", dev, rows)
    if local_topk is None:
        local_topk = _empty((rows, TOPK), torch.int32, dev, stream)
    _need(local_topk, torch.int32, "local_topk", dev, rows * TOPK)
    _call("dsa_cp_topk_localize", dev, _ptr(topk), rows, _ptr(slice_start), _ptr(slice_len), _ptr(local_topk),
          _stream(stream, dev))
    return local_topk


def dsa_cp_attention_merge(o_parts, lse_parts, *, out=None, out_dtype=DTYPE_BF16, lse=None, stream=None):
    """Attention over the union of the ranks' selected positions from their
    parts: o_parts fp32 [G, rows, 64, 512], lse_parts fp32 [G, rows, 64]."""
    _need(o_parts, torch.float32, "o_parts")
    if o_parts.dim() != 4 or tuple(o_parts.shape[2:]) != (MLA_HEADS, LATENT_DIM):
        raise ValueError(f"o_parts must be [G, rows, 64, 512], got {tuple(o_parts.shape)}")
    G, rows, dev = o_parts.shape[0], o_parts.shape[1], o_parts.device
    _need(lse_parts, torch.float32, "lse_parts", dev, G * rows * MLA_HEADS)
    out_t = torch.float32 if out_dtype == DTYPE_F32 else torch.bfloat16
    if out is None:
        out = _empty((rows, MLA_HEADS, LATENT_DIM), out_t, dev, stream)
    _need(out, out_t, "out", dev, rows * MLA_HEADS * LATENT_DIM)
    _opt(lse, torch.float32, "lse", dev, rows * MLA_HEADS)
    _call("dsa_cp_attention_merge", dev, _ptr(o_parts), _ptr(lse_parts), G, rows, _ptr(out), out_dtype, _ptr(lse),
          _stream(stream, dev))
    return out


class LibraryOps:
    """The per-rank steps of the context-parallel split, as library calls."""

    def indexer_topk(self, q, w, idxk_cache, batch, ws=None, dev_status=None, stream=None):
        T = batch.total_q
        topk = _empty((T, TOPK), torch.int32, q.device, stream)
        scores = _empty((T, TOPK), torch.float32, q.device, stream)
        dsa_indexer_topk(q, w, idxk_cache, batch, topk=topk, topk_scores=scores, ws=ws, dev_status=dev_status,
                         stream=stream)
        return topk, scores

    def topk_merge(self, cand_pos, cand_scores, pos_offset, dev_status=None, stream=None):
        return dsa_cp_topk_merge(cand_pos, cand_scores, pos_offset, dev_status=dev_status, stream=stream)

    def topk_localize(self, topk, slice_start, slice_len, stream=None):
        return dsa_cp_topk_localize(topk, slice_start, slice_len, stream=stream)

    def sparse_mla(self, q, local_topk, kv_cache, batch, softmax_scale, ws=None, dev_status=None, stream=None):
        T = batch.total_q
        lse = _empty((T, MLA_HEADS), torch.float32, q.device, stream)
        out = dsa_sparse_mla_decode(q, local_topk, kv_cache, batch, softmax_scale=softmax_scale, out_dtype=DTYPE_F32,
                                    lse=lse, ws=ws, dev_status=dev_status, stream=stream)
        return out, lse

    def attention_merge(self, o_parts, lse_parts, out_dtype, stream=None):
        T = o_parts.shape[1]
        lse = _empty((T, MLA_HEADS), torch.float32, o_parts.device, stream)
        out = dsa_cp_attention_merge(o_parts, lse_parts, out_dtype=out_dtype, lse=lse, stream=stream)
        return out, lse


def _gather_ranks(t, group):
    """[G, *t.shape]: every rank's t, in rank order (the exchange step)."""
    import torch.distributed as dist
    G = dist.get_world_size(group)
    if dist.get_backend(group) == "nccl":
        out = torch.empty((G, *t.shape), dtype=t.dtype, device=t.device)
        dist.all_gather_into_tensor(out, t.contiguous(), group=group)
        return out
    parts = [torch.empty_like(t) for _ in range(G)]
    dist.all_gather(parts, t.contiguous(), group=group)
    return torch.stack(parts)


class ContextParallel:
    """One layer's indexer and sparse MLA for requests whose positions are cut
    into disjoint slices, one per rank of `group` (at most 8 ranks).  This rank
    holds its slice of every request in its own caches, described by `batch`
    as requests of seq_len = slice length with local positions; slice_start
    (int64 [rows], device) gives the global position of each row's local
    position 0, slice_len the slice's length.  Every slice must be longer than
    2048 tokens.  Two exchanges per layer: at most 2048 (score, position) pairs
    per row and rank after the indexer, one [64, 512] fp32 part and its
    log-sum-exp per row and rank after sparse MLA.

    `ops` performs the per-rank steps; it defaults to the library's calls."""

    def __init__(self, group=None, ops=None, gather=None):
        import torch.distributed as dist
        self.group = group
        self.world = dist.get_world_size(group)
        if self.world > CP_MAX_RANKS:
            raise ValueError(f"at most {CP_MAX_RANKS} ranks, the group has {self.world}")
        self.ops = ops if ops is not None else LibraryOps()
        self._gather = gather if gather is not None else (lambda t: _gather_ranks(t, group))

    def indexer_topk(self, q, w, idxk_cache, batch, slice_start, *, share=None, layer_id=0, ws=None,
                     dev_status=None, stream=None):
        """The global top-2048 of every row (global positions, ascending)."""
        local, scores = self.ops.indexer_topk(q, w, idxk_cache, batch, ws=ws, dev_status=dev_status, stream=stream)
        cand_pos = self._gather(local)
        cand_scores = self._gather(scores)
        offsets = self._gather(slice_start)
        topk = self.ops.topk_merge(cand_pos, cand_scores, offsets, dev_status=dev_status, stream=stream)
        if share is not None:
            share.publish(layer_id, topk)
        return topk

    def sparse_mla(self, q, topk, kv_cache, batch, slice_start, slice_len, *, softmax_scale=1.0 / 16,
                   out_dtype=DTYPE_BF16, ws=None, dev_status=None, stream=None):
        """Attention of every row over its global top-2048; returns (out, lse)."""
        local = self.ops.topk_localize(topk, slice_start, slice_len, stream=stream)
        o, lse = self.ops.sparse_mla(q, local, kv_cache, batch, softmax_scale, ws=ws, dev_status=dev_status,
                                     stream=stream)
        return self.ops.attention_merge(self._gather(o), self._gather(lse), out_dtype, stream=stream)
