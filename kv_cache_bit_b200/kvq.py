"""Thin ctypes binding of libkvq (include/kvq.h): the same call names, with
argument marshalling only.  Every step of the quantizer and of decode
attention runs in the library's CUDA kernels; PyTorch is used here only to
hold device memory and to name the current CUDA stream.

Loading fails loudly (ImportError) when libkvq.so has not been built: there
is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "libkvq.so")

KVQ_OK, KVQ_ERR_INVALID_ARG, KVQ_ERR_UNSUPPORTED, KVQ_ERR_CAPACITY, KVQ_ERR_WORKSPACE, KVQ_ERR_CUDA = range(6)
KVQ_NORM_SEP, KVQ_PER_CHANNEL, KVQ_NSN, KVQ_HADAMARD, KVQ_DQ = 1, 2, 4, 8, 16
NORM_SEP, PER_CHANNEL, NSN, HADAMARD, DQ = KVQ_NORM_SEP, KVQ_PER_CHANNEL, KVQ_NSN, KVQ_HADAMARD, KVQ_DQ
BLOCK_TOKENS = 128

EXPORTS = ["kvq_row_bytes", "kvq_tok_params", "kvq_off_words", "kvq_make_signs", "kvq_quantize_block", "kvq_append_token",
           "kvq_decode_workspace_bytes", "kvq_decode_attention", "kvq_decode_attention_noalloc", "kvq_dequantize",
           "kvq_select_signs_workspace_bytes", "kvq_select_signs", "kvq_read_device_errors",
           "kvq_pages_write", "kvq_pages_read", "kvq_pages_attention_workspace_bytes", "kvq_pages_attention",
           "kvq_pages_read_errors", "kvq_status_string"]


class kvq_config(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("bits", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("reserved", ctypes.c_int32), ("signs", ctypes.c_void_p)]


class kvq_cache(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("len", ctypes.c_int64),
                ("codes", ctypes.c_void_p * 2), ("tok", ctypes.c_void_p * 2), ("chan", ctypes.c_void_p * 2),
                ("off", ctypes.c_void_p * 2), ("resid", ctypes.c_void_p * 2)]


class kvq_pages(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("codes", ctypes.c_void_p * 2), ("tok", ctypes.c_void_p * 2)]


class kvq_batch(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("table_stride", ctypes.c_int32),
                ("max_rows", ctypes.c_int32), ("start", ctypes.c_void_p), ("len", ctypes.c_void_p),
                ("table", ctypes.c_void_p)]


class kvq_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libkvq.so not built ({LIB_PATH}); run kv_cache_bit_b200/build.py")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    L.kvq_row_bytes.restype = ctypes.c_int32
    L.kvq_row_bytes.argtypes = [ctypes.c_int32, ctypes.c_int32]
    L.kvq_tok_params.restype = ctypes.c_int32
    L.kvq_tok_params.argtypes = [ctypes.c_uint32]
    L.kvq_off_words.restype = ctypes.c_int32
    L.kvq_off_words.argtypes = [ctypes.c_uint32, ctypes.c_int32]
    L.kvq_make_signs.restype = ctypes.c_int
    L.kvq_make_signs.argtypes = [ctypes.c_uint64, ctypes.c_int32, P]
    L.kvq_quantize_block.restype = ctypes.c_int
    L.kvq_quantize_block.argtypes = [ctypes.POINTER(kvq_config), ctypes.POINTER(kvq_cache), P, P,
                                     ctypes.c_int64, ctypes.c_int64, P]
    L.kvq_append_token.restype = ctypes.c_int
    L.kvq_append_token.argtypes = [ctypes.POINTER(kvq_config), ctypes.POINTER(kvq_cache), P, P, P]
    L.kvq_decode_workspace_bytes.restype = ctypes.c_size_t
    L.kvq_decode_workspace_bytes.argtypes = [ctypes.POINTER(kvq_config), ctypes.POINTER(kvq_cache), ctypes.c_int32]
    L.kvq_decode_attention.restype = ctypes.c_int
    L.kvq_decode_attention.argtypes = [ctypes.POINTER(kvq_config), ctypes.POINTER(kvq_cache), P, ctypes.c_int32,
                                       ctypes.c_float, P, P, ctypes.c_size_t, P]
    L.kvq_decode_attention_noalloc.restype = ctypes.c_int
    L.kvq_decode_attention_noalloc.argtypes = [ctypes.POINTER(kvq_config), ctypes.POINTER(kvq_cache), P,
                                               ctypes.c_int32, ctypes.c_float, P, P]
    L.kvq_dequantize.restype = ctypes.c_int
    L.kvq_dequantize.argtypes = [ctypes.POINTER(kvq_config), ctypes.POINTER(kvq_cache), ctypes.c_int32,
                                 ctypes.c_int64, ctypes.c_int64, P, P]
    L.kvq_select_signs_workspace_bytes.restype = ctypes.c_size_t
    L.kvq_select_signs_workspace_bytes.argtypes = [ctypes.c_int32, ctypes.c_int64]
    L.kvq_select_signs.restype = ctypes.c_int
    L.kvq_select_signs.argtypes = [ctypes.POINTER(kvq_config), P, ctypes.c_int64, P, ctypes.c_int32, P, P, P,
                                   ctypes.c_size_t, P]
    L.kvq_read_device_errors.restype = ctypes.c_int
    L.kvq_read_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int32]
    C, G, B, R = (ctypes.POINTER(t) for t in (kvq_config, kvq_pages, kvq_batch, kvq_rows))
    L.kvq_pages_write.restype = ctypes.c_int
    L.kvq_pages_write.argtypes = [C, G, B, R, R, ctypes.c_int64, P]
    L.kvq_pages_read.restype = ctypes.c_int
    L.kvq_pages_read.argtypes = [C, G, B, R, R, ctypes.c_int64, P]
    L.kvq_pages_attention_workspace_bytes.restype = ctypes.c_size_t
    L.kvq_pages_attention_workspace_bytes.argtypes = [C, G, B, ctypes.c_int64, ctypes.c_int32]
    L.kvq_pages_attention.restype = ctypes.c_int
    L.kvq_pages_attention.argtypes = [C, G, B, R, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_int32,
                                      ctypes.c_int32, R, P, P, ctypes.c_size_t, P]
    L.kvq_pages_read_errors.restype = ctypes.c_int
    L.kvq_pages_read_errors.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int32]
    L.kvq_status_string.restype = ctypes.c_char_p
    L.kvq_status_string.argtypes = [ctypes.c_int]
    return L


lib = _load()


class KvqError(RuntimeError):
    def __init__(self, status: int, call: str):
        super().__init__(f"{call}: {lib.kvq_status_string(status).decode()} (status {status})")
        self.status = status


def _check(status: int, call: str):
    if status != KVQ_OK:
        raise KvqError(status, call)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


# ------------------------------------------------------------------ calls

def kvq_row_bytes(head_dim: int, bits: int) -> int:
    return lib.kvq_row_bytes(head_dim, bits)


def kvq_tok_params(flags: int) -> int:
    return lib.kvq_tok_params(flags)


def kvq_off_words(flags: int, head_dim: int) -> int:
    return lib.kvq_off_words(flags, head_dim)


def kvq_make_signs(seed: int, head_dim: int):
    """Host +-1 signs (numpy int8) from SplitMix64."""
    import numpy as np
    out = np.empty(head_dim, np.int8)
    _check(lib.kvq_make_signs(ctypes.c_uint64(seed), head_dim, out.ctypes.data), "kvq_make_signs")
    return out


def kvq_quantize_block(cfg: "Config", cache: "KVCache", k, v, t0: int, ntok: int, stream=None):
    _check(lib.kvq_quantize_block(ctypes.byref(cfg.c), ctypes.byref(cache.c), _ptr(k), _ptr(v), t0, ntok,
                                  _stream(stream)), "kvq_quantize_block")


def kvq_append_token(cfg: "Config", cache: "KVCache", k_new, v_new, stream=None):
    _check(lib.kvq_append_token(ctypes.byref(cfg.c), ctypes.byref(cache.c), _ptr(k_new), _ptr(v_new),
                                _stream(stream)), "kvq_append_token")


def kvq_decode_workspace_bytes(cfg: "Config", cache: "KVCache", q_heads: int) -> int:
    return lib.kvq_decode_workspace_bytes(ctypes.byref(cfg.c), ctypes.byref(cache.c), q_heads)


def kvq_decode_attention(cfg: "Config", cache: "KVCache", q, q_heads: int, scale: float, out, ws, ws_bytes: int,
                         stream=None):
    _check(lib.kvq_decode_attention(ctypes.byref(cfg.c), ctypes.byref(cache.c), _ptr(q), q_heads, scale,
                                    _ptr(out), _ptr(ws), ws_bytes, _stream(stream)), "kvq_decode_attention")


def kvq_decode_attention_noalloc(cfg: "Config", cache: "KVCache", q, q_heads: int, scale: float, out,
                                 stream=None):
    """Decode attention with the library's own fixed device scratch (no
    workspace argument, no allocation); see include/kvq.h."""
    _check(lib.kvq_decode_attention_noalloc(ctypes.byref(cfg.c), ctypes.byref(cache.c), _ptr(q), q_heads, scale,
                                            _ptr(out), _stream(stream)), "kvq_decode_attention_noalloc")


NOALLOC_SCRATCH_BYTES = 32 << 20


def kvq_dequantize(cfg: "Config", cache: "KVCache", tensor: int, t0: int, ntok: int, out, stream=None):
    _check(lib.kvq_dequantize(ctypes.byref(cfg.c), ctypes.byref(cache.c), tensor, t0, ntok, _ptr(out),
                              _stream(stream)), "kvq_dequantize")


SELECT_MAX_CANDIDATES = 256


def kvq_select_signs_workspace_bytes(n_cand: int, n_blocks: int) -> int:
    return lib.kvq_select_signs_workspace_bytes(n_cand, n_blocks)


def kvq_select_signs(cfg: "Config", x, n_blocks: int, signs, n_cand: int, err, best, ws, ws_bytes: int,
                     stream=None):
    """Sign-pattern selection (see include/kvq.h): x fp16 [n_blocks, 128,
    head_dim], signs int8 [n_cand, head_dim], err float64 [n_cand] and best
    int32 [1] outputs, all device tensors."""
    _check(lib.kvq_select_signs(ctypes.byref(cfg.c), _ptr(x), n_blocks, _ptr(signs), n_cand, _ptr(err), _ptr(best),
                                _ptr(ws), ws_bytes, _stream(stream)), "kvq_select_signs")


def kvq_read_device_errors(clear: bool = True) -> int:
    v = ctypes.c_uint32(0)
    _check(lib.kvq_read_device_errors(ctypes.byref(v), 1 if clear else 0), "kvq_read_device_errors")
    return v.value


# ------------------------------------------------------------------ paged cache

KVQ_F16, KVQ_BF16, KVQ_F32 = 0, 1, 2
PAGE_TOKENS = (16, 32, 64, 128)
_DTYPES = {}


def _paged(call: str, cfg: "Config", pages: "PagedCache", batch: "Batch", *tensors) -> int:
    """Number of rows of the [rows, heads, head_dim] tensors, after the checks
    that only their Python side can make (the library sees bare pointers)."""
    rows = None
    device = pages.device
    if batch.device != device or (cfg.signs_dev is not None and cfg.signs_dev.device != device):
        raise KvqError(KVQ_ERR_INVALID_ARG, call + ": configuration, cache and batch on one device")
    for x, heads in tensors:
        if x is None:
            continue
        shape = x.shape
        if len(shape) != 3 or shape[2] != cfg.head_dim or x.stride(2) != 1 or x.device != device:
            raise KvqError(KVQ_ERR_INVALID_ARG, call + ": tensors are [rows, heads, head_dim] on the cache's device")
        if (heads and shape[1] != heads) or (rows is not None and rows != shape[0]):
            raise KvqError(KVQ_ERR_INVALID_ARG, call + ": heads or rows of the tensors differ")
        rows = shape[0]
    return rows


def _rows(x, call: str):
    """kvq_rows of a [rows, heads, head_dim] tensor (None: a null pointer)."""
    if x is None:
        return None
    kind = _DTYPES.get(x.dtype)
    if kind is None:
        import torch
        _DTYPES.update({torch.float16: KVQ_F16, torch.bfloat16: KVQ_BF16, torch.float32: KVQ_F32})
        kind = _DTYPES.get(x.dtype)
        if kind is None:
            raise KvqError(KVQ_ERR_UNSUPPORTED, call)
    stride = x.stride()
    # (a tensor without rows has no address; nothing is read through this one)
    return kvq_rows(x.data_ptr() or 16, stride[0], stride[1], kind, 0)


_torch = None  # torch and its raw accessors, once a paged call needs them


def _on(pages: "PagedCache", stream, call: str, fn, *args):
    """fn(*args, stream) with the cache's device current; stream None: the
    current stream of that device."""
    global _torch
    if pages.device.type != "cuda":
        raise KvqError(KVQ_ERR_INVALID_ARG, call + ": a cache on a GPU")
    if _torch is None:
        import torch
        torch.cuda.init()
        _torch = (torch, torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice)
    torch, raw_stream, current = _torch
    index = pages.device.index
    if stream is None:
        stream = raw_stream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if current() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != KVQ_OK:
        raise KvqError(status, call)


def kvq_pages_write(cfg: "Config", pages: "PagedCache", batch: "Batch", k, v, stream=None):
    """Quantize rows k, v [rows, kv_heads, head_dim] (fp16 or bf16, any row and
    head strides of whole 16 bytes) into their slots; see include/kvq.h."""
    name = "kvq_pages_write"
    rows = _paged(name, cfg, pages, batch, (k, pages.c.kv_heads), (v, pages.c.kv_heads))
    _on(pages, stream, name, lib.kvq_pages_write, cfg.c, pages.c, batch.c, _rows(k, name), _rows(v, name), rows or 0)


def kvq_pages_read(cfg: "Config", pages: "PagedCache", batch: "Batch", k_out, v_out, stream=None):
    """Rebuild the batch's rows into k_out and v_out [rows, kv_heads, head_dim]
    (fp16, bf16 or fp32; one of them may be None)."""
    name = "kvq_pages_read"
    rows = _paged(name, cfg, pages, batch, (k_out, pages.c.kv_heads), (v_out, pages.c.kv_heads))
    _on(pages, stream, name, lib.kvq_pages_read, cfg.c, pages.c, batch.c, _rows(k_out, name), _rows(v_out, name),
        rows or 0)


def kvq_pages_attention_workspace_bytes(cfg: "Config", pages: "PagedCache", batch: "Batch", rows: int,
                                        q_heads: int) -> int:
    import torch
    with torch.cuda.device(pages.device):
        return lib.kvq_pages_attention_workspace_bytes(cfg.c, pages.c, batch.c, rows, q_heads)


def kvq_pages_attention(cfg: "Config", pages: "PagedCache", batch: "Batch", q, out, lse=None, scale: float = 0.0,
                        causal: bool = True, window: int = 0, ws=None, stream=None):
    """Attention of queries q [rows, q_heads, head_dim] over their sequences
    into out (q's type and shape) and, if given, lse fp32 [rows, q_heads].
    ws: uint8 tensor of kvq_pages_attention_workspace_bytes()."""
    name = "kvq_pages_attention"
    if q is None or out is None:
        raise KvqError(KVQ_ERR_INVALID_ARG, name + ": q and out")
    rows = _paged(name, cfg, pages, batch, (q, 0), (out, 0))
    heads = q.shape[1]
    if out.shape[1] != heads or ws is None or ws.device != pages.device or not ws.is_contiguous():
        raise KvqError(KVQ_ERR_INVALID_ARG, name + ": out of q's shape, a contiguous workspace on the cache's device")
    if lse is not None and (lse.device != pages.device or tuple(lse.shape) != (rows, heads) or
                            lse.element_size() != 4 or not lse.is_floating_point() or not lse.is_contiguous()):
        raise KvqError(KVQ_ERR_INVALID_ARG, name + ": lse is a contiguous float32 [rows, q_heads]")
    _on(pages, stream, name, lib.kvq_pages_attention, cfg.c, pages.c, batch.c, _rows(q, name), heads, rows, scale,
        1 if causal else 0, window, _rows(out, name), _ptr(lse) or None, _ptr(ws), ws.numel() * ws.element_size())


def kvq_pages_read_errors(clear: bool = True) -> int:
    v = ctypes.c_uint32(0)
    _check(lib.kvq_pages_read_errors(ctypes.byref(v), 1 if clear else 0), "kvq_pages_read_errors")
    return v.value


# ------------------------------------------------------------------ plumbing

class Config:
    """kvq_config plus the device copy of the rotation signs it points to."""

    def __init__(self, head_dim: int, bits: int, flags: int, signs=None, device="cuda"):
        import torch
        self.head_dim, self.bits, self.flags = head_dim, bits, flags
        self.signs_dev = None
        if signs is not None:
            self.signs_dev = torch.as_tensor(signs, dtype=torch.int8).to(device).contiguous()
        self.c = kvq_config(head_dim, bits, flags, 0, _ptr(self.signs_dev))


@dataclass
class KVCache:
    """Caller-side allocation of a kvq_cache (torch tensors on the GPU)."""
    c: kvq_cache
    codes: list
    tok: list
    chan: list
    off: list
    resid: list

    @classmethod
    def allocate(cls, cfg: Config, batch: int, kv_heads: int, capacity: int, device="cuda") -> "KVCache":
        import torch
        assert capacity % BLOCK_TOKENS == 0
        rb = kvq_row_bytes(cfg.head_dim, cfg.bits)
        nt = kvq_tok_params(cfg.flags)
        if rb <= 0 or nt <= 0:
            raise KvqError(KVQ_ERR_UNSUPPORTED, "KVCache.allocate")
        nb = capacity // BLOCK_TOKENS
        d = cfg.head_dim
        mk = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)
        codes = [mk((batch, kv_heads, capacity, rb), torch.uint8) for _ in range(2)]
        tok = [mk((batch, kv_heads, capacity, nt), torch.int16) for _ in range(2)]
        pchan = bool(cfg.flags & PER_CHANNEL)
        chan = [mk((batch, kv_heads, nb, d), torch.int16) if pchan else None for _ in range(2)]
        ow = kvq_off_words(cfg.flags, d)
        off = [mk((batch, kv_heads, nb, ow), torch.int16) if cfg.flags & NSN else None for _ in range(2)]
        resid = [mk((batch, kv_heads, BLOCK_TOKENS, d), torch.int16) for _ in range(2)]
        c = kvq_cache(batch, kv_heads, d, capacity, 0,
                      (ctypes.c_void_p * 2)(*[_ptr(x) for x in codes]),
                      (ctypes.c_void_p * 2)(*[_ptr(x) for x in tok]),
                      (ctypes.c_void_p * 2)(*[_ptr(x) for x in chan]),
                      (ctypes.c_void_p * 2)(*[_ptr(x) for x in off]),
                      (ctypes.c_void_p * 2)(*[_ptr(x) for x in resid]))
        return cls(c, codes, tok, chan, off, resid)

    def rows(self, b0: int, b1: int) -> "KVCache":
        """A view of batch rows [b0, b1) sharing this cache's memory (its own
        kvq_cache struct, len copied)."""
        sl = lambda ts: [t[b0:b1] if t is not None else None for t in ts]
        codes, tok, chan, off, resid = sl(self.codes), sl(self.tok), sl(self.chan), sl(self.off), sl(self.resid)
        c = kvq_cache(b1 - b0, self.c.kv_heads, self.c.head_dim, self.c.capacity, self.c.len,
                      (ctypes.c_void_p * 2)(*[_ptr(x) for x in codes]),
                      (ctypes.c_void_p * 2)(*[_ptr(x) for x in tok]),
                      (ctypes.c_void_p * 2)(*[_ptr(x) for x in chan]),
                      (ctypes.c_void_p * 2)(*[_ptr(x) for x in off]),
                      (ctypes.c_void_p * 2)(*[_ptr(x) for x in resid]))
        return KVCache(c, codes, tok, chan, off, resid)

    @property
    def len(self) -> int:
        return self.c.len

    def snapshot(self) -> dict:
        """A host copy of the cache (checkpoint): every buffer and the
        token count.  The cache is plain caller-owned memory, so this is the
        whole state."""
        cp = lambda ts: [t.cpu() if t is not None else None for t in ts]
        return {"len": self.c.len, "codes": cp(self.codes), "tok": cp(self.tok), "chan": cp(self.chan),
                "off": cp(self.off), "resid": cp(self.resid)}

    def restore(self, snap: dict) -> None:
        """Load a snapshot taken from a cache of the same configuration and
        shape (resume)."""
        for name in ("codes", "tok", "chan", "off", "resid"):
            for dst, src in zip(getattr(self, name), snap[name]):
                if (dst is None) != (src is None) or (dst is not None and dst.shape != src.shape):
                    raise KvqError(KVQ_ERR_INVALID_ARG, "KVCache.restore: snapshot of another cache shape")
                if dst is not None:
                    dst.copy_(src)
        self.c.len = snap["len"]

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for group in (self.codes, self.tok, self.chan, self.off, self.resid)
                   for t in group if t is not None)


@dataclass
class PagedCache:
    """Caller-side memory of a kvq_pages pool (torch tensors on the GPU):
    codes[2] uint8 [n_pages, kv_heads, page_tokens, head_dim / 2] and tok[2]
    float16 [n_pages, kv_heads, page_tokens], K then V."""
    c: kvq_pages
    codes: list
    tok: list
    device: object = None

    def __post_init__(self):
        self.device = self.codes[0].device

    @classmethod
    def allocate(cls, cfg: Config, n_pages: int, kv_heads: int, page_tokens: int, device="cuda") -> "PagedCache":
        import torch
        if page_tokens not in PAGE_TOKENS or cfg.bits != 4 or kvq_row_bytes(cfg.head_dim, 4) == 0:
            raise KvqError(KVQ_ERR_UNSUPPORTED, "PagedCache.allocate")
        shape = (n_pages, kv_heads, page_tokens)
        codes = [torch.zeros((*shape, cfg.head_dim // 2), dtype=torch.uint8, device=device) for _ in range(2)]
        tok = [torch.zeros(shape, dtype=torch.float16, device=device) for _ in range(2)]
        return cls.wrap(cfg, codes, tok)

    @classmethod
    def wrap(cls, cfg: Config, codes, tok) -> "PagedCache":
        """A pool over tensors that the caller has."""
        import torch
        n, h, t, half = codes[0].shape
        for x, y in zip(codes, tok):
            if (x.dtype, y.dtype) != (torch.uint8, torch.float16) or x.device != y.device or \
                    x.device != codes[0].device or tuple(x.shape) != (n, h, t, half) or half * 2 != cfg.head_dim or \
                    tuple(y.shape) != (n, h, t) or not x.is_contiguous() or not y.is_contiguous():
                raise KvqError(KVQ_ERR_INVALID_ARG, "PagedCache.wrap")
        c = kvq_pages(n, h, cfg.head_dim, t, (ctypes.c_void_p * 2)(*[_ptr(x) for x in codes]),
                      (ctypes.c_void_p * 2)(*[_ptr(x) for x in tok]))
        return cls(c, list(codes), list(tok))

    def snapshot(self) -> dict:
        """A host copy of the pool (checkpoint); the batch's tables and
        lengths are the caller's."""
        return {"codes": [t.cpu() for t in self.codes], "tok": [t.cpu() for t in self.tok]}

    def restore(self, snap: dict) -> None:
        """Load a snapshot taken from a pool of the same shape (resume)."""
        for name in ("codes", "tok"):
            for dst, src in zip(getattr(self, name), snap[name]):
                if dst.shape != src.shape:
                    raise KvqError(KVQ_ERR_INVALID_ARG, "PagedCache.restore: snapshot of another pool shape")
        for name in ("codes", "tok"):
            for dst, src in zip(getattr(self, name), snap[name]):
                dst.copy_(src)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (*self.codes, *self.tok))


class Batch:
    """kvq_batch over int32 device tensors: start [n_seqs + 1], length [n_seqs]
    and the page table [n_seqs, pages] (rows may be further apart than their
    pages, as in a slice of a larger table).  Their contents may change between
    calls, and between a graph's replays."""

    def __init__(self, start, length, table, max_rows: int = 0):
        import torch
        n = length.shape[0]
        ok = all(x.dtype == torch.int32 and x.device == table.device for x in (start, length, table))
        if not ok or start.dim() != 1 or length.dim() != 1 or table.dim() != 2 or start.shape[0] != n + 1 or \
                table.shape[0] != n or (n and not (start.is_contiguous() and length.is_contiguous())) or \
                (table.shape[1] > 1 and table.stride(1) != 1):
            raise KvqError(KVQ_ERR_INVALID_ARG, "Batch")
        self.start, self.length, self.table = start, length, table
        self.device = table.device
        stride = table.stride(0) if n > 1 else table.shape[1]
        self.c = kvq_batch(n, table.shape[1], stride, max_rows, _ptr(start), _ptr(length), _ptr(table))
