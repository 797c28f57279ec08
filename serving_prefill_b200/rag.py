"""Python binding of the C ABI in include/rag_prefill.h (ctypes).

Argument marshalling only: every step of the hot path runs in the CUDA
kernels of librag.so. Tensors are torch CUDA tensors owned by the caller;
calls are asynchronous on the current torch stream unless one is passed.
There is no CPU fallback: loading fails loudly when librag.so is missing.
"""

from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_double, c_float, c_int32, c_int64, c_size_t, c_void_p

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "librag.so")

RAG_BF16, RAG_F32 = 0, 1
PAGE_SIZE = 16
KERNEL_KINDS = ("pool_write", "attn", "combine", "impact", "topk", "simt_attn", "simt_impact", "rc_plan", "rc_copy",
                "rc_gemm", "rope_table", "kv_decode", "attn_dec", "kv_append", "kv8_append", "rope_cos_sin",
                "kv8_attn", "kv8_combine", "kv8_split_q", "kv8_attn_dec", "rope_q")

STATUS = {
    0: "ok", 1: "invalid argument", 2: "inconsistent shape", 3: "page id outside the pool",
    4: "unsupported configuration", 5: "CUDA runtime error", 6: "device pipeline wait timed out",
    7: "workspace missing or too small", 8: "chunk page count does not match its length",
    9: "a V value beyond the fp16 range was saturated",
    10: "too few free pages for the copy-on-write recompute",
}


class RagError(RuntimeError):
    def __init__(self, status: int, where: str):
        detail = ""
        if status == 5 and _lib is not None:
            detail = f", {_lib.rag_last_cuda_error().decode()}"
        super().__init__(f"{where}: {STATUS.get(status, 'unknown')} (status {status}{detail})")
        self.status = status


class RagKVPool(ctypes.Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("num_layers", c_int32), ("num_pages", c_int32),
                ("num_kv_heads", c_int32), ("page_size", c_int32), ("head_dim", c_int32), ("dtype", c_int32)]


class RagBatch(ctypes.Structure):
    _fields_ = [("num_requests", c_int32), ("num_chunks", c_int32), ("num_page_refs", c_int32),
                ("total_q", c_int32), ("total_doc", c_int32), ("max_q", c_int32), ("max_doc", c_int32),
                ("max_pages", c_int32), ("req_chunk_off", c_void_p), ("chunk_doc_off", c_void_p),
                ("chunk_page_off", c_void_p), ("page_ids", c_void_p), ("q_off", c_void_p)]


class RagKV8Pool(ctypes.Structure):
    _fields_ = [("k", c_void_p), ("v", c_void_p), ("k_scale", c_void_p), ("v_scale", c_void_p),
                ("num_layers", c_int32), ("num_pages", c_int32), ("num_kv_heads", c_int32), ("page_size", c_int32),
                ("head_dim", c_int32)]


class RagAppend(ctypes.Structure):
    _fields_ = [("n_seqs", c_int32), ("total_new", c_int32), ("total_pages", c_int32), ("tok_off", c_void_p),
                ("start", c_void_p), ("page_off", c_void_p), ("page_ids", c_void_p), ("pos0", c_void_p)]


_lib = None

_APPEND_ARGS = [c_int32, POINTER(RagAppend), c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int32, c_void_p,
                c_int64, c_int32, c_void_p, c_void_p, c_void_p]

EXPORTS = {
    "rag_abi_version": (c_int32, []),
    "rag_status_string": (ctypes.c_char_p, [c_int32]),
    "rag_num_sms": (c_int32, []),
    "rag_kv_pool_write": (c_int32, [POINTER(RagKVPool), c_int32, c_void_p, c_int32, c_int32, c_void_p, c_void_p,
                                    c_void_p, c_void_p]),
    "rag_workspace_size": (c_size_t, [POINTER(RagKVPool), POINTER(RagBatch), c_int32]),
    "rag_workspace_init": (c_int32, [c_void_p, c_size_t, c_void_p]),
    "rag_fused_prefill_attn": (c_int32, [POINTER(RagKVPool), c_int32, POINTER(RagBatch), c_void_p, c_int32,
                                         c_void_p, c_void_p, c_float, c_void_p, c_void_p, c_void_p, c_void_p,
                                         c_size_t, c_void_p]),
    "rag_fused_prefill_attn_rope": (c_int32, [POINTER(RagKVPool), c_int32, POINTER(RagBatch), c_void_p, c_int32,
                                              c_void_p, c_void_p, c_float, c_double, c_void_p, c_void_p, c_void_p,
                                              c_void_p, c_size_t, c_void_p]),
    "rag_fused_prefill_attn_static": (c_int32, [POINTER(RagKVPool), c_int32, POINTER(RagBatch), c_void_p,
                                                c_int32, c_void_p, c_void_p, c_float, c_void_p, c_void_p,
                                                c_void_p, c_void_p, c_void_p]),
    "rag_recompute_count": (c_int32, [c_int32, c_double]),
    "rag_impact_topk": (c_int32, [c_void_p, POINTER(RagBatch), c_double, c_int32, c_void_p, c_void_p, c_void_p,
                                  c_void_p]),
    "rag_last_device_error": (c_int32, [c_void_p, c_void_p, c_void_p]),
    "rag_selftest_wait_timeout": (c_int32, [c_void_p, c_int64, c_void_p]),
    "rag_kv_decode": (c_int32, [POINTER(RagKVPool), c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_int32, c_int32,
                                c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p]),
    "rag_rope_cos_sin": (c_int32, [c_double, c_int32, c_int32, c_void_p, c_void_p]),
    "rag_kv_append": (c_int32, [POINTER(RagKVPool)] + _APPEND_ARGS),
    "rag_kv8_append": (c_int32, [POINTER(RagKV8Pool)] + _APPEND_ARGS),
    "rag_kv8_workspace_size": (c_size_t, [POINTER(RagKV8Pool), POINTER(RagBatch), c_int32]),
    "rag_kv8_attn": (c_int32, [POINTER(RagKV8Pool), c_int32, POINTER(RagBatch), c_void_p, c_int32, c_float, c_int32,
                               c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]),
    "rag_recompute_plan_size": (c_size_t, [POINTER(RagBatch), c_int32]),
    "rag_recompute_plan": (c_int32, [POINTER(RagBatch), c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_int32,
                                     c_void_p, c_void_p, c_size_t, c_void_p]),
    "rag_recompute_kv": (c_int32, [POINTER(RagKVPool), c_int32, POINTER(RagBatch), c_int32, c_void_p, c_size_t,
                                   c_void_p, c_int64, c_int32, c_void_p, c_void_p, c_void_p]),
    "rag_recompute_status": (c_int32, [c_void_p, c_void_p, c_void_p]),
    "rag_launch_count": (c_int64, []),
    "rag_last_cuda_error": (ctypes.c_char_p, []),
    "rag_profile_enable": (None, [c_int32]),
    "rag_profile_collect": (c_int32, [c_void_p, c_void_p, c_int32]),
    "rag_profile_peek": (c_int32, [c_void_p, c_void_p, c_int32]),
}


def lib():
    """The loaded librag.so (raises when it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m serving_prefill_b200.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _ptr(t):
    return None if t is None else c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return c_void_p(stream.cuda_stream)


def _check(status: int, where: str):
    if status != 0:
        raise RagError(status, where)


# --------------------------------------------------------------------------- pool

class KVPool:
    """The paged pool [layers][pages][kv_heads][16][head_dim] for K and V. A
    bf16 cache keeps K in bf16 and V in fp16 (the type V enters the product
    with the attention weights in; rag_kv_pool_write and the decode and
    recompute kernels store it so)."""

    def __init__(self, num_layers, num_pages, num_kv_heads, head_dim, dtype=torch.bfloat16, device="cuda",
                 k=None, v=None):
        shape = (num_layers, num_pages, num_kv_heads, PAGE_SIZE, head_dim)
        v_dtype = torch.float16 if dtype == torch.bfloat16 else dtype
        self.k = torch.zeros(shape, dtype=dtype, device=device) if k is None else k
        self.v = torch.zeros(shape, dtype=v_dtype, device=device) if v is None else v
        assert tuple(self.k.shape) == shape and tuple(self.v.shape) == shape
        assert self.k.dtype == dtype and self.v.dtype == v_dtype
        self.c = RagKVPool(self.k.data_ptr(), self.v.data_ptr(), num_layers, num_pages, num_kv_heads, PAGE_SIZE,
                           head_dim, RAG_BF16 if dtype == torch.bfloat16 else RAG_F32)
        self.ref, self.heads, self.dim, self.dev = ctypes.byref(self.c), num_kv_heads, head_dim, self.k.get_device()

    @property
    def num_kv_heads(self):
        return self.c.num_kv_heads


class KV8Pool:
    """The paged pool held in 8 bits: e4m3 codes [layers][pages][kv_heads][16][128]
    for K and V, and one fp32 scale [layers][pages][kv_heads] for each (value =
    code * scale). rag_kv8_append writes it, rag_kv8_attn reads it."""

    def __init__(self, num_layers, num_pages, num_kv_heads, head_dim=128, device="cuda", k=None, v=None,
                 k_scale=None, v_scale=None):
        shape = (num_layers, num_pages, num_kv_heads, PAGE_SIZE, head_dim)
        dt = torch.float8_e4m3fn
        self.k = torch.zeros(shape, dtype=dt, device=device) if k is None else k
        self.v = torch.zeros(shape, dtype=dt, device=device) if v is None else v
        self.k_scale = torch.ones(shape[:3], device=device) if k_scale is None else k_scale
        self.v_scale = torch.ones(shape[:3], device=device) if v_scale is None else v_scale
        for t, sh, d in ((self.k, shape, dt), (self.v, shape, dt), (self.k_scale, shape[:3], torch.float32),
                         (self.v_scale, shape[:3], torch.float32)):
            assert tuple(t.shape) == sh and t.dtype == d and t.is_contiguous() and t.device == self.k.device
        self.c = RagKV8Pool(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
                            num_layers, num_pages, num_kv_heads, PAGE_SIZE, head_dim)
        self.ref, self.heads, self.dim, self.dev = ctypes.byref(self.c), num_kv_heads, head_dim, self.k.get_device()

    @property
    def num_kv_heads(self):
        return self.c.num_kv_heads


# --------------------------------------------------------------------------- batch

class Batch:
    """Batch descriptor: device int32 arrays plus host totals and maxima."""

    def __init__(self, req_chunk_off, chunk_doc_off, chunk_page_off, page_ids, q_off, device="cuda"):
        h = [torch.as_tensor(x, dtype=torch.int32).cpu() for x in
             (req_chunk_off, chunk_doc_off, chunk_page_off, page_ids, q_off)]
        self.host = h
        rc, cd, cp, pid, qo = h
        B = len(rc) - 1
        docs = [int(cd[rc[b + 1]] - cd[rc[b]]) for b in range(B)]
        pages = [int(cp[rc[b + 1]] - cp[rc[b]]) for b in range(B)]
        qs = [int(qo[b + 1] - qo[b]) for b in range(B)]
        self.dev = [t.to(device) if t.numel() > 0 else torch.zeros(1, dtype=torch.int32, device=device) for t in h]
        self.c = RagBatch(B, len(cd) - 1, len(pid), int(qo[-1]) if B else 0, int(cd[-1]) if len(cd) else 0,
                          max(qs, default=0), max(docs, default=0), max(pages, default=0),
                          *[t.data_ptr() for t in self.dev])
        self.doc_lens, self.q_lens = docs, qs
        self.ref = ctypes.byref(self.c)

    @property
    def num_requests(self):
        return self.c.num_requests

    @property
    def total_q(self):
        return self.c.total_q

    @property
    def total_doc(self):
        return self.c.total_doc


class Append:
    """Which sequences one append call grows (rag_append): int32 arrays, moved to
    the device if they are not there yet. total_new bounds the rows of k, v and
    q (the last entry of tok_off when that is on the host and total_new is not
    given)."""

    def __init__(self, tok_off, start, page_off, page_ids, pos0=None, total_new=None, device="cuda"):
        if total_new is None:
            if isinstance(tok_off, torch.Tensor) and tok_off.is_cuda:
                raise ValueError("total_new is needed when tok_off is on the device")
            total_new = int(tok_off[-1])

        def dev(x):
            t = torch.as_tensor(x, dtype=torch.int32)
            t = t if t.is_cuda else t.to(device)
            if t.dim() != 1 or not t.is_contiguous():
                raise ValueError("the arrays of an Append are one-dimensional and contiguous")
            return t if t.numel() else torch.zeros(1, dtype=torch.int32, device=t.device)

        n, n_pages = len(start), len(page_ids)
        if len(tok_off) != n + 1 or len(page_off) != n + 1 or (pos0 is not None and len(pos0) != n):
            raise ValueError("tok_off and page_off have one entry more than start, pos0 as many")
        self.dev = [dev(x) for x in (tok_off, start, page_off, page_ids)] + [None if pos0 is None else dev(pos0)]
        self.c = RagAppend(n, total_new, n_pages, *[None if t is None else t.data_ptr() for t in self.dev])
        self.ref, self.total_new, self.dev_index = ctypes.byref(self.c), total_new, self.dev[0].get_device()
        if any(t is not None and t.get_device() != self.dev_index for t in self.dev):
            raise ValueError("the arrays of an Append are on one device")


# --------------------------------------------------------------------------- entry points

def rag_abi_version() -> int:
    return lib().rag_abi_version()


def rag_num_sms() -> int:
    return lib().rag_num_sms()


def rag_recompute_count(n_doc: int, r: float) -> int:
    return lib().rag_recompute_count(n_doc, r)


def rag_kv_pool_write(pool: KVPool, layer: int, page_ids: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                      device_err: torch.Tensor = None, stream=None):
    n_tokens = k.shape[0]
    _check(lib().rag_kv_pool_write(ctypes.byref(pool.c), layer, _ptr(page_ids), page_ids.numel(), n_tokens,
                                   _ptr(k), _ptr(v), _ptr(device_err), _stream(stream)), "rag_kv_pool_write")


def rag_workspace_size(pool: KVPool, batch: Batch, num_q_heads: int) -> int:
    n = lib().rag_workspace_size(ctypes.byref(pool.c), ctypes.byref(batch.c), num_q_heads)
    if n == 0:
        raise RagError(1, "rag_workspace_size")
    return n


def rag_kv8_workspace_size(pool: KV8Pool, batch: Batch, num_q_heads: int) -> int:
    n = lib().rag_kv8_workspace_size(ctypes.byref(pool.c), ctypes.byref(batch.c), num_q_heads)
    if n == 0:
        raise RagError(1, "rag_kv8_workspace_size")
    return n


def new_workspace(pool, batch: Batch, num_q_heads: int, device="cuda", stream=None) -> torch.Tensor:
    """Workspace for rag_fused_prefill_attn (a KVPool) or rag_kv8_attn (a KV8Pool)."""
    size = rag_kv8_workspace_size if isinstance(pool, KV8Pool) else rag_workspace_size
    n = size(pool, batch, num_q_heads)
    with torch.cuda.stream(stream):   # its memory may still be in use on another one
        ws = torch.empty(n, dtype=torch.uint8, device=device)
    _check(lib().rag_workspace_init(_ptr(ws), n, _stream(stream)), "rag_workspace_init")
    return ws


def rag_fused_prefill_attn(pool: KVPool, layer: int, batch: Batch, q: torch.Tensor, kq: torch.Tensor,
                           vq: torch.Tensor, o: torch.Tensor, workspace: torch.Tensor, impact: torch.Tensor = None,
                           row_lse: torch.Tensor = None, sm_scale: float = 0.0, stream=None):
    num_q_heads = q.shape[1] if q.dim() == 3 else 0
    _check(lib().rag_fused_prefill_attn(ctypes.byref(pool.c), layer, ctypes.byref(batch.c), _ptr(q), num_q_heads,
                                        _ptr(kq), _ptr(vq), sm_scale, _ptr(o), _ptr(row_lse), _ptr(impact),
                                        _ptr(workspace), workspace.numel(), _stream(stream)),
           "rag_fused_prefill_attn")


def rag_fused_prefill_attn_rope(pool: KVPool, layer: int, batch: Batch, q: torch.Tensor, kq: torch.Tensor,
                                vq: torch.Tensor, o: torch.Tensor, workspace: torch.Tensor, rope_base: float,
                                impact: torch.Tensor = None, row_lse: torch.Tensor = None, sm_scale: float = 0.0,
                                stream=None):
    num_q_heads = q.shape[1] if q.dim() == 3 else 0
    _check(lib().rag_fused_prefill_attn_rope(ctypes.byref(pool.c), layer, ctypes.byref(batch.c), _ptr(q),
                                             num_q_heads, _ptr(kq), _ptr(vq), sm_scale, rope_base, _ptr(o),
                                             _ptr(row_lse), _ptr(impact), _ptr(workspace), workspace.numel(),
                                             _stream(stream)), "rag_fused_prefill_attn_rope")


def rag_fused_prefill_attn_static(pool: KVPool, layer: int, batch: Batch, q: torch.Tensor, kq: torch.Tensor,
                                  vq: torch.Tensor, o: torch.Tensor, impact: torch.Tensor = None,
                                  row_lse: torch.Tensor = None, device_err: torch.Tensor = None,
                                  sm_scale: float = 0.0, stream=None):
    """rag_fused_prefill_attn without a workspace: for callers that cannot
    allocate device memory; scratch is the library's fixed 64 MiB device array."""
    num_q_heads = q.shape[1] if q.dim() == 3 else 0
    _check(lib().rag_fused_prefill_attn_static(ctypes.byref(pool.c), layer, ctypes.byref(batch.c), _ptr(q),
                                               num_q_heads, _ptr(kq), _ptr(vq), sm_scale, _ptr(o), _ptr(row_lse),
                                               _ptr(impact), _ptr(device_err), _stream(stream)),
           "rag_fused_prefill_attn_static")


def rag_impact_topk(impact: torch.Tensor, batch: Batch, r: float, k_cap: int, topk_idx: torch.Tensor,
                    topk_val: torch.Tensor = None, k_out: torch.Tensor = None, stream=None):
    _check(lib().rag_impact_topk(_ptr(impact), ctypes.byref(batch.c), r, k_cap, _ptr(topk_idx), _ptr(topk_val),
                                 _ptr(k_out), _stream(stream)), "rag_impact_topk")


def rag_last_device_error(workspace: torch.Tensor, stream=None) -> tuple:
    bits = c_int32(0)
    st = lib().rag_last_device_error(_ptr(workspace), ctypes.byref(bits), _stream(stream))
    return st, bits.value


def rag_selftest_wait_timeout(device_err: torch.Tensor, limit_ns: int, stream=None):
    _check(lib().rag_selftest_wait_timeout(_ptr(device_err), limit_ns, _stream(stream)),
           "rag_selftest_wait_timeout")


def rag_kv_decode(pool: KVPool, layer: int, chunk_tok_off: torch.Tensor, chunk_page_off: torch.Tensor,
                  page_ids: torch.Tensor, bits: int, codes_k: torch.Tensor, codes_v: torch.Tensor,
                  scale_k: torch.Tensor, offset_k: torch.Tensor, scale_v: torch.Tensor, offset_v: torch.Tensor,
                  device_err: torch.Tensor = None, stream=None):
    _check(lib().rag_kv_decode(ctypes.byref(pool.c), layer, chunk_tok_off.numel() - 1, _ptr(chunk_tok_off),
                               _ptr(chunk_page_off), _ptr(page_ids), page_ids.numel(), bits, _ptr(codes_k),
                               _ptr(codes_v), _ptr(scale_k), _ptr(offset_k), _ptr(scale_v), _ptr(offset_v),
                               _ptr(device_err), _stream(stream)), "rag_kv_decode")


def _on(dev: int, stream) -> int:
    """The stream to launch on (its handle): the one given, or the current one of
    device `dev`, where the tensors are. The library launches on the current
    device, so it has to be that one."""
    if dev != torch._C._cuda_getDevice():
        raise RagError(1, f"the tensors are on device {dev}, the current one is {torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def rag_rope_cos_sin(base: float, head_dim: int, n_pos: int, device="cuda", stream=None) -> torch.Tensor:
    """Table of rotations [n_pos][head_dim / 2][2] = (cos, sin) of p * base^(-2j/head_dim).
    Allocated, like everything torch makes, for the stream that writes it."""
    with torch.cuda.stream(stream):
        table = torch.empty(max(n_pos, 1), max(head_dim, 2) // 2, 2, device=device)
    _check(lib().rag_rope_cos_sin(base, head_dim, n_pos, _ptr(table), _on(table.get_device(), stream)),
           "rag_rope_cos_sin")
    return table[:n_pos]


def _row_stride(t, rows, heads, dim, dtype, dev, where) -> int:
    """Elements between the token rows of t [>= rows][heads][dim], each row dense."""
    try:
        n, h, d = t.shape
    except ValueError:
        raise RagError(2, where) from None
    if n < rows or h != heads or d != dim:
        raise RagError(2, where)
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != d and h != 1) or t.dtype is not dtype or t.get_device() != dev:
        raise RagError(1, where)
    return s0 if n > 1 else max(s0, h * d)


def _append(fn, where, pool, dtype, layer, seqs, k, v, rope, q, q_out, device_err, stream):
    rows, heads, dim, dev = seqs.total_new, pool.heads, pool.dim, pool.dev
    ks = _row_stride(k, rows, heads, dim, dtype, dev, where)
    vs = _row_stride(v, rows, heads, dim, dtype, dev, where)
    qs = hq = n_pos = 0
    qp = op = rp = None
    if q is not None:
        if q_out is None:
            raise RagError(1, where)
        shape = q.shape
        hq = shape[1] if len(shape) == 3 else -1
        qs = _row_stride(q, rows, hq, dim, dtype, dev, where)
        if q_out.shape != shape:
            raise RagError(2, where)
        if q_out.dtype is not dtype or not q_out.is_contiguous() or q_out.get_device() != dev:
            raise RagError(1, where)
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise RagError(1, where)
    if rope is not None:
        shape = rope.shape
        n_pos = shape[0]
        if shape != (n_pos, dim // 2, 2) or n_pos == 0:
            raise RagError(2, where)
        if rope.dtype is not torch.float32 or not rope.is_contiguous() or rope.get_device() != dev:
            raise RagError(1, where)
        rp = rope.data_ptr()
    if seqs.dev_index != dev:
        raise RagError(1, where)
    if device_err is not None and (device_err.dtype is not torch.int32 or device_err.numel() == 0
                                   or device_err.get_device() != dev):
        raise RagError(1, where)
    status = fn(pool.ref, layer, seqs.ref, k.data_ptr(), ks, v.data_ptr(), vs, rp, n_pos, qp, qs, hq, op,
                None if device_err is None else device_err.data_ptr(), _on(dev, stream))
    if status != 0:
        raise RagError(status, where)


def rag_kv_append(pool: KVPool, layer: int, seqs: Append, k: torch.Tensor, v: torch.Tensor, rope: torch.Tensor = None,
                  q: torch.Tensor = None, q_out: torch.Tensor = None, device_err: torch.Tensor = None, stream=None):
    """Append new tokens' k, v [rows][kv_heads][head_dim] (rows may be strided, as
    slices of a fused projection are) to their sequences' pages, K rotated by the
    table's rows; q, if given, is rotated into the dense q_out."""
    _append(lib().rag_kv_append, "rag_kv_append", pool, pool.k.dtype, layer, seqs, k, v, rope, q, q_out, device_err,
            stream)


def rag_kv8_append(pool: KV8Pool, layer: int, seqs: Append, k: torch.Tensor, v: torch.Tensor,
                   rope: torch.Tensor = None, q: torch.Tensor = None, q_out: torch.Tensor = None,
                   device_err: torch.Tensor = None, stream=None):
    """rag_kv_append into an 8-bit pool: bf16 k, v (and q), quantised on the way."""
    _append(lib().rag_kv8_append, "rag_kv8_append", pool, torch.bfloat16, layer, seqs, k, v, rope, q, q_out,
            device_err, stream)


def rag_kv8_attn(pool: KV8Pool, layer: int, batch: Batch, q: torch.Tensor, o: torch.Tensor, workspace: torch.Tensor,
                 causal: bool = True, row_lse: torch.Tensor = None, sm_scale: float = 0.0, stream=None):
    """Attention of the query tokens q [total_q][num_q_heads][128] (bf16) over their
    requests' pages of an 8-bit pool, into o; causal: query token j of n_q sees
    the first N - n_q + j + 1 of the request's N cached tokens."""
    where, dev, hq = "rag_kv8_attn", pool.dev, 0
    if q.dim() == 3:
        n, hq, d = q.shape
    if hq == 0 or d != 128 or n < batch.c.total_q or o.shape != q.shape:
        raise RagError(2, where)
    if (q.dtype != torch.bfloat16 or o.dtype != torch.bfloat16 or not q.is_contiguous() or not o.is_contiguous()
            or q.get_device() != dev or o.get_device() != dev or batch.dev[0].get_device() != dev):
        raise RagError(1, where)
    lp = None
    if row_lse is not None:
        if row_lse.shape != (n, hq):
            raise RagError(2, where)
        if row_lse.dtype != torch.float32 or not row_lse.is_contiguous() or row_lse.get_device() != dev:
            raise RagError(1, where)
        lp = row_lse.data_ptr()
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise RagError(7, where)
    status = lib().rag_kv8_attn(pool.ref, layer, batch.ref, q.data_ptr(), hq, sm_scale, 1 if causal else 0,
                                o.data_ptr(), lp, workspace.data_ptr(), workspace.nbytes, _on(dev, stream))
    if status != 0:
        raise RagError(status, where)


def rag_recompute_plan_size(batch: Batch, k_cap: int) -> int:
    n = lib().rag_recompute_plan_size(ctypes.byref(batch.c), k_cap)
    if n == 0:
        raise RagError(1, "rag_recompute_plan_size")
    return n


def rag_recompute_plan(batch: Batch, topk_idx: torch.Tensor, k_cap: int, k: torch.Tensor, free_pages: torch.Tensor,
                       page_ids_out: torch.Tensor, plan: torch.Tensor, x_by_selection: bool = False, stream=None):
    _check(lib().rag_recompute_plan(ctypes.byref(batch.c), _ptr(topk_idx), k_cap, _ptr(k), _ptr(free_pages),
                                    free_pages.numel(), 1 if x_by_selection else 0, _ptr(page_ids_out), _ptr(plan),
                                    plan.numel() * plan.element_size(), _stream(stream)), "rag_recompute_plan")


def rag_recompute_kv(pool: KVPool, layer: int, batch: Batch, k_cap: int, plan: torch.Tensor, x: torch.Tensor,
                     w_k: torch.Tensor, w_v: torch.Tensor, stream=None):
    _check(lib().rag_recompute_kv(ctypes.byref(pool.c), layer, ctypes.byref(batch.c), k_cap, _ptr(plan),
                                  plan.numel() * plan.element_size(), _ptr(x), x.shape[0], x.shape[1], _ptr(w_k),
                                  _ptr(w_v), _stream(stream)), "rag_recompute_kv")


def rag_recompute_status(plan: torch.Tensor, stream=None) -> tuple:
    counts = (c_int32 * 3)()
    st = lib().rag_recompute_status(_ptr(plan), ctypes.cast(counts, c_void_p), _stream(stream))
    return st, (counts[0], counts[1], counts[2])


def rag_launch_count() -> int:
    return lib().rag_launch_count()


def rag_profile_enable(on: bool):
    lib().rag_profile_enable(1 if on else 0)


def rag_profile_peek() -> dict:
    n = len(KERNEL_KINDS)
    ms = (c_double * n)()
    cnt = (c_int64 * n)()
    _check(lib().rag_profile_peek(ctypes.cast(ms, c_void_p), ctypes.cast(cnt, c_void_p), n), "rag_profile_peek")
    return {k: (ms[i], cnt[i]) for i, k in enumerate(KERNEL_KINDS)}


def rag_profile_collect() -> dict:
    n = len(KERNEL_KINDS)
    ms = (c_double * n)()
    cnt = (c_int64 * n)()
    _check(lib().rag_profile_collect(ctypes.cast(ms, c_void_p), ctypes.cast(cnt, c_void_p), n),
           "rag_profile_collect")
    return {k: (ms[i], cnt[i]) for i, k in enumerate(KERNEL_KINDS)}


def topk_capacity(batch: Batch, r: float) -> int:
    """Row length for the top-k outputs: k of the request with the most doc tokens."""
    return max(1, rag_recompute_count(max(batch.doc_lens, default=0), r))
