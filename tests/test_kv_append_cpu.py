"""Refusals of the append entry points, without a GPU: everything the host can
see is rejected before a launch."""

import ctypes

import pytest
import torch

import serving_prefill_b200 as sp
from serving_prefill_b200.rag import RagAppend, RagKV8Pool, RagKVPool, lib

INVALID, SHAPE, UNSUPPORTED = 1, 2, 4


def pool16(dtype=0, head_dim=128, layers=2, heads=8):
    return RagKVPool(0x10000, 0x20000, layers, 64, heads, 16, head_dim, dtype)


def pool8(head_dim=128, page=16, layers=2, pages=64, k=0x10000, ks=0x30000):
    return RagKV8Pool(k, 0x20000, ks, 0x40000, layers, pages, 8, page, head_dim)


def seqs(n=2, total=10, pages=4, tok=0x1000, start=0x2000, po=0x3000, pid=0x4000, pos0=None):
    return RagAppend(n, total, pages, tok, start, po, pid, pos0)


def call(pool, s, fn=None, layer=0, k=0x50000, ks=1024, v=0x60000, vs=1024, rope=0x70000, n_pos=100, q=0x80000,
         qs=4096, hq=32, q_out=0x200000, err=None):
    fn = fn or (lib().rag_kv8_append if isinstance(pool, RagKV8Pool) else lib().rag_kv_append)
    return fn(ctypes.byref(pool) if pool is not None else None, layer, ctypes.byref(s) if s is not None else None, k, ks,
              v, vs, rope, n_pos, q, qs, hq, q_out, err, None)


@pytest.mark.parametrize("pool", [pool16(), pool8()], ids=["bf16", "e4m3"])
def test_arguments_are_refused_before_a_launch(pool):
    assert call(pool, None) == INVALID
    for bad in (dict(layer=2), dict(layer=-1), dict(k=None), dict(v=None), dict(k=0x50008), dict(v=0x60004),
                dict(rope=0x70008), dict(q=0x80004), dict(q_out=0x200008), dict(q_out=None), dict(q=None),
                dict(n_pos=0), dict(ks=1028), dict(vs=1025), dict(qs=4100), dict(q=0x80000, q_out=0x80000, qs=6144)):
        assert call(pool, seqs(), **bad) == INVALID, bad
    for bad in (dict(ks=1016), dict(vs=0), dict(qs=4088), dict(hq=0)):
        assert call(pool, seqs(), **bad) == SHAPE, bad
    for s in (seqs(tok=None), seqs(start=None), seqs(po=None), seqs(pid=None)):
        assert call(pool, s) == INVALID
    for s in (seqs(n=-1), seqs(total=-1), seqs(pages=-1)):
        assert call(pool, s) == SHAPE
    assert call(pool, seqs(n=65537)) == UNSUPPORTED


@pytest.mark.parametrize("pool", [pool16(), pool8(), pool16(dtype=1, head_dim=64)], ids=["bf16", "e4m3", "f32"])
def test_an_empty_call_does_nothing(pool):
    assert call(pool, seqs(n=0)) == 0
    assert call(pool, seqs(total=0)) == 0


def test_pools_are_checked():
    assert call(None, seqs(), fn=lib().rag_kv8_append) == INVALID
    assert call(None, seqs(), fn=lib().rag_kv_append) == INVALID
    assert call(pool8(head_dim=64), seqs()) == UNSUPPORTED
    assert call(pool8(page=32), seqs()) == UNSUPPORTED
    assert call(pool8(k=0x10001), seqs()) == INVALID
    assert call(pool8(ks=None), seqs()) == INVALID
    assert call(pool8(ks=0x30002), seqs()) == INVALID
    assert call(pool8(layers=0), seqs()) == SHAPE
    assert call(pool8(layers=1 << 12, pages=1 << 12), seqs()) == UNSUPPORTED   # 2^27 page blocks
    assert call(pool16(head_dim=64), seqs()) == UNSUPPORTED                    # bf16 needs head_dim 128


def test_outputs_that_overlap_inputs_are_refused():
    """10 tokens: rows of 8 KB of queries, 2 KB of k at 0x50000 and of v at 0x60000."""
    for out in (0x80000 + 16, 0x80000 - 16, 0x80000 + 10 * 8192 - 16,
                0x50000, 0x50000 + 9 * 2048, 0x60000 - 10 * 8192 + 16):
        assert call(pool8(), seqs(), q_out=out) == INVALID, hex(out)
    assert call(pool8(), seqs(), err=0x400002) == INVALID
    assert attend(pool8(), batch(), q=0x400000, o=0x400000) == INVALID
    assert attend(pool8(), batch(), q=0x400000, o=0x400000 + 30 * 32 * 256 - 16) == INVALID


def test_binding_checks_the_error_word_and_the_table():
    pool = sp.KV8Pool(1, 4, 2, device="cpu")
    s = sp.Append([0, 3], [0], [0, 1], [2], device="cpu")
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    for err in (torch.zeros(1), torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(sp.RagError) as e:
            sp.rag_kv8_append(pool, 0, s, k, k, device_err=err)
        assert e.value.status == INVALID
    with pytest.raises(sp.RagError) as e:
        sp.rag_kv8_append(pool, 0, s, k, k, rope=torch.zeros(0, 64, 2))   # no table is rope=None
    assert e.value.status == SHAPE


def test_table_of_rotations_is_checked():
    f = lib().rag_rope_cos_sin
    assert f(1.0, 128, 10, 0x1000, None) == INVALID
    assert f(float("inf"), 128, 10, 0x1000, None) == INVALID
    assert f(1e4, 128, 10, None, None) == INVALID
    assert f(1e4, 128, 10, 0x1008, None) == INVALID
    assert f(1e4, 128, -1, 0x1000, None) == INVALID
    assert f(1e4, 96, 10, 0x1000, None) == UNSUPPORTED
    assert f(1e4, 128, 0, 0x1000, None) == 0


def test_append_arrays_are_checked():
    with pytest.raises(ValueError):
        sp.Append([0, 1], [0, 0], [0, 1], [0], device="cpu")
    with pytest.raises(ValueError):
        sp.Append([0, 1], [0], [0, 1], [0], pos0=[1, 2], device="cpu")
    with pytest.raises(ValueError):
        sp.Append(torch.tensor([[0, 1]]).int(), [0], [0, 1], [0], total_new=1, device="cpu")
    a = sp.Append([0, 3, 7], [0, 5], [0, 1, 2], [4, 9], device="cpu")
    assert (a.c.n_seqs, a.total_new, a.c.total_pages, a.c.pos0) == (2, 7, 2, None)


def test_binding_checks_shapes_types_and_strides():
    pool = sp.KV8Pool(1, 4, 2, device="cpu")
    s = sp.Append([0, 3], [0], [0, 1], [2], device="cpu")
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    for bad in (k[:2], k[:, :1], k[:, :, :64], k.float(), torch.zeros(3, 128, 2, dtype=torch.bfloat16).transpose(1, 2)):
        with pytest.raises(sp.RagError):
            sp.rag_kv8_append(pool, 0, s, bad, k)
        with pytest.raises(sp.RagError):
            sp.rag_kv8_append(pool, 0, s, k, bad)
    with pytest.raises(sp.RagError):
        sp.rag_kv8_append(pool, 0, s, k, k, q=k)                              # no q_out
    with pytest.raises(sp.RagError):
        sp.rag_kv8_append(pool, 0, s, k, k, rope=torch.zeros(5, 32, 2))       # a table of another head_dim
    with pytest.raises(AssertionError):
        sp.KV8Pool(1, 4, 2, device="cpu", k=torch.zeros(1, 4, 2, 16, 128))


# ---------------------------------------------------------------- attention over the 8-bit pool

from serving_prefill_b200.rag import RagBatch  # noqa: E402

WORKSPACE = 7


def batch(B=2, q=(10, 20), docs=(100, 50)):
    pages = [-(-d // 16) for d in docs]
    return RagBatch(B, B, sum(pages), sum(q), sum(docs), max(q), max(docs), max(pages),
                    0x30000, 0x31000, 0x32000, 0x33000, 0x34000)


def attend(pool, b, hq=32, layer=0, q=0x40000, o=0x100000, lse=None, ws=0x80000, ws_bytes=1 << 40, scale=0.0, causal=1):
    return lib().rag_kv8_attn(ctypes.byref(pool), layer, ctypes.byref(b) if b is not None else None, q, hq, scale,
                              causal, o, lse, ws, ws_bytes, None)


def test_attention_refuses_before_a_launch():
    assert attend(pool8(), None) == INVALID
    for bad in (dict(layer=-1), dict(layer=2), dict(q=None), dict(o=None), dict(q=0x40008), dict(o=0x70004),
                dict(lse=0x90002), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert attend(pool8(), batch(), **bad) == INVALID, bad
    assert attend(pool8(), batch(), hq=30) == SHAPE
    assert attend(pool8(), batch(), hq=0) == SHAPE
    assert attend(pool8(), batch(), hq=8 * 129) == UNSUPPORTED       # more than 128 query heads a KV head
    assert attend(pool8(head_dim=64), batch()) == UNSUPPORTED
    assert attend(pool8(page=8), batch()) == UNSUPPORTED
    for bad in (dict(ws=None), dict(ws=0x80080), dict(ws_bytes=4096)):
        assert attend(pool8(), batch(), **bad) == WORKSPACE, bad
    many = batch()
    many.num_requests = 4097
    assert attend(pool8(), many) == UNSUPPORTED
    over = batch()
    over.max_q = 31                                                   # above the total
    assert attend(pool8(), over) == SHAPE
    huge = batch(q=(1 << 24, 1 << 24), docs=(1 << 24, 1 << 24))       # weights past 31 bits
    assert attend(pool8(), huge) == UNSUPPORTED


def test_attention_of_no_queries_does_nothing():
    assert attend(pool8(), batch(B=0, q=(0, 0), docs=(0, 0)), q=None, o=None) == 0
    assert attend(pool8(), batch(q=(0, 0)), q=None, o=None) == 0


def test_attention_workspace_size():
    size = lambda b, hq=32: lib().rag_kv8_workspace_size(ctypes.byref(pool8()), ctypes.byref(b), hq)  # noqa: E731
    assert size(batch(), hq=30) == 0 and size(batch(), hq=8 * 129) == 0
    assert 256 <= size(batch(q=(1, 1), docs=(30, 20))) <= 4096         # short requests: no partial rows
    assert size(batch(q=(1, 1), docs=(3000, 2000))) < size(batch(q=(100, 100), docs=(3000, 2000)))
    need = size(batch(docs=(3000, 2000)))
    assert attend(pool8(), batch(docs=(3000, 2000)), ws_bytes=need - 1) == WORKSPACE


def test_attention_binding_checks():
    pool = sp.KV8Pool(1, 8, 2, device="cpu")
    b = sp.Batch([0, 1], [0, 40], [0, 3], [1, 2, 3], [0, 4], device="cpu")
    q, ws = torch.zeros(4, 8, 128, dtype=torch.bfloat16), torch.zeros(1 << 20, dtype=torch.uint8)
    o = torch.empty_like(q)
    for bad in (q[:3], q[:, :, :64], q.float(), q[0], torch.zeros(4, 128, 8, dtype=torch.bfloat16).transpose(1, 2)):
        with pytest.raises(sp.RagError):
            sp.rag_kv8_attn(pool, 0, b, bad, o, ws)
    for bad in (o[:3], o.float()):
        with pytest.raises(sp.RagError):
            sp.rag_kv8_attn(pool, 0, b, q, bad, ws)
    for lse in (torch.zeros(4, 7), torch.zeros(4, 8, dtype=torch.bfloat16)):
        with pytest.raises(sp.RagError):
            sp.rag_kv8_attn(pool, 0, b, q, o, ws, row_lse=lse)
