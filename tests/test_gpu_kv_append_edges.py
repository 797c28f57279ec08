"""Appends at the edges of what the descriptors may say."""

import numpy as np
import pytest
import torch

import serving_prefill_b200 as sp
from test_gpu_kv_append import Case

pytestmark = pytest.mark.gpu

TOP = (1 << 31) - 1


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32"])
def test_a_sequence_of_two_billion_tokens(kind):
    """A page table of 2^27 + 2 entries. Tokens up to number 2^31 - 2 are stored
    (at a position that pos0 brings into the table); a call that would go past
    2^31 - 1 tokens is reported and stores nothing (token numbers are 32 bits)."""
    case = Case(kind, [0], [40], seed=1)
    pages = torch.zeros((1 << 27) + 2, dtype=torch.int32, device="cuda")
    last = (TOP - 20) // 16
    pages[last:last + 3] = torch.tensor(case.seqs[0][0], dtype=torch.int32)
    fn = sp.rag_kv8_append if kind == "e4m3" else sp.rag_kv_append

    def call(start, n):
        s = sp.Append([0, n], [start], [0, pages.numel()], pages, pos0=[-start])
        fn(case.pool, 1, s, case.k[:n], case.v[:n], rope=case.rope, q=case.q[:n], q_out=case.q_out[:n],
           device_err=case.err)
        torch.cuda.synchronize()
        return int(case.err.item())

    before = case.state()
    q0 = case.q_out.clone()
    for start, n in ((TOP - 10, 20), (TOP, 1), (TOP - 19, 20)):
        case.err.zero_()
        assert call(start, n) == 2, (start, n)
        for a, b in zip(case.state(), before):
            assert a is None or np.array_equal(a, b)
        assert not case.q_out[:n].any()
    case.q_out.copy_(q0)
    case.err.zero_()
    assert call(TOP - 20, 20) == 0
    # the same tokens as a short sequence whose first token has the same slot
    other = Case(kind, [0], [40], seed=1)
    slot = (TOP - 20) % 16
    s = sp.Append([0, 20], [slot], [0, 3], other.seqs[0][0], pos0=[-slot])
    fn(other.pool, 1, s, other.k[:20], other.v[:20], rope=other.rope, q=other.q[:20], q_out=other.q_out[:20],
       device_err=other.err)
    torch.cuda.synchronize()
    assert int(other.err.item()) == 0
    for a, b in zip(case.state(), other.state()):
        assert a is None or np.array_equal(a, b)
    assert torch.equal(case.q_out, other.q_out)


@pytest.mark.parametrize("kind,H,total", [("bf16", 2, 30), ("e4m3", 2, 30), ("e4m3", 32, 700)])
@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("t0", [1, 5, 15, 16, 20])
def test_rows_before_the_first_sequences_are_reported(kind, H, total, with_q, t0):
    """tok_off that does not begin at 0: the rows before it belong to no sequence.
    They are reported, not stored, and their rows of q_out are zero; the sequence
    itself is stored. (700 tokens of 32 heads take the streamed kernel.)"""
    case = Case(kind, [0], [total], H=H, G=1, seed=2)
    fn = sp.rag_kv8_append if kind == "e4m3" else sp.rag_kv_append
    pages = case.seqs[0][0]
    q = dict(q=case.q, q_out=case.q_out) if with_q else {}
    s = sp.Append([t0, total], [0], [0, len(pages)], pages, total_new=total)
    fn(case.pool, 1, s, case.k, case.v, rope=case.rope, device_err=case.err, **q)
    torch.cuda.synchronize()
    assert int(case.err.item()) == 2
    if with_q:
        assert not case.q_out[:t0].any() and case.q_out[t0:].any(-1).all()
    other = Case(kind, [0], [total], H=H, G=1, seed=2)
    s = sp.Append([0, total - t0], [0], [0, len(pages)], pages)
    fn(other.pool, 1, s, other.k[t0:], other.v[t0:], rope=other.rope)
    torch.cuda.synchronize()
    for a, b in zip(case.state(), other.state()):
        assert a is None or np.array_equal(a, b)


def test_what_the_binding_allocates_belongs_to_the_stream_that_writes_it():
    """The current stream still has a write to a freed block ahead of it; a table
    (and a workspace) made on another stream must not take that block."""
    n_pos = 1 << 16
    want = sp.rag_rope_cos_sin(10000.0, 128, n_pos)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    pool = sp.KVPool(1, 4, 2, 128)
    b = sp.Batch([0, 1], [0, 40], [0, 3], [0, 1, 2], [0, 4])
    size = sp.rag_workspace_size(pool, b, 8)
    torch.cuda.empty_cache()
    for make, nbytes in ((lambda: sp.rag_rope_cos_sin(10000.0, 128, n_pos, stream=side), want.nbytes),
                         (lambda: sp.new_workspace(pool, b, 8, stream=side), size)):
        block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(200_000_000)                       # about 0.1 s
        block.fill_(0x55)
        at = block.data_ptr()
        del block
        made = make()
        assert made.data_ptr() != at
        torch.cuda.synchronize()
        if made.dtype == torch.float32:
            assert torch.equal(made, want)
        else:
            assert not made[:4].any()                        # the error word
