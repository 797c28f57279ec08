"""Warps that share a named barrier leave it together when one of them gives up a
wait (a warp that just left would be waited for without a limit)."""

import pytest
import torch

import serving_prefill_b200 as sp
from kv8_support import AttnCase, check

pytestmark = pytest.mark.gpu


def test_warps_of_a_named_barrier_leave_at_one_round():
    """Bit 4 is the waits that gave up; bit 2 would be a warp that left at
    another round. The context stays usable: a step and a prompt follow."""
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for limit_ns in (1, 1000, 1_000_000):
        err.zero_()
        sp.rag.rag_selftest_wait_timeout(err, limit_ns)
        torch.cuda.synchronize()
        assert int(err.item()) == 4
    for n_q in (1, 20):
        case = AttnCase(2, 4, [([300, 77], n_q), ([50], n_q)], seed=n_q)
        check(case.run(), case.reference())
