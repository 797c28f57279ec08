"""Appends of many sequences in one call: several page units, and several tokens,
a block, and more sequences than one round of the search by a warp."""

import numpy as np
import pytest
import torch

import serving_prefill_b200 as sp
from oracle import append as oa
from test_gpu_kv_append import Case

pytestmark = pytest.mark.gpu

# (starts, new tokens): tokens whose slots coincide, begun pages, sequences of no
# tokens; every one leaves units without a page between units with one
MANY = {
    "2048_single": ([0] * 2048, [1] * 2048),
    "4096_single": ([5] * 4096, [1] * 4096),
    "800_of_64": ([7 * i % 16 for i in range(800)], [64] * 800),
    "600_of_60": ([i % 16 for i in range(600)], [60] * 600),
    "480_of_100": ([i % 16 for i in range(480)], [100] * 480),
    "some_empty": ([3 * i % 33 for i in range(4000)], [0 if i % 3 == 1 else 1 + i % 2 for i in range(4000)]),
}


def many(kind, name, H, G, seed=0):
    starts, news = MANY[name]
    return Case(kind, starts, news, H=H, G=G, seed=seed, n_pos=37 * len(news) + 256)


@pytest.mark.parametrize("name", list(MANY))
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "f32_64"])
def test_bits_are_the_fp32_formulas(kind, name):
    case = many(kind, name, 1, 1, seed=len(name))
    before = case.state()
    case.run()
    after = case.state()
    assert int(case.err.item()) == 0
    q, k, v = case.host
    tab = case.table[case.positions()]
    turn = lambda x: np.stack([oa.rotate(x[t].astype(np.float32), tab[t]) for t in range(case.T)])  # noqa: E731
    k32, q32 = turn(k), turn(q)
    want = [None if x is None else x.copy() for x in before]
    oa.append(want[0], want[1], want[2], want[3], case.seqs, k32.astype(np.float64), v, None)
    for i in range(4):
        if want[i] is None:
            continue
        if kind == "e4m3" and i < 2:
            want[i] = oa.to_e4m3(want[i])
        elif i == 0:
            want[i] = torch.from_numpy(want[i]).float().to(case.dt).double().numpy()
        elif kind == "bf16":
            want[i] = torch.from_numpy(want[i]).half().double().numpy()
        np.testing.assert_array_equal(after[i], want[i])
    np.testing.assert_array_equal(case.q_out[:case.T].double().cpu().numpy(),
                                  torch.from_numpy(q32).to(case.dt).double().numpy())


@pytest.mark.parametrize("H", [1, 3, 8])
@pytest.mark.parametrize("name", list(MANY))
def test_one_call_stores_what_calls_of_32_sequences_store(name, H):
    """The same tokens into 8 bits by one call and by calls of 32 sequences, whose
    blocks hold one unit each."""
    one, few = (many("e4m3", name, H, 2, seed=1) for _ in range(2))
    one.run()
    tok, start, po, ids, pos0 = few.arrays
    for s0 in range(0, len(start), 32):
        s1 = min(s0 + 32, len(start))
        t0, t1 = tok[s0], tok[s1]
        part = sp.Append([t - t0 for t in tok[s0:s1 + 1]], start[s0:s1], [x - po[s0] for x in po[s0:s1 + 1]],
                         ids[po[s0]:po[s1]], pos0=pos0[s0:s1])
        sp.rag_kv8_append(few.pool, 1, part, few.k[t0:t1], few.v[t0:t1], rope=few.rope, q=few.q[t0:t1],
                          q_out=few.q_out[t0:t1], device_err=few.err)
    torch.cuda.synchronize()
    assert int(one.err.item()) == 0 and int(few.err.item()) == 0
    for a, b in ((one.pool.k, few.pool.k), (one.pool.v, few.pool.v), (one.pool.k_scale, few.pool.k_scale),
                 (one.pool.v_scale, few.pool.v_scale), (one.q_out, few.q_out)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
