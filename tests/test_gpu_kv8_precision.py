"""The precision of the 8-bit attention's operands, value by value, as the header
states it. Rows that see one key have that key's V as their output and that key's
score as their lse."""

import pytest
import torch

import serving_prefill_b200 as sp
from kv8_support import AttnCase

pytestmark = pytest.mark.gpu

KINDS = pytest.mark.parametrize("n_q", [1, 40], ids=["short", "long"])


def v_of_one_key(n_q, scale):
    """Two requests of one cached token each whose V holds every finite code: the
    output, the codes' values, and the scale as fp32 has it."""
    case = AttnCase(2, 4, [([1], n_q), ([1], n_q)], seed=1)
    codes = torch.arange(128).clamp(max=126).to(torch.uint8)
    codes[1::2] |= 0x80
    for pg in case.pages:
        case.pool.v.view(torch.uint8)[1, pg[0], :, 0] = codes.cuda()
    case.pool.v_scale.fill_(scale)
    o, _ = case.run(causal=False)
    assert sp.rag_last_device_error(case.ws) == (0, 0)
    return o, codes.view(torch.float8_e4m3fn).double(), float(torch.tensor(scale, dtype=torch.float32))


@KINDS
@pytest.mark.parametrize("scale", [1e-8, 3e-8, 1.3 * 2.0 ** -20, 1e-5, 1e-4, 0.3, 1.0009765625, 100.7])
def test_v_under_a_scale_that_is_no_power_of_two(scale, n_q):
    """The weight is 1, so O is V, rounded to bf16 (2^-8 of it). Long blocks: the
    scale is rounded to fp16 (half a step, 2^-11 of it, or 2^-25 below fp16's
    normal range; times the code), then the product (2^-11, or 2^-25). fp32's
    roundings on the way: 2^-20."""
    o, codes, scale = v_of_one_key(n_q, scale)
    want = codes * scale
    tol = want.abs() * (2.0 ** -8 + 2.0 ** -20)
    if n_q > 1:
        tol = tol + codes.abs() * max(scale * 2.0 ** -11, 2.0 ** -25) * (1 + 2.0 ** -7) + want.abs() * 2.0 ** -11 + 2.0 ** -25
    assert ((o - want).abs() <= tol).all(), float(((o - want).abs() / tol).max())


@KINDS
@pytest.mark.parametrize("e", [-24, -20, -16, -15, -9, 0, 7])
def test_v_under_power_of_two_scales(e, n_q):
    """Exact for short blocks, and from 2^-15 on for long ones (e4m3's smallest
    step there is fp16's, 2^-24); below, V is the nearest value of fp16."""
    o, codes, scale = v_of_one_key(n_q, 2.0 ** e)
    want = codes * scale
    exact = want if n_q == 1 or e >= -15 else want.half().double()
    assert torch.equal(exact, want) or e < -15
    assert torch.equal(o, exact.to(torch.bfloat16).double().expand_as(o))


@pytest.mark.parametrize("n_q", [4, 64], ids=["short", "long"])
@pytest.mark.parametrize("top", [1.0, 1.7421875, 1.7578125, 3.0e4, 1e-3])
def test_queries_small_beside_their_rows_largest(top, n_q):
    """The key is 1 in one channel, so the lse is the query's value there times
    the softmax scale. Two e4m3 parts under the row's power of two s, where the
    row's largest is above 224 s: values from 2^-9 of the largest on are exact
    (2^-13 in short blocks, whose low part is kept 16-fold), others are off by
    at most 2^-10 s (2^-14 s). fp32: the factor, the multiply-add and the
    logarithm of the sum, 2^-20 of the score, or 2^-18 of a score near 0."""
    long = n_q > 4
    sm = 4096.0 / top
    case = AttnCase(2, 4, [([1], n_q)], seed=3)
    case.pool.k.view(torch.uint8).zero_()
    case.pool.k.view(torch.uint8)[1, case.pages[0][0], :, 0, 5] = 0x38          # 1.0
    case.pool.k_scale.fill_(1.0)
    case.pool.v_scale.fill_(1.0)
    g = torch.Generator().manual_seed(7)
    rows = n_q * 8
    small = torch.exp2(-(torch.arange(rows).double() % 22)) * (1 + torch.rand(rows, generator=g).double())
    small = (small * top / 2).to(torch.bfloat16)
    q = torch.zeros(rows, 128, dtype=torch.bfloat16)
    q[:, 5], q[:, 0] = small, top
    case.q = q.view(n_q, 8, 128).cuda()
    _, lse = case.run(causal=False, sm_scale=sm)
    got, want = lse.reshape(-1) / sm, small.double()
    largest = torch.maximum(q[:, 0].double(), want)
    fp32 = want.abs() * 2.0 ** -20 + 2.0 ** -18 / sm
    off = largest * (2.0 ** -10 if long else 2.0 ** -14) / 224
    tol = torch.where(want >= largest * (2.0 ** -9 if long else 2.0 ** -13), fp32, fp32 + off)
    assert ((got - want).abs() <= tol).all(), float(((got - want).abs() / tol).max())
    assert off.max() <= largest.max() * (2.0 ** -17 if long else 2.0 ** -21)
