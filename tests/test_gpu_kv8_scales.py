"""Scales at the small end of what the 8-bit attention takes."""

import pytest
import torch

import serving_prefill_b200 as sp
from kv8_support import AttnCase, check

pytestmark = pytest.mark.gpu

SHORT = [([300, 77, 12], 1), ([500, 33], 2), ([90], 1), ([260, 16], 4)]
LONG = [([300, 77, 12], 40), ([500, 33], 70), ([90], 9), ([260, 16], 33), ([5], 20)]


def finite(case, **kw):
    got = case.run(**kw)
    assert sp.rag_last_device_error(case.ws) == (0, 0)
    check(got, case.reference(scale=kw.get("sm_scale", 128.0 ** -0.5)))


@pytest.mark.parametrize("reqs", [SHORT, LONG], ids=["short", "long"])
@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -149, 1e-36, 2.0 ** -65, 2.0 ** -64])
def test_scales_near_the_smallest_number(scale, which, reqs):
    """All pages of a pool, and one page among others, with a scale that fp32
    just holds: the scores (the values) are then 0 within every bound, and
    neither a masked place nor a row sum becomes nan. Queries of zeros too."""
    for some in (False, True):
        case = AttnCase(2, 4, reqs, seed=1)
        case.q[::2] = 0
        for name, host, dev in (("k", case.ks, case.pool.k_scale), ("v", case.vs, case.pool.v_scale)):
            if which in (name, "both"):
                at = torch.zeros_like(host, dtype=torch.bool)
                at[:, case.pages[0][:1] if some else slice(None)] = True
                at &= ~torch.isnan(host)
                host[at] = scale
                dev.copy_(host)
        finite(case)


@pytest.mark.parametrize("reqs", [SHORT, LONG], ids=["short", "long"])
@pytest.mark.parametrize("sm_scale", [1e-45, 1e-38, 1e-20, 2.0 ** -32])
def test_a_softmax_scale_near_zero_weighs_every_visible_key_alike(sm_scale, reqs):
    case = AttnCase(2, 4, reqs, seed=2)
    case.q[::2] = 0
    finite(case, sm_scale=sm_scale)
