"""Attention over the 8-bit pool on the GPU, against fp64."""

import pytest
import torch

import serving_prefill_b200 as sp
from kv8_support import AttnCase, check, reference

pytestmark = pytest.mark.gpu

# (KV heads, query heads a KV head, [(chunk lengths, query tokens)])
PROMPTS = {
    "one_page": (2, 4, [([16], 16)]),
    "ragged": (2, 4, [([100, 33, 1, 15, 17], 10), ([250], 33), ([16, 16, 5], 1)]),
    "two_q_tiles": (1, 4, [([300, 70], 61)]),
    "three_blocks": (2, 8, [([700], 100), ([40, 41], 80)]),
    "mha": (4, 1, [([130, 20], 140), ([7], 3)]),
    "mqa": (1, 32, [([200, 9], 11)]),
    "group_3": (2, 3, [([90, 90], 50), ([33], 20)]),
    "group_5": (1, 5, [([90, 64], 60)]),
    "group_7": (2, 7, [([333], 40), ([20], 19)]),
    "group_128": (1, 128, [([60, 7], 5)]),
    "group_100": (1, 100, [([60, 7], 3)]),
    "long_split": (2, 4, [([1000] * 5, 70)]),
    "many_chunks": (1, 4, [([3 + i % 5 for i in range(90)], 30), ([1], 1)]),
    "self_prompt": (2, 2, [([500], 500)]),
    "more_queries_than_keys": (2, 4, [([5], 40), ([], 7), ([64], 64), ([1], 1)]),
    "no_queries": (2, 4, [([50], 0), ([60], 30), ([], 0)]),
}
SINGLE = {
    "one_token": (8, 4, [([100], 1)]),
    "one_key": (2, 4, [([1], 1)]),
    "step": (8, 4, [([300, 77, 12], 1), ([16], 1), ([900, 1], 1), ([33] * 7, 1)]),
    "mha_step": (32, 1, [([200, 31], 1), ([50], 1)]),
    "group_16": (2, 16, [([500, 10], 1), ([129], 1)]),
    "group_3": (2, 3, [([300, 11], 1), ([128], 1)]),
    "group_7": (4, 7, [([150, 150], 2), ([16], 1)]),
    "four_tokens": (2, 4, [([200, 90], 4), ([3], 2), ([600], 3)]),
    "five_of_three": (1, 3, [([140], 5), ([2], 5)]),
    "sixteen_of_one": (4, 1, [([300, 300], 16), ([10], 16)]),
    "empty_requests": (2, 4, [([], 1), ([40], 1), ([], 2), ([40], 0)]),
    "many_chunks": (2, 4, [([1 + i % 19 for i in range(130)], 1)]),
    "long": (2, 4, [([1024] * 12, 1)]),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", list(PROMPTS))
def test_prompts(name, causal):
    case = AttnCase(*PROMPTS[name], seed=len(name))
    check(case.run(causal), case.reference(causal))
    assert sp.rag_last_device_error(case.ws) == (0, 0)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", list(SINGLE))
def test_short_query_blocks(name, causal):
    case = AttnCase(*SINGLE[name], seed=len(name))
    check(case.run(causal), case.reference(causal))
    assert sp.rag_last_device_error(case.ws) == (0, 0)


@pytest.mark.parametrize("seed", [0, 1])
def test_many_items_a_block_of_every_kind(seed):
    """More work items than SMs, one- and two-tile query blocks and single
    tokens mixed, so that a block walks items of every kind in turn."""
    import random
    r = random.Random(seed)
    reqs = [([r.randint(1, 400) for _ in range(r.randint(1, 5))], r.choice([1, 2, 20, 33, 60, 64, 70, 100, 129]))
            for _ in range(24)]
    case = AttnCase(8, 4, reqs, seed=seed)
    check(case.run(True), case.reference(True))
    assert sp.rag_last_device_error(case.ws) == (0, 0)
