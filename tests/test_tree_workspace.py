"""Workspace of qsa_tree_attention: what a call of a server's largest batch is given serves every smaller one."""
import random

import pytest

from int8_kv_top_gb300 import build as qbuild
from int8_kv_top_gb300 import qsa

DENSE = (2048, 131072, 1 / 16)


@pytest.fixture(scope="module", autouse=True)
def lib():
    qbuild.build()
    return qsa.load()


@pytest.mark.parametrize("big,small,params", [
    ((32, 512, 2000), (16, 256, 2000), None),
    ((64, 512, 16000), (48, 384, 16000), None),
    ((1, 8, 65537), (1, 8, 65536), None),        # past what selects together
    ((100, 100, 30000), (1, 100, 30000), None),  # one token a sequence, and all of them in one
    ((300, 2400, 131072), (270, 2400, 127000), DENSE),
    ((76, 76, 131072), (1, 1, 131072), DENSE),
])
def test_a_smaller_call_needs_no_more(big, small, params):
    assert qsa.qsa_tree_attention_workspace_bytes(*small, params) <= qsa.qsa_tree_attention_workspace_bytes(*big, params)


@pytest.mark.parametrize("params", [None, DENSE, (40, 71, 1 / 16)])
def test_it_grows_with_each_argument(params):
    rng = random.Random(7)
    for _ in range(3000):
        at = [int(2 ** rng.uniform(0, top)) for top in (11, 14, 17)]
        size = qsa.qsa_tree_attention_workspace_bytes(*at, params)
        for i, most in enumerate((65535, 65535, 131072)):
            more = list(at)
            more[i] = min(most, at[i] + rng.choice((1, 7, 128, 1000, at[i])))
            assert qsa.qsa_tree_attention_workspace_bytes(*more, params) >= size, (at, more)


def test_it_stays_small_beside_the_cache():
    # a fixed number of CTAs' parts, and a few bytes a (token, cell) where tokens may select
    assert qsa.qsa_tree_attention_workspace_bytes(1, 8, 500) <= 4 << 20
    assert qsa.qsa_tree_attention_workspace_bytes(32, 1024, 2048) <= 160 << 20
    assert qsa.qsa_tree_attention_workspace_bytes(65535, 65535, 2048) <= 430 << 20
