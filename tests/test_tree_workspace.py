"""Workspace of qsa_tree_attention: what a call of a server's largest batch is given serves every smaller one."""
import ctypes
import os
import random
import subprocess

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


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """dense_plan(held, n_seq, n_tok, max_n_kv, identity_max, with_selected) -> (blocks, pairs, runs, parts_most)."""
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(f'''#include "{os.path.join(qbuild.CSRC, "tree_plan.cuh")}"
extern "C" void plan(const int* held, const int* at, int* out) {{
  qsa::PlanHeld h;
  for (int i = 0; i < qsa::kPlanSizesN; ++i) h.n[i] = held[i];
  const qsa::DensePlan p = qsa::dense_plan(h, at[0], at[1], at[2], at[3], at[4] != 0);
  out[0] = p.blocks; out[1] = p.pairs; out[2] = p.runs; out[3] = (int)qsa::parts_most(at[0], at[1], at[2]);
}}''')
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-o", str(d / "plan.so"), str(d / "plan.cpp")], check=True)
    f = ctypes.CDLL(str(d / "plan.so")).plan

    def call(held, *at):
        out = (ctypes.c_int * 4)()
        f((ctypes.c_int * 7)(*held), (ctypes.c_int * 5)(*at), out)
        return tuple(out)

    return call


SIZES = (1, 2, 3, 4, 5, 6, 8)  # pairs of a cluster
GB300 = (76, 36, 23, 15, 13, 8, 7)


def shapes(seed, n):
    rng = random.Random(seed)
    for _ in range(n):
        n_seq = int(2 ** rng.uniform(0, 11))
        yield (n_seq, min(65535, max(1, int(n_seq * 2 ** rng.uniform(-1, 8)))), int(2 ** rng.uniform(0, 17)),
               rng.choice((5, 2051, 131072)), rng.randrange(2))


def test_a_plan_writes_inside_the_workspace(plan):
    for at in shapes(8, 20000):
        blocks, pairs, runs, most = plan(GB300, *at)
        assert pairs == 1 or runs == 1
        assert pairs * runs == 1 or 2 * blocks * pairs * runs <= most, at


@pytest.mark.parametrize("held", [(76, 36, 23, 15, 0, 0, 0), (60, 28, 0, 12, 0, 0, 0), (4, 0, 0, 0, 0, 0, 0)])
def test_a_plan_launches_clusters_that_the_gpu_holds(plan, held):
    # a GPU (or a part of one) that takes clusters of 8 CTAs at most, or of 2
    largest = 0
    for at in shapes(9, 20000):
        _, pairs, _, _ = plan(held, *at)
        assert held[SIZES.index(pairs)] > 0, at
        largest = max(largest, plan(GB300, *at)[1])
    assert largest == 8  # a GB300 takes clusters of 16 for some of them


def test_sizes_that_the_call_refuses_need_none():
    for args in ((65536, 65536, 50), (1, 65536, 50), (65536, 1, 50), (2**31 - 1, 2**31 - 1, 2**31 - 1), (3, 2**31 - 1, 9000)):
        assert qsa.qsa_tree_attention_workspace_bytes(*args) == 0
    assert qsa.qsa_tree_attention_workspace_bytes(65535, 65535, 131072) > 0
