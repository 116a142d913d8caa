"""GPU parity: qsa_tree_attention where few selected tokens a sequence take a cluster of CTAs each (the decode
layer's kernel over the visible cells) beside the tensor-core attention of the others, against the definition in
64 bits."""
import numpy as np
import pytest
import torch

from int8_kv_top_gb300 import qsa, synth
from tests.drafts_testutil import make_batch, reference, run_tree
from tests.qsa_testutil import REL_L2_TOL, rel_l2

pytestmark = pytest.mark.gpu
SCALE = 1 / 16


def check(pool, seqs, params=None, gate=None, with_ids=True, max_n_kv=None):
    ids, out = run_tree(pool, seqs, max_n_kv, params, gate, with_ids)
    qsa.qsa_check_device_status()
    ref, ref_ids, bound = reference(pool, seqs, *(params or (2048, 2051, SCALE)), gate=gate)
    got = out.double().cpu().numpy()
    if with_ids:
        np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
    assert (np.abs(got - ref) <= bound).all() and rel_l2(got, ref) <= REL_L2_TOL
    return got


@pytest.mark.parametrize("specs", [
    [(2052, 1)], [(2051, 1), (2050, 1), (2052, 1)], [(2100, 3), (2500, 1), (9000, 2)], [(3000, 2)] * 9,
    [(2049, [-1, 0, 1, 2]), (100, 2), (0, 1)],  # a chain that crosses the budget
    [(20000, 2), (2300, 3)],                    # clusters of 16
])
@pytest.mark.parametrize("gated,with_ids", [(False, True), (True, True), (True, False)])
def test_few_selected_tokens(specs, gated, with_ids):
    pool, seqs = make_batch(specs, seed=51, gap=2)
    gate = synth.gate_input(pool["q"].shape[0], seed=63) if gated else None
    check(pool, seqs, gate=gate, with_ids=with_ids)


@pytest.mark.parametrize("params", [(40, 71, SCALE), (1, 5, SCALE), (64, 63, 0.11), (7, 100, SCALE), (1, 1, 0.5)])
def test_small_budgets(params):
    pool, seqs = make_batch([(60, 4), (0, 3), (140, 2), (3, 1), (500, 3), (6, 4)], seed=52)
    check(pool, seqs, params=params)


def test_any_mask_pattern():
    pool, seqs = make_batch([(2300, 4), (2049, 4), (2048, 4), (70, 4)], seed=53)
    pool["tree"] = np.random.default_rng(53).integers(0, 1 << 32, pool["tree"].shape, dtype=np.uint32)
    check(pool, seqs)


def test_wide_masks_with_stray_bits():
    pool, seqs = make_batch([(2300, 3), (2600, 2)], seed=54, words=8)
    pool["tree"] = pool["tree"].copy()
    want = run_tree(pool, seqs)
    pool["tree"][:3, 0] |= np.uint32(0xFFFFFFF8)
    pool["tree"][:, 1:] = 0xFFFFFFFF
    got = run_tree(pool, seqs)
    qsa.qsa_check_device_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_cells_that_nobody_sees_may_hold_anything(bad):
    pool, seqs = make_batch([(2100, 4), (2600, 4)], seed=55)
    for c0, _, pos0, t0 in seqs:
        pool["tree"][t0:t0 + 4, 0] &= ~np.uint32(1 << 2)
        pool["ksc"][c0 + pos0 + 2] = bad
        pool["vsc"][c0 + pos0 + 2] = bad
    check(pool, seqs)


def test_exact_ties_go_to_the_lower_cell():
    pool, seqs = make_batch([(200, 3)], seed=57)
    for k in ("kq", "ksc"):
        pool[k][50:203] = pool[k][50]
    check(pool, seqs, params=(120, 150, SCALE))


def test_large_logits():
    pool, seqs = make_batch([(2200, 3), (5000, 2)], seed=58)
    pool["q"] = (pool["q"].astype(np.float32) * 12).astype(np.float16)
    ids, out = run_tree(pool, seqs)
    qsa.qsa_check_device_status()
    ref, ref_ids, bound = reference(pool, seqs)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


def test_padding_leaves_its_rows():
    pool, seqs = make_batch([(2100, 3), (30, 2), (2200, 1)], seed=59)
    pool["q"] = np.concatenate([pool["q"], pool["q"][:4]])
    pool["tree"] = np.concatenate([pool["tree"], pool["tree"][:4]])
    padded = np.concatenate([seqs, [[0, 0, 0, 6], [7, 0, 9, 8]]]).astype(np.int32)
    ids, out = run_tree(pool, padded, max_n_kv=2201)
    qsa.qsa_check_device_status()
    assert torch.isnan(out[6:]).all() and (ids[6:] == -7).all()
    ref, ref_ids, bound = reference(dict(pool, q=pool["q"][:6], tree=pool["tree"][:6]), seqs)
    assert (np.abs(out[:6].double().cpu().numpy() - ref) <= bound).all()
    np.testing.assert_array_equal(ids[:6].cpu().numpy(), ref_ids)


@pytest.mark.parametrize("how", ["cells", "pool", "negative", "words", "max_n_kv", "pos0"])
def test_a_bad_sequence_is_skipped_and_flagged(how):
    specs = [(2100, 3), (2200, 3), (2150, 3)]
    pool, seqs = make_batch(specs, seed=60, words=1)
    bad, max_n_kv, rows = seqs.copy(), 2300, range(3, 6)
    if how == "cells":
        bad[1, 1] = 2202
    elif how == "pool":
        bad[1, 0] = len(pool["kq"]) - 100
    elif how == "negative":
        bad[1, 0] = -5
    elif how == "pos0":
        bad[1, 2] = -1
    elif how == "words":  # more tokens than mask bits: 40 in one sequence, and many sequences of one token
        pool, seqs = make_batch([(2200, 40)] + [(2100, 1)] * 14, seed=60)
        pool["tree"] = pool["tree"][:, :1]
        bad, rows = seqs, range(40)
    else:
        max_n_kv = 2202
    ids, out = run_tree(pool, bad, max_n_kv=max_n_kv)
    with pytest.raises(qsa.QSAError) as e:
        qsa.qsa_check_device_status()
    assert e.value.code == qsa.QSA_ERR_DEVICE
    assert torch.isnan(out[list(rows)]).all() and (ids[list(rows)] == -7).all()
    use = sorted(set(range(len(pool["q"]))) - set(rows))
    ref, ref_ids, bound = reference(pool, seqs, rows=set(use))
    assert (np.abs(out.double().cpu().numpy()[use] - ref[use]) <= bound[use]).all()
    np.testing.assert_array_equal(ids.cpu().numpy()[use], ref_ids[use])


def test_same_bits_on_other_streams_and_in_graphs():
    specs = [(2300, 3), (700, 2), (9000, 2)]
    pool, seqs = make_batch(specs, seed=61)
    want_ids, want = run_tree(pool, seqs)
    n_tok = pool["q"].shape[0]
    dev = {k: torch.from_numpy(v).cuda() for k, v in pool.items() if k != "tree"}
    tree, table = torch.from_numpy(pool["tree"].view(np.int32)).cuda(), torch.from_numpy(seqs).cuda()
    need = qsa.qsa_tree_attention_workspace_bytes(3, n_tok, 9002)

    def buffers():
        return (torch.full((n_tok, 2, 2048), -7, dtype=torch.int32, device="cuda"), torch.zeros_like(want),
                torch.empty(max(need, 1), dtype=torch.uint8, device="cuda"))

    def call(ids, out, ws):
        qsa.qsa_tree_attention(dev["q"], dev["kq"], dev["vq"], dev["ksc"], dev["vsc"], len(pool["kq"]), table, 3, n_tok, tree,
                               9002, ids, out, ws)

    sets, streams = [buffers() for _ in range(3)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, b in zip(streams, sets):
        with torch.cuda.stream(s):
            for _ in range(5):
                call(*b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(*sets[2])
    sets[2][1].zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    qsa.qsa_check_device_status()
    for ids, out, _ in sets:
        assert torch.equal(out, want) and torch.equal(ids, want_ids)
