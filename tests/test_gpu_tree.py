"""GPU parity: qsa_tree_attention against the definition in 64 bits: drafted trees over committed
cells, identity and selected tokens, odd sizes, masks that leave a token nothing, NaN cells that no
token sees, padding, streams, graphs, and sequences that break the contract."""
import numpy as np
import pytest
import torch

from int8_kv_top_gb300 import qsa, synth
from tests.drafts_testutil import make_batch, reference, run_tree, tree_masks
from tests.qsa_testutil import REL_L2_TOL, rel_l2

pytestmark = pytest.mark.gpu
SCALE = 1 / 16


def check(pool, seqs, max_n_kv=None, params=None, gate=None, with_ids=True, rows=None):
    topk, idmax, scale = params if params else (2048, 2051, SCALE)
    ids, out = run_tree(pool, seqs, max_n_kv, params, gate, with_ids)
    qsa.qsa_check_device_status()
    ref, ref_ids, bound = reference(pool, seqs, topk, idmax, scale, gate, rows)
    got = out.double().cpu().numpy()
    use = np.arange(len(got)) if rows is None else np.array(sorted(rows))
    if with_ids:
        np.testing.assert_array_equal(ids.cpu().numpy()[use], ref_ids[use])
    assert np.isfinite(got).all()
    over = np.abs(got[use] - ref[use]) - bound[use]
    assert over.max() <= 0, f"{over.max():.3e} over the bound at {np.unravel_index(over.argmax(), over.shape)}"
    r = rel_l2(got[use], ref[use])
    assert r <= REL_L2_TOL, f"rel L2 {r:.3e}"
    return got


@pytest.mark.parametrize("pos0,n", [(0, 1), (1, 1), (0, 2), (5, 3), (63, 1), (64, 10), (127, 11), (128, 20), (500, 8),
                                    (1000, 21), (1984, 61), (2047, 4), (300, 64), (77, 200)])
def test_one_tree_under_the_threshold(pos0, n):
    pool, seqs = make_batch([(pos0, n)], seed=pos0 + n, gap=2)
    check(pool, seqs)


@pytest.mark.parametrize("pos0,n", [(2050, 5), (2051, 1), (2051, 9), (3000, 7), (8192, 4)])
def test_one_tree_with_selection(pos0, n):
    # at 2050 committed cells a chain crosses the 2051/2052 budget inside the tree
    pool, seqs = make_batch([(pos0, list(range(-1, n - 1)))], seed=pos0 + n, gap=1)
    check(pool, seqs)


def test_ragged_batch_mixed():
    pool, seqs = make_batch([(0, 7), (2040, 33), (130, 64), (4000, 5), (1, 1), (1999, 12), (2600, 40), (64, 0), (9, 30)],
                            seed=5, gap=4)
    check(pool, seqs)


def test_gated_batch():
    pool, seqs = make_batch([(100, 12), (2045, 10), (2500, 3)], seed=6)
    check(pool, seqs, gate=synth.gate_input(pool["q"].shape[0], seed=61))


def test_without_ids():
    pool, seqs = make_batch([(2100, 6), (40, 6)], seed=7)
    check(pool, seqs, with_ids=False)


@pytest.mark.parametrize("params", [(40, 71, SCALE), (1, 5, SCALE), (64, 63, 0.11), (7, 100, SCALE)])
def test_small_budgets(params):
    pool, seqs = make_batch([(60, 30), (0, 90), (140, 10), (3, 9), (0, 8)], seed=8)
    check(pool, seqs, params=params)


def test_dense_over_long_caches():
    # a threshold above every context: all visible cells, at lengths that split over many CTAs
    pool, seqs = make_batch([(5000, 13), (12345, 3), (20, 5)], seed=9)
    check(pool, seqs, params=(2048, 131072, SCALE))


@pytest.mark.parametrize("specs,params,gated", [
    ([(9000, 16)], None, True),                            # selected tokens
    ([(4500, 12), (0, 3), (9000, 10)], None, False),       # short sequences: pairs without a tile
    ([(7000, 30)], (2048, 131072, SCALE), True),           # two blocks, the second ends inside its rows
    ([(20000, 2)] + [(5, 1), (300, 4)] * 4, (2048, 131072, SCALE), False),
    ([(6000, 1)], (2048, 131072, SCALE), False),
])
def test_blocks_shared_by_many_pairs(specs, params, gated):
    # few sequences over long caches: a block's cells are split over pairs of CTAs and the parts joined afterwards
    pool, seqs = make_batch(specs, seed=31)
    if (0, 3) in specs:
        pool["tree"][13] = 0  # sees nothing
    torch.full((128 << 20,), 255, dtype=torch.uint8, device="cuda")  # freed at once: the workspace starts with NaN
    gate = synth.gate_input(pool["q"].shape[0], seed=62) if gated else None
    first = check(pool, seqs, params=params, gate=gate)
    for _ in range(2):
        again = run_tree(pool, seqs, None, params, gate)[1]
        assert np.array_equal(again.double().cpu().numpy(), first)


def test_many_short_trees():
    rng = np.random.default_rng(10)
    pool, seqs = make_batch([(int(rng.integers(0, 300)), int(rng.integers(1, 26))) for _ in range(60)], seed=10)
    check(pool, seqs)


def test_mask_words_wider_than_the_trees_and_stray_bits():
    pool, seqs = make_batch([(50, 20), (9, 70)], seed=11, words=8)
    want = run_tree(pool, seqs)[1]
    pool["tree"] = pool["tree"].copy()
    pool["tree"][:20, 0] |= np.uint32(0xFFF00000)  # bits past the sequence's 20 tokens are ignored
    pool["tree"][:20, 1:] = 0xFFFFFFFF
    pool["tree"][20:, 2] |= np.uint32(0xFFFFFFC0)
    got = run_tree(pool, seqs)[1]
    qsa.qsa_check_device_status()
    assert torch.equal(got, want)
    check(pool, seqs)


def test_any_mask_pattern():
    # not a tree at all: random bits, later tokens visible to earlier ones, tokens that do not see themselves
    pool, seqs = make_batch([(70, 40), (2040, 33), (2300, 33)], seed=12)
    rng = np.random.default_rng(12)
    pool["tree"] = rng.integers(0, 1 << 32, pool["tree"].shape, dtype=np.uint32)
    check(pool, seqs)


def test_tokens_that_see_nothing_get_zeros():
    pool, seqs = make_batch([(0, 12), (0, 1), (3, 5)], seed=13)
    pool["tree"][[0, 4, 11, 12]] = 0
    got = check(pool, seqs)
    assert (got[[0, 4, 11, 12]] == 0).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_cells_that_nobody_sees_may_hold_anything(bad):
    specs = [(100, 30), (2045, 40), (2600, 30)]
    pool, seqs = make_batch(specs, seed=14)
    for (c0, _, pos0, t0), (_, n) in zip(seqs, specs):
        pool["tree"][t0:t0 + n, 0] &= ~np.uint32((1 << 3) | (1 << 17))
        for j in (3, 17):
            pool["ksc"][c0 + pos0 + j] = bad
            pool["vsc"][c0 + pos0 + j] = bad
    check(pool, seqs)


def test_exact_ties_go_to_the_lower_cell():
    # every drafted cell and many committed ones are copies of one another: the ranking is all ties
    specs = [(200, 24)]
    pool, seqs = make_batch(specs, seed=15)
    for k in ("kq", "ksc"):
        pool[k][50:224] = pool[k][50]
    check(pool, seqs, params=(120, 150, SCALE))


def test_large_logits():
    # queries far from unit size: the running maximum moves by much more than the rescale threshold
    pool, seqs = make_batch([(900, 20), (2200, 6)], seed=16)
    pool["q"] = (pool["q"].astype(np.float32) * 12).astype(np.float16)
    ids, out = run_tree(pool, seqs)
    qsa.qsa_check_device_status()
    ref, ref_ids, bound = reference(pool, seqs)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


def test_padding_sequences_and_tokens_leave_their_rows():
    pool, seqs = make_batch([(100, 10), (2100, 4), (30, 6)], seed=17)
    pool["q"] = np.concatenate([pool["q"], pool["q"][:5]])
    pool["tree"] = np.concatenate([pool["tree"], pool["tree"][:5]])
    padded = np.concatenate([seqs, [[0, 0, 0, 20], [7, 0, 9, 25]]]).astype(np.int32)
    ids, out = run_tree(pool, padded, max_n_kv=2104)
    qsa.qsa_check_device_status()
    assert torch.isnan(out[20:]).all() and (ids[20:] == -7).all()
    # the batch's size may change how a row's cells are split over CTAs, hence the last bits: held to the definition
    ref, ref_ids, bound = reference(dict(pool, q=pool["q"][:20], tree=pool["tree"][:20]), seqs)
    assert (np.abs(out[:20].double().cpu().numpy() - ref) <= bound).all()
    np.testing.assert_array_equal(ids[:20].cpu().numpy(), ref_ids)


@pytest.mark.parametrize("how", ["cells", "pool", "negative", "words", "max_n_kv", "pos0"])
def test_a_bad_sequence_is_skipped_and_flagged(how):
    pool, seqs = make_batch([(100, 10), (200, 40), (2100, 3)], seed=18)
    bad, max_n_kv = seqs.copy(), 2103
    if how == "cells":
        bad[1, 1] = 239            # 200 + 40 tokens do not fit
    elif how == "pool":
        bad[1, 0] = len(pool["kq"]) - 100
    elif how == "negative":
        bad[1, 0] = -5
    elif how == "pos0":
        bad[1, 2] = -1
    elif how == "words":
        pool["tree"] = pool["tree"][:, :1]   # 40 tokens, 32 bits
    else:
        pool, bad = make_batch([(100, 10), (2200, 40), (2000, 3)], seed=18)
        seqs = bad
    skipped = slice(10, 50)
    ids, out = run_tree(pool, bad, max_n_kv=max_n_kv)
    with pytest.raises(qsa.QSAError) as e:
        qsa.qsa_check_device_status()
    assert e.value.code == qsa.QSA_ERR_DEVICE
    assert torch.isnan(out[skipped]).all() and (ids[skipped] == -7).all()
    rows = set(range(10)) | set(range(50, 53))
    ref, ref_ids, bound = reference(pool, seqs, rows=rows)
    use = sorted(rows)
    assert (np.abs(out.double().cpu().numpy()[use] - ref[use]) <= bound[use]).all()
    np.testing.assert_array_equal(ids.cpu().numpy()[use], ref_ids[use])


@pytest.mark.parametrize("pos0", [100, 2100])
def test_tables_whose_rows_go_back_are_flagged(pos0):
    # first token rows 0, 40, 0, 40, ...: every other entry goes back; the listed blocks would be many times the rows'
    pool, _ = make_batch([(pos0, 40)], seed=26)
    seqs = np.array([[0, pos0 + 40, pos0, 40 * (i & 1)] for i in range(300)], np.int32)
    run_tree(pool, seqs, max_n_kv=pos0 + 40)
    with pytest.raises(qsa.QSAError) as e:
        qsa.qsa_check_device_status()
    assert e.value.code == qsa.QSA_ERR_DEVICE
    check(*make_batch([(pos0, 40)], seed=27))  # the device goes on


@pytest.mark.parametrize("n_seq", [7, 8, 40])
def test_trees_of_equal_and_of_no_length(n_seq):
    # sequences without drafted tokens among the others, on both sides of where the blocks are listed first
    pool, seqs = make_batch([(300 if i % 3 else 0, 0 if i % 4 == 1 else 25) for i in range(n_seq)], seed=28)
    check(pool, seqs)


def test_a_chain_equals_the_batched_prefill():
    # a chain of drafted tokens is what a prefill of the same tokens computes
    pool, seqs = make_batch([(1990, list(range(-1, 24))), (300, list(range(-1, 39)))], seed=19)
    out = check(pool, seqs)
    dev = {k: torch.from_numpy(v).cuda() for k, v in pool.items() if k != "tree"}
    n_tok = pool["q"].shape[0]
    want = torch.empty(n_tok, 24, 256, dtype=torch.float16, device="cuda")
    ws = torch.empty(qsa.qsa_flash_prefill_batched_workspace_bytes(2, n_tok, 2015), dtype=torch.uint8, device="cuda")
    qsa.qsa_flash_prefill_batched(dev["q"], dev["kq"], dev["vq"], dev["ksc"], dev["vsc"], pool["kq"].shape[0],
                                  torch.from_numpy(seqs).cuda(), 2, n_tok, 2015, None, want, ws)
    qsa.qsa_check_device_status()
    assert rel_l2(out, want.double().cpu().numpy()) <= 2 * REL_L2_TOL  # each side within its own tolerance


def test_repeated_calls_give_the_same_bits():
    pool, seqs = make_batch([(1500, 30), (2500, 8), (7000, 9)], seed=20)
    params = (2048, 2051, SCALE)
    first = run_tree(pool, seqs, params=params)
    for _ in range(3):
        again = run_tree(pool, seqs, params=params)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])


@pytest.mark.parametrize("specs", [[(700, 17), (2300, 6)], [(9000, 16)], [(5000, 30), (7000, 12)]])
def test_on_another_stream_and_in_graphs(specs):
    pool, seqs = make_batch(specs, seed=21)
    want_ids, want = run_tree(pool, seqs)
    n_tok, n_pool, n_seq, max_n_kv = pool["q"].shape[0], pool["kq"].shape[0], len(specs), max(p + n for p, n in specs)
    dev = {k: torch.from_numpy(v).cuda() for k, v in pool.items() if k != "tree"}
    tree = torch.from_numpy(pool["tree"].view(np.int32)).cuda()
    table = torch.from_numpy(seqs).cuda()
    need = qsa.qsa_tree_attention_workspace_bytes(n_seq, n_tok, max_n_kv)

    def buffers():
        return (torch.full((n_tok, 2, 2048), -7, dtype=torch.int32, device="cuda"), torch.zeros_like(want),
                torch.empty(max(need, 1), dtype=torch.uint8, device="cuda"))

    def call(ids, out, ws):
        qsa.qsa_tree_attention(dev["q"], dev["kq"], dev["vq"], dev["ksc"], dev["vsc"], n_pool, table, n_seq, n_tok, tree,
                               max_n_kv, ids, out, ws)

    torch.cuda.synchronize()
    sets = [buffers() for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, b in zip(streams, sets):      # two calls at once, a workspace each
        with torch.cuda.stream(s):
            for _ in range(5):
                call(*b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(*sets[2])
    for b in sets[2:]:
        b[1].zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    qsa.qsa_check_device_status()
    for ids, out, _ in sets:
        assert torch.equal(out, want) and torch.equal(ids, want_ids)


def test_a_graph_follows_its_tables():
    # a captured call reads lengths, masks and positions from the device: the same graph serves the next step
    pool, seqs = make_batch([(700, 17), (1200, 6)], seed=22)
    other, _ = make_batch([(700, 17), (1200, 6)], seed=23)
    n_tok = pool["q"].shape[0]
    dev = {k: torch.from_numpy(v).cuda() for k, v in pool.items() if k != "tree"}
    tree = torch.from_numpy(pool["tree"].view(np.int32)).cuda()
    table = torch.from_numpy(seqs).cuda()
    out = torch.zeros(n_tok, 24, 256, dtype=torch.float16, device="cuda")
    need = qsa.qsa_tree_attention_workspace_bytes(2, n_tok, 2000)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")

    def call():
        qsa.qsa_tree_attention(dev["q"], dev["kq"], dev["vq"], dev["ksc"], dev["vsc"], pool["kq"].shape[0], table, 2,
                               n_tok, tree, 2000, None, out, ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    nxt = seqs.copy()
    nxt[:, 2] -= (40, 700)               # shorter contexts, other trees
    table.copy_(torch.from_numpy(nxt))
    tree.copy_(torch.from_numpy(other["tree"].view(np.int32)))
    g.replay()
    torch.cuda.synchronize()
    qsa.qsa_check_device_status()
    ref, _, bound = reference(dict(pool, tree=other["tree"]), nxt)
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


def test_cells_past_four_gigabytes():
    # a pool of 9 million cells: byte offsets of its codes pass 32 bits
    n_pool, pos0, n = 9_000_000, 400, 9
    small, seqs = make_batch([(pos0, n)], seed=24, slack=0)
    ref, _, bound = reference(small, seqs)
    first = n_pool - (pos0 + n)
    dev = {}
    for k in ("kq", "vq", "ksc", "vsc"):
        t = torch.from_numpy(small[k])
        big = torch.empty((n_pool,) + t.shape[1:], dtype=t.dtype, device="cuda")
        big[first:] = t.cuda()
        dev[k] = big
    out = torch.zeros(n, 24, 256, dtype=torch.float16, device="cuda")
    need = qsa.qsa_tree_attention_workspace_bytes(1, n, pos0 + n)
    qsa.qsa_tree_attention(torch.from_numpy(small["q"]).cuda(), dev["kq"], dev["vq"], dev["ksc"], dev["vsc"], n_pool,
                           torch.tensor([[first, pos0 + n, pos0, 0]], dtype=torch.int32, device="cuda"), 1, n,
                           torch.from_numpy(small["tree"].view(np.int32)).cuda(), pos0 + n, None, out,
                           torch.empty(max(need, 1), dtype=torch.uint8, device="cuda"))
    qsa.qsa_check_device_status()
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()


def test_a_context_past_65536_cells():
    pool, seqs = make_batch([(70000, 3)], seed=25)
    check(pool, seqs)


def test_tree_masks_of_a_small_tree():
    np.testing.assert_array_equal(tree_masks([-1, 0, 0, 1, -1], 1)[:, 0], [0b1, 0b11, 0b101, 0b1011, 0b10000])
