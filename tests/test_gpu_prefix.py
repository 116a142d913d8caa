"""GPU parity: qsa_prefix_attention against the definition in 64 bits: prefixes and own cells of every kind of length, drafted
trees, selection over both, padding, streams, graphs, and tables that break the contract."""
import numpy as np
import pytest
import torch

from int8_kv_top_gb300 import qsa, synth
from tests.drafts_testutil import reference
from tests.prompts_testutil import bounds_of, on_gpu, run_shared, shared_batch, verified
from tests.qsa_testutil import REL_L2_TOL, rel_l2

pytestmark = pytest.mark.gpu
SMALL = (40, 71, 1 / 16)  # topk, identity_max: selection over few cells


FAR = 40000  # as max_prefix: few tokens then take the kernels of many, whatever their prefixes are


def check(groups, seed=1, params=None, gate=False, causal=False, words=None, rows=None, with_ids=True, max_prefix=None):
    b, ref, flat = shared_batch(groups, seed, words, causal)
    g = synth.gate_input(len(b["q"]), seed=seed + 50) if gate else None
    ids, out = run_shared(b, params, g, with_ids, bounds=max_prefix and (max_prefix, bounds_of(b)[1]))
    qsa.qsa_check_device_status()
    p = params or (2048, 2051, 1 / 16)
    want, want_ids, bound = reference(ref, flat, *p, gate=g, rows=rows)
    got = out.double().cpu().numpy()
    pick = sorted(rows) if rows is not None else slice(None)
    if with_ids:
        np.testing.assert_array_equal(ids.cpu().numpy()[pick], want_ids[pick])
    got, want, bound = got[pick], want[pick], bound[pick]
    assert np.isfinite(got).all()
    off = np.abs(got - want)
    assert (off <= bound).all(), (off - bound).max()
    assert rel_l2(got, want) <= REL_L2_TOL
    return b, out


@pytest.mark.parametrize("shared", [0, 1, 15, 127, 128, 129, 300])
@pytest.mark.parametrize("own", [0, 1, 15, 16, 17, 64, 200])
def test_decoding_identity(shared, own):
    check([(shared, [(own, 1), (own + 3, 1), (0, 1)])], seed=shared + own)


@pytest.mark.parametrize("n_seq", [1, 2, 20, 21, 22, 43, 64, 170])
def test_blocks_of_tokens(n_seq):
    # 21 1/3 tokens fill a block: sequences cross its border, and the border between a pair's CTAs
    rng = np.random.default_rng(n_seq)
    check([(200, [(int(x), 1) for x in rng.integers(0, 90, n_seq)])], seed=n_seq, causal=True)


@pytest.mark.parametrize("groups", [
    [(150, [(10, 1)] * 5), (0, [(300, 1)] * 3), (77, [(0, 1)] * 30)],
    [(0, [(5, 2), (70, 1)]), (260, [(1, 3)])],
    [(130, []), (40, [(9, 1)] * 2), (50, [])],
    [(500, [(0, 16)] * 3 + [(33, 1)]), (129, [(64, 30), (2, 2)])],
    [(100, [(7, 256), (0, 1)])],
    [(64, [(20, 5), (3, 0), (40, 7)])],
    [(1700, [(100, 12)] * 9), (300, [(900, 6)] * 4)],
], ids=range(7))
@pytest.mark.parametrize("gate", [False, True])
def test_prefixes_and_drafts_identity(groups, gate):
    check(groups, seed=7, gate=gate)


def test_no_prefix_table_at_all():
    b, ref, flat = shared_batch([(0, [(50, 1), (3, 2), (200, 1)])], 3)
    b["prefixes"] = np.zeros((0, 4), np.int32)
    _, out = run_shared(b, bounds=(0, 201))
    qsa.qsa_check_device_status()
    want, _, bound = reference(ref, flat)
    assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("groups", [
    [(60, [(5, 1), (11, 1), (10, 1), (200, 1)])],                       # about the threshold, on both sides
    [(71, [(0, 1)] * 3), (70, [(0, 1)] * 3), (72, [(0, 1)] * 2)],
    [(128, [(0, 1), (30, 1)]), (127, [(0, 1), (30, 1)]), (129, [(60, 1)])],
    [(500, [(40, 1)] * 50)],
    [(0, [(400, 1), (20, 1)]), (1000, [(3, 1), (128, 1)])],
    [(300, [(20, 9)] * 5), (30, [(10, 40), (100, 3)])],
    [(2100, [(2100, 4), (1, 8)])],                                      # several chunks of maxima
    [(200, [(50, 33), (0, 70)])],
], ids=range(8))
@pytest.mark.parametrize("gate", [False, True])
def test_selection(groups, gate):
    check(groups, seed=11, params=SMALL, gate=gate)


def test_selection_with_the_defaults():
    check([(2000, [(50, 1), (51, 1), (300, 1)]), (2600, [(7, 1), (500, 2)])], seed=5)


@pytest.mark.parametrize("causal", [False, True])
def test_without_ids_and_masks(causal):
    check([(400, [(30, 3), (2, 1), (90, 6)])], seed=6, params=SMALL, causal=causal, with_ids=False)


def test_long_prefix_many_tokens():
    rng = np.random.default_rng(8)
    groups = [(9000, [(int(x), 1) for x in rng.integers(10, 400, 60)])]
    rows = {0, 20, 21, 42, 59}
    check(groups, seed=8, rows=rows)
    check(groups, seed=8, params=(2048, 1 << 17, 1 / 16), rows=rows, causal=True)


@pytest.mark.parametrize("n_seq", [3, 76, 77])
@pytest.mark.parametrize("shared", [8000, 16200, 16300, 32500, 33000])
def test_selection_at_the_borders_of_the_kernels(n_seq, shared):
    # rows of scores on an SM of their own and two on an SM, of up to 8,192, 16,384, 32,768 and 65,536 columns
    check([(shared, [(30 + i, 1) for i in range(n_seq)])], seed=n_seq, rows={0, n_seq - 1})


def test_long_own_cells():
    check([(300, [(9000, 1), (40, 1)])], seed=9, rows={0, 1}, params=(2048, 1 << 17, 1 / 16))
    check([(300, [(9000, 1), (40, 1)])], seed=9, rows={0, 1})


def test_equal_scores_go_to_the_lower_cell():
    # the same key in every cell of prefix and own cells: the first topk cells, prefix first
    b, ref, flat = shared_batch([(90, [(40, 1), (5, 1)])], 12)
    for pool in (b, ref):
        pool["kq"][:] = 3
        pool["ksc"][:] = np.where(np.isnan(pool["ksc"]), pool["ksc"], np.float16(0.01))
    ids, _ = run_shared(b, SMALL)
    qsa.qsa_check_device_status()
    assert (ids.cpu().numpy() == np.arange(40)).all()


@pytest.mark.parametrize("n_seq", [3, 80])  # 1,024 threads a row, and 512
@pytest.mark.parametrize("shared,own", [(700, 900), (1, 1500), (1280, 300), (1100, 2600)])
@pytest.mark.parametrize("far", [0, 25])
def test_many_equal_scores_go_to_the_lower_cells(n_seq, shared, own, far):
    # one key in every cell, more of them than are ranked one by one: the first topk cells, from the prefix over the gap
    # into the own ones.  With `far`, that many of the last own cells have a key twice as large, or small: chosen, or not
    topk = 1200
    if n_seq > 3:
        own = own // 3 + 200 if shared > 800 else own
    b, _, _ = shared_batch([(shared, [(own, 1)] * n_seq)], 14, causal=True)
    b["kq"][:] = 3
    b["ksc"][:] = np.where(np.isnan(b["ksc"]), b["ksc"], np.float16(0.01))
    for first, _, held, _ in b["seqs"]:
        b["kq"][first + held - far:first + held] = 6
    ids, _ = run_shared(b, (topk, topk + 50, 1 / 16))
    qsa.qsa_check_device_status()
    got = ids.cpu().numpy()
    n_kv = shared + own + 1
    up = b["q"].astype(np.float64).reshape(n_seq, 2, 12 * 256).sum(-1) > 0  # the sign of a row's scores
    lows = np.concatenate([np.arange(shared + own - far), [n_kv - 1]])
    highs = np.arange(shared + own - far, shared + own)
    assert n_kv > topk + 50 and len(lows) > topk
    for t in range(n_seq):
        for g in range(2):
            want = np.sort(np.concatenate([highs, lows[:topk - far]])) if up[t, g] else lows[:topk]
            np.testing.assert_array_equal(got[t, g], want)


def test_a_token_that_sees_nothing_gets_zeros():
    b, _, _ = shared_batch([(0, [(0, 2), (0, 1)])], 13)
    b["tree"][:] = [[0], [2], [0]]
    _, out = run_shared(b)
    qsa.qsa_check_device_status()
    assert (out[0] == 0).all() and (out[2] == 0).all() and (out[1] != 0).any()


@pytest.mark.parametrize("params", [None, SMALL])
@pytest.mark.parametrize("parents", [[-1], [-1, -1, -1], [-1] * 12])
def test_unseen_own_cells_may_hold_anything(params, parents):
    # a drafted cell that nobody sees, of infinities and NaN, beside seen ones
    b, ref, flat = shared_batch([(100, [(33, parents + [-1]), (20, parents)])], 14)
    n = len(parents)
    row = int(b["seqs"][0][0]) + 33 + n
    b["ksc"][row], b["vsc"][row] = np.nan, np.inf
    b["tree"][n] &= ~np.uint32(1 << n)
    ref["tree"][n] = b["tree"][n]
    _, out = run_shared(b, params)
    qsa.qsa_check_device_status()
    want, _, bound = reference(ref, flat, *(params or (2048, 2051, 1 / 16)))
    assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()


def test_far_larger_logits_late_in_the_row():
    # the running maximum grows by far more than its slack, in the prefix's and in the own cells
    b, ref, flat = shared_batch([(300, [(120, 1), (300, 5)])], 15)
    grow = np.linspace(0.2, 6, 300).astype(np.float16)[:, None, None]
    at, own = int(b["prefixes"][0][0]), [(int(s[0]), int(s[2])) for s in b["seqs"]]
    b["ksc"][at:at + 300] *= grow
    for i, (c0, pos0) in enumerate(own):
        b["ksc"][c0:c0 + pos0] *= grow[:pos0]
        f0 = int(flat[i][0])
        ref["ksc"][f0:f0 + 300] = b["ksc"][at:at + 300]
        ref["ksc"][f0 + 300:f0 + 300 + pos0] = b["ksc"][c0:c0 + pos0]
    _, out = run_shared(b)
    qsa.qsa_check_device_status()
    want, _, bound = reference(ref, flat)
    assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("groups", [[(300, [(50, 1), (60, 1)])], [(300, [(50, 5), (60, 5)])], [(0, [(50, 1), (2000, 1)])], [(0, [(50, 5), (60, 5)])],
                                    [(900, [(9, 1)] * 30)]], ids=["one token", "drafts", "own cells", "own drafts", "a block"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nan_reaches_its_row_and_no_other(groups, value):
    b, _, _ = shared_batch(groups, 41)
    _, good = run_shared(b)
    for h, d in ((3, 7), (14, 200)):
        b["q"][1, h, d] = value
    _, out = run_shared(b)
    qsa.qsa_check_device_status()
    hit = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    hit[1, [3, 14]] = True
    assert out[hit].isnan().all() and torch.equal(out[~hit], good[~hit])


@pytest.mark.parametrize("shared", [0, 1, 15, 127, 128, 129, 300])
@pytest.mark.parametrize("own", [0, 17, 200])
def test_decoding_identity_as_of_many(shared, own):
    check([(shared, [(own, 1), (own + 3, 1), (0, 1)])], seed=shared + own, max_prefix=FAR)


@pytest.mark.parametrize("n_seq", [1, 20, 21, 22, 43, 64, 170])
def test_blocks_of_tokens_as_of_many(n_seq):
    rng = np.random.default_rng(n_seq)
    check([(200, [(int(x), 1) for x in rng.integers(0, 90, n_seq)])], seed=n_seq, causal=True, max_prefix=FAR)


@pytest.mark.parametrize("groups", [
    [(150, [(10, 1)] * 5), (0, [(300, 1)] * 3), (77, [(0, 1)] * 30)],
    [(0, [(5, 2), (70, 1)]), (260, [(1, 3)])],
    [(130, []), (40, [(9, 1)] * 2), (50, [])],
    [(500, [(40, 1)] * 50)],
    [(60, [(5, 1), (11, 1), (10, 1), (200, 1)])],
], ids=range(5))
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("params", [None, SMALL])
def test_prefixes_as_of_many(groups, gate, params):
    check(groups, seed=7, gate=gate, params=params, max_prefix=FAR)


@pytest.mark.parametrize("max_prefix", [None, FAR])
@pytest.mark.parametrize("n_seq,shared,own", [(1, 1, 0), (1, 100, 30), (1, 300, 90), (1, 2000, 40), (1, 3000, 2000), (3, 900, 10), (5, 1900, 140), (8, 1500, 130),
                                              (11, 40, 300), (20, 600, 50), (40, 100, 20)])
def test_few_tokens_are_shared_out(n_seq, shared, own, max_prefix):
    # one to many CTAs a token, whose parts a cluster or the last launch joins: the same result within its rounding
    dense = (2048, 1 << 17, 1 / 16)
    check([(shared, [(own + 7 * i, 1) for i in range(n_seq)])], seed=60 + n_seq, params=dense, with_ids=False, max_prefix=max_prefix)


@pytest.mark.parametrize("max_prefix", [None, FAR])
@pytest.mark.parametrize("how", ["cells", "n_kv", "prefix past the pool", "prefix cells<0"])
def test_bad_tables_of_single_tokens(how, max_prefix):
    b, ref, flat = shared_batch([(90, [(20, 1), (31, 1)]), (40, [(5, 1), (60, 1)]), (30, [(10, 1)])], 17)
    bounds = (max_prefix or 90, bounds_of(b)[1])
    if how == "cells":
        b["seqs"][2][1] = 5
    elif how == "n_kv":
        b["seqs"][2][:3] = [0, 200, 150]
    else:
        b["prefixes"][1][:2] = [len(b["kq"]) - 39, 40] if how == "prefix past the pool" else [0, -1]
    _, out = run_shared(b, fill=7.0, bounds=bounds)
    with pytest.raises(qsa.QSAError) as e:
        qsa.qsa_check_device_status()
    assert e.value.code == qsa.QSA_ERR_DEVICE
    want, _, bound = reference(ref, flat)
    got = out.double().cpu().numpy()
    gone = {2} if how in ("cells", "n_kv") else {2, 3}
    for s in range(5):
        assert (got[s] == 7).all() if s in gone else (np.abs(got[s] - want[s]) <= bound[s]).all(), s


def test_nan_reaches_its_row_of_many():
    b, _, _ = shared_batch([(900, [(9, 1)] * 30)], 43)
    bounds = (FAR, bounds_of(b)[1])
    _, good = run_shared(b, bounds=bounds)
    b["q"][1, 3, 7] = np.nan
    _, out = run_shared(b, bounds=bounds)
    qsa.qsa_check_device_status()
    hit = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    hit[1, 3] = True
    assert out[hit].isnan().all() and torch.equal(out[~hit], good[~hit])


@pytest.mark.parametrize("params", [None, SMALL])
def test_same_bits_of_many_in_graphs(params):
    sets = [device_batch([(1200, [(50, 1)] * 30)], 21 + i, params) for i in range(2)]
    for *_, call in sets:
        call()
    torch.cuda.synchronize()
    want = [(s[3]["out"].clone(), s[3]["ids"].clone()) for s in sets]
    for s in sets:
        s[3]["out"].zero_()
        s[3]["ids"].fill_(-7)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for *_, call in sets:
            call()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    qsa.qsa_check_device_status()
    for s, (out, ids) in zip(sets, want):
        assert torch.equal(s[3]["out"], out) and torch.equal(s[3]["ids"], ids)


@pytest.mark.parametrize("tokens", [1, 5])
@pytest.mark.parametrize("where", ["prefix", "own"])
def test_a_cell_of_nan_among_far_larger_scores_reaches_every_row(tokens, where):
    # the part with the NaN has a maximum far below the other part's: its weight is 0 but for the NaN
    b, _, _ = shared_batch([(300, [(64, tokens)])], 42)
    prefix, own = int(b["prefixes"][0, 0]), int(b["seqs"][0, 0])
    big, nan = ((own, 64), prefix + 5) if where == "prefix" else ((prefix, 300), own + 5)
    b["q"][:] = 4
    b["kq"][big[0]:big[0] + big[1]] = 127
    b["ksc"][nan] = np.nan
    _, out = run_shared(b)
    qsa.qsa_check_device_status()
    assert out.isnan().all()


@pytest.mark.parametrize("params", [None, SMALL])
@pytest.mark.parametrize("tokens", [1, 6])
def test_padding_and_rows_that_are_nobodys(params, tokens):
    groups = [(90, [(20, tokens), (31, tokens), (8, tokens)]), (40, [(5, tokens), (60, tokens)])]
    b, ref, flat = shared_batch(groups, 16)
    b["seqs"][1][1] = 0  # padding: its rows are left as they are
    ids, out = run_shared(b, params, fill=7.0)
    qsa.qsa_check_device_status()
    want, _, bound = reference(ref, flat, *(params or (2048, 2051, 1 / 16)))
    got = out.double().cpu().numpy()
    left = slice(tokens, 2 * tokens)
    assert (got[left] == 7).all() and (ids[left] == -7).all()
    for rows in (slice(0, tokens), slice(2 * tokens, None)):
        assert (np.abs(got[rows] - want[rows]) <= bound[rows]).all()


@pytest.mark.parametrize("params", [None, SMALL])
@pytest.mark.parametrize("how", ["first<0", "past the pool", "pos0<0", "cells", "n_kv", "rows", "prefix past the pool", "prefix cells<0",
                                 "prefix too long", "prefix order", "prefix first<0"])
def test_bad_tables_are_flagged_and_skipped(how, params):
    groups = [(90, [(20, 2), (31, 2)]), (40, [(5, 2), (60, 2)]), (30, [(10, 2)])]
    b, ref, flat = shared_batch(groups, 17)
    bounds = bounds_of(b)
    seqs, prefixes, n_pool = b["seqs"], b["prefixes"], len(b["kq"])
    gone = {2}
    if how == "first<0":
        seqs[2][0] = -1
    elif how == "past the pool":
        seqs[2][0] = n_pool - 4
    elif how == "pos0<0":
        seqs[2][2] = -2
    elif how == "cells":
        seqs[2][1] = 6
    elif how == "n_kv":
        seqs[2][1:3] = [200, 150]
        seqs[2][0] = 0
    elif how == "rows":
        seqs[3][3] = 3
        gone = {1, 2, 3}
    else:
        gone = {2, 3}
        if how == "prefix past the pool":
            prefixes[1][0] = n_pool - 39
        elif how == "prefix cells<0":
            prefixes[1][1] = -1
        elif how == "prefix too long":
            prefixes[1][1], prefixes[1][0] = 91, 0
        elif how == "prefix order":
            prefixes[1][2] = 5
            gone = {2, 3, 4}
        else:
            prefixes[1][0] = -3
    ids, out = run_shared(b, params, fill=7.0, bounds=bounds)
    with pytest.raises(qsa.QSAError) as e:
        qsa.qsa_check_device_status()
    assert e.value.code == qsa.QSA_ERR_DEVICE
    want, _, bound = reference(ref, flat, *(params or (2048, 2051, 1 / 16)))
    got = out.double().cpu().numpy()
    for s in range(5):
        r = slice(2 * s, 2 * s + 2)
        if s in gone:
            if how not in ("rows", "prefix order"):
                assert (got[r] == 7).all(), s
        else:
            assert (np.abs(got[r] - want[r]) <= bound[r]).all(), s


def device_batch(groups, seed, params, gate=False):
    b, ref, flat = shared_batch(groups, seed)
    d = on_gpu({k: v for k, v in b.items() if k != "tree"})
    d["tree"] = torch.from_numpy(b["tree"].view(np.int32)).cuda()
    max_prefix, max_n_kv = bounds_of(b)
    n_tok = len(b["q"])
    need = qsa.qsa_prefix_attention_workspace_bytes(len(b["prefixes"]), len(b["seqs"]), n_tok, max_prefix, max_n_kv, params)
    d |= {"ws": torch.empty(need, dtype=torch.uint8, device="cuda"), "out": torch.zeros(n_tok, 24, 256, dtype=torch.float16, device="cuda"),
          "ids": torch.full((n_tok, 2, params[0] if params else 2048), -7, dtype=torch.int32, device="cuda")}

    def call(stream=None):
        qsa.qsa_prefix_attention(d["q"], d["kq"], d["vq"], d["ksc"], d["vsc"], len(b["kq"]), d["prefixes"], len(b["prefixes"]), d["seqs"],
                                 len(b["seqs"]), n_tok, d["tree"], max_prefix, max_n_kv, d["ids"], d["out"], d["ws"], params=params, stream=stream)

    return b, ref, flat, d, call


@pytest.mark.parametrize("params,groups", [(None, [(700, [(50, 1)] * 30)]), (None, [(300, [(20, 8)] * 4)]), (SMALL, [(700, [(50, 1)] * 30)]),
                                           (SMALL, [(300, [(20, 8)] * 4)])])
def test_same_bits_on_streams_and_in_graphs(params, groups):
    sets = [device_batch(groups, 21 + i, params) for i in range(3)]
    for *_, call in sets:
        call()
    torch.cuda.synchronize()
    want = [(s[3]["out"].clone(), s[3]["ids"].clone()) for s in sets]
    ref, _, bound = reference(sets[0][1], sets[0][2], *(params or (2048, 2051, 1 / 16)))
    assert (np.abs(want[0][0].double().cpu().numpy() - ref) <= bound).all()

    def cleared():
        for s in sets:
            s[3]["out"].zero_()
            s[3]["ids"].fill_(-7)

    def same():
        torch.cuda.synchronize()
        qsa.qsa_check_device_status()
        for s, (out, ids) in zip(sets, want):
            assert torch.equal(s[3]["out"], out) and torch.equal(s[3]["ids"], ids)

    cleared()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):  # at the same time, a workspace each
        for s, st in zip(sets, streams):
            s[4](st)
    same()
    cleared()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for *_, call in sets:
            call()
    graph.replay()
    graph.replay()
    same()


def test_a_graph_follows_its_tables():
    # lengths and masks are read on the device: one captured call serves the next step too
    b, ref, flat, d, call = device_batch([(200, [(30, 1), (60, 1)]), (90, [(10, 1)])], 31, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    want, _, bound = reference(ref, flat)
    graph.replay()
    assert (np.abs(d["out"].double().cpu().numpy() - want) <= bound).all()
    d["prefixes"][0, 1] = 150  # the same sequences behind the first 150 cells
    for s in (0, 1):
        f0, n = int(flat[s][0]), int(flat[s][1])
        sub = {k: np.concatenate([ref[k][f0:f0 + 150], ref[k][f0 + 200:f0 + n]]) for k in ("kq", "vq", "ksc", "vsc")}
        sub |= {"q": ref["q"][s:s + 1], "tree": ref["tree"][s:s + 1]}
        w, _, bd = reference(sub, np.array([(0, n - 50, n - 51, 0)], np.int32))
        graph.replay()
        assert (np.abs(d["out"][s].double().cpu().numpy() - w[0]) <= bd[0]).all()
    qsa.qsa_check_device_status()


def test_a_large_workspace_serves_smaller_calls():
    big = qsa.qsa_prefix_attention_workspace_bytes(4, 64, 300, 2000, 3000, SMALL)
    ws = torch.full((big,), 0xFF, dtype=torch.uint8, device="cuda")
    for i, groups in enumerate([[(300, [(20, 8)] * 4)], [(700, [(50, 1)] * 30)], [(0, [(9, 1)])], [(30, [(2, 1)] * 3), (1500, [(900, 5)])]]):
        b, ref, flat = shared_batch(groups, 41 + i)
        _, out = run_shared(b, SMALL, ws=ws)
        qsa.qsa_check_device_status()
        want, _, bound = reference(ref, flat, *SMALL)
        assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("params", [None, SMALL])
def test_many_sequences_and_prefixes(params):
    # more than the searches hold in shared memory, and prefixes than are planned one by one
    rng = np.random.default_rng(71)
    groups = [(int(rng.integers(0, 150)), [(int(x), 1) for x in rng.integers(0, 40, 4)]) for _ in range(300)]
    rows = set(int(x) for x in rng.integers(0, 1200, 60)) | {0, 1199}
    check(groups, seed=71, params=params, rows=rows, gate=True)


def test_the_most_tokens():
    n, shared = 65535, 70
    rng = np.random.default_rng(72)
    pool = shared_batch([(shared, [(n, 1)])], 72, gap=0, slack=0)[0]
    first = int(pool["seqs"][0][0])
    b = dict(pool, q=rng.standard_normal((n, 24, 256), np.float32).astype(np.float16), tree=None,
             seqs=np.stack([first + np.arange(n), np.ones(n), np.zeros(n), np.arange(n)], 1).astype(np.int32))
    ids, out = run_shared(b, with_ids=False, bounds=(shared, shared + 1))
    qsa.qsa_check_device_status()
    at = int(pool["prefixes"][0][0])
    for t in (0, 1, 21, 32767, n - 2, n - 1):
        cells = np.concatenate([at + np.arange(shared), [first + t]])
        one = {k: pool[k][cells] for k in ("kq", "vq", "ksc", "vsc")} | {"q": b["q"][t:t + 1], "tree": np.array([[1]], np.uint32)}
        w, _, bd = reference(one, np.array([(0, shared + 1, shared, 0)], np.int32))
        assert (np.abs(out[t].double().cpu().numpy() - w[0]) <= bd[0]).all(), t


def test_a_prefix_longer_than_the_other_calls_take():
    check([(140000, [(40, 1), (3, 2)])], seed=73, params=(2048, 1 << 20, 1 / 16), with_ids=False)


@pytest.mark.parametrize("gate", [False, True])
def test_own_cells_alone(gate):
    check([(0, [(20, 1), (300, 1), (0, 1)])], seed=74, gate=gate)          # one CTA has all of a token's cells
    check([(0, [(20, 1), (1900, 1), (0, 1)])], seed=75, gate=gate)         # several share them
    check([(0, [(20, 8), (300, 5)])], seed=76, gate=gate)                  # on the tensor-core kernel
    check([(0, [(20, 1), (300, 1), (90, 2)])], seed=77, params=SMALL, gate=gate)


def test_overlapping_rows_are_flagged_and_harm_nobody_elses_memory():
    # first token rows that run back and forth: flagged; nothing is said of the rows, but what lies around the outputs stays
    b, _, _ = shared_batch([(200, [(20, 1)] * 40), (90, [(10, 1)] * 40), (300, [(5, 1)] * 40)], 78)
    rng = np.random.default_rng(78)
    for how in range(4):
        seqs = b["seqs"].copy()
        seqs[1:, 3] = rng.permutation(seqs[1:, 3]) if how < 2 else rng.integers(-5, 130, len(seqs) - 1)
        prefixes = b["prefixes"].copy()
        if how == 3:
            prefixes[1:, 2] = [80, 40]
        d = on_gpu({k: v for k, v in b.items() if k in ("q", "kq", "vq", "ksc", "vsc")})
        s, p = torch.from_numpy(seqs).cuda(), torch.from_numpy(prefixes).cuda()
        tree = torch.from_numpy(b["tree"].view(np.int32)).cuda()
        for params in (None, SMALL):
            n, topk = 120, params[0] if params else 2048
            out = torch.full((n + 2, 24, 256), 7.0, dtype=torch.float16, device="cuda")
            ids = torch.full((n + 2, 2, topk), -7, dtype=torch.int32, device="cuda")
            need = qsa.qsa_prefix_attention_workspace_bytes(3, n, n, 300, 330, params)
            ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
            qsa.qsa_prefix_attention(d["q"], d["kq"], d["vq"], d["ksc"], d["vsc"], len(b["kq"]), p, 3, s, n, n, tree, 300, 330, ids[1:],
                                     out[1:], ws[:need], params=params)
            with pytest.raises(qsa.QSAError) as e:
                qsa.qsa_check_device_status()
            assert e.value.code == qsa.QSA_ERR_DEVICE
            assert (out[0] == 7).all() and (out[-1] == 7).all() and (ids[0] == -7).all() and (ids[-1] == -7).all()
            assert (ws[need:] == 0x5A).all()


@pytest.mark.parametrize("own", [10, 3000])
def test_broken_orders_leave_ids_that_are_cells(own):
    # first sequences and first rows that run backwards, over a workspace of large scores: what is selected is among the cells,
    # once each, and nothing is written around the outputs
    n, shared = 64, 200
    b, _, _ = shared_batch([(shared, [(own, 1)] * 2), (90, [(own, 1)] * 10), (300, [(own, 1)] * 52)], 79)
    rows = 0
    for how in range(6):
        seqs, prefixes = b["seqs"].copy(), b["prefixes"].copy()
        if how < 3:
            prefixes[1, 2] = (-1, 70, 1)[how]
            prefixes[2, 2] = (2, 12, 0)[how]
        elif how < 5:
            seqs[10:14, 3], seqs[40:45, 3] = ([13, 12, 11, 10], [44, 41, 43, 40, 45]) if how == 3 else ([11, 10, 13, 12], [42] * 5)
        else:
            seqs[20, 3] = 1 << 20
        d = on_gpu({k: v for k, v in b.items() if k in ("q", "kq", "vq", "ksc", "vsc")})
        s, p = torch.from_numpy(seqs).cuda(), torch.from_numpy(prefixes).cuda()
        out = torch.full((n + 2, 24, 256), 7.0, dtype=torch.float16, device="cuda")
        ids = torch.full((n + 2, 2, 40), -7, dtype=torch.int32, device="cuda")
        most = 300 + own + 1
        need = qsa.qsa_prefix_attention_workspace_bytes(3, n, n, 300, most, SMALL)
        ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        qsa.qsa_prefix_attention(d["q"], d["kq"], d["vq"], d["ksc"], d["vsc"], len(b["kq"]), p, 3, s, n, n, None, 300, most, ids[1:], out[1:],
                                 ws[:need], params=SMALL)
        with pytest.raises(qsa.QSAError) as e:
            qsa.qsa_check_device_status()
        assert e.value.code == qsa.QSA_ERR_DEVICE
        assert (out[0] == 7).all() and (out[-1] == 7).all() and (ids[0] == -7).all() and (ids[-1] == -7).all()
        assert (ws[need:] == 0x5A).all()
        got = ids[1:-1].cpu().numpy()
        for t in range(n):  # a sequence's second token sees a cell of NaN: nothing is said of its ids
            lo, hi = 0, n - 1
            while lo < hi:  # the sequence that the call finds for the row
                mid = (lo + hi + 1) // 2
                lo, hi = (mid, hi) if seqs[mid, 3] <= t else (lo, mid - 1)
            if t != seqs[lo, 3]:
                got[t] = -7
        got = got[(got != -7).any(-1)]
        rows += len(got)
        assert (got >= 0).all() and (got < most).all() and (np.diff(got, axis=-1) > 0).all(), how
    assert rows > 100


def test_tensors_of_the_wrong_kind_are_refused():
    b, _, _, d, call = device_batch([(20, [(3, 1)])], 51, None)
    for name, bad in (("q", d["q"].float()), ("q", d["q"][:, :, ::2]), ("kq", d["kq"][:-1]), ("vsc", d["vsc"].cpu()), ("seqs", d["seqs"].long()),
                      ("tree", d["tree"].long()), ("out", d["out"].cpu()), ("ids", d["ids"][:, :, :100])):
        keep, d[name] = d[name], bad
        with pytest.raises(qsa.QSAError) as e:
            call()
        assert e.value.code == qsa.QSA_ERR_INVALID_ARG and name in str(e.value)
        d[name] = keep
    call()
    qsa.qsa_check_device_status()


def test_a_step_of_a_server():
    """Fork a sequence, draft behind the shared prompt, attend, verify, commit, end one sequence, compact, and decode on."""
    rng = np.random.default_rng(61)
    b, ref, flat = shared_batch([(150, [(30, [-1, 0, 0, 1])])], 61)
    n_own, T = 30, 4
    base, shared0 = int(b["seqs"][0][0]), int(b["prefixes"][0][0])
    pool = {k: np.concatenate([b[k], np.zeros((400, *b[k].shape[1:]), b[k].dtype)]) for k in ("kq", "vq", "ksc", "vsc")}
    d = on_gpu(pool)
    n_pool, first_free = len(pool["kq"]), len(b["kq"])
    kv = (d["kq"], d["ksc"], d["vq"], d["vsc"])
    # the sequence's own cells, its four drafted ones among them, forked twice
    forks = [base, first_free + 20, first_free + 200]
    runs = torch.tensor([[base, f, n_own + T, 0] for f in forks[1:]], dtype=torch.int32, device="cuda")
    qsa.qsa_cache_copy(*kv, n_pool, runs, 2, n_own + T)
    seqs = torch.tensor([[f, n_own + T, n_own, T * i] for i, f in enumerate(forks)], dtype=torch.int32, device="cuda")
    prefixes = torch.from_numpy(b["prefixes"]).cuda()
    q = torch.from_numpy(np.tile(b["q"], (3, 1, 1))).cuda()
    tree = torch.from_numpy(np.tile(b["tree"], (3, 1)).view(np.int32)).cuda()
    out = torch.zeros(3 * T, 24, 256, dtype=torch.float16, device="cuda")
    max_n_kv = 150 + n_own + T
    ws = torch.empty(qsa.qsa_prefix_attention_workspace_bytes(1, 3, 3 * T, 150, max_n_kv, SMALL), dtype=torch.uint8, device="cuda")
    ids = torch.zeros(3 * T, 2, 40, dtype=torch.int32, device="cuda")
    qsa.qsa_prefix_attention(q, d["kq"], d["vq"], d["ksc"], d["vsc"], n_pool, prefixes, 1, seqs, 3, 3 * T, tree, 150, max_n_kv, ids, out, ws,
                             params=SMALL)
    qsa.qsa_check_device_status()
    want, _, bound = reference(ref, flat, *SMALL)
    for i in range(3):
        assert (np.abs(out[T * i:T * i + T].double().cpu().numpy() - want) <= bound).all()
    # the target's answers settle a path of each fork; the last token of a full path leaves no room, so two at most are taken
    vocab, cap = 50, 2
    p = rng.dirichlet(np.ones(vocab) * 0.3, 3 * T).astype(np.float32)
    dr = rng.dirichlet(np.ones(vocab) * 0.3, 3 * T).astype(np.float32)
    parent, token = np.tile([-1, 0, 0, 1], 3).astype(np.int32), np.argsort(p, 1)[np.repeat([0, 4, 8], 4), -1].astype(np.int32)
    u, u_end = (rng.random(n, np.float32) * np.float32(0.3) for n in (3 * T, 3))
    t = on_gpu(dict(p=p, dr=dr, parent=parent, token=token, u=u, u_end=u_end))
    path = torch.zeros(3, cap, dtype=torch.int32, device="cuda")
    n_path, after = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    qsa.qsa_tree_verify(t["p"], t["dr"], vocab, t["token"], t["parent"], t["u"], t["u_end"], seqs, 3, 3 * T, path, n_path, after)
    qsa.qsa_cache_commit(*kv, n_pool, seqs, 3, path, n_path)
    ways = []
    for i in range(3):
        r = slice(T * i, T * i + T)
        way, x = verified(p[r], dr[r], token[r], parent[r], u[r], u_end[i], cap)
        assert path[i, :n_path[i]].tolist() == way and int(after[i]) == x
        ways.append(way)
    # the second fork ends; prefix, first and third move together; one more token each, its K/V copied from cell 0 of the own cells
    table = torch.stack([seqs[0], seqs[2]]).clone()
    table[:, 2] += torch.stack([n_path[0], n_path[2]])
    table[:, 3] = torch.tensor([0, 1])
    used = torch.zeros(1, dtype=torch.int32, device="cuda")
    cws = torch.empty(qsa.qsa_cache_compact_workspace_bytes(n_pool, 1, 2), dtype=torch.uint8, device="cuda")
    qsa.qsa_cache_compact(*kv, n_pool, prefixes, 1, table, 2, prefixes, table, used, cws)
    assert int(used) == 150 + 2 * (n_own + T)
    rows = table.tolist()
    qsa.qsa_cache_copy(*kv, n_pool, torch.tensor([[r[0], r[0] + r[2], 1, 0] for r in rows], dtype=torch.int32, device="cuda"), 2, 1)
    q2 = torch.from_numpy(synth.layer_inputs(2, 2, seed=62)["q"]).cuda()
    out2, ids2 = out[:2].clone(), ids[:2].clone()
    qsa.qsa_prefix_attention(q2, d["kq"], d["vq"], d["ksc"], d["vsc"], n_pool, prefixes, 1, table, 2, 2, None, 150, max_n_kv, ids2, out2, ws,
                             params=SMALL)
    qsa.qsa_check_device_status()
    for i, way in enumerate((ways[0], ways[2])):
        cells = np.concatenate([shared0 + np.arange(150), base + np.arange(n_own), base + n_own + np.array(way), [base]])
        one = {k: pool[k][cells] for k in ("kq", "vq", "ksc", "vsc")} | {"q": q2[i:i + 1].cpu().numpy(), "tree": np.array([[1]], np.uint32)}
        w, wi, bd = reference(one, np.array([(0, len(cells), len(cells) - 1, 0)], np.int32), *SMALL)
        np.testing.assert_array_equal(ids2[i].cpu().numpy(), wi[0])
        assert (np.abs(out2[i].double().cpu().numpy() - w[0]) <= bd[0]).all()
