"""GPU: qsa_tree_attention where its parts meet: hand-over between the CTAs of a pair under load, rows far below
their maximum, workspaces of other sizes, tables that break the contract, on each of its paths."""
import numpy as np
import pytest
import torch

from int8_kv_top_gb300 import qsa
from tests.drafts_testutil import make_batch, reference, run_tree

pytestmark = pytest.mark.gpu
SCALE = 1 / 16


def test_many_calls_give_the_same_bits():
    # long runs of tiles on every pair, beside calls on another stream that change what the SMs do meanwhile
    pool, seqs = make_batch([(5000, 30), (300, 25), (7100, 44), (2600, 9)], seed=41)
    params = (2048, 131072, SCALE)
    first = run_tree(pool, seqs, params=params, with_ids=False)[1]
    ref, _, bound = reference(pool, seqs, *params)
    assert (np.abs(first.double().cpu().numpy() - ref) <= bound).all()
    dev = {k: torch.from_numpy(v).cuda() for k, v in pool.items() if k != "tree"}
    tree = torch.from_numpy(pool["tree"].view(np.int32)).cuda()
    n_tok, table = pool["q"].shape[0], torch.from_numpy(seqs).cuda()
    ws = torch.empty(qsa.qsa_tree_attention_workspace_bytes(4, n_tok, 7144, params), dtype=torch.uint8, device="cuda")
    outs = torch.full((60, *first.shape), float("nan"), dtype=torch.float16, device="cuda")
    side, noise = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    for i in range(60):
        with torch.cuda.stream(side):
            noise = noise @ noise * 1e-2
        qsa.qsa_tree_attention(dev["q"], dev["kq"], dev["vq"], dev["ksc"], dev["vsc"], pool["kq"].shape[0], table, 4, n_tok,
                               tree, 7144, None, outs[i], ws, params=params)
    torch.cuda.synchronize()
    qsa.qsa_check_device_status()
    assert all(torch.equal(o, first) for o in outs)


@pytest.mark.parametrize("n,n_seq", [(2000, 1), (2000, 90), (9000, 76), (131072, 1)])
@pytest.mark.parametrize("at", [0.0, 0.6, 1.0])
@pytest.mark.parametrize("binades", [18.3, 22.6, 25.5, 28.0])
def test_cells_far_below_the_largest(binades, at, n, n_seq):
    # One cell with V = 0 (a sink), `binades` above all others: the output is the others' share alone, n 2^-binades of
    # their mean.  A row's maximum is held as 2^7 or more, so an other cell's P is 2^(7 - binades) or more and off by at
    # most 2^-25 (half of fp16's smallest step; 2^-11 of itself where that is more); sums of n in fp32 add n 2^-24, and
    # 16 stands for the few roundings of a logit of 18 to 28 in fp32, in units of 2^-24 of it.  q.k^ and v^ are exact.
    rng = np.random.default_rng(int(binades * 10))
    ln2, sink = np.log(2.0), round(at * (n - 2))  # a cell before the drafted one
    v = rng.integers(0, 65, (n, 2, 256)).astype(np.int8)
    v[sink] = 0
    dev = {"kq": torch.zeros(n, 2, 256, dtype=torch.int8, device="cuda"), "vq": torch.from_numpy(v).cuda(),
           "ksc": torch.full((n, 2, 4), 2.0 ** -7, dtype=torch.float16, device="cuda"),
           "vsc": torch.full((n, 2, 4), 0.5, dtype=torch.float16, device="cuda")}
    dev["kq"][sink] = 64
    dev["ksc"][sink] = binades * ln2 / (SCALE * 256 * 64)
    q = torch.ones(n_seq, 24, 256, dtype=torch.float16, device="cuda")
    seqs = torch.tensor([[0, n, n - 1, i] for i in range(n_seq)], dtype=torch.int32, device="cuda")
    tree = torch.ones(n_seq, 1, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    params = (2048, 131072, SCALE)
    need = qsa.qsa_tree_attention_workspace_bytes(n_seq, n_seq, n, params)
    qsa.qsa_tree_attention(q, dev["kq"], dev["vq"], dev["ksc"], dev["vsc"], n, seqs, n_seq, n_seq, tree, n, None, out,
                           torch.empty(max(need, 1), dtype=torch.uint8, device="cuda"), params=params)
    qsa.qsa_check_device_status()
    z = SCALE * 256 * 64 * float(dev["ksc"][sink, 0, 0])
    want = np.repeat(0.5 * v.sum(0, dtype=np.float64) / (np.exp(z) + n - 1), 12, axis=0)
    p = 2.0 ** (7 - z / ln2)
    rel = max(2.0 ** -25 / p, 2.0 ** -11) + n * 2.0 ** -24 + 16 * z * 2.0 ** -24
    off = np.abs(out.double().cpu().numpy() - want)
    assert (off <= want * (rel + 2.0 ** -11) + 2.0 ** -25).all(), f"{(off / want).max():.3e} off, {rel:.3e} allowed"


@pytest.mark.parametrize("path,n", [("clusters", 3), ("together", 20)])  # few tokens a sequence, and many
@pytest.mark.parametrize("how", ["first row", "next row"])
def test_first_rows_that_break_the_table(how, path, n):
    # the table's first sequence starts behind row 0; a sequence's tokens end behind the call's rows.  Either is
    # skipped and flagged, whichever way the selected tokens would have taken
    pool, seqs = make_batch([(2200, n), (2300, n)], seed=42, slack=40)
    bad = seqs.copy()
    if how == "first row":
        bad[0, 3], skipped, kept = 1, slice(0, n), range(n, 2 * n)
    else:
        bad = np.concatenate([seqs, [[0, 50, 10, 2 * n + 5]]]).astype(np.int32)
        skipped, kept = slice(n, 2 * n), range(n)
    ids, out = run_tree(pool, bad, max_n_kv=2400)
    with pytest.raises(qsa.QSAError) as e:
        qsa.qsa_check_device_status()
    assert e.value.code == qsa.QSA_ERR_DEVICE
    assert torch.isnan(out[skipped]).all() and (ids[skipped] == -7).all()
    ref, ref_ids, bound = reference(pool, seqs, rows=set(kept))
    use = list(kept)
    assert (np.abs(out.double().cpu().numpy()[use] - ref[use]) <= bound[use]).all()
    np.testing.assert_array_equal(ids.cpu().numpy()[use], ref_ids[use])


@pytest.mark.parametrize("params", [None, (2048, 131072, SCALE)])
def test_one_workspace_for_every_smaller_call(params):
    # the workspace of a server's largest batch, between guards, serves calls of all kinds; each writes inside what its
    # own query says
    calls = [[(1950, 8)] * 16, [(9000, 5)] * 3, [(16000, 16)], [(700, 30), (4000, 9), (0, 1)], [(300, 4)] * 40, [(2500, 2)] * 5]
    whole = qsa.qsa_tree_attention_workspace_bytes(40, 160, 16016, params)
    ws = torch.full((whole + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    for i, specs in enumerate(calls):
        pool, seqs = make_batch(specs, seed=70 + i)
        n_tok, max_n_kv = pool["q"].shape[0], max(p + n for p, n in specs)
        need = qsa.qsa_tree_attention_workspace_bytes(len(specs), n_tok, max_n_kv, params)
        assert need <= whole
        ws.fill_(0x5A)
        dev = {k: torch.from_numpy(v).cuda() for k, v in pool.items() if k != "tree"}
        out = torch.zeros(n_tok, 24, 256, dtype=torch.float16, device="cuda")
        qsa.qsa_tree_attention(dev["q"], dev["kq"], dev["vq"], dev["ksc"], dev["vsc"], len(pool["kq"]),
                               torch.from_numpy(seqs).cuda(), len(specs), n_tok, torch.from_numpy(pool["tree"].view(np.int32)).cuda(),
                               max_n_kv, None, out, ws[:whole], params=params)
        qsa.qsa_check_device_status()
        assert (ws[need:] == 0x5A).all()
        ref, _, bound = reference(pool, seqs, *(params or (2048, 2051, SCALE)))
        assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all(), specs


def random_pool(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = lambda: torch.randint(-127, 128, (n, 2, 256), generator=g, device="cuda", dtype=torch.int8)
    scales = lambda: (torch.rand(n, 2, 4, generator=g, device="cuda") * 0.015 + 0.005).half()
    return {"kq": codes(), "vq": codes(), "ksc": scales(), "vsc": scales()}


@pytest.mark.parametrize("n_seq,pos0,params", [
    (65535, 3, None),                # as many sequences as a call takes, one token each
    (257, 100, (40, 71, SCALE)),     # as many tokens: trees of 255, selecting together
    (32768, 90, (40, 71, SCALE)),    # two tokens each, a cluster for each of them
])
def test_the_largest_calls(n_seq, pos0, params):
    each = 65535 // n_seq
    n_tok = each * n_seq
    rng = np.random.default_rng(n_seq)
    base = rng.integers(0, pos0 + 1, n_seq)  # committed cells, 0 among them
    size = base + each
    cell0 = np.concatenate([[0], np.cumsum(size)[:-1]])
    seqs = np.stack([cell0, size, base, np.arange(n_seq) * each], 1).astype(np.int32)
    words = (each + 31) // 32
    masks = np.zeros((n_tok, words), np.uint32)
    row = np.arange(n_tok) % each
    for w in range(words):  # chains
        left = np.clip(row + 1 - 32 * w, 0, 32)
        masks[:, w] = ((np.uint64(1) << left.astype(np.uint64)) - np.uint64(1)).astype(np.uint32)
    pool = random_pool(int(size.sum()), n_seq)
    g = torch.Generator(device="cuda").manual_seed(n_seq)
    q = torch.randn(n_tok, 24, 256, generator=g, device="cuda").half()
    topk, max_n_kv = (params or (2048,))[0], int(size.max())
    ids = torch.full((n_tok, 2, topk), -7, dtype=torch.int32, device="cuda") if params else None
    out = torch.full_like(q, float("nan"))
    need = qsa.qsa_tree_attention_workspace_bytes(n_seq, n_tok, max_n_kv, params)
    qsa.qsa_tree_attention(q, pool["kq"], pool["vq"], pool["ksc"], pool["vsc"], len(pool["kq"]), torch.from_numpy(seqs).cuda(),
                           n_seq, n_tok, torch.from_numpy(masks.view(np.int32)).cuda(), max_n_kv, ids, out,
                           torch.empty(max(need, 1), dtype=torch.uint8, device="cuda"), params=params)
    qsa.qsa_check_device_status()
    assert torch.isfinite(out).all()
    for s in sorted({0, 1, n_seq // 2, n_seq - 2, n_seq - 1, *rng.integers(0, n_seq, 8)}):
        a, b = int(cell0[s]), int(cell0[s] + size[s])
        t = slice(s * each, (s + 1) * each)
        one = {k: v[a:b].cpu().numpy() for k, v in pool.items()} | {"q": q[t].cpu().numpy(), "tree": masks[t]}
        ref, ref_ids, bound = reference(one, np.array([[0, b - a, base[s], 0]]), *(params or (2048, 2051, SCALE)))
        assert (np.abs(out[t].double().cpu().numpy() - ref) <= bound).all(), s
        if params:
            np.testing.assert_array_equal(ids[t].cpu().numpy(), ref_ids)
