"""GPU parity: qsa_tree_verify against its definition in whole numbers, entry for entry."""
import numpy as np
import pytest
import torch

from int8_kv_top_gb300 import qsa
from tests.prompts_testutil import verified

pytestmark = pytest.mark.gpu


def softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def batch(counts, vocab, seed, bush=3, near=0.4, peak=3.0):
    """p, d, token, parent, u, u_end and first rows of sequences with `counts` tokens."""
    rng = np.random.default_rng(seed)
    n = sum(counts)
    p = softmax(rng.normal(size=(n, vocab)) * peak)
    d = softmax(near * rng.normal(size=(n, vocab)) * peak + np.log(p.astype(np.float64) + 1e-30))
    first = np.concatenate([[0], np.cumsum(counts)[:-1]]).astype(int)
    parent = np.concatenate([[-1] + [int(rng.integers(max(0, i - bush), i)) for i in range(1, t)] for t in counts if t] or [[]]).astype(np.int32)
    token = np.zeros(n, np.int32)
    for r0, t in zip(first, counts):
        for k in range(1, t):
            row = d[r0 + parent[r0 + k]].astype(np.float64)
            token[r0 + k] = rng.choice(vocab, p=row / row.sum())
    return dict(p=p, d=d, token=token, parent=parent, u=rng.random(n, np.float32), u_end=rng.random(len(counts), np.float32), first=first)


def run(b, n_seq, vocab, cap, points=False, stride=None, offset=0, cells=None):
    n = len(b["token"])

    def rows(x):
        if x is None:
            return None
        wide = torch.full((n * (stride or vocab) + offset,), float("nan"), device="cuda")
        v = wide[offset:].view(n, stride or vocab)
        v[:, :vocab] = torch.from_numpy(x).cuda()
        return v

    seqs = np.zeros((n_seq, 4), np.int32)
    seqs[:, 1] = 10 if cells is None else cells
    seqs[:, 3] = b["first"]
    path = torch.full((n_seq, cap), -7, dtype=torch.int32, device="cuda")
    n_path, after = (torch.full((n_seq,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    t = {k: torch.from_numpy(np.ascontiguousarray(b[k])).cuda() for k in ("token", "parent", "u", "u_end")}
    qsa.qsa_tree_verify(rows(b["p"]), None if points else rows(b["d"]), vocab, t["token"], t["parent"], t["u"], t["u_end"],
                        torch.from_numpy(seqs).cuda(), n_seq, n, path, n_path, after)
    return path.cpu().numpy(), n_path.cpu().numpy(), after.cpu().numpy()


def check(b, counts, got, cap, points=False):
    path, n_path, after = got
    for s, (r0, t) in enumerate(zip(b["first"], counts)):
        if t == 0:
            assert n_path[s] == 0 and after[s] == -1
            continue
        r = slice(r0, r0 + t)
        way, x = verified(b["p"][r], None if points else b["d"][r], b["token"][r], b["parent"][r], b["u"][r], b["u_end"][s], cap)
        assert n_path[s] == len(way) and path[s, :len(way)].tolist() == way, s
        assert (path[s, len(way):] == -7).all()
        assert after[s] == x, (s, after[s], x)


@pytest.mark.parametrize("points", [False, True])
@pytest.mark.parametrize("counts,vocab,bush", [([1], 1, 1), ([1, 2], 2, 1), ([5], 3, 4), ([8], 100, 1), ([256], 77, 9), ([3, 0, 7, 1, 0], 1023, 3),
                                               ([16] * 3, 1024, 4), ([30, 2, 11], 1025, 6), ([6] * 40, 4099, 5), ([12], 32768, 12),
                                               ([4, 9], 131071, 5), ([3] * 200, 300, 2), ([5], 262144, 4)])
def test_against_the_definition(points, counts, vocab, bush):
    for seed, near in ((1, 0.4), (2, 2.0)):
        b = batch(counts, vocab, seed, bush, near)
        cap = max(max(counts), 1)
        check(b, counts, run(b, len(counts), vocab, cap, points), cap, points)
    qsa.qsa_check_device_status()


@pytest.mark.parametrize("points", [False, True])
def test_many_refusals_at_one_token(points):
    # bushes under the root, drafted from a distribution far from the target's: several masses in a row, repeated tokens among them
    counts, vocab = [40, 25, 60], 50
    b = batch(counts, vocab, 3, bush=1, near=3.0)
    for r0, t in zip(b["first"], counts):
        b["parent"][r0 + 1:r0 + t] = 0
    b["u"][:] = np.maximum(b["u"], 0.6)
    check(b, counts, run(b, 3, vocab, 60, points), 60, points)
    qsa.qsa_check_device_status()


@pytest.mark.parametrize("stride,offset", [(104, 0), (104, 4), (101, 0), (104, 1), (107, 3)])
def test_strides_and_alignment(stride, offset):
    counts = [9, 4, 13]
    b = batch(counts, 101, 4)
    check(b, counts, run(b, 3, 101, 13, stride=stride, offset=offset), 13)


@pytest.mark.parametrize("cap", [1, 2, 5])
def test_a_short_path_buffer_ends_the_walk(cap):
    counts = [12] * 6
    b = batch(counts, 64, 5, bush=1, near=0.1)
    got = run(b, 6, 64, cap)
    assert got[1].max() == cap
    check(b, counts, got, cap)


@pytest.mark.parametrize("points", [False, True])
def test_degenerate_rows(points):
    counts, vocab = [3] * 8, 10
    b = batch(counts, vocab, 6)
    b["parent"][:] = np.tile([-1, 0, 0], 8)
    b["u"][:] = 0.999
    p, d = b["p"].reshape(8, 3, vocab), b["d"].reshape(8, 3, vocab)
    p[0] = d[0]                       # equal: nothing is refused
    p[1] = 0                          # no mass at all
    p[2, :, :] = np.eye(vocab, dtype=np.float32)[4]  # one entry has all of it
    p[3, 0, 2], d[3, 0, 5] = np.nan, np.nan
    p[4, 0, 1], p[4, 0, 7] = -0.5, 1.5
    d[5] = 1                          # more than a distribution: nothing is left of the row
    d[6] = 0                          # a drafter that could not have drawn these
    b["u_end"][:] = [0, 0.5, 0.999, 0, 1 - 2.0 ** -24, 0.3, 2.0 ** -60, 0.7]
    got = run(b, 8, vocab, 3, points)
    check(b, counts, got, 3, points)
    assert got[2][1] == -1 and got[2][2] == 4
    qsa.qsa_check_device_status()


@pytest.mark.parametrize("how", ["token", "token<0", "parent", "parent<0", "root", "rows", "order", "count"])
def test_a_bad_sequence_is_flagged_and_gets_no_path(how):
    counts, vocab = [4, 300 if how == "count" else 5, 6], 33
    b = batch([4, counts[1], 6], vocab, 7)
    r = b["first"][1]
    if how == "token":
        b["token"][r + 2] = vocab
    elif how == "token<0":
        b["token"][r + 2] = -1
    elif how == "parent":
        b["parent"][r + 2] = 2
    elif how == "parent<0":
        b["parent"][r + 2] = -1
    elif how == "root":
        b["parent"][r] = 0
    elif how == "rows":
        b["first"] = np.array([0, r + 7, r + 5])
    elif how == "order":
        b["first"] = np.array([0, -1, r + 5])
    path, n_path, after = run(b, 3, vocab, 8)
    with pytest.raises(qsa.QSAError) as e:
        qsa.qsa_check_device_status()
    assert e.value.code == qsa.QSA_ERR_DEVICE
    assert n_path[1] == 0 and after[1] == -1 and (path[1] == -7).all()
    good = [2] if how in ("rows", "order") else [0, 2]
    for s in good:
        r0, t = b["first"][s], counts[s]
        way, x = verified(b["p"][r0:r0 + t], b["d"][r0:r0 + t], b["token"][r0:r0 + t], b["parent"][r0:r0 + t], b["u"][r0:r0 + t], b["u_end"][s], 8)
        assert n_path[s] == len(way) and after[s] == x


def test_padding_sequences_and_rows_behind_the_last():
    counts = [4, 5, 6]
    b = batch(counts, 50, 8)
    got = run(b, 3, 50, 6, cells=[10, 0, 10])
    assert got[1][1] == 0 and got[2][1] == -1
    check(b, [4, 0, 6], got, 6)
    qsa.qsa_check_device_status()


def test_no_tokens():
    n_path, after = (torch.full((2,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    seqs = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    qsa.qsa_tree_verify(None, None, 10, None, None, None, torch.zeros(2, device="cuda"), seqs, 2, 0,
                        torch.zeros(2, 1, dtype=torch.int32, device="cuda"), n_path, after)
    qsa.qsa_check_device_status()
    assert n_path.tolist() == [0, 0] and after.tolist() == [-1, -1]


@pytest.mark.parametrize("points", [False, True])
def test_the_first_token_has_the_targets_distribution(points):
    # 20,000 sequences with two candidates from the same distribution; the token behind the root is an accepted one or `next`.  Counts
    # of a sample of n are off by a standard deviation sqrt(n p (1 - p)); six of them are passed with a chance of 2e-9.
    rng = np.random.default_rng(11)
    n_seq, vocab = 20000, 9
    p, d = softmax(rng.normal(size=vocab)), softmax(rng.normal(size=vocab))
    q = rng.choice(vocab, (n_seq, 3), p=d.astype(np.float64) / d.sum(dtype=np.float64)).astype(np.int32)
    if points:
        q[:, 1:] = [3, 5]
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    rows = np.repeat(p[None], 3 * n_seq, 0)
    seqs = np.stack([np.zeros(n_seq), np.full(n_seq, 4), np.zeros(n_seq), 3 * np.arange(n_seq)], 1).astype(np.int32)
    path = torch.zeros(n_seq, 3, dtype=torch.int32, device="cuda")
    n_path, after = (torch.zeros(n_seq, dtype=torch.int32, device="cuda") for _ in range(2))
    qsa.qsa_tree_verify(dev(rows), None if points else dev(np.repeat(d[None], 3 * n_seq, 0)), vocab, dev(q.reshape(-1)),
                        dev(np.tile([-1, 0, 0], n_seq).astype(np.int32)), dev(rng.random(3 * n_seq, np.float32)),
                        dev(rng.random(n_seq, np.float32)), dev(seqs), n_seq, 3 * n_seq, path, n_path, after)
    qsa.qsa_check_device_status()
    path, n_path, after = path.cpu().numpy(), n_path.cpu().numpy(), after.cpu().numpy()
    first = np.where(n_path > 1, q[np.arange(n_seq), path[:, 1]], after)
    count = np.bincount(first, minlength=vocab)
    want = p.astype(np.float64) / p.sum(dtype=np.float64)
    assert (np.abs(count - n_seq * want) < 6 * np.sqrt(n_seq * want * (1 - want)) + 1).all(), (count, n_seq * want)


def test_verify_feeds_the_commit():
    # path and n_path go to qsa_cache_commit as they are
    rng = np.random.default_rng(12)
    counts, vocab = [6, 9, 3], 40
    b = batch(counts, vocab, 13, near=0.1)
    seqs = torch.tensor([[0, 30, 20, 0], [30, 40, 25, 6], [70, 20, 11, 15]], dtype=torch.int32, device="cuda")
    kq = torch.from_numpy(rng.integers(-127, 128, (90, 2, 256), dtype=np.int8)).cuda()
    sc = torch.rand(90, 2, 4, device="cuda").half()
    vq, vsc, before = kq.clone(), sc.clone(), kq.cpu().numpy()
    path = torch.full((3, 9), -1, dtype=torch.int32, device="cuda")
    n_path, after = (torch.zeros(3, dtype=torch.int32, device="cuda") for _ in range(2))
    t = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in b.items() if k != "first"}
    qsa.qsa_tree_verify(t["p"], t["d"], vocab, t["token"], t["parent"], t["u"], t["u_end"], seqs, 3, 18, path, n_path, after)
    qsa.qsa_cache_commit(kq, sc, vq, vsc, 90, seqs, 3, path, n_path)
    qsa.qsa_check_device_status()
    for s, (c0, _, pos0, r0) in enumerate(seqs.tolist()):
        way, _ = verified(b["p"][r0:], b["d"][r0:], b["token"][r0:r0 + counts[s]], b["parent"][r0:r0 + counts[s]], b["u"][r0:], b["u_end"][s], 9)
        for i, k in enumerate(way):
            np.testing.assert_array_equal(kq[c0 + pos0 + i].cpu().numpy(), before[c0 + pos0 + k])


UNIT = 2.0 ** -44


def plainly(b, r0, t, points, u_end):
    """(path, left-over row, its sum, refusals of it, least margin of a decision over its bound) in 64-bit floating point."""
    p, d = b["p"][r0:r0 + t].astype(np.float64), b["d"][r0:r0 + t].astype(np.float64)
    u, parent, token, vocab = b["u"][r0:r0 + t].astype(np.float64), b["parent"][r0:r0 + t], b["token"][r0:r0 + t], p.shape[1]
    way, w, c, r, margin = [0], p[0], 1.0, 0, np.inf
    for k in range(1, t):
        if parent[k] != way[-1]:
            continue
        x = token[k]
        base = np.eye(1, vocab, x)[0] if points else d[way[-1]]
        # an entry is rounded to a unit (half a unit each for p and d at the first refusal, one for each later product), and what
        # is left of c is the sum of vocab of them, times d at the next refusal
        off = (2 * r + 2) * UNIT * (1 + vocab * base[x]) + 2.0 ** -50
        margin = min(margin, abs(u[k] * c * base[x] - w[x]) / off)
        if u[k] * c * base[x] < w[x]:
            way, w, c, r = way + [k], p[k], 1.0, 0
            continue
        if points:
            c, w = c - w[x], np.where(np.arange(vocab) == x, 0.0, w)
        else:
            w = np.maximum(w - c * base, 0.0)
            c = w.sum()
        r += 1
    return way, w, r, margin


@pytest.mark.parametrize("points", [False, True])
@pytest.mark.parametrize("counts,vocab,bush,near", [([9] * 12, 131071, 3, 0.4), ([30, 2, 11] * 3, 100003, 6, 1.0), ([20] * 4, 262144, 12, 2.0)])
def test_large_vocabularies_against_plain_arithmetic_in_64_bits(points, counts, vocab, bush, near):
    b = batch(counts, vocab, 11, bush, near)
    path, n_path, after = run(b, len(counts), vocab, max(counts), points)
    qsa.qsa_check_device_status()
    close = 0
    for s, (r0, t) in enumerate(zip(b["first"], counts)):
        way, w, r, margin = plainly(b, r0, t, points, b["u_end"][s])
        if margin <= 1:  # a decision that the rounding may turn
            close += 1
            continue
        assert path[s, :n_path[s]].tolist() == way, s
        up = np.cumsum(w)
        at, x = float(b["u_end"][s]) * up[-1], after[s]
        off = 2 * vocab * (2 * r + 2) * UNIT  # of the running sum, and of the total
        assert up[x] > at - off and (x == 0 or up[x - 1] <= at + off), (s, x)
        assert w[x] > 0
    assert close <= 1
