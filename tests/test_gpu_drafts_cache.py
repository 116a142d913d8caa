"""GPU parity: qsa_prep_batched, qsa_cache_read and qsa_cache_commit, and a whole drafting step of the
three with the tree attention, against the formulas in 64 bits and the oracle's quantiser."""
import numpy as np
import pytest
import torch

import oracle
from int8_kv_top_gb300 import qsa, synth
from tests.drafts_testutil import reference, tree_masks
from tests.qsa_testutil import rel_l2

pytestmark = pytest.mark.gpu
DEFAULT_ROPE = (10000.0, 256, 1e-6, (32, 48, 48))


def prep_reference(raw, gamma, pos, rope):
    """RMS norm with gain and rotation of rows [n][heads][256] in 64 bits."""
    base, rd, eps, sec = rope
    x = raw.astype(np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma.astype(np.float64)
    axes = np.repeat([0, 1, 2], sec) if pos.shape[1] == 3 else np.zeros(rd // 2, int)
    th = (pos[:, axes].astype(np.float64) * base ** (-2.0 * np.arange(rd // 2) / rd))[:, None]
    a, b = y[..., :rd // 2], y[..., rd // 2:rd]
    out = y.copy()
    out[..., :rd // 2] = a * np.cos(th) - b * np.sin(th)
    out[..., rd // 2:rd] = b * np.cos(th) + a * np.sin(th)
    # an element is off by the fp16 rounding (2^-11 of it, or half the smallest step) and by the fp32 steps
    # before it: the norm (about 12 roundings), cos and sin (2^-22) and the angle (2^-30 rad here, or
    # |pos| 2^-52 rad for the frequency's own rounding), all relative to the pair's size
    size = np.abs(y)
    pair = size.copy()
    pair[..., :rd // 2] = pair[..., rd // 2:rd] = size[..., :rd // 2] + size[..., rd // 2:rd]
    off = np.abs(pos).max(-1).astype(np.float64)[:, None, None] * 2.0 ** -51
    return out, np.abs(out) * 2.0 ** -11 + 2.0 ** -25 + pair * (16 * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -29 + off)


def random_cache(n_pool, rng):
    return {"kq": rng.integers(-127, 128, (n_pool, 2, 256), dtype=np.int8), "vq": rng.integers(-127, 128, (n_pool, 2, 256), dtype=np.int8),
            "ksc": rng.uniform(0.005, 0.02, (n_pool, 2, 4)).astype(np.float16), "vsc": rng.uniform(0.005, 0.02, (n_pool, 2, 4)).astype(np.float16)}


def on_gpu(d):
    return {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in d.items()}


def check_prep(T, pos, rope=None, pad=(), seed=0, fused=False, with_kcur=True):
    rng = np.random.default_rng(seed)
    inp = synth.prep_inputs(T, seed=300 + seed)
    n_pool = 3 * T + 4
    cells = rng.permutation(n_pool)[:T].astype(np.int32)
    cells[list(pad)] = -1
    before = random_cache(n_pool, rng)
    dev, cache = on_gpu(inp), on_gpu(before)
    if fused:  # a token's q, k and v rows beside one another, and other columns behind them
        wide = torch.full((T, 28 * 256 + 64), float("nan"), dtype=torch.float16, device="cuda")
        wide[:, :6144] = dev["q_raw"].view(T, -1)
        wide[:, 6144:6656] = dev["k_raw"].view(T, -1)
        wide[:, 6656:7168] = dev["v_raw"].view(T, -1)
        dev["q_raw"], dev["k_raw"], dev["v_raw"] = wide[:, :6144], wide[:, 6144:6656], wide[:, 6656:7168]
    qcur = torch.full((T, 24, 256), float("nan"), dtype=torch.float16, device="cuda")
    kcur = torch.full((T, 2, 256), float("nan"), dtype=torch.float16, device="cuda") if with_kcur else None
    qsa.qsa_prep_batched(dev["q_raw"], dev["k_raw"], dev["v_raw"], dev["q_gamma"], dev["k_gamma"],
                         torch.from_numpy(pos).cuda(), torch.from_numpy(cells).cuda(), T, n_pool, qcur, kcur, cache["kq"],
                         cache["ksc"], cache["vq"], cache["vsc"], rope=rope)
    qsa.qsa_check_device_status()
    use = cells >= 0
    r = rope or DEFAULT_ROPE
    p2 = pos.reshape(T, -1)
    want, bound = prep_reference(inp["q_raw"], inp["q_gamma"], p2, r)
    got = qcur.cpu().numpy()
    assert (np.abs(got[use].astype(np.float64) - want[use]) <= bound[use]).all()
    assert np.isnan(got[~use]).all()
    after = {k: v.cpu().numpy() for k, v in cache.items()}
    if with_kcur:
        want, bound = prep_reference(inp["k_raw"], inp["k_gamma"], p2, r)
        got = kcur.cpu().numpy()
        assert (np.abs(got[use].astype(np.float64) - want[use]) <= bound[use]).all()
        assert np.isnan(got[~use]).all()
        kq, ksc = oracle.quantize(got[use])
        np.testing.assert_array_equal(after["kq"][cells[use]], kq)
        np.testing.assert_array_equal(after["ksc"][cells[use]].view(np.uint16), ksc.view(np.uint16))
    vq, vsc = oracle.quantize(inp["v_raw"][use])
    np.testing.assert_array_equal(after["vq"][cells[use]], vq)
    np.testing.assert_array_equal(after["vsc"][cells[use]].view(np.uint16), vsc.view(np.uint16))
    other = np.ones(n_pool, bool)
    other[cells[use]] = False
    for k in before:
        np.testing.assert_array_equal(after[k][other].view(np.uint8), before[k][other].view(np.uint8))


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 64, 333, 1500])
@pytest.mark.parametrize("fused", [False, True])
def test_prep_batched(T, fused):
    pos = np.random.default_rng(T).integers(0, 40000, T).astype(np.int32)
    check_prep(T, pos, seed=T, fused=fused, pad=range(T - T // 5, T))


@pytest.mark.parametrize("rd", [16, 32, 64, 128, 256])
def test_prep_batched_three_axes(rd):
    third = rd // 2 // 8 * 3
    pos = np.random.default_rng(rd).integers(0, 5000, (37, 3)).astype(np.int32)
    check_prep(37, pos, rope=(500000.0, rd, 1e-5, (rd // 2 - 2 * third, third, third)), seed=rd, with_kcur=rd != 64)
    check_prep(5, pos[:5], rope=(10000.0, rd, 1e-5, (0, rd // 2, 0)), seed=rd + 1)


@pytest.mark.parametrize("pos", [[0, 1, -1], [131071, 131072, 131073], [2**24 + 1, 2**31 - 1, -2**31], [-40000, 999999, 10**9]])
def test_prep_batched_far_positions(pos):
    check_prep(3, np.array(pos, np.int32), seed=3)


def test_prep_batched_rows_of_zeros_and_extremes():
    T = 4
    inp = synth.prep_inputs(T, seed=9)
    inp["k_raw"][0], inp["v_raw"][0], inp["q_raw"][0] = 0, 0, 0
    inp["v_raw"][1] = np.float16(65504)
    inp["v_raw"][2] = np.float16(6e-8)
    inp["v_raw"][3, :, ::2] = -65504
    dev, cache = on_gpu(inp), on_gpu(random_cache(8, np.random.default_rng(1)))
    qcur, kcur = (torch.empty(T, h, 256, dtype=torch.float16, device="cuda") for h in (24, 2))
    qsa.qsa_prep_batched(dev["q_raw"], dev["k_raw"], dev["v_raw"], dev["q_gamma"], dev["k_gamma"],
                         torch.arange(T, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda"),
                         T, 8, qcur, kcur, cache["kq"], cache["ksc"], cache["vq"], cache["vsc"])
    qsa.qsa_check_device_status()
    for rows, c, sc in ((kcur.cpu().numpy(), "kq", "ksc"), (inp["v_raw"], "vq", "vsc")):
        codes, scales = oracle.quantize(rows)
        np.testing.assert_array_equal(cache[c][:T].cpu().numpy(), codes)
        np.testing.assert_array_equal(cache[sc][:T].cpu().numpy().view(np.uint16), scales.view(np.uint16))
    assert (qcur[0] == 0).all()


def test_prep_batched_matches_the_one_sequence_prep():
    T, pos0 = 50, 1000
    inp = synth.prep_inputs(T, seed=10)
    dev = on_gpu(inp)
    got = []
    for batched in (False, True):
        cache = on_gpu(random_cache(pos0 + T, np.random.default_rng(2)))
        q, k = (torch.empty(T, h, 256, dtype=torch.float16, device="cuda") for h in (24, 2))
        if batched:
            at = torch.arange(pos0, pos0 + T, dtype=torch.int32, device="cuda")
            qsa.qsa_prep_batched(dev["q_raw"], dev["k_raw"], dev["v_raw"], dev["q_gamma"], dev["k_gamma"], at, at, T,
                                 pos0 + T, q, k, cache["kq"], cache["ksc"], cache["vq"], cache["vsc"])
        else:
            qsa.qsa_prep(dev["q_raw"], dev["k_raw"], dev["v_raw"], dev["q_gamma"], dev["k_gamma"], T, pos0, pos0 + T, q, k,
                         cache["kq"], cache["ksc"], cache["vq"], cache["vsc"])
        qsa.qsa_check_device_status()
        got.append((q, k, cache))
    (q0, k0, c0), (q1, k1, c1) = got
    # both are one fp16 rounding from values that agree to fp32: a rounding border apart at most
    assert rel_l2(q1.float().cpu(), q0.float().cpu()) <= 2.0 ** -13 and rel_l2(k1.float().cpu(), k0.float().cpu()) <= 2.0 ** -13
    assert torch.equal(c0["vq"], c1["vq"]) and torch.equal(c0["vsc"], c1["vsc"])
    assert ((c0["kq"].int() - c1["kq"].int()).abs() <= 1).all()


def test_prep_batched_flags_cells_outside_the_pool():
    T = 6
    inp = synth.prep_inputs(T, seed=11)
    dev, before = on_gpu(inp), random_cache(10, np.random.default_rng(3))
    for bad in (10, -2, 2**31 - 1, -2**31):
        cache = on_gpu(before)
        q = torch.full((T, 24, 256), float("nan"), dtype=torch.float16, device="cuda")
        cells = torch.tensor([3, 1, bad, 5, -1, 7], dtype=torch.int64).to(torch.int32).cuda()
        qsa.qsa_prep_batched(dev["q_raw"], dev["k_raw"], dev["v_raw"], dev["q_gamma"], dev["k_gamma"],
                             torch.arange(T, dtype=torch.int32, device="cuda"), cells, T, 10, q, None, cache["kq"], cache["ksc"],
                             cache["vq"], cache["vsc"])
        with pytest.raises(qsa.QSAError) as e:
            qsa.qsa_check_device_status()
        assert e.value.code == qsa.QSA_ERR_DEVICE
        assert torch.isnan(q[2]).all() and torch.isnan(q[4]).all() and not torch.isnan(q[[0, 1, 3, 5]]).any()
        vq, _ = oracle.quantize(inp["v_raw"][[0, 1, 3, 5]])
        np.testing.assert_array_equal(cache["vq"][[3, 1, 5, 7]].cpu().numpy(), vq)
        for i in (0, 2, 4, 6, 8, 9):
            np.testing.assert_array_equal(cache["vq"][i].cpu().numpy(), before["vq"][i])


# ----------------------------------------------------------------------------------- read
def read_reference(codes, scales):
    """fp16 rounding of code * scale, which float32 holds exactly."""
    return (codes.astype(np.float32) * np.repeat(scales.astype(np.float32), 64, axis=-1)).astype(np.float16)


@pytest.mark.parametrize("n,n_pool", [(1, 1), (1, 9), (7, 20), (64, 64), (1001, 5000), (40000, 30000)])
def test_cache_read(n, n_pool):
    rng = np.random.default_rng(n)
    pool = random_cache(n_pool, rng)
    pool["kq"][0], pool["ksc"][0] = -128, np.float16(6e-8)          # codes the quantiser does not make, subnormal scales
    pool["vsc"][-1] = [[np.inf, 0.0, -0.0, 500.0], [np.float16(6e-8), 1.0, -2.0, 65504.0]]
    cells = rng.integers(0, n_pool, n).astype(np.int32)              # repeats among them
    cells[0], cells[-1] = 0, n_pool - 1
    skip = rng.random(n) < (0.1 if n > 2 else 0.0)
    cells[skip] = -1
    dev = on_gpu(pool)
    at = torch.from_numpy(cells).cuda()
    k16, v16 = (torch.full((n, 2, 256), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    qsa.qsa_cache_read(dev["kq"], dev["ksc"], dev["vq"], dev["vsc"], n_pool, at, n, k16, v16)
    qsa.qsa_check_device_status()
    with np.errstate(all="ignore"):
        for got, c, s in ((k16, "kq", "ksc"), (v16, "vq", "vsc")):
            want = read_reference(pool[c][cells], pool[s][cells])
            want[skip] = 7.0
            np.testing.assert_array_equal(got.cpu().numpy(), want)
    for which in range(2):  # one of the two alone, the other's arrays not given
        alone = torch.full((n, 2, 256), 7.0, dtype=torch.float16, device="cuda")
        if which == 0:
            qsa.qsa_cache_read(dev["kq"], dev["ksc"], None, None, n_pool, at, n, alone, None)
        else:
            qsa.qsa_cache_read(None, None, dev["vq"], dev["vsc"], n_pool, at, n, None, alone)
        qsa.qsa_check_device_status()
        assert np.array_equal(alone.cpu().numpy(), (k16, v16)[which].cpu().numpy(), equal_nan=True)


def test_cache_read_flags_cells_outside_the_pool():
    pool = on_gpu(random_cache(5, np.random.default_rng(1)))
    for bad in (5, -2, 2**31 - 1):
        out = torch.full((3, 2, 256), 7.0, dtype=torch.float16, device="cuda")
        cells = torch.tensor([1, bad, 4], dtype=torch.int32, device="cuda")
        qsa.qsa_cache_read(pool["kq"], pool["ksc"], None, None, 5, cells, 3, out, None)
        with pytest.raises(qsa.QSAError) as e:
            qsa.qsa_check_device_status()
        assert e.value.code == qsa.QSA_ERR_DEVICE
        assert (out[1] == 7).all() and (out[0] != 7).any() and (out[2] != 7).any()


def test_cache_read_past_four_gigabytes():
    n_pool = 9_000_000
    kq = torch.zeros(n_pool, 2, 256, dtype=torch.int8, device="cuda")
    ksc = torch.zeros(n_pool, 2, 4, dtype=torch.float16, device="cuda")
    kq[-1], ksc[-1], kq[8_500_000], ksc[8_500_000] = 3, 0.5, -7, 0.25
    out = torch.empty(2, 2, 256, dtype=torch.float16, device="cuda")
    qsa.qsa_cache_read(kq, ksc, None, None, n_pool, torch.tensor([n_pool - 1, 8_500_000], dtype=torch.int32, device="cuda"), 2, out, None)
    qsa.qsa_check_device_status()
    assert (out[0] == 1.5).all() and (out[1] == -1.75).all()


# ----------------------------------------------------------------------------------- commit
def commit_reference(pool, seqs, path, n_path):
    new = {k: v.copy() for k, v in pool.items()}
    for (c0, n, pos0, _), p, m in zip(seqs, path, n_path):
        if n > 0 and m > 0:
            for k in new:
                new[k][c0 + pos0:c0 + pos0 + m] = pool[k][c0 + pos0 + p[:m]]
    return new


def run_commit(pool, seqs, path, n_path):
    dev = on_gpu(pool)
    qsa.qsa_cache_commit(dev["kq"], dev["ksc"], dev["vq"], dev["vsc"], len(pool["kq"]), torch.from_numpy(seqs).cuda(), len(seqs),
                         torch.from_numpy(path).cuda(), torch.from_numpy(n_path).cuda())
    return dev


@pytest.mark.parametrize("n_seq,t_max,cap", [(1, 1, 1), (1, 8, 5), (3, 17, 9), (40, 64, 33), (2, 256, 256), (300, 5, 5)])
def test_commit(n_seq, t_max, cap):
    rng = np.random.default_rng(n_seq + t_max)
    seqs, path, n_path, c0 = [], [], [], 0
    for s in range(n_seq):
        t, pos0 = (t_max, 3) if s == 0 else (int(rng.integers(1, t_max + 1)), int(rng.integers(0, 50)))
        m = min(cap, t) if s == 0 else int(rng.integers(0, min(cap, t) + 1))
        p = np.sort(rng.choice(t, m, replace=False))
        if s == 0 and m > 1:  # the longest shift: the path's last cells
            p = np.arange(t - m, t)
        path.append(np.concatenate([p, np.full(cap - m, -9)]))
        n_path.append(m)
        n = pos0 + t + int(rng.integers(0, 4))
        seqs.append((c0, n, pos0, 0))
        c0 += n
    seqs, path, n_path = np.array(seqs, np.int32), np.array(path, np.int32), np.array(n_path, np.int32)
    pool = random_cache(c0, rng)
    dev = run_commit(pool, seqs, path, n_path)
    qsa.qsa_check_device_status()
    want = commit_reference(pool, seqs, path, n_path)
    for k in pool:
        np.testing.assert_array_equal(dev[k].cpu().numpy().view(np.uint8), want[k].view(np.uint8))


@pytest.mark.parametrize("how", ["order", "twice", "negative", "past", "count", "count<0", "cells", "pool"])
def test_commit_leaves_and_flags_a_bad_sequence(how):
    rng = np.random.default_rng(4)
    pool = random_cache(60, rng)
    seqs = np.array([(0, 20, 5, 0), (20, 20, 5, 0), (40, 20, 5, 0), (50, 0, 3, 0)], np.int32)  # the last: padding
    path = np.array([[1, 3, 7, 9]] * 4, np.int32)
    n_path = np.array([4, 4, 3, 4], np.int32)
    if how == "order":
        path[1] = [1, 7, 3, 9]
    elif how == "twice":
        path[1] = [1, 3, 3, 9]
    elif how == "negative":
        path[1] = [-1, 3, 7, 9]
    elif how == "past":
        path[1] = [1, 3, 7, 15]
    elif how == "count":
        n_path[1] = 5
    elif how == "count<0":
        n_path[1] = -1
    elif how == "cells":
        seqs[1, 1] = -20
    else:
        seqs[1, 0] = 41
    dev = run_commit(pool, seqs, path, n_path)
    with pytest.raises(qsa.QSAError) as e:
        qsa.qsa_check_device_status()
    assert e.value.code == qsa.QSA_ERR_DEVICE
    n_good = np.array([4, 0, 3, 0], np.int32)
    want = commit_reference(pool, seqs, path, n_good)
    for k in pool:
        np.testing.assert_array_equal(dev[k].cpu().numpy().view(np.uint8), want[k].view(np.uint8))


# ----------------------------------------------------------------------------------- a whole step
@pytest.mark.parametrize("pos0s", [(40, 700, 1990), (2046, 2600, 0)])
def test_a_drafting_step(pos0s):
    """Draft, attend, commit, and decode on: an accepted path's tokens get what decoding them one by one gives,
    and the committed cache is what one-by-one decoding leaves."""
    rng = np.random.default_rng(sum(pos0s))
    parents = [[-1, 0, 0, 1, 2, 4, 3], [-1, -1, 1, 2, 0], [-1, 0, 1, 2, 1, 4, 5, 5]]
    paths = [[0, 2, 4, 5], [1, 2, 3], [0, 1, 4, 5, 7]]
    n_tok = sum(map(len, parents))
    raw = synth.prep_inputs(n_tok, seed=33)
    base = random_cache(sum(pos0s) + n_tok + 3 * 4, rng)
    n_pool = len(base["kq"])
    seqs, cells, pos, masks, c0, t0 = [], [], [], [], 0, 0
    for p0, par in zip(pos0s, parents):
        seqs.append((c0, p0 + len(par) + 4, p0, t0))
        depth = []
        for q in par:
            depth.append(depth[q] + 1 if q >= 0 else 0)
        cells += [c0 + p0 + i for i in range(len(par))]
        pos += [p0 + d for d in depth]
        masks.append(tree_masks(par, 1))
        c0 += p0 + len(par) + 4
        t0 += len(par)
    seqs = np.array(seqs, np.int32)
    dev, cache = on_gpu(raw), on_gpu(base)
    table, tree = torch.from_numpy(seqs).cuda(), torch.from_numpy(np.concatenate(masks).view(np.int32)).cuda()
    max_n_kv = max(pos0s) + 8
    q, out = (torch.empty(n_tok, 24, 256, dtype=torch.float16, device="cuda") for _ in range(2))
    need = qsa.qsa_tree_attention_workspace_bytes(3, n_tok, max_n_kv)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    args = (dev["q_raw"], dev["k_raw"], dev["v_raw"], dev["q_gamma"], dev["k_gamma"])
    qsa.qsa_prep_batched(*args, torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.tensor(cells, dtype=torch.int32, device="cuda"),
                         n_tok, n_pool, q, None, cache["kq"], cache["ksc"], cache["vq"], cache["vsc"])
    qsa.qsa_tree_attention(q, cache["kq"], cache["vq"], cache["ksc"], cache["vsc"], n_pool, table, 3, n_tok, tree, max_n_kv, None, out, ws)
    path = np.zeros((3, 5), np.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = p
    qsa.qsa_cache_commit(cache["kq"], cache["ksc"], cache["vq"], cache["vsc"], n_pool, table, 3, torch.from_numpy(path).cuda(),
                         torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda"))
    # the attention itself, on what the prep wrote
    after = {k: v.cpu().numpy() for k, v in cache.items()}
    # one by one: prep at the path's own positions and cells, then a decode over the committed cells
    one = on_gpu(base)
    for i, (p0, p) in enumerate(zip(pos0s, paths)):
        rows = torch.tensor([int(seqs[i][3]) + j for j in p], device="cuda")
        m = len(p)
        at = torch.arange(p0, p0 + m, dtype=torch.int32, device="cuda")
        qi = torch.empty(m, 24, 256, dtype=torch.float16, device="cuda")
        qsa.qsa_prep_batched(dev["q_raw"][rows], dev["k_raw"][rows], dev["v_raw"][rows], dev["q_gamma"], dev["k_gamma"], at,
                             at + int(seqs[i][0]), m, n_pool, qi, None, one["kq"], one["ksc"], one["vq"], one["vsc"])
        assert torch.equal(qi, q[rows])
        lo = int(seqs[i][0])
        sub = {k: one[k][lo:lo + p0 + m].contiguous() for k in one}
        xp = torch.empty(m, 24, 256, dtype=torch.float32, device="cuda")
        qsa.qsa_decode_layer(qi, sub["kq"], sub["vq"], sub["ksc"], sub["vsc"], p0 + m, m, p0, None, xp)
        qsa.qsa_check_device_status()
        assert rel_l2(out[rows].float().cpu(), xp.cpu()) <= 2e-3  # each within 1e-3 of the exact result
        for k in one:
            np.testing.assert_array_equal(after[k][lo:lo + p0 + m].view(np.uint8), one[k][lo:lo + p0 + m].cpu().numpy().view(np.uint8))
