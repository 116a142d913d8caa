"""GPU parity: qsa_cache_copy and qsa_cache_compact against their definitions, byte by byte."""
import numpy as np
import pytest
import torch

from int8_kv_top_gb300 import qsa
from tests.prompts_testutil import compacted, moved, on_gpu, random_cache, same_bytes

pytestmark = pytest.mark.gpu


def table(rows):
    return np.array([list(r) + [0] * (4 - len(r)) for r in rows], np.int32).reshape(-1, 4)


def run_copy(pool, runs, max_cells=None, stream=None):
    dev = on_gpu(pool)
    t = torch.from_numpy(table(runs)).cuda()
    qsa.qsa_cache_copy(dev["kq"], dev["ksc"], dev["vq"], dev["vsc"], len(pool["kq"]), t, len(runs),
                       max_cells if max_cells is not None else max(r[2] for r in runs), stream=stream)
    return dev


@pytest.mark.parametrize("lengths", [[1], [0, 1, 0, 2], [63, 64, 65], [500] * 3, list(range(40)), [3] * 1024, [1] * 1025, [2, 0, 5] * 800, [4100, 1, 700]],
                         ids=lambda x: f"{len(x)}x{max(x)}")
def test_copy(lengths):
    rng = np.random.default_rng(len(lengths))
    far = max(lengths) + 7
    runs, dst = [], far
    for n in lengths:
        dst += int(rng.integers(0, 3))
        runs.append((int(rng.integers(0, far - n + 1)), dst, n))
        dst += n
    pool = random_cache(dst + 3, rng)
    order = rng.permutation(len(runs))
    dev = run_copy(pool, [runs[i] for i in order])
    qsa.qsa_check_device_status()
    same_bytes(dev, moved(pool, runs))


def test_a_run_onto_itself_changes_nothing():
    pool = random_cache(300, np.random.default_rng(1))
    dev = run_copy(pool, [(10, 10, 200), (220, 260, 40)])
    qsa.qsa_check_device_status()
    same_bytes(dev, moved(pool, [(220, 260, 40)]))


@pytest.mark.parametrize("bad", [(-1, 100, 5), (0, -1, 5), (0, 100, -1), (196, 100, 5), (0, 196, 5), (0, 100, 31), (2 ** 31 - 1, 100, 30),
                                 (0, 2 ** 31 - 1, 30)])
def test_copy_skips_and_flags_a_bad_run(bad):
    pool = random_cache(200, np.random.default_rng(2))
    good = [(0, 150, 20), (30, 100, 30)]
    dev = run_copy(pool, [good[0], bad, good[1]], max_cells=30)
    with pytest.raises(qsa.QSAError) as e:
        qsa.qsa_check_device_status()
    assert e.value.code == qsa.QSA_ERR_DEVICE
    same_bytes(dev, moved(pool, good))


def test_most_runs():
    n = 65535
    pool = random_cache(2 * n, np.random.default_rng(3))
    runs = [(i, 2 * n - 1 - i, 1) for i in range(n)]
    dev = run_copy(pool, runs)
    qsa.qsa_check_device_status()
    want = {k: v.copy() for k, v in pool.items()}
    for k in want:
        want[k][n:] = pool[k][:n][::-1]
    same_bytes(dev, want)


# ---------------------------------------------------------------- compaction
def run_compact(pool, prefixes, seqs, in_place=False, stream=None, ws=None):
    dev = on_gpu(pool)
    a, b = torch.from_numpy(prefixes).cuda(), torch.from_numpy(seqs).cuda()
    ao, bo = (a, b) if in_place else (torch.full_like(a, -5), torch.full_like(b, -5))
    used = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    if ws is None:
        need = qsa.qsa_cache_compact_workspace_bytes(len(pool["kq"]), len(prefixes), len(seqs))
        ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    qsa.qsa_cache_compact(dev["kq"], dev["ksc"], dev["vq"], dev["vsc"], len(pool["kq"]), a if len(prefixes) else None, len(prefixes), b,
                          len(seqs), ao if len(prefixes) else None, bo, used, ws, stream=stream)
    return dev, ao.cpu().numpy(), bo.cpu().numpy(), int(used)


def holes(lengths, gaps, rng, n_prefix=0, end=0):
    rows, at = [], 0
    for n, g in zip(lengths, gaps):
        at += g
        rows.append((at, n, int(rng.integers(0, 99)), int(rng.integers(0, 99))))
        at += n
    rows = [rows[i] for i in rng.permutation(len(rows))]
    return table(rows[:n_prefix]), table(rows[n_prefix:]), max(at + end, 1)


@pytest.mark.parametrize("name,lengths,gaps,n_prefix,end", [
    ("one at its place", [70], [0], 0, 5), ("one far away", [200], [10000], 0, 0), ("by one cell", [700], [1], 0, 0),
    ("by a chunk", [640], [64], 0, 0), ("nearly a chunk", [1000], [63], 1, 9), ("first stays", [100, 100], [0, 1], 1, 0),
    ("all stay", [64, 64, 30], [0, 0, 0], 0, 70), ("none has cells", [0, 0, 0], [0, 3, 9], 1, 4), ("some have none", [0, 5, 0, 70], [3, 0, 2, 1], 1, 1),
    ("single cells", [1] * 500, [1] * 500, 3, 0), ("single cells, side by side", [1] * 300, [2] + [0] * 299, 0, 0),
    ("large hole behind", [64, 64, 64], [0, 500, 0], 0, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(name, lengths, gaps, n_prefix, end, in_place):
    rng = np.random.default_rng(len(name))
    prefixes, seqs, n_pool = holes(lengths, gaps, rng, n_prefix, end)
    pool = random_cache(n_pool, rng)
    dev, a, b, used = run_compact(pool, prefixes, seqs, in_place)
    qsa.qsa_check_device_status()
    want, (wa, wb), n = compacted(pool, (prefixes, seqs))
    assert used == n
    np.testing.assert_array_equal(a, wa)
    np.testing.assert_array_equal(b, wb)
    same_bytes(dev, want)


@pytest.mark.parametrize("seed", range(6))
def test_compact_random(seed):
    rng = np.random.default_rng(100 + seed)
    n = int(rng.integers(1, 400))
    lengths, gaps = rng.integers(0, [5, 70, 300][seed % 3], n), rng.integers(0, [3, 200][seed % 2], n) * (rng.random(n) < 0.6)
    prefixes, seqs, n_pool = holes([int(x) for x in lengths], [int(x) for x in gaps], rng, int(rng.integers(0, n)), int(rng.integers(0, 90)))
    pool = random_cache(n_pool, rng)
    dev, a, b, used = run_compact(pool, prefixes, seqs)
    qsa.qsa_check_device_status()
    want, (wa, wb), total = compacted(pool, (prefixes, seqs))
    assert used == total
    np.testing.assert_array_equal(a, wa)
    np.testing.assert_array_equal(b, wb)
    same_bytes(dev, want)


def test_compact_entries_without_cells_in_both_tables():
    # at the first cell of a run before and behind it in the tables, between runs, inside one, and behind all
    rng = np.random.default_rng(12)
    prefixes = table([(50, 0, 1, 2), (90, 7, 3, 4), (33, 0, 5, 6)])
    seqs = table([(50, 20, 7, 8), (50, 0, 9, 10), (90, 0, 11, 12), (30, 10, 13, 14), (200, 0, 15, 16), (0, 0, 17, 18)])
    pool = random_cache(200, rng)
    for in_place in (False, True):
        dev, a, b, used = run_compact(pool, prefixes, seqs, in_place)
        qsa.qsa_check_device_status()
        assert used == 37 and list(a[:, 0]) == [10, 30, 10] and list(b[:, 0]) == [10, 30, 37, 0, 37, 0]
        want, (wa, wb), n = compacted(pool, (prefixes, seqs))
        assert n == 37
        np.testing.assert_array_equal(a, wa)
        np.testing.assert_array_equal(b, wb)
        same_bytes(dev, want)


def test_compact_many_runs():
    rng = np.random.default_rng(9)
    prefixes, seqs, n_pool = holes([1] * 65535, [int(x) for x in rng.integers(0, 2, 65535)], rng, 35)
    pool = random_cache(n_pool, rng)
    dev, a, b, used = run_compact(pool, prefixes, seqs)
    qsa.qsa_check_device_status()
    want, (wa, wb), total = compacted(pool, (prefixes, seqs))
    assert used == total == 65535
    np.testing.assert_array_equal(a, wa)
    np.testing.assert_array_equal(b, wb)
    same_bytes(dev, want)


@pytest.mark.parametrize("bad", [(-1, 5), (10, -1), (296, 5), (120, 10), (100, 20), (90, 200), (2 ** 31 - 1, 9)],
                         ids=["first<0", "cells<0", "past the pool", "inside another", "the same run", "around others", "far"])
def test_a_broken_table_moves_nothing(bad):
    rng = np.random.default_rng(4)
    pool = random_cache(300, rng)
    prefixes, seqs = table([(20, 30, 1, 2)]), table([(100, 20, 3, 4), (*bad, 5, 6), (119, 11, 0, 0) if bad == (120, 10) else (140, 7, 8, 9)])
    dev, a, b, used = run_compact(pool, prefixes, seqs)
    with pytest.raises(qsa.QSAError) as e:
        qsa.qsa_check_device_status()
    assert e.value.code == qsa.QSA_ERR_DEVICE
    assert used == -1
    np.testing.assert_array_equal(a, prefixes)
    np.testing.assert_array_equal(b, seqs)
    same_bytes(dev, pool)


def test_nothing_to_compact_uses_no_cells():
    used = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    qsa.qsa_cache_compact(None or 0, 0, 0, 0, 10, None, 0, None, 0, None, None, used, None)
    assert int(used) == 0


def test_copy_and_compact_on_a_stream_and_in_a_graph():
    # fork, end the first sequence, compact: captured once and replayed over pools that change in between
    rng = np.random.default_rng(5)
    n_pool = 5000
    pools = [random_cache(n_pool, rng) for _ in range(3)]
    runs = [(100, 3000, 700), (300, 3900, 555)]
    seqs = table([(300, 900, 1, 0), (3000, 700, 2, 1), (3900, 555, 3, 2)])
    dev = on_gpu(pools[0])
    t, s = torch.from_numpy(table(runs)).cuda(), torch.from_numpy(seqs).cuda()
    out, used = torch.zeros_like(s), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(qsa.qsa_cache_compact_workspace_bytes(n_pool, 0, 3), dtype=torch.uint8, device="cuda")

    def step():
        qsa.qsa_cache_copy(dev["kq"], dev["ksc"], dev["vq"], dev["vsc"], n_pool, t, 2, 700)
        qsa.qsa_cache_compact(dev["kq"], dev["ksc"], dev["vq"], dev["vsc"], n_pool, None, 0, s, 3, None, out, used, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for pool in pools:
        for k in pool:
            dev[k].copy_(torch.from_numpy(pool[k]))
        graph.replay()
        qsa.qsa_check_device_status()
        want, (w,), n = compacted(moved(pool, runs), (seqs,))
        assert int(used) == n
        np.testing.assert_array_equal(out.cpu().numpy(), w)
        same_bytes(dev, want)


def test_compact_far_into_a_large_pool():
    # byte offsets past 32 bits: 9.5 million cells (4.9 GB of codes each), the last of them moved to the front
    n_pool = 9_500_000
    dev = {"kq": torch.zeros(n_pool, 2, 256, dtype=torch.int8, device="cuda"), "ksc": torch.zeros(n_pool, 2, 4, dtype=torch.float16, device="cuda")}
    dev |= {"vq": torch.zeros_like(dev["kq"]), "vsc": torch.zeros_like(dev["ksc"])}
    small = random_cache(100, np.random.default_rng(6))
    for k in small:
        dev[k][n_pool - 100:] = torch.from_numpy(small[k]).cuda()
    runs = torch.tensor([[n_pool - 100, n_pool - 300, 100, 0]], dtype=torch.int32, device="cuda")
    qsa.qsa_cache_copy(dev["kq"], dev["ksc"], dev["vq"], dev["vsc"], n_pool, runs, 1, 100)
    seqs = torch.tensor([[n_pool - 300, 100, 0, 0], [n_pool - 100, 100, 0, 0]], dtype=torch.int32, device="cuda")
    used = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(qsa.qsa_cache_compact_workspace_bytes(n_pool, 0, 2), dtype=torch.uint8, device="cuda")
    qsa.qsa_cache_compact(dev["kq"], dev["ksc"], dev["vq"], dev["vsc"], n_pool, None, 0, seqs, 2, None, seqs, used, ws)
    qsa.qsa_check_device_status()
    assert int(used) == 200 and seqs[:, 0].tolist() == [0, 100]
    for k in small:
        for at in (0, 100, n_pool - 100):
            np.testing.assert_array_equal(dev[k][at:at + 100].cpu().numpy(), small[k])
