"""Definitions of the operators for sequences that share a prompt, for the tests: cell runs, compaction, and the
verification of drafted trees in whole numbers."""
from __future__ import annotations

import numpy as np
import torch

UNIT = 1 << 44  # units of a probability


def random_cache(n_pool, rng):
    return {"kq": rng.integers(-127, 128, (n_pool, 2, 256), dtype=np.int8), "vq": rng.integers(-127, 128, (n_pool, 2, 256), dtype=np.int8),
            "ksc": rng.uniform(0.005, 0.02, (n_pool, 2, 4)).astype(np.float16), "vsc": rng.uniform(0.005, 0.02, (n_pool, 2, 4)).astype(np.float16)}


def on_gpu(d):
    return {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in d.items()}


def same_bytes(dev, want):
    for k, v in want.items():
        np.testing.assert_array_equal(dev[k].cpu().numpy().view(np.uint8), v.view(np.uint8), err_msg=k)


def moved(pool, runs):
    """The pool with cells a .. a + n of every run (a, b, n) at b, all read before any is written."""
    new = {k: v.copy() for k, v in pool.items()}
    for a, b, n in runs:
        for k in new:
            new[k][b:b + n] = pool[k][a:a + n]
    return new


def compacted(pool, tables):
    """(pool, tables with their new first cells, cells in use)."""
    at, runs, to = 0, [], {}
    for a, n in sorted((int(r[0]), int(r[1])) for t in tables for r in t if r[1] > 0):
        runs.append((a, at, n))
        to[a] = at
        at += n
    out = [t.copy() for t in tables]
    for t in out:
        for r in t:
            if r[1] > 0:
                r[0] = to[int(r[0])]
    return moved(pool, runs), out, at


def units(x) -> list:
    """fp32 probabilities in units of 2^-44, rounded half to even; outside [0, 1] the nearer end, NaN 0."""
    x = np.nan_to_num(np.asarray(x, np.float32), nan=0.0).clip(0, 1).astype(np.float64)
    return np.rint(x * UNIT).astype(np.int64)  # 24 bits times a power of two: exact before the rounding


def verified(p, d, token, parent, u, u_end, cap):
    """(path, next) of one sequence: p and d [T][vocab] fp32 (d may be None)."""
    def clip(x):
        return float(np.clip(np.nan_to_num(np.float32(x), nan=0.0), 0, 1))

    way, w, mass, refused, out = [0], units(p[0]), [UNIT], 0, set()
    for k in range(1, len(token)):
        if parent[k] != way[-1] or len(way) >= cap:
            continue
        x, cur = int(token[k]), way[-1]
        wx = (clip(p[cur][x]) if refused == 0 else int(w[x]) / UNIT) if d is not None else (0.0 if x in out else clip(p[cur][x]))
        c = 1.0 if refused == 0 else mass[-1] / UNIT
        if float(u[k]) * (1.0 if d is None else clip(d[cur][x])) * c < wx:
            way.append(k)
            w, mass, refused, out = units(p[k]), [UNIT], 0, set()
            continue
        if d is None:
            mass.append(max(mass[-1] - (0 if x in out else int(units(p[cur][x]))), 0))
            out.add(x)
            w = w.copy()
            w[x] = 0
        else:
            df = units(d[cur])
            if refused == 0:
                w = np.maximum(w - df, 0)
            else:
                w = np.array([max(int(a) - ((mass[-1] * int(b)) >> 44), 0) for a, b in zip(w, df)], np.int64)
            mass.append(min(int(w.sum()), 4 * UNIT - 1))
        refused += 1
    if int(w.sum()) == 0:
        w = units(p[way[-1]])
    up = np.cumsum(w)
    total = int(up[-1])
    if total == 0:
        return way, -1
    u = float(np.float32(u_end))
    u64 = 0 if not u > 0 else (1 << 64) - 1 if u >= 1 else int(u * 2.0 ** 64)
    return way, int(np.searchsorted(up, (u64 * total) >> 64, side="right"))
