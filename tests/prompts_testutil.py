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
    """(pool, tables with their new first cells, cells in use): all entries in the order of their first cells, equal ones in
    the tables' order; one without cells goes where a run in its place would."""
    at, runs = 0, []
    out = [t.copy() for t in tables]
    for r in sorted((r for t in out for r in t), key=lambda r: int(r[0])):  # rows are views of `out`; the sort is stable
        runs.append((int(r[0]), at, int(r[1])))
        r[0] = at
        at += int(r[1])
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


# ---------------------------------------------------------------- attention behind prefixes
def shared_batch(groups, seed: int, words: int | None = None, causal: bool = False, gap: int = 3, slack: int = 2):
    """groups: (prefix cells, [(own committed cells, tokens or their parents), ...]) -> the call's arrays, and the same batch as
    a tree call has it, every sequence's prefix in front of its own cells (for drafts_testutil.reference).  Runs lie in a
    shuffled order with `gap` cells of NaN scales before each and `slack` of them behind a sequence's."""
    from int8_kv_top_gb300 import synth
    from tests.drafts_testutil import random_parents, tree_masks

    rng = np.random.default_rng(seed)
    parts = ("kq", "vq", "ksc", "vsc")

    def nans(n):
        return {"kq": np.full((n, 2, 256), 127, np.int8), "vq": np.full((n, 2, 256), -127, np.int8),
                "ksc": np.full((n, 2, 4), np.nan, np.float16), "vsc": np.full((n, 2, 4), np.nan, np.float16)}

    def cells(n, s):
        inp = synth.layer_inputs(1, max(n, 1), seed=seed * 1000 + s)
        return {k: inp[k][:n] for k in parts}

    runs, prefixes, seqs, qs, masks, flat, flat_seqs, t0, f0, no = [], [], [], [], [], [], [], 0, 0, 0
    for n_shared, members in groups:
        shared = cells(n_shared, no)
        prefixes.append([0, n_shared, len(seqs), 0])
        runs.append((prefixes[-1], shared, 0))
        no += 1
        for pos0, par in members:
            par = (list(range(-1, par - 1)) if causal else random_parents(par, rng)) if isinstance(par, int) else list(par)
            own = cells(pos0 + len(par), no)
            seqs.append([0, pos0 + len(par) + slack, pos0, t0])
            runs.append((seqs[-1], own, slack))
            qs.append(synth.layer_inputs(max(len(par), 1), 1, seed=seed * 1000 + 500 + no)["q"][:len(par)])
            masks.append(par)
            flat.append({k: np.concatenate([shared[k], own[k]]) for k in parts})
            flat_seqs.append((f0, n_shared + pos0 + len(par), n_shared + pos0, t0))
            f0 += n_shared + pos0 + len(par)
            t0 += len(par)
            no += 1
    words = words or max(1, (max(len(m) for m in masks) + 31) // 32)
    tree = np.concatenate([tree_masks(m, words) for m in masks])
    pool, at = [], 0
    for i in rng.permutation(len(runs)):
        entry, data, more = runs[i]
        pool += [nans(gap), data, nans(more)]
        entry[0] = at + gap
        at += gap + len(data["kq"]) + more
    pool.append(nans(1))
    pool = {k: np.concatenate([x[k] for x in pool]) for k in parts}
    q = np.concatenate(qs)
    ref = {k: np.concatenate([x[k] for x in flat]) for k in parts} | {"q": q, "tree": tree}
    return ({**pool, "q": q, "tree": None if causal else tree.copy(), "prefixes": np.array(prefixes, np.int32),
             "seqs": np.array(seqs, np.int32)}, ref, np.array(flat_seqs, np.int32))


def bounds_of(b):
    """(longest prefix, most cells that a token of a valid sequence may see)."""
    n_tok, seqs, prefixes = len(b["q"]), b["seqs"], b["prefixes"]
    most = 1
    for s, e in enumerate(seqs):
        t = (int(seqs[s + 1][3]) if s + 1 < len(seqs) else n_tok) - int(e[3])
        mine = [int(p[1]) for p in prefixes if p[2] <= s]
        most = max(most, (mine[-1] if mine else 0) + int(e[2]) + t)
    return max([int(p[1]) for p in prefixes], default=0), most


def run_shared(b, params=None, gate=None, with_ids=True, stream=None, fill=float("nan"), bounds=None, ws=None):
    """One call on fresh device copies: (ids or None, out) as device tensors."""
    from int8_kv_top_gb300 import qsa

    dev = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in b.items() if v is not None and k != "tree"}
    tree = None if b["tree"] is None else torch.from_numpy(np.ascontiguousarray(b["tree"]).view(np.int32)).cuda()
    n_tok, n_seq, n_prefix = len(b["q"]), len(b["seqs"]), len(b["prefixes"])
    max_prefix, max_n_kv = bounds or bounds_of(b)
    ids = torch.full((n_tok, 2, params[0] if params else 2048), -7, dtype=torch.int32, device="cuda") if with_ids else None
    out = torch.full((n_tok, 24, 256), fill, dtype=torch.float16, device="cuda")
    if ws is None:
        need = qsa.qsa_prefix_attention_workspace_bytes(n_prefix, n_seq, n_tok, max_prefix, max_n_kv, params)
        ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever it is read before it is written
    qsa.qsa_prefix_attention(dev["q"], dev["kq"], dev["vq"], dev["ksc"], dev["vsc"], len(b["kq"]), dev["prefixes"] if n_prefix else None,
                             n_prefix, dev["seqs"], n_seq, n_tok, tree, max_prefix, max_n_kv, ids, out, ws, params=params,
                             gate=None if gate is None else torch.from_numpy(gate).cuda(), stream=stream)
    return ids, out
