"""Drafted-token trees for the tests: pools, seqs tables and masks, and the operators' results in
64 bits (exact selection by the oracle's integer keys)."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from int8_kv_top_gb300 import qsa, synth

HPG, GROUPS, HEADS, D = 12, 2, 24, 256


def tree_masks(parents, words: int) -> np.ndarray:
    """Mask rows [n][words] uint32 of one tree: a token sees itself and all its ancestors (parent -1: none)."""
    rows = []
    for i, p in enumerate(parents):
        rows.append((rows[p] if p >= 0 else 0) | (1 << i))
    return np.array([[(m >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for m in rows], np.uint32).reshape(-1, words)


def random_parents(n: int, rng, back: int = 9):
    return [int(rng.integers(max(-1, i - back), i)) for i in range(n)]


def make_batch(specs, seed: int, words: int | None = None, gap: int = 0, slack: int = 3):
    """specs: (committed cells, drafted tokens or their parents) per sequence -> pool dict (with q and tree) and
    the seqs table.  `gap` cells with NaN scales lie before every sequence and `slack` such cells behind its
    drafted ones: nothing may read them."""
    rng = np.random.default_rng(seed)
    parts = {k: [] for k in ("kq", "vq", "ksc", "vsc")}
    trees, seqs, qs, c0, t0 = [], [], [], 0, 0

    def add(piece):
        for k in parts:
            parts[k].append(piece[k])
        return len(piece["kq"])

    def nans(n):
        return {"kq": np.full((n, 2, D), 127, np.int8), "vq": np.full((n, 2, D), -127, np.int8),
                "ksc": np.full((n, 2, 4), np.nan, np.float16), "vsc": np.full((n, 2, 4), np.nan, np.float16)}

    parents = [random_parents(t, rng) if isinstance(t, int) else list(t) for _, t in specs]
    if words is None:
        words = (max((len(p) for p in parents), default=1) + 31) // 32 or 1
    for i, ((pos0, _), par) in enumerate(zip(specs, parents)):
        n = len(par)
        c0 += add(nans(gap))
        inp = synth.layer_inputs(max(n, 1), max(pos0 + n, 1), seed=seed * 100 + i)
        for k in parts:
            inp[k] = inp[k][:pos0 + n]
        used = add(inp)
        used += add(nans(slack))
        seqs.append((c0, used, pos0, t0))
        qs.append(inp["q"][:n])
        trees.append(tree_masks(par, words))
        c0 += used
        t0 += n
    pool = {k: np.concatenate(v) for k, v in parts.items()}
    pool["q"] = np.concatenate(qs)
    pool["tree"] = np.concatenate(trees)
    return pool, np.array(seqs, np.int32)


def visible_cells(pool, seqs, s: int, row: int) -> np.ndarray:
    """Cells of sequence s that token row sees, ascending (cell indices within the sequence)."""
    c0, n, pos0, t0 = (int(x) for x in seqs[s])
    t1 = int(seqs[s + 1][3]) if s + 1 < len(seqs) else pool["q"].shape[0]
    bits = [j for j in range(t1 - t0) if j // 32 < pool["tree"].shape[1] and (int(pool["tree"][row][j // 32]) >> (j % 32)) & 1]
    return np.array(list(range(pos0)) + [pos0 + j for j in bits], np.int64)


def reference(pool, seqs, topk=2048, identity_max=2051, sm_scale=1 / 16, gate=None, rows=None):
    """(out [n_tok][24][256] float64, ids [n_tok][2][topk] with -7 where not written, bound [n_tok][24][256]).

    `bound` is how far a result held in the kernels' types may be from it at most, element by element.
    fp16 roundings are off by at most half a step, e = 2^-11 relative: k^ moves a logit by at most
    E = sm_scale sum |q k^| (e + 256 2^-24) (its rounding and the fp32 sum over 256 dims), which moves every
    p by a factor within e^(+-2E) after normalising; P, V^ and the output round once each; n fp32 additions
    add n 2^-24; and a P under 2^-24 loses at most 2^-25 against a row sum of at least 1."""
    n_tok = pool["q"].shape[0]
    out = np.zeros((n_tok, HEADS, D))
    bound = np.zeros((n_tok, HEADS, D))
    ids = np.full((n_tok, GROUPS, topk), -7, np.int64)
    e = 2.0 ** -11
    for s in range(len(seqs)):
        c0, n_cells, pos0, t0 = (int(x) for x in seqs[s])
        t1 = int(seqs[s + 1][3]) if s + 1 < len(seqs) else n_tok
        if n_cells == 0:
            continue
        kv = {k: pool[k][c0:c0 + n_cells] for k in ("kq", "vq", "ksc", "vsc")}
        k64 = kv["kq"].astype(np.float64) * np.repeat(kv["ksc"].astype(np.float64), 64, axis=-1)
        v64 = kv["vq"].astype(np.float64) * np.repeat(kv["vsc"].astype(np.float64), 64, axis=-1)
        for row in range(t0, t1):
            if rows is not None and row not in rows:
                continue
            vis = visible_cells(pool, seqs, s, row)
            for g in range(GROUPS):
                use = vis
                if len(vis) > identity_max:
                    kept, _ = oracle.cell_set(pool["q"][row], kv["kq"][vis], kv["ksc"][vis], len(vis), g, topk=topk,
                                              identity_max=identity_max, sm_scale=sm_scale)
                    use = vis[kept]
                    ids[row, g] = use
                if len(use) == 0:
                    continue
                h = slice(g * HPG, (g + 1) * HPG)
                q = pool["q"][row, h].astype(np.float64)
                z = q @ k64[use, g].T * sm_scale
                p = np.exp(z - z.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                out[row, h] = p @ v64[use, g]
                E = sm_scale * (np.abs(q) @ np.abs(k64[use, g]).T).max(-1, keepdims=True) * (e + 256 * 2.0 ** -24)
                A = p @ np.abs(v64[use, g])
                n = len(use)
                bound[row, h] = (np.abs(out[row, h]) * e + A * (2 * e + e * e + np.expm1(2 * E) + n * 2.0 ** -24)
                                 + n * 2.0 ** -25 * np.abs(v64[use, g]).max() + 2.0 ** -25)
    if gate is not None:
        sig = 1.0 / (1.0 + np.exp(-gate.astype(np.float64)))
        out, bound = out * sig, bound * sig + 2.0 ** -25
    return out, ids, bound


def run_tree(pool, seqs, max_n_kv=None, params=None, gate=None, with_ids=True, stream=None, fill=float("nan")):
    """One call on fresh device copies: (ids or None, out) as device tensors."""
    dev = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in pool.items() if k != "tree"}
    tree = torch.from_numpy(np.ascontiguousarray(pool["tree"]).view(np.int32)).cuda()
    n_tok = pool["q"].shape[0]
    topk = params[0] if params else 2048
    if max_n_kv is None:
        nxt = [int(x[3]) for x in seqs[1:]] + [n_tok]
        max_n_kv = max([1] + [int(x[2]) + b - int(x[3]) for x, b in zip(seqs, nxt) if x[1] > 0])
    ids = torch.full((n_tok, 2, topk), -7, dtype=torch.int32, device="cuda") if with_ids else None
    out = torch.full((n_tok, HEADS, D), fill, dtype=torch.float16, device="cuda")
    need = qsa.qsa_tree_attention_workspace_bytes(len(seqs), n_tok, max_n_kv, params)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    g = torch.from_numpy(gate).cuda() if gate is not None else None
    qsa.qsa_tree_attention(dev["q"], dev["kq"], dev["vq"], dev["ksc"], dev["vsc"], pool["kq"].shape[0],
                           torch.from_numpy(np.ascontiguousarray(seqs)).cuda(), len(seqs), n_tok, tree, max_n_kv, ids, out,
                           ws, params=params, gate=g, stream=stream)
    return ids, out
