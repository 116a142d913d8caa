"""Workloads of the operators for answers that share a prompt: attention of a batch over shared prefixes and over
each sequence's own cells of the int8 KV cache, the verification of drafted tokens, copies of runs of cells, and
compaction of the pool.

A case is a dict of plain values; `prepare` makes its inputs on the GPU from a seed, `run` makes one
pass through the operator and returns its outputs, and `exact` gives the same outputs from the
definitions in 64 bits.  With `own` false `run` computes the plain form out of elementary torch
operations; with `own` true it makes the library's calls.
"""
import math
import random

import torch

own = False

HEADS, GROUPS, HPG, DIM, BLOCK = 24, 2, 12, 256, 64
SM_SCALE = 0.0625
DEFAULT_IDENTITY = 2051  # at or under this many visible cells a token attends to all of them
DEFAULT_TOPK = 2048
CELL_BYTES = 2 * GROUPS * (DIM + 2 * DIM // BLOCK)  # int8 K and V codes and their fp16 scales
LONG_DENSE = 131072


# ----------------------------------------------------------------------------------- cases
def _attend(name, n_prefix, n_seq, prefix, held, drafted, shape, dense=False, gate=False):
    """`prefix`, `held` and `drafted`: least and most shared cells, own committed cells, and tokens a sequence."""
    return {"name": name, "op": "attend", "n_prefix": n_prefix, "n_seq": n_seq, "x_lo": prefix[0], "x_hi": prefix[1],
            "p_lo": held[0], "p_hi": held[1], "t_lo": drafted[0], "t_hi": drafted[1],
            "identity_max": LONG_DENSE if dense else DEFAULT_IDENTITY, "topk": DEFAULT_TOPK, "gate": gate, "shape": shape}


def listed():
    return [
        # a few answers to one short prompt, decoded token by token: latency counts
        _attend("8 answers to 1800", 1, 8, (1800, 1800), (5, 150), (1, 1), 1),
        # many samples of one long document, selection switched off by its threshold: dense attention
        _attend("64 samples of 30000, all cells", 1, 64, (30000, 30000), (100, 600), (1, 1), 2, dense=True),
        # a serving batch behind one long system prompt: every token selects its cells
        _attend("48 chats behind 16000", 1, 48, (16000, 16000), (50, 900), (1, 1), 3, gate=True),
        # three prompts with drafts of every size: some sequences select, some do not
        _attend("40 drafts behind 3 prompts", 3, 40, (900, 12000), (0, 400), (1, 16), 4),
        # one chat's chain of drafted tokens against a small vocabulary
        {"name": "verify 1", "op": "verify", "n_seq": 1, "t_lo": 8, "t_hi": 8, "vocab": 32768, "points": False, "bush": 1, "shape": 5},
        # a serving batch of drafted trees, a large odd vocabulary
        {"name": "verify 64", "op": "verify", "n_seq": 64, "t_lo": 4, "t_hi": 24, "vocab": 131071, "points": False, "bush": 3, "shape": 6},
        # drafts looked up in the prompt: no probabilities of their own
        {"name": "verify 48 looked up", "op": "verify", "n_seq": 48, "t_lo": 2, "t_hi": 12, "vocab": 100003, "points": True, "bush": 2, "shape": 7},
        # a sequence forked into three
        {"name": "copy 3", "op": "copy", "n_run": 3, "c_lo": 500, "c_hi": 500, "shape": 8},
        # a beam step: each kept beam's own cells copied for its continuations
        {"name": "copy 96", "op": "copy", "n_run": 96, "c_lo": 40, "c_hi": 3000, "shape": 9},
        # a small pool after one sequence has ended
        {"name": "compact 8", "op": "compact", "n_prefix": 0, "n_seq": 8, "c_lo": 60, "c_hi": 300, "hole": 200, "shape": 10},
        # a server's pool after many sequences have ended, prefixes among those that stay
        {"name": "compact 500", "op": "compact", "n_prefix": 12, "n_seq": 488, "c_lo": 10, "c_hi": 900, "hole": 300, "shape": 11},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {"attend": (3e8, 5.0e10), "verify": (9e7, 1e18), "copy": (3.2e8, 1e18), "compact": (4.6e8, 1e18)}
    while True:
        op = rng.choice(("attend", "attend", "attend", "verify", "copy", "compact"))
        shape = rng.randrange(1 << 20)
        if op == "attend":
            n_seq, t_hi, x_hi, p_hi = _log(rng, 1, 100), _log(rng, 1, 40), _log(rng, 1, 31000), _log(rng, 1, 2000)
            c = _attend("", rng.randint(1, min(n_seq, 6)), n_seq, (x_hi // rng.choice((1, 2, 8)), x_hi),
                        (p_hi // rng.choice((1, 3, 20)), p_hi), (max(1, t_hi // rng.choice((1, 4))), t_hi), shape,
                        dense=rng.random() < 0.4, gate=rng.random() < 0.4)
            if n_seq * t_hi * (x_hi + p_hi + t_hi) > 6e6:  # the plain form pads sequences to the longest
                continue
        elif op == "verify":
            t_hi = _log(rng, 1, 60)
            c = {"op": op, "n_seq": _log(rng, 1, 64), "t_lo": max(1, t_hi // rng.choice((1, 4))), "t_hi": t_hi,
                 "vocab": _log(rng, 100, 131071), "points": rng.random() < 0.4, "bush": rng.randint(1, 4), "shape": shape}
            if c["n_seq"] * t_hi * c["vocab"] > 2.1e8:
                continue
        elif op == "copy":
            c_hi = _log(rng, 1, 4000)
            c = {"op": op, "n_run": _log(rng, 1, 300), "c_lo": c_hi // rng.choice((1, 3, 50)), "c_hi": c_hi, "shape": shape}
        else:
            c_hi = _log(rng, 2, 2000)
            c = {"op": op, "n_prefix": rng.randint(0, 5), "n_seq": _log(rng, 1, 500), "c_lo": c_hi // rng.choice((1, 3, 50)),
                 "c_hi": c_hi, "hole": _log(rng, 1, 2000), "shape": shape}
        c.pop("name", None)
        w = work(c)
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def _layout(case):
    """Prefixes [first pool cell, cells, first sequence], sequences [first pool cell, cells, committed cells, first token
    row, tokens, prefix], the token count and the pool's size.  Runs lie in any order with gaps between them."""
    rng = random.Random(case["shape"])
    n_seq, n_prefix = case["n_seq"], case["n_prefix"]
    starts = [0] + sorted(rng.sample(range(1, n_seq), n_prefix - 1))
    prefixes = [[0, rng.randint(case["x_lo"], case["x_hi"]), s] for s in starts]
    seqs, row0 = [], 0
    for s in range(n_seq):
        t, p = rng.randint(case["t_lo"], case["t_hi"]), rng.randint(case["p_lo"], case["p_hi"])
        seqs.append([0, p + t + rng.randint(0, 40), p, row0, t, sum(x <= s for x in starts) - 1])
        row0 += t
    cell = 0
    for r in rng.sample(prefixes + seqs, n_prefix + n_seq):
        r[0] = cell + rng.randint(0, 30)
        cell = r[0] + r[1]
    return prefixes, seqs, row0, cell


def _holes(case):
    """Runs [first pool cell, cells] in the order of a table, and the pool's size."""
    rng = random.Random(case["shape"])
    runs, cell = [], 0
    for i in range(case["n_prefix"] + case["n_seq"]):
        # some runs lie side by side, and the first ones stay where they are
        cell += 0 if i < 2 or rng.random() < 0.3 else rng.randint(0, 2 * case["hole"])
        runs.append([cell, rng.randint(case["c_lo"], case["c_hi"])])
        cell += runs[-1][1]
    rng.shuffle(runs)
    return runs, cell + rng.randint(0, case["hole"])


def _copies(case):
    """Runs [source, destination, cells] and the pool's size; sources repeat and overlap, destinations do not."""
    rng = random.Random(case["shape"])
    cells = [rng.randint(case["c_lo"], case["c_hi"]) for _ in range(case["n_run"])]
    far = max(cells) + sum(cells) // 3
    runs, dst = [], far
    for n in cells:
        dst += rng.randint(0, 3)
        runs.append([rng.randint(0, far - n), dst, n])
        dst += n
    rng.shuffle(runs)
    return runs, dst


def work(case):
    if case["op"] == "attend":
        prefixes, seqs, n_tok, _ = _layout(case)
        b = n_tok * HEADS * DIM * 2 * (3 if case["gate"] else 2) + sum(x[1] for x in prefixes) * CELL_BYTES
        f = 0
        for _, _, p, _, t, x in seqs:
            b += (p + t) * CELL_BYTES
            n_kv = prefixes[x][1] + p + (t + 1) // 2
            if n_kv > case["identity_max"]:
                b += t * GROUPS * case["topk"] * 4
                f += t * GROUPS * n_kv * DIM * 2  # the score of a group: its summed queries
                n_kv = case["topk"]
            f += t * HEADS * n_kv * DIM * 4
        return {"bytes": b, "flops": f}
    if case["op"] == "verify":
        rows = case["n_seq"] * (1 if case["points"] else 2)
        return {"bytes": rows * case["vocab"] * 4 + case["n_seq"] * case["t_hi"] * 16, "flops": 3 * rows * case["vocab"]}
    if case["op"] == "copy":
        return {"bytes": 2 * CELL_BYTES * sum(r[2] for r in _copies(case)[0]), "flops": 0}
    at, moved = 0, 0
    for first, cells in sorted(_holes(case)[0]):
        moved += cells if first != at else 0
        at += cells
    return {"bytes": 2 * CELL_BYTES * moved + 32 * (case["n_seq"] + case["n_prefix"]), "flops": 0}


# ----------------------------------------------------------------------------------- inputs
def _pool(n, gen):
    """Codes and scales as a quantised cache holds them: codes over the whole range, scales of one magnitude."""
    def codes():
        return torch.randint(-127, 128, (n, GROUPS, DIM), generator=gen, device="cuda", dtype=torch.int8)

    def scales():
        return (torch.rand(n, GROUPS, DIM // BLOCK, generator=gen, device="cuda") * 0.015 + 0.005).half()

    return {"n_pool": n, "kq": codes(), "ksc": scales(), "vq": codes(), "vsc": scales()}


def _ints(rows, width):
    return torch.tensor([r[:width] + [0] * (width - len(r)) for r in rows], dtype=torch.int32, device="cuda").reshape(-1, width)


def _parents(t, bush, rng):
    """A drafted tree behind its root; with bush 1 a chain."""
    return [-1] + [rng.randint(max(0, i - bush), i - 1) for i in range(1, t)]


def _masks(parents, words):
    """Ancestor bits: a token sees itself and what its parent sees."""
    rows = []
    for i, p in enumerate(parents):
        rows.append((rows[p] if p >= 0 else 0) | (1 << i))
    out = [[(m >> (32 * k)) & 0xFFFFFFFF for k in range(words)] for m in rows]
    return [[x - (1 << 32) if x >= 1 << 31 else x for x in r] for r in out]


def _probabilities(n, vocab, gen, like=None):
    """Rows as a softmax of a peaked distribution gives them; with `like`, near those rows, as a good drafter's."""
    z = torch.randn(n, vocab, generator=gen, device="cuda") * 3
    if like is not None:
        z = 0.4 * z + torch.log(like[:, :vocab])
    wide = (vocab + 3) // 4 * 4  # rows start on 16 bytes
    out = torch.zeros(n, wide, device="cuda")
    e = torch.exp(z - z.amax(1, keepdim=True))
    out[:, :vocab] = e / e.sum(1, keepdim=True)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + case["shape"])
    rng = random.Random(seed * 7919 + case["shape"])
    if case["op"] == "attend":
        prefixes, seqs, n_tok, n_pool = _layout(case)
        t_max = max(r[4] for r in seqs)
        words = (t_max + 31) // 32
        masks = [m for r in seqs for m in _masks(_parents(r[4], 9, rng), words)]
        q, gate = (torch.randn(n_tok, HEADS, DIM, generator=gen, device="cuda").half() for _ in range(2))
        return _pool(n_pool, gen) | {
            "op": "attend", "q": q, "gate": gate if case["gate"] else None, "prefixes": _ints(prefixes, 4), "n_prefix": len(prefixes),
            "seqs": _ints(seqs, 4), "n_seq": len(seqs), "n_tok": n_tok, "t_max": t_max,
            # one token a sequence sees its own cell: no masks needed
            "tree": torch.tensor(masks, dtype=torch.int32, device="cuda") if t_max > 1 else None,
            "max_prefix": max(x[1] for x in prefixes), "max_own": max(r[2] + r[4] for r in seqs),
            "max_n_kv": max(prefixes[r[5]][1] + r[2] + r[4] for r in seqs),
            "ids": torch.full((n_tok, GROUPS, case["topk"]), -1, dtype=torch.int32, device="cuda"),
            "out": torch.zeros(n_tok, HEADS, DIM, dtype=torch.float16, device="cuda"),
            "params": (case["topk"], case["identity_max"], SM_SCALE)}
    if case["op"] == "verify":
        n_seq, vocab = case["n_seq"], case["vocab"]
        counts = [rng.randint(case["t_lo"], case["t_hi"]) for _ in range(n_seq)]
        parents = [p for t in counts for p in _parents(t, case["bush"], rng)]
        first = [sum(counts[:s]) for s in range(n_seq)]
        n = len(parents)
        p = _probabilities(n, vocab, gen)
        d = None if case["points"] else _probabilities(n, vocab, gen, like=p)
        up = torch.tensor([max(0, x) + first[s] for s, t in enumerate(counts) for x in parents[first[s]:first[s] + t]], device="cuda")
        # a drafted token is a sample of its parent's draft; one that is looked up is often a likely one
        weight = (p[:, :vocab] ** 2 if d is None else d[:, :vocab])[up]
        at = torch.rand(n, 1, generator=gen, device="cuda") * weight.sum(1, keepdim=True)
        token = torch.searchsorted(weight.cumsum(1), at)[:, 0].clamp(max=vocab - 1).to(torch.int32)
        u = torch.rand(n + n_seq, generator=gen, device="cuda")
        return {"op": "verify", "p": p, "d": d, "vocab": vocab, "token": token, "u": u[:n], "u_end": u[n:].clone(), "n_seq": n_seq, "n_tok": n,
                "parent": torch.tensor(parents, dtype=torch.int32, device="cuda"), "t_max": max(counts),
                "seqs": _ints([[0, 1000, 0, r] for r in first], 4),
                "path": torch.full((n_seq, max(counts)), -1, dtype=torch.int32, device="cuda"),
                "n_path": torch.zeros(n_seq, dtype=torch.int32, device="cuda"), "next": torch.zeros(n_seq, dtype=torch.int32, device="cuda")}
    if case["op"] == "copy":
        runs, n_pool = _copies(case)
        return _pool(n_pool, gen) | {"op": "copy", "runs": _ints(runs, 4), "n_run": len(runs), "max_cells": max(r[2] for r in runs)}
    runs, n_pool = _holes(case)
    n_prefix = case["n_prefix"]
    seqs = [[r[0], r[1], r[1] // 2, i] for i, r in enumerate(runs[n_prefix:])]
    prefixes = [[r[0], r[1], i] for i, r in enumerate(runs[:n_prefix])]
    s = _pool(n_pool, gen) | {"op": "compact", "prefixes": _ints(prefixes, 4), "n_prefix": n_prefix, "seqs": _ints(seqs, 4),
                              "n_seq": len(seqs), "used": torch.zeros(1, dtype=torch.int32, device="cuda")}
    return s | {"prefixes_out": s["prefixes"].clone(), "seqs_out": s["seqs"].clone()}


# ----------------------------------------------------------------------------------- plain forms
def _values(codes, scales):
    """The cache's values, as the prefill attends to them and the read-back gives them."""
    return (codes.float() * scales.float().repeat_interleave(BLOCK, -1)).half().float()


def _plain_attend(s):
    n_seq, n_tok, t_max, x_max, o_max = s["n_seq"], s["n_tok"], s["t_max"], s["max_prefix"], s["max_own"]
    topk, identity_max, scale = s["params"]
    dev = s["q"].device
    x_first, x_cells, x_seq, _ = s["prefixes"].long().unbind(1)
    first, _, held, row0 = s["seqs"].long().unbind(1)
    seq = torch.arange(n_seq, device=dev)
    mine = torch.searchsorted(x_seq, seq, right=True) - 1                       # each sequence's prefix
    count = torch.cat([row0[1:], row0.new_full((1,), n_tok)]) - row0
    tok, shared, kept = torch.arange(t_max, device=dev), torch.arange(x_max, device=dev), torch.arange(o_max, device=dev)
    real = tok[None] < count[:, None]                                           # [S, T]
    row = (row0[:, None] + tok).clamp(max=n_tok - 1)
    at = torch.cat([x_first[mine][:, None] + shared, first[:, None] + kept], 1).clamp(max=s["n_pool"] - 1)  # [S, X + O]
    drafted = kept[None] - held[:, None]
    if s["tree"] is None:
        bit = drafted[:, None] <= tok[None, :, None]
    else:
        word = (drafted >> 5).clamp(0, s["tree"].shape[1] - 1)
        bits = s["tree"][row].gather(2, word[:, None, :].expand(n_seq, t_max, o_max))
        bit = ((bits >> (drafted & 31).to(torch.int32)[:, None, :]) & 1) > 0
    inside = (drafted >= 0) & (drafted < count[:, None])
    seen_own = (drafted < 0)[:, None] | (inside[:, None] & bit)
    seen_shared = (shared[None] < x_cells[mine][:, None])[:, None].expand(n_seq, t_max, x_max)
    seen = torch.cat([seen_shared, seen_own], 2) & real[..., None]               # [S, T, X + O]
    n_kv = seen.sum(-1)
    seen = seen[:, None].expand(n_seq, GROUPS, t_max, x_max + o_max)
    q = s["q"][row].view(n_seq, t_max, GROUPS, HPG, DIM)
    if s["max_n_kv"] > identity_max:
        chooses = (n_kv > identity_max) & real
        exact_k = s["kq"][at].double() * s["ksc"][at].double().repeat_interleave(BLOCK, -1)
        score = torch.matmul(q.double().sum(3).transpose(1, 2), exact_k.permute(0, 2, 3, 1)) * scale
        score = score.masked_fill(~seen, -math.inf)
        best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :topk]
        chosen = torch.zeros(score.shape, dtype=torch.bool, device=dev).scatter_(3, best, True)
        seen = torch.where(chooses[:, None, :, None], chosen, seen)
        ids = torch.where(best < x_max, best, best - x_max + x_cells[mine][:, None, None, None])
        s["ids"][row[chooses]] = ids.sort(-1).values.transpose(1, 2)[chooses].to(torch.int32)
    k = _values(s["kq"][at], s["ksc"][at]).permute(0, 2, 3, 1)
    logit = torch.matmul(q.float().transpose(1, 2).reshape(n_seq, GROUPS, t_max * HPG, DIM), k) * scale
    logit = logit.view(n_seq, GROUPS, t_max, HPG, -1).masked_fill(~seen[:, :, :, None], -math.inf)
    top = logit.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(logit - top)
    v = _values(s["vq"][at], s["vsc"][at]).transpose(1, 2)
    o = torch.matmul(p.view(n_seq, GROUPS, t_max * HPG, -1), v).view(n_seq, GROUPS, t_max, HPG, DIM)
    o = o / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.transpose(1, 2).reshape(n_seq, t_max, HEADS, DIM)
    if s["gate"] is not None:
        o = o / (1 + torch.exp(-s["gate"][row].float()))
    s["out"][row[real]] = o[real].half()
    return s["out"], s["ids"]


def _plain_verify(s):
    """All sequences at once, their drafted tokens in order: a child of the token that was accepted last is tried."""
    n_seq, n_tok, vocab = s["n_seq"], s["n_tok"], s["vocab"]
    p, d = s["p"][:, :vocab], None if s["d"] is None else s["d"][:, :vocab]
    row0 = s["seqs"][:, 3].long()
    count = torch.cat([row0[1:], row0.new_full((1,), n_tok)]) - row0
    seq = torch.arange(n_seq, device=p.device)
    at, n = torch.zeros_like(row0), torch.ones_like(row0)
    w, mass = p[row0].double(), torch.ones(n_seq, 1, dtype=torch.float64, device=p.device)  # 64 bits: sums over a vocabulary
    s["path"][:, 0] = 0
    for k in range(1, s["t_max"]):
        row = (row0 + k).clamp(max=n_tok - 1)
        tried = ((k < count) & (s["parent"][row] == at))[:, None]
        x = s["token"][row].long()[:, None]
        u = s["u"][row].double()[:, None]
        base = torch.zeros_like(w).scatter_(1, x, 1.0) if d is None else d[row0 + at].double()
        taken = tried & (u * mass * base.gather(1, x) < w.gather(1, x))
        left = (w * (1 - base) if d is None else (w - mass * base).clamp(min=0))
        left_mass = mass - w.gather(1, x) if d is None else left.sum(1, keepdim=True)
        w = torch.where(taken, p[row].double(), torch.where(tried, left, w))
        mass = torch.where(taken, torch.ones_like(mass), torch.where(tried, left_mass, mass))
        here = torch.where(taken[:, 0], n, n - 1)
        s["path"][seq, here] = torch.where(taken[:, 0], torch.full_like(s["n_path"], k), s["path"][seq, here])
        at, n = torch.where(taken[:, 0], torch.full_like(at, k), at), n + taken[:, 0]
    w = torch.where(w.sum(1, keepdim=True) > 0, w, p[row0 + at].double())
    up = w.cumsum(1)
    s["next"].copy_((up <= s["u_end"].double()[:, None] * up[:, -1:]).sum(1))
    s["n_path"].copy_(n)
    return s["path"], s["n_path"], s["next"]


def _plain_copy(s):
    src, dst, cells, _ = s["runs"].long().unbind(1)
    step = torch.arange(s["max_cells"], device=src.device)
    use = step[None] < cells[:, None]
    a, b = (src[:, None] + step)[use], (dst[:, None] + step)[use]
    s["kq"][b], s["ksc"][b] = s["kq"][a], s["ksc"][a]
    s["vq"][b], s["vsc"][b] = s["vq"][a], s["vsc"][a]
    return s["kq"], s["ksc"], s["vq"], s["vsc"]


def _plain_compact(s):
    table = torch.cat([s["prefixes"][:, :2], s["seqs"][:, :2]]).long()
    order = torch.sort(table[:, 0]).indices
    first, cells = table[order].unbind(1)
    end = cells.cumsum(0)
    cell = torch.arange(s["n_pool"], device=end.device)
    run = torch.searchsorted(end, cell, right=True)
    use = run < len(end)
    run = run.clamp(max=len(end) - 1)
    a = torch.where(use, first[run] + cell - (end - cells)[run], cell)
    s["kq"][cell], s["ksc"][cell] = s["kq"][a], s["ksc"][a]
    s["vq"][cell], s["vsc"][cell] = s["vq"][a], s["vsc"][a]
    to = torch.empty_like(end).scatter_(0, order, end - cells).to(torch.int32)
    s["prefixes_out"][:, 0], s["seqs_out"][:, 0] = to[:s["n_prefix"]], to[s["n_prefix"]:]
    s["used"].copy_(end[-1:])
    return s["kq"], s["ksc"], s["vq"], s["vsc"], s["prefixes_out"], s["seqs_out"], s["used"]


# ----------------------------------------------------------------------------------- the library's calls
def _workspace(s, need):
    if "ws" not in s:  # a program keeps one workspace for its calls
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    return s["ws"]


def _own_attend(s):
    from int8_kv_top_gb300 import qsa

    ws = s["ws"] if "ws" in s else _workspace(s, qsa.qsa_prefix_attention_workspace_bytes(
        s["n_prefix"], s["n_seq"], s["n_tok"], s["max_prefix"], s["max_n_kv"], params=s["params"]))
    qsa.qsa_prefix_attention(s["q"], s["kq"], s["vq"], s["ksc"], s["vsc"], s["n_pool"], s["prefixes"], s["n_prefix"], s["seqs"],
                             s["n_seq"], s["n_tok"], s["tree"], s["max_prefix"], s["max_n_kv"], s["ids"], s["out"], ws,
                             params=s["params"], gate=s["gate"])
    return s["out"], s["ids"]


def _own_verify(s):
    from int8_kv_top_gb300 import qsa

    qsa.qsa_tree_verify(s["p"], s["d"], s["vocab"], s["token"], s["parent"], s["u"], s["u_end"], s["seqs"], s["n_seq"], s["n_tok"],
                        s["path"], s["n_path"], s["next"])
    return s["path"], s["n_path"], s["next"]


def _own_copy(s):
    from int8_kv_top_gb300 import qsa

    qsa.qsa_cache_copy(s["kq"], s["ksc"], s["vq"], s["vsc"], s["n_pool"], s["runs"], s["n_run"], s["max_cells"])
    return s["kq"], s["ksc"], s["vq"], s["vsc"]


def _own_compact(s):
    from int8_kv_top_gb300 import qsa

    ws = s["ws"] if "ws" in s else _workspace(s, qsa.qsa_cache_compact_workspace_bytes(s["n_pool"], s["n_prefix"], s["n_seq"]))
    qsa.qsa_cache_compact(s["kq"], s["ksc"], s["vq"], s["vsc"], s["n_pool"], s["prefixes"], s["n_prefix"], s["seqs"], s["n_seq"],
                          s["prefixes_out"], s["seqs_out"], s["used"], ws)
    return s["kq"], s["ksc"], s["vq"], s["vsc"], s["prefixes_out"], s["seqs_out"], s["used"]


def run(state):
    if own:
        return {"attend": _own_attend, "verify": _own_verify, "copy": _own_copy, "compact": _own_compact}[state["op"]](state)
    return {"attend": _plain_attend, "verify": _plain_verify, "copy": _plain_copy, "compact": _plain_compact}[state["op"]](state)


# ----------------------------------------------------------------------------------- 64-bit results
def _exact_values(codes, scales):
    return (codes.double().view(-1, GROUPS, DIM // BLOCK, BLOCK) * scales.double()[..., None]).view(-1, GROUPS, DIM)


def _exact_attend(s):
    topk, identity_max, scale = s["params"]
    table, prefixes = s["seqs"].tolist(), s["prefixes"].tolist()
    masks = None if s["tree"] is None else s["tree"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, (first, _, p, r0) in enumerate(table):
        r1 = table[i + 1][3] if i + 1 < len(table) else s["n_tok"]
        x0, x, _, _ = [e for e in prefixes if e[2] <= i][-1]
        cells = torch.cat([torch.arange(x0, x0 + x), torch.arange(first, first + p + r1 - r0)]).cuda()
        n = len(cells)
        k, v = _exact_values(s["kq"][cells], s["ksc"][cells]), _exact_values(s["vq"][cells], s["vsc"][cells])
        see = torch.zeros(r1 - r0, n, dtype=torch.bool)
        see[:, :x + p] = True
        for t in range(r1 - r0):
            for j in range(r1 - r0):
                see[t, x + p + j] = j <= t if masks is None else bool((masks[r0 + t][j >> 5] >> (j & 31)) & 1)
        see = see.cuda()
        chooses = see.sum(1) > identity_max
        q = s["q"][r0:r1].double()
        for g in range(GROUPS):
            use = see
            if bool(chooses.any()):
                total = torch.einsum("thd,cd->tc", q[:, g * HPG:(g + 1) * HPG], k[:, g])
                total = torch.where(see, total, torch.full_like(total, -math.inf))
                least = total.topk(topk, dim=1).values[:, -1:]
                use = torch.where(chooses[:, None], total >= least, see)
            # what a token attends to are the cache's fp16 values
            dots = torch.einsum("thd,cd->thc", q[:, g * HPG:(g + 1) * HPG], k[:, g].half().double()) * scale
            dots = torch.where(use[:, None], dots, torch.full_like(dots, -math.inf))
            out[r0:r1, g * HPG:(g + 1) * HPG] = torch.einsum("thc,cd->thd", torch.softmax(dots, -1), v[:, g].half().double())
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"].double())
    return out, None


def _exact_verify(s):
    """Sequence by sequence: the children of the token that was accepted last, one after another."""
    vocab, row0, parent, u = s["vocab"], s["seqs"][:, 3].tolist(), s["parent"].tolist(), s["u"].double().tolist()
    token, u_end = s["token"].tolist(), s["u_end"].double().tolist()
    path, n_path, after = s["path"].clone(), [], []
    for i, r0 in enumerate(row0):
        t = (row0[i + 1] if i + 1 < len(row0) else s["n_tok"]) - r0
        way, w, mass = [0], s["p"][r0, :vocab].double(), 1.0
        for k in range(1, t):
            if parent[r0 + k] != way[-1]:
                continue
            x, d = token[r0 + k], 1.0 if s["d"] is None else float(s["d"][r0 + way[-1], token[r0 + k]])
            if u[r0 + k] * mass * d < float(w[x]):
                way, w, mass = way + [k], s["p"][r0 + k, :vocab].double(), 1.0
            elif s["d"] is None:
                w = w.clone()
                mass, w[x] = mass - float(w[x]), 0.0
            else:
                w = torch.relu(w - s["d"][r0 + way[-1], :vocab].double() * mass)
                mass = float(w.sum())
        if float(w.sum()) <= 0:
            w = s["p"][r0 + way[-1], :vocab].double()
        up = torch.cumsum(w, 0)
        after.append(int(torch.searchsorted(up, up[-1:] * u_end[i], right=True)))
        path[i, :len(way)] = torch.tensor(way, dtype=torch.int32)
        n_path.append(len(way))
    return path, torch.tensor(n_path, dtype=torch.int32), torch.tensor(after, dtype=torch.int32)


def _exact_moved(s, runs):
    """Runs (source, destination, cells), read before any is written."""
    out = []
    for name in ("kq", "ksc", "vq", "vsc"):
        x = s[name].clone()
        for a, b, n in runs:
            x[b:b + n] = s[name][a:a + n]
        out.append(x)
    return out


def _exact_compact(s):
    at, runs, to = 0, [], {}
    for a, n in sorted(r[:2] for r in s["prefixes"].tolist() + s["seqs"].tolist()):
        runs.append((a, at, n))
        to[a] = at
        at += n
    tables = [s["prefixes"].tolist(), s["seqs"].tolist()]
    moved = [torch.tensor([[to[r[0]]] + r[1:] for r in t], dtype=torch.int32).reshape(-1, 4) for t in tables]
    return (*_exact_moved(s, runs), *moved, torch.tensor([at], dtype=torch.int32))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    if case["op"] == "verify":
        return _exact_verify(s)
    if case["op"] == "copy":
        return tuple(_exact_moved(s, [r[:3] for r in s["runs"].tolist()]))
    return _exact_compact(s)
