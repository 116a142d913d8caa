"""Workloads of the drafted-token operators: attention of token trees over the int8 KV cache, the
batched prep that writes the cache, reading cells back, and committing an accepted path.

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
def _tree(name, n_seq, t, p, shape, identity_max=DEFAULT_IDENTITY, topk=DEFAULT_TOPK, gate=False):
    return {"name": name, "op": "tree", "n_seq": n_seq, "t_lo": t[0], "t_hi": t[1], "p_lo": p[0], "p_hi": p[1],
            "identity_max": identity_max, "topk": topk, "gate": gate, "shape": shape}


def listed():
    return [
        # one chat with a small draft over a short context: launch latency is what counts
        _tree("tree 8 after 500", 1, (8, 8), (500, 500), 1),
        # one sequence, a wide draft just under the selection threshold
        _tree("tree 61 after 1984", 1, (61, 61), (1984, 1984), 2),
        # a serving batch of short contexts with drafts of every size, odd ones among them
        _tree("32 trees after 64-1984", 32, (4, 64), (64, 1984), 3, gate=True),
        # one long chat: every drafted token selects its own 2048 cells
        _tree("tree 16 after 8192", 1, (16, 16), (8192, 8192), 4),
        # a serving batch of mixed contexts: some sequences select, some do not
        _tree("24 trees after 200-16000", 24, (1, 32), (200, 16000), 5),
        # selection switched off by its threshold: dense attention over long caches
        _tree("4 dense trees after 30000", 4, (33, 48), (29000, 31000), 6, identity_max=LONG_DENSE),
        # the prep of one draft step of a small batch, plain positions
        {"name": "prep 64", "op": "prep", "n_tok": 64, "axes": 1, "rotary": 256, "far": 30000, "pad": 3, "shape": 7},
        # a prompt chunk of many images and texts: three position axes, rows taken out of fused projections
        {"name": "prep 8191", "op": "prep", "n_tok": 8191, "axes": 3, "rotary": 128, "far": 130000, "pad": 0, "shape": 8},
        # one short prefix read back
        {"name": "read 2051", "op": "read", "n": 2051, "pool": 4096, "shape": 9},
        # the prefixes of a batch read back, in the order that their pages were handed out
        {"name": "read 131072", "op": "read", "n": 131072, "pool": 200000, "shape": 10},
        # one chat's accepted path moved into place
        {"name": "commit 1", "op": "commit", "n_seq": 1, "t_hi": 16, "cap": 8, "slack": 40, "shape": 11},
        # a large batch's accepted paths, from none to many tokens each
        {"name": "commit 512", "op": "commit", "n_seq": 512, "t_hi": 64, "cap": 33, "slack": 40, "shape": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {"tree": (6.0e8, 1.6e11), "prep": (2.6e8, 1e18), "read": (4.1e8, 1e18), "commit": (4.0e7, 1e18)}
    while True:
        op = rng.choice(("tree", "tree", "tree", "prep", "read", "commit"))
        shape = rng.randrange(1 << 20)
        if op == "tree":
            t_hi = _log(rng, 1, 200)
            p_hi = _log(rng, 1, 31000)
            dense = rng.random() < 0.25
            c = _tree("", _log(rng, 1, 32), (max(1, t_hi // rng.choice((1, 3, 10))), t_hi),
                      (p_hi // rng.choice((1, 2, 20)), p_hi), shape, gate=rng.random() < 0.4,
                      identity_max=LONG_DENSE if dense else DEFAULT_IDENTITY)
        elif op == "prep":
            n = _log(rng, 1, 8000)
            c = {"op": op, "n_tok": n, "axes": rng.choice((1, 3)), "rotary": rng.choice((16, 32, 64, 128, 256)),
                 "far": _log(rng, 100, 130000), "pad": rng.randrange(0, max(1, n // 8) + 1), "shape": shape}
        elif op == "read":
            n = _log(rng, 1, 130000)
            c = {"op": op, "n": n, "pool": n + _log(rng, 1, 60000), "shape": shape}
        else:
            t_hi = _log(rng, 1, 64)
            c = {"op": op, "n_seq": _log(rng, 1, 500), "t_hi": t_hi, "cap": max(1, t_hi // 2), "slack": rng.randrange(0, 60),
                 "shape": shape}
        c.pop("name", None)
        w = work(c)
        if op == "tree" and c["n_seq"] * t_hi * (p_hi + t_hi) > 1.25e7:  # the plain form pads sequences to the longest
            continue
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return c


def _seq_table(case):
    """Per sequence [first pool cell, cells, committed cells, first token row], the token count and the pool's size."""
    rng = random.Random(case["shape"])
    rows, row0, cell0 = [], 0, 0
    for _ in range(case["n_seq"]):
        t = rng.randint(case.get("t_lo", 1), case["t_hi"])
        p = rng.randint(case.get("p_lo", 0), case.get("p_hi", 2 * case.get("slack", 0)))
        cells = p + t + rng.randint(0, 70)
        rows.append([cell0, cells, p, row0, t])
        row0 += t
        cell0 += cells
    return rows, row0, cell0


def work(case):
    if case["op"] == "tree":
        rows, n_tok, _ = _seq_table(case)
        b = n_tok * HEADS * DIM * 2 * (3 if case["gate"] else 2)
        f = 0
        for _, _, p, _, t in rows:
            n_kv = p + min(t, 4)
            b += (p + t) * CELL_BYTES
            if n_kv > case["identity_max"]:
                b += t * GROUPS * case["topk"] * 4
                f += t * GROUPS * n_kv * DIM * 2  # the score of a group: its summed queries
                n_kv = case["topk"]
            f += t * HEADS * n_kv * DIM * 4
        return {"bytes": b, "flops": f}
    if case["op"] == "prep":
        n = case["n_tok"] - case["pad"]
        # raw rows and q out; the cells written, read back once and returned as fp16 rows
        return {"bytes": n * ((HEADS * 2 + 2 * GROUPS) * DIM * 2 + 2 * CELL_BYTES + 2 * GROUPS * DIM * 2),
                "flops": n * (HEADS + GROUPS) * DIM * 8}
    if case["op"] == "read":
        return {"bytes": case["n"] * (CELL_BYTES + 2 * GROUPS * DIM * 2 + 4), "flops": case["n"] * 2 * GROUPS * DIM}
    moved = case["n_seq"] * min(case["cap"], case["t_hi"]) // 2 + 1
    return {"bytes": 2 * moved * CELL_BYTES, "flops": 0}


# ----------------------------------------------------------------------------------- inputs
def _pool(n, gen):
    """Codes and scales as a quantised cache holds them: codes over the whole range, scales of one magnitude."""
    def codes():
        return torch.randint(-127, 128, (n, GROUPS, DIM), generator=gen, device="cuda", dtype=torch.int8)

    def scales():
        return (torch.rand(n, GROUPS, DIM // BLOCK, generator=gen, device="cuda") * 0.015 + 0.005).half()

    return {"kq": codes(), "ksc": scales(), "vq": codes(), "vsc": scales()}


def _normal(shape, gen, dtype=torch.float16):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _tree_masks(rows, words, rng):
    """Ancestor bits of random trees: a token sees itself and what its parent sees; some trees are plain chains."""
    out = []
    for _, _, _, _, t in rows:
        chain = rng.random() < 0.2
        masks = []
        for i in range(t):
            parent = i - 1 if chain else rng.randint(max(-1, i - 9), i - 1)
            masks.append((masks[parent] if parent >= 0 else 0) | (1 << i))
        for m in masks:
            w = [(m >> (32 * k)) & 0xFFFFFFFF for k in range(words)]
            out.append([x - (1 << 32) if x >= 1 << 31 else x for x in w])
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + case["shape"])
    rng = random.Random(seed * 7919 + case["shape"])
    if case["op"] == "tree":
        rows, n_tok, n_pool = _seq_table(case)
        words = (max(r[4] for r in rows) + 31) // 32
        s = _pool(n_pool, gen)
        s |= {"op": "tree", "n_pool": n_pool, "n_seq": len(rows), "n_tok": n_tok, "t_max": max(r[4] for r in rows),
              "max_n_kv": max(r[2] + r[4] for r in rows), "q": _normal((n_tok, HEADS, DIM), gen),
              "seqs": torch.tensor([r[:4] for r in rows], dtype=torch.int32, device="cuda"),
              "tree": _tree_masks(rows, words, rng), "gate": _normal((n_tok, HEADS, DIM), gen) if case["gate"] else None,
              "ids": torch.full((n_tok, GROUPS, case["topk"]), -1, dtype=torch.int32, device="cuda"),
              "out": torch.zeros(n_tok, HEADS, DIM, dtype=torch.float16, device="cuda"),
              "params": (case["topk"], case["identity_max"], SM_SCALE)}
        return s
    if case["op"] == "prep":
        n, rd = case["n_tok"], case["rotary"]
        n_pool = 2 * n + 5
        # q, k and v rows lie beside one another in a token's fused projection
        fused = _normal((n, (HEADS + 2 * GROUPS) * DIM), gen)
        cells = torch.randperm(n_pool, generator=gen, device="cuda")[:n].to(torch.int32)
        if case["pad"]:
            cells[n - case["pad"]:] = -1
        at = torch.randint(0, case["far"], (n, case["axes"]), generator=gen, device="cuda", dtype=torch.int32)
        s = {"kq": torch.zeros(n_pool, GROUPS, DIM, dtype=torch.int8, device="cuda"),
             "ksc": torch.zeros(n_pool, GROUPS, DIM // BLOCK, dtype=torch.float16, device="cuda")}
        s |= {"vq": s["kq"].clone(), "vsc": s["ksc"].clone()}
        third = rd // 2 // 8 * 3
        sections = (rd // 2 - 2 * third, third, third) if case["axes"] == 3 else (rd // 2, 0, 0)
        s |= {"op": "prep", "n_tok": n, "n_pool": n_pool, "fused": fused, "cells": cells, "pos": at,
              "rope": (10000.0, rd, 1e-6, sections),
              "q_gamma": 1 + 0.1 * _normal((DIM,), gen, torch.float32), "k_gamma": 1 + 0.1 * _normal((DIM,), gen, torch.float32),
              "qcur": torch.zeros(n, HEADS, DIM, dtype=torch.float16, device="cuda"),
              "k16": torch.zeros(n, GROUPS, DIM, dtype=torch.float16, device="cuda"),
              "v16": torch.zeros(n, GROUPS, DIM, dtype=torch.float16, device="cuda")}
        return s
    if case["op"] == "read":
        s = _pool(case["pool"], gen)
        # runs of 64 consecutive cells, as sequences are given their part of a pool, in any order
        at = torch.randperm((case["pool"] + 63) // 64, generator=gen, device="cuda")
        cells = (at[:, None] * 64 + torch.arange(64, device="cuda")).reshape(-1)
        cells = cells[cells < case["pool"]][:case["n"]].to(torch.int32).contiguous()
        s |= {"op": "read", "n": case["n"], "n_pool": case["pool"], "cells": cells,
              "k16": torch.zeros(case["n"], GROUPS, DIM, dtype=torch.float16, device="cuda"),
              "v16": torch.zeros(case["n"], GROUPS, DIM, dtype=torch.float16, device="cuda")}
        return s
    rows, _, n_pool = _seq_table(case)
    s = _pool(n_pool, gen)
    path, n_path = [], []
    for r in rows:
        n = rng.randint(0, min(case["cap"], r[4])) if len(rows) > 1 else min(case["cap"], r[4])
        p = sorted(rng.sample(range(r[4]), n))
        path.append(p + [0] * (case["cap"] - n))
        n_path.append(n)
    s |= {"op": "commit", "n_pool": n_pool, "n_seq": len(rows), "seqs": torch.tensor([r[:4] for r in rows], dtype=torch.int32, device="cuda"),
          "path": torch.tensor(path, dtype=torch.int32, device="cuda"), "n_path": torch.tensor(n_path, dtype=torch.int32, device="cuda")}
    return s


# ----------------------------------------------------------------------------------- plain forms
def _values(codes, scales, dtype):
    return codes.to(dtype) * scales.to(dtype).repeat_interleave(BLOCK, -1)


def _plain_tree(s):
    n_seq, n_tok, t_max, c_max = s["n_seq"], s["n_tok"], s["t_max"], s["max_n_kv"]
    topk, identity_max, scale = s["params"]
    dev = s["q"].device
    first, _, pos0, row0 = s["seqs"].long().unbind(1)
    count = torch.cat([row0[1:], row0.new_full((1,), n_tok)]) - row0
    tok, cell = torch.arange(t_max, device=dev), torch.arange(c_max, device=dev)
    real = tok[None] < count[:, None]                                           # [S, T]
    row = (row0[:, None] + tok).clamp(max=n_tok - 1)
    at = (first[:, None] + cell).clamp(max=s["n_pool"] - 1)                      # [S, C]
    drafted = cell[None] - pos0[:, None]
    word = (drafted >> 5).clamp(0, s["tree"].shape[1] - 1)
    bits = s["tree"][row].gather(2, word[:, None, :].expand(n_seq, t_max, c_max))
    bit = ((bits >> (drafted & 31).to(torch.int32)[:, None, :]) & 1) > 0
    inside = (drafted >= 0) & (drafted < count[:, None])
    seen = ((drafted < 0)[:, None] | (inside[:, None] & bit)) & real[..., None]  # [S, T, C]
    n_kv = seen.sum(-1)
    seen = seen[:, None].expand(n_seq, GROUPS, t_max, c_max)
    q = s["q"][row].view(n_seq, t_max, GROUPS, HPG, DIM)
    if c_max > identity_max:
        chooses = (n_kv > identity_max) & real
        k64 = _values(s["kq"][at], s["ksc"][at], torch.float64).permute(0, 2, 3, 1)
        score = torch.matmul(q.double().sum(3).transpose(1, 2), k64) * scale
        score = score.masked_fill(~seen, -math.inf)
        best = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :topk]
        kept = torch.zeros(score.shape, dtype=torch.bool, device=dev).scatter_(3, best, True)
        seen = torch.where(chooses[:, None, :, None], kept, seen)
        s["ids"][row[chooses]] = best.sort(-1).values.transpose(1, 2)[chooses].to(torch.int32)
    k = _values(s["kq"][at], s["ksc"][at], torch.float32).permute(0, 2, 3, 1)
    logit = torch.matmul(q.float().transpose(1, 2).reshape(n_seq, GROUPS, t_max * HPG, DIM), k) * scale
    logit = logit.view(n_seq, GROUPS, t_max, HPG, c_max).masked_fill(~seen[:, :, :, None], -math.inf)
    top = logit.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(logit - top)
    v = _values(s["vq"][at], s["vsc"][at], torch.float32).transpose(1, 2)
    o = torch.matmul(p.view(n_seq, GROUPS, t_max * HPG, c_max), v).view(n_seq, GROUPS, t_max, HPG, DIM)
    o = o / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.transpose(1, 2).reshape(n_seq, t_max, HEADS, DIM)
    if s["gate"] is not None:
        o = o / (1 + torch.exp(-s["gate"][row].float()))
    s["out"][row[real]] = o[real].half()
    return s["out"], s["ids"]


def _plain_quantise(x):
    b = x.view(*x.shape[:-1], DIM // BLOCK, BLOCK)
    scale = (b.abs().amax(-1) / 127).half()
    ratio = b / scale.float()[..., None].clamp(min=1e-30)
    code = torch.trunc(ratio + torch.copysign(torch.full_like(ratio, 0.5), ratio)).clamp(-127, 127)
    return code.view(x.shape).to(torch.int8), scale


def _plain_prep(s):
    n = s["n_tok"]
    base, rd, eps, sections = s["rope"]
    x = s["fused"].float().view(n, HEADS + 2 * GROUPS, DIM)
    qk, v = x[:, :HEADS + GROUPS], x[:, HEADS + GROUPS:]
    y = qk / torch.sqrt((qk * qk).mean(-1, keepdim=True) + eps)
    gamma = torch.cat([s["q_gamma"].expand(HEADS, DIM), s["k_gamma"].expand(GROUPS, DIM)])
    y = y * gamma
    pair = torch.arange(rd // 2, device=x.device, dtype=torch.float64)
    axis = (pair >= sections[0]).long() + (pair >= sections[0] + sections[1]).long()
    pos = s["pos"].double()
    pos = pos.expand(n, 3)[:, axis] if pos.shape[1] == 1 else pos[:, axis]
    angle = pos * base ** (-2 * pair / rd)  # in 64 bits: far positions
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    a, b = y[..., :rd // 2], y[..., rd // 2:rd]
    y = torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., rd:]], -1).half()
    use = s["cells"] >= 0
    cells = s["cells"][use].long()
    s["qcur"][use] = y[use, :HEADS]
    for_k, for_v = y[use, HEADS:].float(), v[use]
    s["kq"][cells], s["ksc"][cells] = _plain_quantise(for_k)
    s["vq"][cells], s["vsc"][cells] = _plain_quantise(for_v)
    s["k16"][use] = _values(s["kq"][cells], s["ksc"][cells], torch.float32).half()
    s["v16"][use] = _values(s["vq"][cells], s["vsc"][cells], torch.float32).half()
    return s["qcur"], s["k16"], s["v16"]


def _plain_read(s):
    at = s["cells"].long()
    s["k16"].copy_(_values(s["kq"][at], s["ksc"][at], torch.float32))
    s["v16"].copy_(_values(s["vq"][at], s["vsc"][at], torch.float32))
    return s["k16"], s["v16"]


def _plain_commit(s):
    start = (s["seqs"][:, 0] + s["seqs"][:, 2]).long()[:, None]
    step = torch.arange(s["path"].shape[1], device=start.device)
    use = step[None] < s["n_path"][:, None]
    src, dst = (start + s["path"].long())[use], (start + step)[use]
    s["kq"][dst], s["ksc"][dst] = s["kq"][src], s["ksc"][src]
    s["vq"][dst], s["vsc"][dst] = s["vq"][src], s["vsc"][src]
    return s["kq"], s["ksc"], s["vq"], s["vsc"]


# ----------------------------------------------------------------------------------- the library's calls
def _own_tree(s):
    from int8_kv_top_gb300 import qsa

    if "ws" not in s:  # a program keeps one workspace for its calls
        need = qsa.qsa_tree_attention_workspace_bytes(s["n_seq"], s["n_tok"], s["max_n_kv"], params=s["params"])
        s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    qsa.qsa_tree_attention(s["q"], s["kq"], s["vq"], s["ksc"], s["vsc"], s["n_pool"], s["seqs"], s["n_seq"], s["n_tok"],
                           s["tree"], s["max_n_kv"], s["ids"], s["out"], s["ws"], params=s["params"], gate=s["gate"])
    return s["out"], s["ids"]


def _own_prep(s):
    from int8_kv_top_gb300 import qsa

    f = s["fused"]
    k0, v0 = HEADS * DIM, (HEADS + GROUPS) * DIM
    qsa.qsa_prep_batched(f[:, :k0], f[:, k0:v0], f[:, v0:], s["q_gamma"], s["k_gamma"], s["pos"], s["cells"], s["n_tok"],
                         s["n_pool"], s["qcur"], None, s["kq"], s["ksc"], s["vq"], s["vsc"], rope=s["rope"])
    qsa.qsa_cache_read(s["kq"], s["ksc"], s["vq"], s["vsc"], s["n_pool"], s["cells"], s["n_tok"], s["k16"], s["v16"])
    return s["qcur"], s["k16"], s["v16"]


def _own_read(s):
    from int8_kv_top_gb300 import qsa

    qsa.qsa_cache_read(s["kq"], s["ksc"], s["vq"], s["vsc"], s["n_pool"], s["cells"], s["n"], s["k16"], s["v16"])
    return s["k16"], s["v16"]


def _own_commit(s):
    from int8_kv_top_gb300 import qsa

    qsa.qsa_cache_commit(s["kq"], s["ksc"], s["vq"], s["vsc"], s["n_pool"], s["seqs"], s["n_seq"], s["path"], s["n_path"])
    return s["kq"], s["ksc"], s["vq"], s["vsc"]


def run(state):
    if own:
        return {"tree": _own_tree, "prep": _own_prep, "read": _own_read, "commit": _own_commit}[state["op"]](state)
    return {"tree": _plain_tree, "prep": _plain_prep, "read": _plain_read, "commit": _plain_commit}[state["op"]](state)


# ----------------------------------------------------------------------------------- 64-bit results
def _exact_values(codes, scales):
    return (codes.double().view(-1, GROUPS, DIM // BLOCK, BLOCK) * scales.double()[..., None]).view(-1, GROUPS, DIM)


def _exact_tree(s):
    topk, identity_max, scale = s["params"]
    table = s["seqs"].tolist()
    masks = s["tree"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, (first, _, p, r0) in enumerate(table):
        r1 = table[i + 1][3] if i + 1 < len(table) else s["n_tok"]
        n = p + r1 - r0
        k = _exact_values(s["kq"][first:first + n], s["ksc"][first:first + n])
        v = _exact_values(s["vq"][first:first + n], s["vsc"][first:first + n])
        see = torch.zeros(r1 - r0, n, dtype=torch.bool)
        see[:, :p] = True
        for t in range(r1 - r0):
            for j in range(r1 - r0):
                see[t, p + j] = bool((masks[r0 + t][j >> 5] >> (j & 31)) & 1)
        see = see.cuda()
        chooses = see.sum(1) > identity_max
        q = s["q"][r0:r1].double()
        for g in range(GROUPS):
            dots = torch.einsum("thd,cd->thc", q[:, g * HPG:(g + 1) * HPG], k[:, g]) * scale
            use = see
            if bool(chooses.any()):
                total = torch.where(see, dots.sum(1), torch.full_like(dots[:, 0], -math.inf))
                least = total.topk(topk, dim=1).values[:, -1:]
                use = torch.where(chooses[:, None], total >= least, see)
            dots = torch.where(use[:, None], dots, torch.full_like(dots, -math.inf))
            w = torch.softmax(dots, -1)
            out[r0:r1, g * HPG:(g + 1) * HPG] = torch.einsum("thc,cd->thd", w, v[:, g])
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"].double())
    return out, None


def _exact_quantised(x):
    b = x.reshape(-1, GROUPS, DIM // BLOCK, BLOCK)
    scale = (b.abs().amax(-1, keepdim=True) / 127).half().double()
    steps = b / torch.where(scale > 0, scale, torch.ones_like(scale))
    code = torch.where(steps >= 0, torch.floor(steps + 0.5), torch.ceil(steps - 0.5)).clamp(-127, 127)
    return (code * scale).reshape(-1, GROUPS, DIM)


def _exact_prep(s):
    base, rd, eps, sections = s["rope"]
    n, h = s["n_tok"], rd // 2
    x = s["fused"].double().view(n, -1, DIM)
    pos = s["pos"].double()
    axes = [0] * sections[0] + [1] * sections[1] + [2] * sections[2]
    angle = torch.stack([pos[:, a if pos.shape[1] == 3 else 0] * math.pow(base, -2.0 * i / rd) for i, a in enumerate(axes)], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def turned(rows, gamma):
        y = rows * torch.rsqrt(rows.square().mean(-1, keepdim=True) + eps) * gamma.double()
        z = torch.complex(y[..., :h].contiguous(), y[..., h:rd].contiguous()) * turn
        return torch.cat([z.real, z.imag, y[..., rd:]], -1)

    use = (s["cells"] >= 0)[:, None, None]
    q = turned(x[:, :HEADS], s["q_gamma"])
    k = _exact_quantised(turned(x[:, HEADS:HEADS + GROUPS], s["k_gamma"]).half().double())
    v = _exact_quantised(x[:, HEADS + GROUPS:])
    return q * use, k * use, v * use


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tree":
        return _exact_tree(s)
    if case["op"] == "prep":
        return _exact_prep(s)
    if case["op"] == "read":
        at = s["cells"].long()
        return _exact_values(s["kq"][at], s["ksc"][at]), _exact_values(s["vq"][at], s["vsc"][at])
    return None  # cells are moved as they are
