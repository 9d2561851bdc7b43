"""Workloads of the tree-drafting operators: rotary positions, the layout of a draft tree, attention of a
draft tree over a KV cache, and the commit of its accepted path.

``listed()`` gives fixed cases, ``draw(rng)`` more of the same ranges. ``prepare(case, seed)`` makes the
inputs on the GPU, ``run(state)`` makes one pass: with ``own`` false in plain torch operations (fp32; fp64
for angles), with ``own`` true through the library's entry points. ``exact(case, seed)`` evaluates the
definitions in float64, and ``work(case)`` counts the bytes and operations one pass cannot do without.

Definitions.
- A draft tree has nodes 0..N-1; node 0 is the root (the pending token), ``parents[i] < i`` is node i's
  parent (-1: a root). Depth is the number of edges to the root. Node i sees itself and its ancestors.
- Layout: parents -> depth[b][i] and visibility words mask[b][i][w] (bit j - 64 w of word w: node i sees
  node j). Nodes at or past n_nodes[b] are padding: depth 0, no bits.
- Attention: row (i, g) of KV head h attends to cache rows [0, len[b]) and to the tree's own K/V rows j
  whose bit is set; softmax over both with scale 1/sqrt(d). Rows of padding nodes are left as they were.
- Commit: from node 0, step to the lowest-indexed child whose token is the argmax at the current node, until
  there is none; a = number of steps. The path's K/V rows go to cache rows len..len+a; committed tokens are
  the path's tokens and the argmax at its end; len grows by a + 1.
- Rotary: pair p of the first rot dims of a head is turned by pos * f_p and scaled by a gain; pairs are
  (p, p + rot/2) or (2p, 2p + 1); pos = len[b] + offset[b][t]. The inverse turns back (the gradient).
"""
import math

import numpy as np
import torch

own = False

VOCAB = 151936
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = {"fp16": F16, "bf16": BF16, "fp32": F32}


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # the tiny decoder's tree step: two sequences of about a hundred tokens, 9 nodes
        {"name": "attention tiny", "op": "attention", "batch": 2, "kv_heads": 2, "group": 2, "dim": 64, "lo": 64, "hi": 104,
         "nodes": 9, "ragged": False, "type": "fp16"},
        # one chat sequence early in its answer, a small tree: latency counts
        {"name": "attention b1 1k", "op": "attention", "batch": 1, "kv_heads": 8, "group": 4, "dim": 128, "lo": 1024,
         "hi": 1024, "nodes": 16, "ragged": False, "type": "fp16"},
        # one sequence at 4096 cached keys with a full block of 33 nodes (the attention microbenchmark's shape)
        {"name": "attention b1 4k", "op": "attention", "batch": 1, "kv_heads": 8, "group": 4, "dim": 128, "lo": 4096,
         "hi": 4096, "nodes": 33, "ragged": False, "type": "fp16"},
        # a serving batch of 16 ragged sequences, 1k to 8k, trees of different sizes padded to 33
        {"name": "attention b16 ragged", "op": "attention", "batch": 16, "kv_heads": 8, "group": 4, "dim": 128, "lo": 1024,
         "hi": 8191, "nodes": 33, "ragged": True, "type": "fp16"},
        # four long documents, the largest tree of one block
        {"name": "attention b4 32k", "op": "attention", "batch": 4, "kv_heads": 8, "group": 4, "dim": 128, "lo": 32768,
         "hi": 32768, "nodes": 64, "ragged": False, "type": "bf16"},
        # q, k and v of one tree block between the projection and the attention
        {"name": "rotary tree block", "op": "rotary", "batch": 1, "tokens": 33, "heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "base": 1024, "interleaved": False, "scaling": "none", "append": True, "tree": True, "inverse": False,
         "from": "fp32", "to": "fp16"},
        # a 32k prompt at far positions of a context stretched four times
        {"name": "rotary 32k stretched", "op": "rotary", "batch": 1, "tokens": 32768, "heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "base": 98304, "interleaved": False, "scaling": "by_index", "append": False, "tree": False,
         "inverse": False, "from": "bf16", "to": "bf16"},
        # gradients of a partly rotated head with neighbouring pairs, odd number of tokens
        {"name": "rotary gradient", "op": "rotary", "batch": 3, "tokens": 1333, "heads": 16, "kv_heads": 4, "dim": 128,
         "rot": 64, "base": 0, "interleaved": True, "scaling": "by_parts", "append": False, "tree": False, "inverse": True,
         "from": "fp32", "to": "fp32"},
        # the accepted path of one sequence, all layers of the 36-layer shape
        {"name": "commit b1", "op": "commit", "batch": 1, "layers": 36, "kv_heads": 8, "dim": 128, "nodes": 33, "accept": 6,
         "cap": 512, "ragged": False},
        # the same for a ragged batch of 16 with trees of up to 64 nodes
        {"name": "commit b16", "op": "commit", "batch": 16, "layers": 36, "kv_heads": 8, "dim": 128, "nodes": 64,
         "accept": 10, "cap": 384, "ragged": True},
        # the tree of one sequence, once a step
        {"name": "layout b1", "op": "layout", "batch": 1, "nodes": 33, "ragged": False},
        # a batch of wide trees
        {"name": "layout b64 wide", "op": "layout", "batch": 64, "nodes": 256, "ragged": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "rotary", "rotary", "commit", "commit", "layout"])
    if op == "attention":
        d, g, hkv = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 4, 5, 8]), rng.choice([1, 2, 4, 8, 8])
        nodes = rng.randint(1, 96)
        batch = _log(rng, 1, 24)
        most_keys = 4 * 32768 * 8 * 128 // (batch * hkv * d)  # K/V elements of the largest listed case
        most_keys = min(most_keys, 4 * 32768 * 8 * 4 * 64 * 128 // (batch * hkv * g * nodes * d))  # and its products
        hi = _log(rng, 24, max(25, min(32768, most_keys) - nodes))
        return {"op": op, "batch": batch, "kv_heads": hkv, "group": g, "dim": d, "lo": max(0, int(hi * rng.uniform(0, 1))),
                "hi": hi, "nodes": nodes, "ragged": rng.random() < 0.5, "type": rng.choice(["fp16", "fp16", "bf16"])}
    if op == "rotary":
        d = rng.choice([64, 128])
        rot = rng.choice([d, d, d // 2, d // 4])
        heads, kv = rng.choice([(32, 8), (16, 4), (8, 8), (20, 4), (4, 2)])
        batch = _log(rng, 1, 16)
        tokens = _log(rng, 1, 32768 * 40 * 128 // (2 * batch * (heads + kv) * d))
        append = tokens <= 4096 and rng.random() < 0.5
        inverse = not append and rng.random() < 0.4
        kinds = [("fp32", "fp16")] if append else [("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "fp16")]
        a, b = rng.choice(kinds)
        return {"op": op, "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv, "dim": d, "rot": rot,
                "base": rng.choice([0, _log(rng, 1, 1000000)]) if not append else _log(rng, 1, 2000),
                "interleaved": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "by_parts", "by_index"]),
                "append": append, "tree": append and tokens <= 256, "inverse": inverse, "from": a, "to": b}
    if op == "commit":
        nodes = rng.randint(2, 96)
        return {"op": op, "batch": _log(rng, 1, 16), "layers": rng.choice([2, 12, 24, 36]), "kv_heads": rng.choice([2, 4, 8]),
                "dim": rng.choice([64, 128]), "nodes": nodes, "accept": rng.randint(0, min(12, nodes - 1)),
                "cap": rng.randint(160, 384), "ragged": rng.random() < 0.5}
    return {"op": op, "batch": _log(rng, 1, 64), "nodes": rng.randint(1, 256), "ragged": rng.random() < 0.5}


# ---- sizes that follow from a case -------------------------------------------------------------

def _lens(c):
    """Cache lengths of an attention case: spread evenly from lo to hi, in a mixed order."""
    b = c["batch"]
    if b == 1:
        return [c["hi"]]
    return [c["lo"] + (c["hi"] - c["lo"]) * ((i * 7 + 3) % b) // (b - 1) for i in range(b)]


def _node_counts(c):
    """Live nodes of each sequence's tree: all, or between half and all of them."""
    n, b = c["nodes"], c["batch"]
    least = max(1, n // 2, c.get("accept", 0) + 1)
    return [n - (i * 5 % (n - least + 1)) for i in range(b)] if c["ragged"] else [n] * b


def _accepts(c):
    """Accepted steps of each sequence: the case's, one less for every third."""
    return [max(0, c["accept"] - (i % 3 == 2)) for i in range(c["batch"])]


def work(c):
    if c["op"] == "attention":
        lens, counts = _lens(c), _node_counts(c)
        h, g, d = c["kv_heads"], c["group"], c["dim"]
        keys = sum(n + t for n, t in zip(lens, counts))
        rows = sum(counts) * h * g
        words = sum(counts) * ((c["nodes"] + 63) // 64)
        seen = sum(t * (n + min(t, 5)) for n, t in zip(lens, counts))  # tree rows see a handful of nodes
        return {"bytes": 2 * keys * h * d * 2 + 2 * rows * d * 2 + 8 * words, "flops": 4 * seen * h * g * d}
    if c["op"] == "rotary":
        size = {"fp16": 2, "bf16": 2, "fp32": 4}
        tokens = c["batch"] * c["tokens"]
        heads = c["heads"] + (2 if c["append"] else 1) * c["kv_heads"]
        values = tokens * heads * c["dim"]
        return {"bytes": values * (size[c["from"]] + size[c["to"]]) + (4 * tokens if c["tree"] else 0),
                "flops": 3 * tokens * (c["heads"] + c["kv_heads"]) * c["rot"]}
    if c["op"] == "commit":
        rows = sum(a + 1 for a in _accepts(c))
        return {"bytes": 4 * rows * c["layers"] * c["kv_heads"] * c["dim"] * 2 + 5 * 4 * c["batch"] * c["nodes"], "flops": 0}
    words = (c["nodes"] + 63) // 64
    return {"bytes": c["batch"] * c["nodes"] * (8 + 8 * words), "flops": 0}


# ---- inputs --------------------------------------------------------------------------------------

def _trees(counts, nodes, accepts, rng):
    """Parents, tokens and argmaxes of one tree per sequence. A main path of at least ``accepts[b]`` steps is
    spread over the nodes, the others hang on random earlier nodes, mostly near the end; the argmaxes follow the
    main path for accepts[b] steps. Now and then a later sibling repeats the path's token."""
    b = len(counts)
    parents = np.full((b, nodes), -1, np.int32)
    tokens = rng.integers(0, VOCAB - 1, (b, nodes)).astype(np.int32)
    argmax = rng.integers(0, VOCAB - 1, (b, nodes)).astype(np.int32)
    for s in range(b):
        n, a = counts[s], accepts[s]
        steps = min(n - 1, max(a, min(n - 1, 2 + n // 6)))
        path = [0] + sorted(int(x) + 1 for x in rng.permutation(n - 1)[:steps])
        on_path = set(path)
        for j in range(1, len(path)):
            parents[s, path[j]] = path[j - 1]
        for i in range(1, n):
            if i not in on_path:
                parents[s, i] = int(rng.integers(max(0, i - 8), i)) if rng.random() < 0.7 else int(rng.integers(0, i))
        for j in range(a):
            argmax[s, path[j]] = tokens[s, path[j + 1]]
            later = [i for i in range(path[j + 1] + 1, n) if parents[s, i] == path[j]]
            if later and rng.random() < 0.3:
                tokens[s, later[0]] = tokens[s, path[j + 1]]
        argmax[s, path[a]] = VOCAB - 1  # no node holds this token
        parents[s, n:] = rng.integers(-1, nodes, nodes - n)  # padding is never read
    return parents, tokens, argmax


def _visible(parents, counts):
    """[B][N][N] truth values: node i sees node j (host)."""
    b, n = parents.shape
    see = np.zeros((b, n, n), bool)
    for s in range(b):
        for i in range(counts[s]):
            p = parents[s, i]
            if p >= 0:
                see[s, i] = see[s, p]
            see[s, i, i] = True
    return see


def _words(see):
    """Visibility as int64 words [B][N][W], bit j of word w = node 64 w + j."""
    b, n, _ = see.shape
    w = (n + 63) // 64
    bits = np.zeros((b, n, w * 64), np.uint8)
    bits[:, :, :n] = see
    return np.packbits(bits, axis=2, bitorder="little").view("<i8").reshape(b, n, w).copy()


def prepare(c, seed):
    rng = np.random.default_rng([seed, 17])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 13)

    def normal(shape, dtype):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)

    def put(x):
        return torch.from_numpy(np.ascontiguousarray(x)).cuda()

    s = {"case": c, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if c["op"] == "attention":
        b, h, g, d, n = c["batch"], c["kv_heads"], c["group"], c["dim"], c["nodes"]
        t, lens, counts = TYPES[c["type"]], _lens(c), _node_counts(c)
        cap = (max(lens) + n + 63) // 64 * 64
        parents, _, _ = _trees(counts, n, [0] * b, rng)
        s["q"] = normal((b, h, n * g, d), t)
        s["k_cache"], s["v_cache"] = normal((b, h, cap, d), t), normal((b, h, cap, d), t)
        s["k_blk"], s["v_blk"] = normal((b, h, n, d), t), normal((b, h, n, d), t)
        s["len"], s["n_nodes"] = put(np.array(lens, np.int32)), put(np.array(counts, np.int32))
        s["mask"] = put(_words(_visible(parents, counts)))
        s["out"] = torch.zeros((b * n, h * g * d), dtype=t, device="cuda")
        s["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    elif c["op"] == "rotary":
        b, t, h, kv, d = c["batch"], c["tokens"], c["heads"], c["kv_heads"], c["dim"]
        src, dst = TYPES[c["from"]], TYPES[c["to"]]
        base = [max(0, c["base"] - 37 * i) for i in range(b)]
        s["len"] = put(np.array(base, np.int32))
        s["offsets"] = None
        if c["tree"]:
            parents, _, _ = _trees([t] * b, t, [0] * b, rng)
            s["offsets"] = put((_visible(parents, [t] * b).sum(2) - 1).astype(np.int32))
        if c["append"]:  # one projection's output: q, k and v side by side; k and v go to the cache
            s["qkv"] = normal((b, t, h + 2 * kv, d), src)
            s["q_out"] = torch.zeros((b, kv, t * (h // kv), d), dtype=dst, device="cuda")
            cap = max(base) + t + 3
            s["k_cache"] = torch.zeros((b, kv, cap, d), dtype=dst, device="cuda")
            s["v_cache"] = torch.zeros_like(s["k_cache"])
        else:
            s["q"], s["k"] = normal((b, t, h, d), src), normal((b, t, kv, d), src)
            s["q_out"] = torch.empty((b, t, h, d), dtype=dst, device="cuda")
            s["k_out"] = torch.empty((b, t, kv, d), dtype=dst, device="cuda")
    elif c["op"] == "commit":
        b, n, counts = c["batch"], c["nodes"], _node_counts(c)
        parents, tokens, argmax = _trees(counts, n, _accepts(c), rng)
        shape = (c["layers"], b, c["kv_heads"], c["cap"], c["dim"])
        s["k_cache"], s["v_cache"] = normal(shape, F16), normal(shape, F16)
        blk = (c["layers"], b, c["kv_heads"], n, c["dim"])
        s["k_blk"], s["v_blk"] = normal(blk, F16), normal(blk, F16)
        s["parents"], s["tokens"], s["argmax"] = put(parents), put(tokens), put(argmax)
        s["len"] = put(np.array([c["cap"] - 2 - n - 5 * i % 17 for i in range(b)], np.int32).clip(0))
        s["n_nodes"] = put(np.array(counts, np.int32))
        for k, shape in (("new_len", (b,)), ("pending", (b,)), ("accept_len", (b,)), ("path", (b, n)), ("committed", (b, n))):
            s[k] = torch.zeros(shape, dtype=torch.int32, device="cuda")
    else:
        b, n, counts = c["batch"], c["nodes"], _node_counts(c)
        s["parents"] = put(_trees(counts, n, [0] * b, rng)[0])
        s["n_nodes"] = put(np.array(counts, np.int32))
        s["depth"] = torch.zeros((b, n), dtype=torch.int32, device="cuda")
        s["mask"] = torch.zeros((b, n, (n + 63) // 64), dtype=torch.int64, device="cuda")
    return s


# ---- the plain forms ------------------------------------------------------------------------------

def _closure(parents, live):
    """[B][N][N] fp32, 1 where node i sees node j: the parent relation closed by repeated squaring (N <= 256)."""
    n = parents.shape[1]
    at = torch.arange(n, device=parents.device)
    up = ((parents[:, :, None] == at) & live[:, :, None] & live[:, None, :]).float()
    up = up + torch.eye(n, device=parents.device) * live[:, :, None]
    twice = lambda m: torch.matmul(m, m).clamp(max=1.0)  # noqa: E731
    return twice(twice(twice(twice(twice(twice(twice(twice(up))))))))


def _live(s):
    n = s["parents"].shape[1]
    return torch.arange(n, device="cuda") < s["n_nodes"][:, None]


def _plain_layout(s):
    see = _closure(s["parents"], _live(s)) > 0
    b, n, _ = see.shape
    w = (n + 63) // 64
    bits = torch.zeros((b, n, w * 64), dtype=torch.int64, device="cuda")
    bits[:, :, :n] = see
    s["depth"].copy_((see.sum(2) - 1).clamp(min=0))
    s["mask"].copy_((bits.view(b, n, w, 64) << torch.arange(64, device="cuda")).sum(3))
    return {"depth": s["depth"], "mask": s["mask"]}


def _plain_attention(s):
    c = s["case"]
    b, h, g, d, n = c["batch"], c["kv_heads"], c["group"], c["dim"], c["nodes"]
    cap = s["k_cache"].shape[2]
    q = s["q"].float() / math.sqrt(d)
    old = torch.arange(cap, device="cuda") < s["len"][:, None]                      # [B][cap]
    j = torch.arange(n, device="cuda")
    see = ((s["mask"][:, :, j // 64] >> (j % 64)) & 1).bool().repeat_interleave(g, 1)  # [B][N g][N]
    live = (j < s["n_nodes"][:, None]).repeat_interleave(g, 1)                      # [B][N g]
    see = see & (j < s["n_nodes"][:, None])[:, None, :]
    low = float("-inf")
    sc = torch.matmul(q, s["k_cache"].float().transpose(2, 3)).masked_fill(~old[:, None, None, :], low)
    sb = torch.matmul(q, s["k_blk"].float().transpose(2, 3)).masked_fill(~see[:, None], low)
    top = torch.maximum(sc.amax(3, keepdim=True), sb.amax(3, keepdim=True))
    top = torch.where(top == low, torch.zeros_like(top), top)
    pc, pb = torch.exp(sc - top), torch.exp(sb - top)
    v = torch.where(old[:, None, :, None], s["v_cache"].float(), 0.0)
    o = torch.matmul(pc, v) + torch.matmul(pb, s["v_blk"].float())
    total = pc.sum(3, keepdim=True) + pb.sum(3, keepdim=True)
    o = torch.where(total > 0, o / total, 0.0).to(s["out"].dtype)
    o = o.view(b, h, n, g, d).permute(0, 2, 1, 3, 4).reshape(b, n, h * g * d)
    out = s["out"].view(b, n, h * g * d)
    out.copy_(torch.where(live.view(b, n, g)[:, :, :1], o, out))
    return s["out"]


#: The stretched contexts of the rotary cases: four times 32768 positions.
STRETCH = {"factor": 4.0, "original": 32768, "slow": 1.0, "fast": 32.0}
THETA = 1.0e6


def _frequencies(c, device):
    """fp64 angles per position and the gain of the rotated pairs."""
    rot = c["rot"]
    p = torch.arange(rot // 2, dtype=torch.float64, device=device)
    f = torch.pow(torch.tensor(THETA, dtype=torch.float64, device=device), -2.0 * p / rot)
    k = STRETCH["factor"]
    if c["scaling"] == "none":
        return f, 1.0
    if c["scaling"] == "linear":
        return f / k, 1.0
    if c["scaling"] == "by_parts":  # by the rotations that a pair makes over the original context
        r = STRETCH["original"] * f / (2 * math.pi)
        keep = ((r - STRETCH["slow"]) / (STRETCH["fast"] - STRETCH["slow"])).clamp(0, 1)
    else:  # by_index: a ramp over the pair's index, between the whole indexes around those rotations
        at = lambda r: rot * math.log(STRETCH["original"] / (2 * math.pi * r)) / (2 * math.log(THETA))  # noqa: E731
        lo, hi = max(math.floor(at(STRETCH["fast"])), 0), min(math.ceil(at(STRETCH["slow"])), rot - 1)
        keep = 1 - ((p - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f * (keep + (1 - keep) / k), 0.1 * math.log(k) + 1


def _plain_turn(x, cos, sin, c):
    """x [B][T][heads][d] fp32; cos, sin [B][T][rot/2] fp32, the gain in them."""
    rot = c["rot"]
    cos, sin = cos[:, :, None], sin[:, :, None]
    if c["interleaved"]:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((x1 * cos - x2 * sin, x2 * cos + x1 * sin), dim=-1).flatten(-2)
    else:
        x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((x1 * cos - x2 * sin, x2 * cos + x1 * sin), dim=-1)
    return torch.cat((y, x[..., rot:]), dim=-1)


def _plain_rotary(s):
    c = s["case"]
    b, t, h, kv, d = c["batch"], c["tokens"], c["heads"], c["kv_heads"], c["dim"]
    f, gain = _frequencies(c, "cuda")
    off = s["offsets"] if s["offsets"] is not None else torch.arange(t, device="cuda")[None]
    ang = (s["len"][:, None] + off).double()[:, :, None] * f
    cos, sin = (torch.cos(ang) * gain).float(), (torch.sin(ang) * (-gain if c["inverse"] else gain)).float()
    if not c["append"]:
        s["q_out"].copy_(_plain_turn(s["q"].float(), cos, sin, c))
        s["k_out"].copy_(_plain_turn(s["k"].float(), cos, sin, c))
        return {"q": s["q_out"], "k": s["k_out"]}
    x = s["qkv"].float()
    q = _plain_turn(x[:, :, :h], cos, sin, c).view(b, t, kv, h // kv, d).permute(0, 2, 1, 3, 4)
    s["q_out"].copy_(q.reshape(b, kv, t * (h // kv), d))
    k = _plain_turn(x[:, :, h:h + kv], cos, sin, c).to(BF16).to(F16)  # the cache's bf16 values in fp16
    v = x[:, :, h + kv:].to(BF16).to(F16)
    rows = (s["len"][:, None] + torch.arange(t, device="cuda")).long()[:, :, None].expand(b, t, kv)
    at = (torch.arange(b, device="cuda")[:, None, None], torch.arange(kv, device="cuda")[None, None], rows)
    s["k_cache"][at] = k
    s["v_cache"][at] = v
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_commit(s):
    c = s["case"]
    b, n = s["parents"].shape
    at, live = torch.arange(n, device="cuda"), _live(s)
    see = _closure(s["parents"], live) > 0
    above = s["parents"].clamp(min=0).long()
    child = live & (s["parents"] >= 0) & (s["parents"] < at)
    hit = child & (s["tokens"] == torch.gather(s["argmax"], 1, above.clamp(max=n - 1)))
    twin = (s["parents"][:, :, None] == s["parents"][:, None, :]) & hit[:, None, :] & (at[None, :] < at[:, None])
    good = (hit & ~twin.any(2)) | (at == 0)
    taken = good & live & ~(see & ~good[:, None, :]).any(2) & see[:, :, 0]  # every ancestor is taken too
    a = taken.sum(1) - 1
    order = torch.where(taken, at, n).sort(1).values                        # the path, then n
    on = at <= a[:, None]
    s["path"].copy_(torch.where(on, order, -1))
    last = order.gather(1, a[:, None])
    final = s["argmax"].gather(1, last)
    toks = s["tokens"].gather(1, torch.cat((order[:, 1:], order[:, :1]), 1).clamp(max=n - 1))
    s["committed"].copy_(torch.where(at < a[:, None], toks, torch.where(at == a[:, None], final, -1)))
    s["accept_len"].copy_(a)
    s["pending"].copy_(final[:, 0])
    s["new_len"].copy_(s["len"] + a + 1)
    seq, step = on.nonzero(as_tuple=True)
    row, node = s["len"][seq].long() + step, order[seq, step]
    s["k_cache"][:, seq, :, row] = s["k_blk"][:, seq, :, node]
    s["v_cache"][:, seq, :, row] = s["v_blk"][:, seq, :, node]
    return {k: s[k] for k in ("k_cache", "v_cache", "accept_len", "path", "committed", "pending", "new_len")}


# ---- the library's calls ----------------------------------------------------------------------------

def _own_attention(s):
    from shared_kv_draft_b200 import orthrus
    orthrus.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["k_blk"], s["v_blk"], s["len"], s["mask"], s["out"],
                           s["workspace"], n_nodes=s["n_nodes"], status=s["status"])
    return s["out"]


def _own_rotary(s):
    from shared_kv_draft_b200 import orthrus
    c = s["case"]
    more = {} if c["scaling"] == "none" else STRETCH
    rope = orthrus.rope(c["dim"], c["rot"], THETA, interleaved=c["interleaved"], scaling=c["scaling"], **more)
    if not c["append"]:
        orthrus.rotary(rope, [(s["q"], s["q_out"]), (s["k"], s["k_out"])], len=s["len"], offsets=s["offsets"],
                       inverse=c["inverse"], status=s["status"])
        return {"q": s["q_out"], "k": s["k_out"]}
    b, t, h, kv, d = c["batch"], c["tokens"], c["heads"], c["kv_heads"], c["dim"]
    q, k, v = s["qkv"].split((h, kv, kv), 2)
    to_cache = orthrus.ROTARY_APPEND | orthrus.ROTARY_BF16_VALUES
    orthrus.rotary(rope, [(q, s["q_out"].view(b, kv, t, h // kv, d).permute(0, 2, 1, 3, 4)),
                          (k, s["k_cache"].transpose(1, 2), to_cache),
                          (v, s["v_cache"].transpose(1, 2), to_cache | orthrus.ROTARY_COPY)],
                   len=s["len"], offsets=s["offsets"], status=s["status"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_commit(s):
    from shared_kv_draft_b200 import orthrus
    orthrus.tree_commit(s["parents"], s["tokens"], s["argmax"], s["k_blk"], s["v_blk"], s["k_cache"], s["v_cache"], s["len"],
                        s["new_len"], s["pending"], s["accept_len"], s["path"], s["committed"], n_nodes=s["n_nodes"],
                        status=s["status"])
    return {k: s[k] for k in ("k_cache", "v_cache", "accept_len", "path", "committed", "pending", "new_len")}


def _own_layout(s):
    from shared_kv_draft_b200 import orthrus
    orthrus.tree_layout(s["parents"], s["depth"], s["mask"], n_nodes=s["n_nodes"], status=s["status"])
    return {"depth": s["depth"], "mask": s["mask"]}


def run(s):
    op = s["case"]["op"]
    if own:
        return {"attention": _own_attention, "rotary": _own_rotary, "commit": _own_commit, "layout": _own_layout}[op](s)
    return {"attention": _plain_attention, "rotary": _plain_rotary, "commit": _plain_commit, "layout": _plain_layout}[op](s)


# ---- the definitions in float64 -------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "attention":
        b, h, g, d, n = c["batch"], c["kv_heads"], c["group"], c["dim"], c["nodes"]
        words = s["mask"].cpu().numpy().view(np.uint8)
        see = np.unpackbits(words, axis=2, bitorder="little")[:, :, :n].astype(bool)
        out = s["out"].double().view(b, n, h, g, d)
        for i in range(b):
            m, t = _lens(c)[i], _node_counts(c)[i]
            seen = torch.from_numpy(np.concatenate([np.ones((t, m), bool), see[i, :t, :t]], 1)).cuda()
            for x in range(h):
                keys = torch.cat([s["k_cache"][i, x, :m], s["k_blk"][i, x, :t]]).double()
                vals = torch.cat([s["v_cache"][i, x, :m], s["v_blk"][i, x, :t]]).double()
                rows = s["q"][i, x].double().view(n, g, d)[:t]
                z = torch.einsum("tgd,kd->tgk", rows, keys) * d ** -0.5
                z = z.masked_fill(~seen[:, None, :], float("-inf"))
                out[i, :t, x] = torch.einsum("tgk,kd->tgd", torch.softmax(z, 2), vals)
        return out.view(b * n, h * g * d)
    if c["op"] == "rotary":
        b, t, h, kv, d, rot = (c[k] for k in ("batch", "tokens", "heads", "kv_heads", "dim", "rot"))
        f, gain = _frequencies(c, "cpu")
        off = torch.arange(t).expand(b, t) if s["offsets"] is None else s["offsets"].cpu()
        where = (s["len"].cpu()[:, None] + off).double()
        turn = torch.polar(torch.full((), float(gain), dtype=torch.float64), where[:, :, None] * f).cuda()[:, :, None]
        turn = turn.conj() if c["inverse"] else turn

        def turned(x):
            x = x.double()
            pairs = x[..., :rot].unflatten(-1, (rot // 2, 2)) if c["interleaved"] else \
                x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            z = z if c["interleaved"] else z.transpose(-1, -2)
            return torch.cat([z.flatten(-2), x[..., rot:]], -1)

        if not c["append"]:
            return {"q": turned(s["q"]), "k": turned(s["k"])}
        x = s["qkv"]
        q = turned(x[:, :, :h]).view(b, t, kv, h // kv, d).permute(0, 2, 1, 3, 4).reshape(b, kv, t * (h // kv), d)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for i in range(b):
            m = int(s["len"][i])
            kc[i, :, m:m + t] = turned(x[:, :, h:h + kv])[i].transpose(0, 1)
            vc[i, :, m:m + t] = x[i, :, h + kv:].double().transpose(0, 1)
        return {"q": q, "k_cache": kc, "v_cache": vc}
    if c["op"] == "commit":
        par, tok, arg = (s[k].cpu().tolist() for k in ("parents", "tokens", "argmax"))
        n, old, counts = c["nodes"], s["len"].cpu().tolist(), _node_counts(c)
        kc, vc = s["k_cache"], s["v_cache"]
        got = {k: [] for k in ("accept_len", "path", "committed", "pending", "new_len")}
        for i in range(c["batch"]):
            path = [0]
            while True:
                here = [j for j in range(1, counts[i]) if par[i][j] == path[-1] and tok[i][j] == arg[i][path[-1]]]
                if not here:
                    break
                path.append(min(here))
            a, final = len(path) - 1, arg[i][path[-1]]
            for j, node in enumerate(path):
                kc[:, i, :, old[i] + j] = s["k_blk"][:, i, :, node]
                vc[:, i, :, old[i] + j] = s["v_blk"][:, i, :, node]
            got["accept_len"].append(a)
            got["path"].append(path + [-1] * (n - a - 1))
            got["committed"].append([tok[i][j] for j in path[1:]] + [final] + [-1] * (n - a - 1))
            got["pending"].append(final)
            got["new_len"].append(old[i] + a + 1)
        return {"k_cache": kc.double(), "v_cache": vc.double(),
                **{k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in got.items()}}
    parents = s["parents"].cpu().numpy()
    see = _visible(parents, _node_counts(c))
    return {"depth": torch.from_numpy(np.maximum(see.sum(2) - 1, 0).astype(np.int32)), "mask": torch.from_numpy(_words(see))}
