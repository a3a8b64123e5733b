"""Cases of the drafted-token (speculative) decode step: the operators' plain
forms in torch and the framework's calls, on the same inputs.

One step of a serving loop that verifies drafted tokens:

``plan``    block tables and slot mappings from the requests' lengths: blocks
            for the new tokens are taken from the free queue, every new token
            gets its position and slot (``plan_step``).
``tree``    attention of the drafted tokens over the paged cache: every token
            sees its sequence's cached tokens, its own ancestors in the draft
            tree and itself (``decode_tree``).
``accept``  the accepted path's K/V rows move to the positions behind the
            cached tokens, in every layer's caches (``accept_tree``).

Sizes of a case (lengths, tokens per request, trees) follow from the case
alone; the seed sets the order of the requests, the physical blocks and the
values.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one decode step of the continuous-batching batch: a token per request
        dict(name="plan-decode", op="plan", n=256, block=16, lens="uniform", lo=1, hi=4096,
             new_lo=1, new_hi=1),
        # a verify step: up to 64 drafted tokens per request, ragged
        dict(name="plan-draft", op="plan", n=128, block=16, lens="lognormal", lo=1, hi=8192,
             new_lo=1, new_hi=64),
        # admission of many prompts' chunks at once, some requests idle
        dict(name="plan-prompts", op="plan", n=2048, block=16, lens="uniform", lo=0, hi=6000,
             new_lo=0, new_hi=2048),
        # one user, a short history and a small tree: latency
        dict(name="tree-one", op="tree", dtype="bf16", n=1, hkv=8, group=4, dim=128, block=16,
             lens="uniform", lo=200, hi=200, nodes_lo=8, nodes_hi=8),
        # multi-head batch, one head per kv head
        dict(name="tree-mha", op="tree", dtype="bf16", n=32, hkv=32, group=1, dim=128, block=16,
             lens="uniform", lo=128, hi=2048, nodes_lo=16, nodes_hi=16),
        # grouped-query batch with lognormal lengths and ragged trees
        dict(name="tree-gqa", op="tree", dtype="bf16", n=128, hkv=8, group=4, dim=128, block=16,
             lens="lognormal", lo=1, hi=8000, nodes_lo=1, nodes_hi=64),
        # long contexts
        dict(name="tree-long", op="tree", dtype="bf16", n=4, hkv=8, group=8, dim=128, block=32,
             lens="uniform", lo=131000, hi=131000, nodes_lo=32, nodes_hi=32),
        # fp32 caches
        dict(name="tree-f32", op="tree", dtype="f32", n=16, hkv=8, group=4, dim=128, block=16,
             lens="uniform", lo=128, hi=2048, nodes_lo=1, nodes_hi=24),
        # head dim, group and block size off the powers of two
        dict(name="tree-odd", op="tree", dtype="bf16", n=24, hkv=8, group=5, dim=96, block=24,
             lens="uniform", lo=1, hi=3000, nodes_lo=1, nodes_hi=48),
        # one user, one layer: latency
        dict(name="accept-one", op="accept", dtype="bf16", n=1, hkv=8, dim=128, block=16,
             layers=1, lens="uniform", lo=200, hi=200, nodes_lo=8, nodes_hi=8),
        # a batch, all layers of a model part in one call
        dict(name="accept-batch", op="accept", dtype="bf16", n=128, hkv=8, dim=128, block=16,
             layers=16, lens="uniform", lo=1, hi=1000, nodes_lo=1, nodes_hi=64),
        # fp32 caches, odd sizes
        dict(name="accept-f32", op="accept", dtype="f32", n=33, hkv=4, dim=80, block=24,
             layers=4, lens="uniform", lo=0, hi=500, nodes_lo=1, nodes_hi=100),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "tree", "tree", "accept"])
    block = rng.choice([4, 8, 16, 16, 24, 32, 64])
    if op == "plan":
        n = _log(rng, 1, 4096)
        # at most the tokens of the largest listed batch
        new_hi = min(_log(rng, 1, 2048), 2 * 2048 * 1024 // n)
        hi = min(_log(rng, 16, 8192), 4 * 2048 * 6000 // n)
        return dict(op=op, n=n, block=block, lens=rng.choice(["uniform", "lognormal"]),
                    lo=rng.randint(0, min(hi, 16)), hi=hi, new_lo=rng.randint(0, 1), new_hi=new_hi)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    size = 4 if dtype == "f32" else 2
    dim = rng.choice([16, 32, 64, 64, 80, 96, 112, 128, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
    nodes = _log(rng, 1, 128)
    lens = rng.choice(["uniform", "lognormal"])
    if op == "accept":
        layers = _log(rng, 1, 16)
        n = _log(rng, 1, 128)
        hi = _log(rng, 16, 1000)
        # at most the largest listed batch's caches
        while n > 1 and n * (hi + nodes + 2 * block) * layers * hkv * dim * size > 4e9:
            n = n // 2
        return dict(op=op, dtype=dtype, n=n, hkv=hkv, dim=dim, block=block, layers=layers,
                    lens=lens, lo=0, hi=hi, nodes_lo=rng.randint(1, nodes), nodes_hi=nodes)
    group = rng.choice([1, 2, 3, 4, 4, 5, 8, 8, 16])
    n = _log(rng, 1, 128)
    hi = _log(rng, 16, 131000)
    flops = 2e11 if dtype == "f32" else 1e12
    while (n * (hi + nodes) * hkv * dim * size > 1e9
           or n * (hi + nodes) * nodes * hkv * group * max(dim, 128) * 4 > flops):
        if n > 1 and (hi < 64 or rng.random() < 0.5):
            n = (n + 1) // 2
        elif hi > 16:
            hi = hi // 2 + 1
        else:
            nodes = (nodes + 1) // 2
    return dict(op=op, dtype=dtype, n=n, hkv=hkv, group=group, dim=dim, block=block, lens=lens,
                lo=rng.randint(0, min(hi, 16)), hi=hi, nodes_lo=rng.randint(1, nodes),
                nodes_hi=nodes)


# ---- sizes: from the case alone ------------------------------------------------

def _sizes(case):
    """Per request: cached tokens, new tokens (nodes), and for trees the
    parents and the deepest accepted node."""
    keys = ("op", "n", "block", "lens", "lo", "hi", "new_lo", "new_hi", "nodes_lo", "nodes_hi")
    rng = random.Random("/".join(str(case.get(k)) for k in keys))
    tree = case["op"] != "plan"
    new_lo, new_hi = (case["nodes_lo"], case["nodes_hi"]) if tree else (case["new_lo"],
                                                                        case["new_hi"])
    out = []
    for _ in range(case["n"]):
        if case["lens"] == "uniform":
            length = rng.randint(case["lo"], case["hi"])
        else:
            length = max(case["lo"], min(case["hi"], int(rng.lognormvariate(
                math.log(max(2, case["hi"] / 8)), 1.0))))
        new = rng.randint(new_lo, new_hi)
        parents, leaf = None, -1
        if tree:
            # the first node is the last verified token; most others continue
            # one of the latest nodes, some branch further up
            parents = [-1]
            for j in range(1, new):
                parents.append(rng.randint(max(0, j - 4), j - 1) if rng.random() < 0.7
                               else rng.randint(-1 if rng.random() < 0.1 else 0, j - 1))
            leaf = rng.randint(0, new - 1) if rng.random() < 0.95 else -1
        out.append((length, new, parents, leaf))
    return out


def _path(parents, leaf):
    path = []
    while leaf >= 0:
        path.append(leaf)
        leaf = parents[leaf]
    return path[::-1]


def work(case):
    sizes = _sizes(case)
    tokens = sum(s[1] for s in sizes)
    block = case["block"]
    if case["op"] == "plan":
        # (a request's spare blocks vary with the seed: blocks as without any)
        grow = sum(-(-(c + n) // block) - -(-c // block) for c, n, _, _ in sizes)
        return {"bytes": 12 * case["n"] + 16 * case["n"] + 8 * grow + 16 * tokens, "flops": 0}
    size = 4 if case["dtype"] == "f32" else 2
    row = case["hkv"] * case["dim"] * size
    if case["op"] == "accept":
        moved = sum(sum(a != j for j, a in enumerate(_path(p, leaf))) for _, _, p, leaf in sizes)
        return {"bytes": 4 * moved * row * case["layers"] + 4 * tokens * 2 + 16 * case["n"],
                "flops": 0}
    keys = sum(c + n for c, n, _, _ in sizes)
    seen = sum((c + 1) * n for c, n, _, _ in sizes)
    blocks = sum(-(-(c + n) // block) for c, n, _, _ in sizes)
    return {"bytes": 2 * keys * row + 2 * tokens * case["group"] * row + 4 * tokens + 4 * blocks
            + 8 * case["n"],
            "flops": 4 * case["dim"] * case["hkv"] * case["group"] * seen}


# ---- inputs --------------------------------------------------------------------

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def prepare(case, seed):
    sizes = _sizes(case)
    random.Random(seed).shuffle(sizes)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    block, n = case["block"], case["n"]
    lens, new = [s[0] for s in sizes], [s[1] for s in sizes]
    if case["op"] == "plan":
        # some requests still hold blocks of rejected tokens
        rng = random.Random(seed + 1)
        held = [-(-c // block) + rng.choice([0, 0, 0, 1, 2]) for c in lens]
        width = max(max(-(-c // block) + 2, -(-(c + m) // block)) for c, m in zip(lens, new)) + 1
        grow = sum(max(0, -(-(c + m) // block) - h) for c, m, h in zip(lens, new, held))
        used, head = sum(held), rng.randint(0, 50)
        num_blocks = used + head + grow + rng.randint(0, 100) + 1
        perm = torch.randperm(num_blocks, device="cuda", generator=gen).int()
        state = {"tables": _tables(perm, held, width), "free": perm[used:].contiguous(),
                 "head": _i32([head]), "held": _i32(held), "num_blocks": num_blocks}
        tokens = sum(new) + 3              # the loop's bound: a few more than this step has
        state["new"] = _i32(new)
        # the step's output buffers, kept by a serving loop
        like = {"seq_lens": (n, torch.int32), "blocks_held": (n, torch.int32),
                "free_head": (1, torch.int32), "query_start_loc": (n + 1, torch.int32),
                "block_start": (n + 1, torch.int32), "slot_mapping": (tokens, torch.int64),
                "positions": (tokens, torch.int32), "seq_ids": (tokens, torch.int32)}
        state["buffers"] = {k: torch.empty(m, dtype=t, device="cuda") for k, (m, t) in like.items()}
        return {"case": case, "lens": _i32(lens), **state}
    dtype, hkv, dim = DTYPES[case["dtype"]], case["hkv"], case["dim"]
    counts = [-(-(c + m) // block) for c, m in zip(lens, new)]
    num_blocks = sum(counts) + 1
    perm = torch.randperm(num_blocks, device="cuda", generator=gen).int()
    shape = (num_blocks, hkv, block, dim)
    state = {"case": case, "tables": _tables(perm, counts, max(counts) + 1),
             "lens": _i32([c + m for c, m in zip(lens, new)]), "start": _i32(_starts(new)),
             "parents": _i32([p for s in sizes for p in s[2]]), "max_q": max(new),
             "max_len": max(c + m for c, m in zip(lens, new)),
             "max_depth": max(len(_path(s[2], j)) for s in sizes for j in range(s[1]))}

    def values(shape, scale=1.0):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        x.normal_(0.0, scale, generator=gen)
        return x

    if case["op"] == "accept":
        shape = (case["layers"],) + shape
        state["leaf"] = _i32([s[3] for s in sizes])
        state["k"], state["v"] = values(shape), values(shape)
        return state
    state["k"], state["v"] = values(shape), values(shape)
    state["q"] = values((sum(new), hkv * case["group"], dim), 2.0)
    return state


def _tables(perm, counts, width):
    """Row i: the next counts[i] entries of perm, then -1."""
    start, count = _i32(_starts(counts))[:-1, None], _i32(counts)[:, None]
    col = torch.arange(width, dtype=torch.int32, device="cuda")
    at = (start + col).clamp(max=perm.numel() - 1).long()
    return torch.where(col < count, perm[at], torch.full_like(at, -1, dtype=torch.int32))


# ---- one pass --------------------------------------------------------------------

def run(state):
    return {"plan": _plan, "tree": _tree, "accept": _accept}[state["case"]["op"]](state)


def _plan(s):
    if own:
        import paged_kv_cache_109_gb300 as pa
        p = pa.StepPlan(**s["buffers"])
        pa.plan_step(s["lens"], s["new"], s["tables"], s["held"], s["free"], s["head"],
                     s["num_blocks"], s["case"]["block"], p)
        return {"tables": s["tables"], **s["buffers"]}
    block, tables = s["case"]["block"], s["tables"]
    total = s["lens"] + s["new"]
    held = torch.maximum(s["held"], (total + block - 1) // block)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = torch.cat([zero, s["new"].cumsum(0, dtype=torch.int32)])
    taken = torch.cat([zero, (held - s["held"]).cumsum(0, dtype=torch.int32)])
    col = torch.arange(tables.shape[1], dtype=torch.int32, device="cuda")
    fresh = (col >= s["held"][:, None]) & (col < held[:, None])
    at = (s["head"] + taken[:-1, None] + col - s["held"][:, None]).clamp(0, s["free"].numel() - 1)
    tables.copy_(torch.where(fresh, s["free"][at.long()], tables))
    token = torch.arange(s["buffers"]["slot_mapping"].numel(), dtype=torch.int32, device="cuda")
    seq = torch.searchsorted(start, token, right=True).clamp(max=s["case"]["n"]) - 1
    live = token < start[-1]
    pos = s["lens"][seq] + token - start[seq]
    entry = tables[seq, (pos // block).clamp(0, tables.shape[1] - 1).long()]
    slot = entry.long() * block + pos % block
    none = torch.full_like(token, -1)
    return {"tables": tables, "seq_lens": total, "blocks_held": held,
            "free_head": s["head"] + taken[-1:], "query_start_loc": start, "block_start": taken,
            "slot_mapping": torch.where(live, slot, none.long()),
            "positions": torch.where(live, pos, none),
            "seq_ids": torch.where(live, seq.int(), none)}


def _ancestors(s):
    """[n, nodes, nodes]: node k is node j or one of its ancestors, and each
    request's parents by node (0 past its last node)."""
    n, m = s["case"]["n"], s["max_q"]
    node = torch.arange(m, device="cuda")
    count = (s["start"][1:] - s["start"][:-1])[:, None]
    at = (s["start"][:-1, None] + node).clamp(max=s["parents"].numel() - 1).long()
    up = torch.where(node < count, s["parents"][at], torch.full_like(at, -1, dtype=torch.int32))
    reach = torch.eye(m, device="cuda").expand(n, m, m) + (up[:, :, None] == node)
    for _ in range(max(1, (s["max_depth"] - 1).bit_length())):
        reach = (reach @ reach > 0).float()           # paths of twice the length
    return reach > 0, node < count


def _tree(s):
    case = s["case"]
    if own:
        import paged_kv_cache_109_gb300 as pa
        return pa.decode_tree(s["q"], s["start"], s["parents"], s["k"], s["v"], s["tables"],
                              s["lens"], s["max_q"], s["max_len"])
    n, m, hkv, group, dim, block = (case["n"], s["max_q"], case["hkv"], case["group"],
                                    case["dim"], case["block"])
    count = s["start"][1:] - s["start"][:-1]
    cached = (s["lens"] - count)[:, None, None]
    pos = torch.arange(s["max_len"], device="cuda")
    entry = s["tables"][:, pos // block].clamp(min=0).long()
    keys = s["k"][entry, :, pos % block].float().permute(0, 2, 1, 3)     # [n, hkv, len, dim]
    vals = s["v"][entry, :, pos % block].float().permute(0, 2, 1, 3)
    reach, _ = _ancestors(s)
    node = (pos - cached).clamp(0, m - 1).expand(n, m, -1)
    seen = (pos < cached) | ((pos < s["lens"][:, None, None]) & reach.gather(2, node))
    at = (s["start"][:-1, None] + torch.arange(m, device="cuda")).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at.long()].float().view(n, m, hkv, group, dim).permute(0, 2, 3, 1, 4)
    score = (q.reshape(n, hkv, group * m, dim) @ keys.transpose(2, 3)) * (1.0 / math.sqrt(dim))
    score = score.view(n, hkv, group, m, -1).masked_fill_(~seen[:, None, None], -math.inf)
    score -= score.amax(-1, keepdim=True).clamp(min=-3e38)
    score.exp_()
    total = score.sum(-1, keepdim=True)
    out = (score.view(n, hkv, group * m, -1) @ vals).view(n, hkv, group, m, dim) / total
    row = torch.arange(s["q"].shape[0], dtype=torch.int32, device="cuda")
    seq = torch.searchsorted(s["start"], row, right=True) - 1
    out = out.permute(0, 3, 1, 2, 4)[seq, (row - s["start"][seq]).long()]
    return out.reshape(s["q"].shape).to(s["q"].dtype)


def _accept(s):
    if own:
        import paged_kv_cache_109_gb300 as pa
        lens, rows = pa.accept_tree(s["leaf"], s["parents"], s["start"], s["lens"], s["k"],
                                    s["v"], s["tables"], s["max_q"])
        return {"lens": lens, "rows": rows, "k": s["k"], "v": s["v"]}
    block, m = s["case"]["block"], s["max_q"]
    reach, real = _ancestors(s)
    count = s["start"][1:] - s["start"][:-1]
    cached = s["lens"] - count
    at = s["leaf"].clamp(min=0).long()[:, None, None].expand(-1, 1, m)
    on = reach.gather(1, at)[:, 0] & real & (s["leaf"] >= 0)[:, None]    # nodes of the path
    depth = on.int().cumsum(1) - 1
    seq, node = on.nonzero(as_tuple=True)
    rank = depth[seq, node]
    src, dst = (cached[seq] + node).long(), (cached[seq] + rank).long()
    sb, db = s["tables"][seq, src // block].long(), s["tables"][seq, dst // block].long()
    s["k"][:, db, :, dst % block] = s["k"][:, sb, :, src % block]
    s["v"][:, db, :, dst % block] = s["v"][:, sb, :, src % block]
    rows = torch.full_like(s["parents"], -1)
    rows[(s["start"][seq] + rank).long()] = (s["start"][seq] + node).int()
    return {"lens": cached + on.sum(1, dtype=torch.int32), "rows": rows, "k": s["k"], "v": s["v"]}


# ---- the definition in 64 bits -------------------------------------------------------

def exact(case, seed):
    """Attention of each drafted token over its visible keys, one request and
    kv head at a time.  The other operators move or count whole values."""
    if case["op"] != "tree":
        return None
    s = prepare(case, seed)
    group, dim, block = case["group"], case["dim"], case["block"]
    lens, start, parents = s["lens"].tolist(), s["start"].tolist(), s["parents"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, length in enumerate(lens):
        q0, q1 = start[i], start[i + 1]
        nodes = q1 - q0
        hidden = torch.ones(nodes, nodes, dtype=torch.bool)
        for j in range(nodes):
            hidden[j, _path(parents[q0:q1], j)] = False
        hidden = hidden.cuda().repeat_interleave(group, 0)               # rows (node, head)
        blocks = s["tables"][i, :-(-length // block)].long()
        for g in range(case["hkv"]):
            k = s["k"][blocks, g].reshape(-1, dim)[:length].double()
            v = s["v"][blocks, g].reshape(-1, dim)[:length].double()
            q = s["q"][q0:q1, g * group:(g + 1) * group].double().reshape(-1, dim)
            w = q @ k.T / math.sqrt(dim)
            w[:, length - nodes:][hidden] = -math.inf
            w = torch.softmax(w, 1)
            out[q0:q1, g * group:(g + 1) * group] = (w @ v).view(nodes, group, dim)
    return out
