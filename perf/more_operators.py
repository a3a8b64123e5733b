"""Cases of the steps around paged attention that keep a serving loop on the
GPU: the operators' plain forms in torch and the framework's calls, on the same
inputs.

``rope``     a layer's projected rows to its attention: queries and keys are
             normed for each head and rotated by their positions (on one axis
             or several), the keys and values go to their cache slots, all in
             one pass (``rope_write``).
``verify``   drafted tokens against the target's probabilities, from given
             random numbers: the deepest token that holds and the one that
             follows it (``verify_tree``).
``release``  the blocks that requests no longer need go back to the free queue
             (``release_blocks``).
``branch``   the life of parallel candidates: prompts are forked, sharing their
             full blocks, a partly filled one copied in every layer, and the
             candidates' blocks go back (``fork_blocks``, ``release_blocks``
             with reference counts).

Sizes of a case follow from the case alone; the seed sets the order of the
requests, the physical blocks and the values.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one user's next token: latency
        dict(name="rope-one", op="rope", dtype="bf16", n=1, pad=0, hq=32, hkv=8, dim=128, rot=128,
             axes=1, order="sections", pairs="halves", norm=True, block=16, far=4096),
        # a decode step of the continuous-batching batch with a prompt's chunk in it
        dict(name="rope-step", op="rope", dtype="bf16", n=2303, pad=1, hq=32, hkv=8, dim=128,
             rot=128, axes=1, order="sections", pairs="halves", norm=True, block=16, far=6144),
        # chunks of several long prompts, no norms
        dict(name="rope-prompts", op="rope", dtype="bf16", n=16384, pad=0, hq=64, hkv=8, dim=128,
             rot=128, axes=1, order="sections", pairs="halves", norm=False, block=32, far=131072),
        # images and text on three axes, a part of the head rotated, neighbouring
        # pairs, fp32, odd sizes
        dict(name="rope-axes", op="rope", dtype="f32", n=5001, pad=7, hq=15, hkv=5, dim=80, rot=48,
             axes=3, order="cyclic", pairs="neighbours", norm=True, block=24, far=20000),
        # one user, a chain of drafted tokens: latency
        dict(name="verify-one", op="verify", dtype="bf16", n=1, vocab=32000, shape="chain",
             nodes_lo=6, nodes_hi=6, draft=True, greedy=0.0),
        # a batch of short chains
        dict(name="verify-chains", op="verify", dtype="bf16", n=64, vocab=131072, shape="chain",
             nodes_lo=5, nodes_hi=5, draft=True, greedy=0.0),
        # ragged trees, some requests greedy
        dict(name="verify-trees", op="verify", dtype="bf16", n=128, vocab=131072, shape="tree",
             nodes_lo=1, nodes_hi=40, draft=True, greedy=0.1),
        # tokens drafted without probabilities, fp32, an odd vocabulary
        dict(name="verify-lookup", op="verify", dtype="f32", n=48, vocab=100003, shape="tree",
             nodes_lo=1, nodes_hi=16, draft=False, greedy=0.2),
        # a few of a decode batch's requests end
        dict(name="release-few", op="release", n=256, block=16, lo=1, hi=4096, done=0.05),
        # many requests cancelled at once, drafted blocks trimmed
        dict(name="release-many", op="release", n=2048, block=16, lo=1, hi=6000, done=0.5),
        # one prompt, four candidates, one layer: latency
        dict(name="branch-one", op="branch", dtype="bf16", n=8, prompts=1, children=4, hkv=8,
             dim=128, block=16, layers=1, lo=200, hi=200),
        # several candidates of many prompts, all layers of a model part
        dict(name="branch-batch", op="branch", dtype="bf16", n=128, prompts=24, children=4, hkv=8,
             dim=128, block=16, layers=16, lo=1, hi=2048),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "verify", "verify", "release", "branch"])
    block = rng.choice([4, 8, 16, 16, 24, 32, 64])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    size = 4 if dtype == "f32" else 2
    if op == "rope":
        dim = rng.choice([16, 32, 64, 64, 80, 96, 112, 128, 128, 128, 192, 256])
        hkv = rng.choice([1, 2, 3, 4, 8, 8, 16])
        hq = hkv * rng.choice([1, 2, 3, 4, 4, 5, 8])
        n = _log(rng, 1, 16384)
        while n * (hq + 2 * hkv) * dim * size > 16384 * 80 * 128 * 2:
            n = (n + 1) // 2
        axes = rng.choice([1, 1, 2, 3])
        return dict(op=op, dtype=dtype, n=n, pad=rng.choice([0, 0, min(n - 1, 5)]), hq=hq, hkv=hkv,
                    dim=dim, rot=rng.choice([dim, dim, dim // 2, dim - 4]), axes=axes,
                    order=rng.choice(["sections", "cyclic"]),
                    pairs=rng.choice(["halves", "neighbours"]), norm=rng.random() < 0.7,
                    block=block, far=_log(rng, max(n, 128), 1000000))
    if op == "verify":
        vocab = _log(rng, 1000, 160000)
        n = _log(rng, 1, 128)
        shape = rng.choice(["chain", "tree"])
        nodes = _log(rng, 1, 10) if shape == "chain" else _log(rng, 1, 40)
        # at most the largest listed batch's logits
        while n * (nodes + 1) * vocab * size > 128 * 41 * 131072 * 2 or n * vocab > 128 * 131072:
            n = (n + 1) // 2
        return dict(op=op, dtype=dtype, n=n, vocab=vocab, shape=shape,
                    nodes_lo=rng.randint(1, nodes), nodes_hi=nodes, draft=rng.random() < 0.6,
                    greedy=rng.choice([0.0, 0.0, 0.2, 1.0]))
    if op == "release":
        n = _log(rng, 1, 4096)
        hi = min(_log(rng, 16, 8192), 2048 * 6000 // n)
        return dict(op=op, n=n, block=block, lo=rng.randint(0, min(hi, 16)), hi=hi,
                    done=rng.choice([0.02, 0.1, 0.5, 1.0]))
    dim = rng.choice([16, 32, 64, 64, 80, 96, 112, 128, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
    layers, prompts, children = _log(rng, 1, 16), _log(rng, 1, 64), _log(rng, 1, 8)
    hi = _log(rng, 16, 2048)
    # at most the largest listed batch's caches
    while prompts * (hi + children * block) * layers * hkv * dim * size > 1.6e9:
        prompts, hi = (prompts + 1) // 2, hi if prompts > 1 else hi // 2
    return dict(op=op, dtype=dtype, n=prompts * (1 + children) + rng.randint(0, 9), prompts=prompts,
                children=children, hkv=hkv, dim=dim, block=block, layers=layers, lo=0, hi=hi)


# ---- sizes: from the case alone ------------------------------------------------

def _rng(case, keys):
    return random.Random("/".join(str(case[k]) for k in keys.split()))


def _trees(case):
    """Per request the parents of its nodes; node 0 is the token that was
    sampled last and the root of all others."""
    rng = _rng(case, "op n shape nodes_lo nodes_hi")
    out = []
    for _ in range(case["n"]):
        m = rng.randint(case["nodes_lo"], case["nodes_hi"])
        if case["shape"] == "chain":
            out.append(list(range(-1, m - 1)))
            continue
        parents = [-1]
        for j in range(1, m):
            # up to four continuations of a node, most of them of early ones
            free = [p for p in range(max(0, j - 9), j) if parents.count(p) < 4]
            parents.append(rng.choice(free))
        out.append(parents)
    return out


def _levels(trees):
    """(nodes on the longest path, most children of a node)."""
    deep = wide = 0
    for parents in trees:
        depth = []
        for p in parents:
            depth.append(1 if p < 0 else depth[p] + 1)
        deep = max([deep] + depth)
        wide = max([wide] + [parents.count(p) for p in set(parents) if p >= 0])
    return deep, wide


def _visited(case):
    """Rows that a walk down the trees reads: a drafted token holds about twice
    in three times (a greedy request's half as often)."""
    rng = _rng(case, "op n shape nodes_lo nodes_hi greedy")
    rows = inner = 0
    for parents in _trees(case):
        hold = 0.33 if rng.random() < case["greedy"] else 0.67
        cur = 0
        while True:
            rows += 1
            kids = [j for j, p in enumerate(parents) if p == cur]
            inner += bool(kids)
            took = [j for j in kids if rng.random() < hold]
            if not took:
                break
            cur = took[0]
    return rows, inner


def _lengths(case):
    """release: per request tokens kept and blocks held."""
    rng = _rng(case, "op n block lo hi done")
    out = []
    for _ in range(case["n"]):
        length = rng.randint(case["lo"], case["hi"])
        held = -(-length // case["block"]) + rng.choice([0, 0, 0, 1, 2])
        out.append((0 if rng.random() < case["done"] else length, held))
    return out


def _prompts(case):
    rng = _rng(case, "op n prompts block lo hi")
    return [rng.randint(case["lo"], case["hi"]) for _ in range(case["prompts"])]


def work(case):
    if case["op"] == "rope":
        size = 4 if case["dtype"] == "f32" else 2
        live = case["n"] - case["pad"]
        elems = live * (case["hq"] + 2 * case["hkv"]) * case["dim"]
        turned = live * (case["hq"] + case["hkv"]) * case["dim"]
        return {"bytes": 2 * elems * size + case["n"] * (8 + 4 * case["axes"]),
                "flops": turned * (7 if case["norm"] else 3)}
    if case["op"] == "verify":
        size = 4 if case["dtype"] == "f32" else 2
        rows, inner = _visited(case)
        if case["draft"]:
            rows += inner
        # (a greedy request needs no noise)
        noise = 4 * case["vocab"] * case["n"] * (1 - case["greedy"])
        return {"bytes": int(rows * case["vocab"] * size + noise),
                "flops": 4 * rows * case["vocab"]}
    block = case["block"]
    if case["op"] == "release":
        freed = sum(h - -(-t // block) for t, h in _lengths(case))
        return {"bytes": 16 * case["n"] + 8 * freed + 8, "flops": 0}
    lens, kids = _prompts(case), case["children"]
    entries = sum(-(-t // block) for t in lens) * kids
    full = sum(t // block for t in lens) * kids
    tail = sum(t % block for t in lens) * kids
    size = 4 if case["dtype"] == "f32" else 2
    row = case["hkv"] * case["dim"] * size * 2 * case["layers"]
    # fork: table entries and counts read and written, tails copied; release:
    # entries read, counts read and written
    return {"bytes": 8 * entries + 8 * full + 2 * tail * row + 12 * entries + 32 * case["n"],
            "flops": 0}


# ---- inputs --------------------------------------------------------------------

def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _tables(perm, counts, width):
    """Row i: the next counts[i] entries of perm, then -1."""
    start, count = _i32(_starts(counts))[:-1, None], _i32(counts)[:, None]
    col = torch.arange(width, dtype=torch.int32, device="cuda")
    at = (start + col).clamp(max=perm.numel() - 1).long()
    return torch.where(col < count, perm[at], torch.full_like(at, -1, dtype=torch.int32))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"rope": _rope_state, "verify": _verify_state, "release": _release_state,
            "branch": _branch_state}[case["op"]](case, seed, gen)


def _sections(case):
    """Pairs of each axis: about a quarter of them turn with time."""
    half, axes = case["rot"] // 2, case["axes"]
    if axes == 1:
        return None
    part = 3 * half // 8 if axes == 3 else half // 2
    if case["order"] == "cyclic":
        part = half // axes
    return (half - part * (axes - 1),) + (part,) * (axes - 1)


def _rope_state(case, seed, gen):
    dtype, n, axes = DTYPES[case["dtype"]], case["n"], case["axes"]
    hq, hkv, dim, block = case["hq"], case["hkv"], case["dim"], case["block"]
    live = n - case["pad"]
    num_blocks = -(-live * 5 // (4 * block)) + 1

    def values(*shape):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        return x.normal_(generator=gen)

    qkv = values(n, (hq + 2 * hkv) * dim)               # the projection's result
    q, k, v = qkv.split([hq * dim, hkv * dim, hkv * dim], 1)
    pos = torch.randint(0, case["far"], (axes, n), device="cuda", generator=gen).int()
    if axes > 1:
        # patches of images: rows and columns count from the frame's place
        side = torch.randint(0, 64, (axes - 1, n), device="cuda", generator=gen).int()
        text = torch.rand(n, device="cuda", generator=gen) < 0.3
        pos[1:] = torch.where(text, pos[:1], pos[:1] + side)
    slots = torch.randperm(num_blocks * block, device="cuda", generator=gen)[:n]
    if slots.numel() < n:
        slots = torch.cat([slots, slots.new_full((n - slots.numel(),), -1)])
    pos[:, live:] = -1                                  # the plan's bound is above the step's tokens
    slots[live:] = -1
    rot = case["rot"]
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))
    state = {"case": case, "live": live, "sections": _sections(case),
             "q": q.unflatten(1, (hq, dim)), "k": k.unflatten(1, (hkv, dim)),
             "v": v.unflatten(1, (hkv, dim)), "pos": pos[0].contiguous() if axes == 1 else pos,
             "inv": inv.float(), "slots": slots, "out": values(n, hq, dim),
             "k_cache": values(num_blocks, hkv, block, dim),
             "v_cache": values(num_blocks, hkv, block, dim), "q_weight": None, "k_weight": None}
    if case["norm"]:
        for name in ("q_weight", "k_weight"):
            state[name] = (1 + 0.2 * values(dim).float()).to(dtype)
    return state


def _verify_state(case, seed, gen):
    dtype, n, vocab = DTYPES[case["dtype"]], case["n"], case["vocab"]
    trees = _trees(case)
    random.Random(seed).shuffle(trees)
    start = _starts([len(t) for t in trees])
    total = start[-1]
    parents = [p for t in trees for p in t]
    temps = torch.rand(n, device="cuda", generator=gen) * 0.6 + 0.6
    temps[torch.rand(n, device="cuda", generator=gen) < case["greedy"]] = 0.0
    logits = torch.empty((total, vocab), dtype=dtype, device="cuda")
    draft = torch.empty_like(logits) if case["draft"] else None
    # row of the parent, and which of its children a node is
    up = [start[i] + max(p, 0) for i, t in enumerate(trees) for p in t]
    seen, rank = {}, []
    for u, p in zip(up, parents):
        rank.append(seen.get(u, 0) if p >= 0 else 0)
        if p >= 0:
            seen[u] = rank[-1] + 1
    seq = torch.tensor([i for i, t in enumerate(trees) for _ in t], device="cuda")
    up_t, rank_t = torch.tensor(up, device="cuda"), torch.tensor(rank, device="cuda")
    tokens = torch.zeros(total, dtype=torch.int32, device="cuda")
    step = max(1, (1 << 28) // vocab)
    for r in range(0, total, step):
        rows = slice(r, min(total, r + step))
        x = torch.empty((rows.stop - r, vocab), dtype=torch.float32, device="cuda")
        x.normal_(0.0, 2.5, generator=gen)
        logits[rows] = x.to(dtype)
        if draft is not None:
            # the draft model: close to the target, not the same
            x.add_(torch.empty_like(x).normal_(0.0, 0.6, generator=gen))
            draft[rows] = x.to(dtype)
    for r in range(0, total, step):
        rows = slice(r, min(total, r + step))
        heat = temps[seq[rows], None].clamp(min=0.05)
        if draft is not None:
            # each token is drawn from the draft's distribution at its parent
            e = torch.empty((rows.stop - r, vocab), dtype=torch.float32, device="cuda")
            e.exponential_(generator=gen)
            tokens[rows] = (draft[up_t[rows]].float() / heat - e.log()).argmax(1).int()
        else:
            # the likeliest tokens of something like the target
            x = logits[up_t[rows]].float()
            x.add_(torch.empty_like(x).normal_(0.0, 0.6, generator=gen))
            top = x.topk(8, dim=1).indices
            tokens[rows] = top.gather(1, (rank_t[rows] % 8)[:, None])[:, 0].int()
    deep, wide = _levels(trees)
    noise = torch.empty((n, vocab), dtype=torch.float32, device="cuda")
    return {"case": case, "logits": logits, "draft": draft, "tokens": tokens,
            "parents": _i32(parents), "start": _i32(start), "temps": temps, "deep": deep,
            "wide": wide, "max_q": max(len(t) for t in trees),
            "uniforms": torch.rand(total, device="cuda", generator=gen),
            "noise": noise.exponential_(generator=gen)}


def _release_state(case, seed, gen):
    lens = _lengths(case)
    random.Random(seed).shuffle(lens)
    held = [h for _, h in lens]
    used, spare = sum(held), case["n"] // 3
    perm = torch.randperm(used + spare, device="cuda", generator=gen).int()
    free = torch.full((used + spare,), -1, dtype=torch.int32, device="cuda")
    free[used:] = perm[used:]                           # blocks in use left the queue's front
    n = case["n"]
    return {"case": case, "lens": _i32([t for t, _ in lens]), "held": _i32(held),
            "tables": _tables(perm, held, max(held) + 2), "free": free, "head": _i32([used]),
            "num_blocks": used + spare, "held_out": torch.empty(n, dtype=torch.int32, device="cuda"),
            "head_out": torch.empty(1, dtype=torch.int32, device="cuda")}


def _branch_state(case, seed, gen):
    dtype, n, block = DTYPES[case["dtype"]], case["n"], case["block"]
    prompts, kids = _prompts(case), case["children"]
    order = list(range(n))
    random.Random(seed).shuffle(order)                  # rows of the batch
    lens, src = [0] * n, [-1] * n
    for p, t in enumerate(prompts):
        lens[order[p]] = t
        for c in range(kids):
            src[order[len(prompts) + p * kids + c]] = order[p]
    held = [-(-t // block) for t in lens]
    used = sum(held)
    num_blocks = used + len(prompts) * kids + 3
    perm = torch.randperm(num_blocks, device="cuda", generator=gen).int()
    free = torch.full((num_blocks,), -1, dtype=torch.int32, device="cuda")
    free[used:] = perm[used:]
    counts = torch.zeros(num_blocks, dtype=torch.int32, device="cuda")
    counts[perm[:used].long()] = 1
    shape = (case["layers"], num_blocks, case["hkv"], block, case["dim"])
    state = {"case": case, "src": _i32(src), "lens": _i32(lens), "held": _i32(held),
             "tables": _tables(perm, held, max(held) + 2), "free": free, "head": _i32([used]),
             "ref_cnt": counts, "rows": torch.tensor([i for i in range(n) if src[i] >= 0],
                                                     device="cuda"),
             "k": torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen),
             "v": torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)}
    for name, m in (("lens_fork", n), ("held_fork", n), ("head_fork", 1), ("held_out", n),
                    ("head_out", 1)):
        state[name] = torch.empty(m, dtype=torch.int32, device="cuda")
    return state


# ---- one pass --------------------------------------------------------------------

def run(state):
    return {"rope": _rope, "verify": _verify, "release": _release,
            "branch": _branch}[state["case"]["op"]](state)


def _axis_of_pair(case, sections):
    """Axis of each rotated pair."""
    half = case["rot"] // 2
    if sections is None:
        return [0] * half
    if case["order"] == "sections":
        return [a for a, m in enumerate(sections) for _ in range(m)]
    axes = len(sections)
    return [j % axes if j < axes * sections[j % axes] else 0 for j in range(half)]


def _rope(s):
    case = s["case"]
    if own:
        import paged_kv_cache_109_gb300 as pa
        pa.rope_write(s["q"], s["k"], s["v"], s["pos"], s["inv"], s["slots"], s["k_cache"],
                      s["v_cache"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                      sections=s["sections"], cyclic=case["order"] == "cyclic",
                      neighbours=case["pairs"] == "neighbours", out=s["out"])
        return {"out": s["out"], "k": s["k_cache"], "v": s["v_cache"]}
    live, rot, block = s["live"], case["rot"], case["block"]
    pos = s["pos"].view(case["axes"], -1)[:, :live]
    axis = torch.tensor(_axis_of_pair(case, s["sections"]), device="cuda")
    angle = pos[axis].T.double() * s["inv"].double()                # [live, rot / 2]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, weight):
        x = x[:live].float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        if case["pairs"] == "halves":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        a, b = a * cos - b * sin, a * sin + b * cos
        front = torch.cat([a, b], -1) if case["pairs"] == "halves" else torch.stack([a, b], -1).flatten(-2)
        return torch.cat([front, x[..., rot:]], -1).to(s["out"].dtype)

    s["out"][:live] = turned(s["q"], s["q_weight"])
    at, off = s["slots"][:live] // block, s["slots"][:live] % block
    s["k_cache"][at, :, off] = turned(s["k"], s["k_weight"])
    s["v_cache"][at, :, off] = s["v"][:live]
    return {"out": s["out"], "k": s["k_cache"], "v": s["v_cache"]}


def _verify(s):
    if own:
        import paged_kv_cache_109_gb300 as pa
        leaf, token = pa.verify_tree(s["logits"], s["tokens"], s["parents"], s["start"],
                                     s["uniforms"], s["noise"], s["max_q"],
                                     draft_logits=s["draft"], temperature=s["temps"])
        return {"leaf": leaf, "token": token}
    # 64 bits: a token next to another's border must fall on the right side
    n, vocab = s["case"]["n"], s["case"]["vocab"]
    start, parents, tokens = s["start"][:-1].long(), s["parents"], s["tokens"].long()
    count = s["start"][1:].long() - start
    node = torch.arange(s["max_q"], device="cuda")
    real = node < count[:, None]
    at = (start[:, None] + node).clamp(max=parents.numel() - 1)
    up = torch.where(real, parents[at].long(), torch.full_like(at, -1))     # [n, nodes]
    cold, column = s["temps"] <= 0, torch.arange(vocab, device="cuda")
    heat = torch.where(cold, torch.ones_like(s["temps"]), s["temps"]).double()[:, None]

    def chances(x, rows):
        x = x[rows].double()
        first = torch.where(x == x.amax(1, keepdim=True), column, vocab).amin(1, keepdim=True)
        first = torch.zeros_like(x).scatter_(1, first, 1.0)
        return torch.where(cold[:, None], first, torch.softmax(x / heat, 1))

    cur = torch.zeros(n, dtype=torch.long, device="cuda")
    done = torch.zeros(n, dtype=torch.bool, device="cuda")
    rest = torch.zeros((n, vocab), dtype=torch.float64, device="cuda")
    one = torch.arange(n, device="cuda")
    for _ in range(s["deep"]):
        p = chances(s["logits"], start + cur)
        q = None if s["draft"] is None else chances(s["draft"], start + cur)
        child = real & (up == cur[:, None]) & (node > 0)
        rank = child.int().cumsum(1)
        left, share = p, torch.ones(n, dtype=torch.float64, device="cuda")
        took = torch.full((n,), -1, dtype=torch.long, device="cuda")
        spent = torch.zeros(n, dtype=torch.float64, device="cuda")
        for c in range(1, s["wide"] + 1):
            is_c = child & (rank == c)
            has = is_c.any(1) & (took < 0)
            j = is_c.int().argmax(1)
            row = (start + j).clamp(max=parents.numel() - 1)
            t, u = tokens[row], s["uniforms"][row].double()
            hold_q = torch.ones_like(share) if q is None else q[one, t]
            hold = torch.where(cold, left[one, t] > 0, u * hold_q * share < left[one, t])
            took = torch.where(has & hold, j, took)
            out = has & ~hold
            if q is None:
                gone = left.scatter(1, t[:, None], 0.0)
            else:
                spent = torch.where(out, spent + share, spent)
                gone = torch.where(cold[:, None], p, (p - spent[:, None] * q).clamp(min=0))
            left = torch.where(out[:, None], gone, left)
            share = torch.where(out, left.sum(1), share)
        stop = ~done & (took < 0)
        rest = torch.where(stop[:, None], torch.where(share[:, None] > 0, left, p), rest)
        done |= stop
        cur = torch.where(took >= 0, took, cur)
    race = torch.where(cold[:, None], rest, rest / s["noise"].double())
    return {"leaf": cur.int(), "token": race.argmax(1).int()}


def _drop(tables, held, keep, ref_cnt, free, head, num_blocks):
    """Plain release: (blocks held after, the queue's front after); ref_cnt and
    free are updated."""
    col = torch.arange(tables.shape[1], dtype=torch.int32, device="cuda")
    drop = ((col >= keep[:, None]) & (col < held[:, None])).flatten()
    ids = torch.where(drop, tables.flatten(), torch.full_like(col[:1], num_blocks)).long()
    freed = drop
    if ref_cnt is not None:
        counts = torch.cat([ref_cnt, ref_cnt.new_zeros(1)])
        counts.index_add_(0, ids, -drop.int())
        ref_cnt.copy_(counts[:num_blocks])
        flat = torch.arange(ids.numel(), device="cuda")
        last = torch.full((num_blocks + 1,), -1, device="cuda").scatter_reduce(0, ids, flat, "amax")
        freed = drop & (counts[ids] == 0) & (last[ids] == flat)
    rank = freed.cumsum(0) - 1
    front = head.long() - freed.sum()
    wide = torch.cat([free, free.new_zeros(1)])
    wide.scatter_(0, torch.where(freed, front + rank, torch.full_like(rank, free.numel())),
                  torch.where(freed, tables.flatten(), torch.zeros_like(tables.flatten())))
    free.copy_(wide[:-1])
    return torch.minimum(held, keep), front.int()


def _release(s):
    if own:
        import paged_kv_cache_109_gb300 as pa
        pa.release_blocks(s["lens"], s["tables"], s["held"], s["free"], s["head"],
                          s["num_blocks"], s["case"]["block"], blocks_held_out=s["held_out"],
                          free_head_out=s["head_out"])
        return {"held": s["held_out"], "head": s["head_out"], "free": s["free"]}
    block = s["case"]["block"]
    held, head = _drop(s["tables"], s["held"], (s["lens"] + block - 1) // block, None, s["free"],
                       s["head"], s["num_blocks"])
    return {"held": held, "head": head, "free": s["free"]}


def _branch(s):
    out = {k: s[k] for k in ("tables", "free", "ref_cnt", "k", "v")}
    block, num_blocks = s["case"]["block"], s["k"].shape[1]
    if own:
        import paged_kv_cache_109_gb300 as pa
        pa.fork_blocks(s["src"], s["lens"], s["tables"], s["held"], s["ref_cnt"], s["free"],
                       s["head"], s["k"], s["v"], seq_lens_out=s["lens_fork"],
                       blocks_held_out=s["held_fork"], free_head_out=s["head_fork"])
        # the candidates end: the lengths before the fork say what stays
        pa.release_blocks(s["lens"], s["tables"], s["held_fork"], s["free"], s["head_fork"],
                          num_blocks, block, ref_cnt=s["ref_cnt"], blocks_held_out=s["held_out"],
                          free_head_out=s["head_out"])
        return {"lens": s["lens_fork"], "held_fork": s["held_fork"], "head_fork": s["head_fork"],
                "held": s["held_out"], "head": s["head_out"], **out}
    rows, tables, counts = s["rows"], s["tables"], s["ref_cnt"]
    src = s["src"][rows].long()
    length = s["lens"][src]
    full, tail = length // block, (length % block > 0)
    col = torch.arange(tables.shape[1], dtype=torch.int32, device="cuda")
    fresh = s["free"][(s["head"] + tail.int().cumsum(0) - 1).clamp(0, num_blocks - 1).long()]
    shared, own_tail = col < full[:, None], (col == full[:, None]) & tail[:, None]
    old = tables[src]
    tables[rows] = torch.where(shared, old, torch.where(own_tail, fresh[:, None], tables[rows]))
    wide = torch.cat([counts, counts.new_zeros(1)])
    none = torch.full_like(old, num_blocks).long()
    wide.index_add_(0, torch.where(shared, old.long(), none).flatten(), shared.flatten().int())
    wide.index_fill_(0, torch.where(tail, fresh.long(), none[:, 0]), 1)
    counts.copy_(wide[:num_blocks])
    # a child without a tail copies a block onto itself
    from_block = old.gather(1, full[:, None].clamp(max=old.shape[1] - 1).long())[:, 0].long()
    to_block = torch.where(tail, fresh.long(), s["free"][-1:].long())
    from_block = torch.where(tail, from_block, to_block)
    moved = (torch.arange(block, device="cuda") < (length % block)[:, None])[None, :, None, :, None]
    for cache in (s["k"], s["v"]):
        cache[:, to_block] = torch.where(moved, cache[:, from_block], cache[:, to_block])
    lens_fork = s["lens"].index_copy(0, rows, length)
    held_fork = s["held"].index_copy(0, rows, (length + block - 1) // block)
    head_fork = s["head"] + tail.sum().int()
    held, head = _drop(tables, held_fork, (s["lens"] + block - 1) // block, counts, s["free"],
                       head_fork, num_blocks)
    return {"lens": lens_fork, "held_fork": held_fork, "head_fork": head_fork, "held": held,
            "head": head, **out}


# ---- the definition in 64 bits -------------------------------------------------------

def exact(case, seed):
    """``rope``: each pair as a complex number, turned by exp(i angle).
    ``verify``: the walk of each request, token by token.  The others move or
    count whole values."""
    if case["op"] == "rope":
        return _exact_rope(prepare(case, seed))
    if case["op"] == "verify":
        return _exact_verify(prepare(case, seed))
    return None


def _exact_rope(s):
    case = s["case"]
    rot, block, half = case["rot"], case["block"], case["rot"] // 2
    pos = s["pos"].view(case["axes"], -1)
    angle = torch.zeros((case["n"], half), dtype=torch.float64, device="cuda")
    for j, a in enumerate(_axis_of_pair(case, s["sections"])):
        angle[:, j] = pos[a].double() * float(s["inv"][j])
    turn = torch.polar(torch.ones_like(angle), angle)
    live = list(range(case["n"] - case["pad"]))
    first = torch.arange(half, device="cuda")
    lo, hi = (first, first + half) if case["pairs"] == "halves" else (2 * first, 2 * first + 1)

    def rows(x, weight):
        y = x.double()
        if weight is not None:
            y = y / (y.square().sum(-1, keepdim=True) / case["dim"] + 1e-6).sqrt() * weight.double()
        z = torch.complex(y[..., lo], y[..., hi]) * turn[:, None]
        y = y.clone()
        y[..., lo], y[..., hi] = z.real, z.imag
        return y[:len(live)]

    out, k, v = s["out"].double(), s["k_cache"].double(), s["v_cache"].clone()
    out[:len(live)] = rows(s["q"], s["q_weight"])
    slots = s["slots"][:len(live)]
    head = torch.arange(case["hkv"], device="cuda")
    where = (slots.div(block, rounding_mode="floor")[:, None], head, slots.remainder(block)[:, None])
    k[where] = rows(s["k"], s["k_weight"])
    v[where] = s["v"][:len(live)]
    return {"out": out, "k": k, "v": v}


def _exact_verify(s):
    starts, parents = s["start"].tolist(), s["parents"].tolist()
    tokens, uniforms, temps = s["tokens"].tolist(), s["uniforms"].tolist(), s["temps"].tolist()
    leaves, follow = [], []
    for i, heat in enumerate(temps):
        q0, m = starts[i], starts[i + 1] - starts[i]
        cur, found = 0, None
        while found is None:
            row = q0 + cur
            kids = [j for j in range(m) if parents[q0 + j] == cur]
            if heat <= 0:
                best = int((s["logits"][row] == s["logits"][row].max()).nonzero()[0, 0])
                took = [j for j in kids if tokens[q0 + j] == best]
                if took:
                    cur = took[0]
                else:
                    found = best
                continue
            w = (s["logits"][row].double() / heat).exp()
            p = w / w.sum()
            left, q, c = p, None, 0.0
            if s["draft"] is not None:
                w = (s["draft"][row].double() / heat).exp()
                q = w / w.sum()
            took = -1
            for j in kids:
                t, total = tokens[q0 + j], float(left.sum())
                ask = uniforms[q0 + j] * total * (1.0 if q is None else float(q[t]))
                if ask < float(left[t]):
                    took = j
                    break
                left = left.clone()
                if q is None:
                    left[t] = 0.0
                else:
                    c += total if c else 1.0
                    left = (p - c * q).clamp(min=0)
            if took >= 0:
                cur = took
                continue
            if float(left.sum()) <= 0:
                left = p
            found = int((left / s["noise"][i].double()).argmax())
        leaves.append(cur)
        follow.append(found)
    return {"leaf": _i32(leaves), "token": _i32(follow)}
