"""Plain 64-bit forms of the drafted-step calls (pa_plan_step, pa_decode_tree,
pa_accept_tree), and random batches for their tests."""
import math

import numpy as np
import torch

from paged_kv_cache_109_gb300.block_pool import BlockPool


def path_of(parents, node):
    """Ancestors of ``node`` and itself, ascending."""
    out = []
    while node >= 0:
        out.append(node)
        node = int(parents[node])
    return out[::-1]


def random_parents(rng, n, kind="mixed"):
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":                       # every node continues the cached tokens
        return [-1] * n
    if kind == "forest":
        return [int(rng.integers(-1, j)) for j in range(n)]
    return [-1 if j == 0 else int(rng.integers(max(0, j - 3) if rng.random() < 0.7 else 0, j))
            for j in range(n)]


class Batch:
    """Host tensors of one verify step: per sequence ``ctx`` cached tokens and
    ``nodes`` drafted ones.  Positions at and behind T_i in the blocks, and the
    spare blocks, hold NaN, which no output may show."""

    def __init__(self, ctx, nodes, hkv, group, d, bs, dtype, seed, kind="mixed", scale=None,
                 spare=2):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.nodes, self.bs, self.group = list(ctx), list(nodes), bs, group
        n = len(self.ctx)
        lens = [c + m for c, m in zip(ctx, nodes)]
        need = [-(-t // bs) for t in lens]
        nb = sum(need) + spare
        perm = rng.permutation(nb).tolist()
        width, pos, rows = max(need, default=0) + 1, 0, []
        for k in need:
            rows.append(perm[pos:pos + k] + [-1] * (width - k))
            pos += k
        self.tables = torch.tensor(rows, dtype=torch.int32).view(n, width)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.start = torch.tensor([0] + list(np.cumsum(nodes)), dtype=torch.int32)
        self.par = [random_parents(rng, m, kind) for m in nodes]
        self.parents = torch.tensor([p for ps in self.par for p in ps], dtype=torch.int32)
        self.total = int(self.start[-1])
        self.max_q, self.max_len = max(nodes, default=0), max(lens, default=0)
        self.scale = 1 / math.sqrt(d) if scale is None else scale
        self.k = torch.randn(nb, hkv, bs, d, generator=g).to(dtype)
        self.v = torch.randn(nb, hkv, bs, d, generator=g).to(dtype)
        held = torch.full((nb * bs,), True)
        for i, t in enumerate(lens):
            for b in range(need[i]):
                s0 = rows[i][b] * bs
                held[s0:s0 + min(bs, t - b * bs)] = False
        for c in (self.k, self.v):
            c.transpose(1, 2)[held.view(nb, bs)] = float("nan")
        self.q = torch.randn(self.total, hkv * group, d, generator=g).to(dtype)

    def to(self, dev):
        return [x.to(dev) for x in (self.q, self.start, self.parents, self.k, self.v, self.tables,
                                    self.lens)]

    def run(self, pa, dev, **kw):
        q, start, parents, k, v, tables, lens = self.to(dev)
        return pa.decode_tree(q, start, parents, k, v, tables, lens, self.max_q, self.max_len,
                              self.scale, **kw)


def tree_reference(b):
    """(out, bound) in 64 bits: softmax over the visible keys, and per element
    the largest error the kernels' roundings can leave (before the rounding of
    the output itself, which the tolerance takes from the type).

    With A = sum_t p_t |v_t|: a score's fp32 dot product of D terms is off by
    at most D 2^-24 sum |q||k| scale (its scaling and the subtraction of the
    maximum by two more such roundings: the + 4), which moves each weight and
    the weights' sum by that share (2 ds A).  The sums over n keys add n 2^-24
    each (2 n 2^-24 A).  exp2's own error (2^-22, approximate unit), the
    rescales by it and the merge add 2^-19 A.  bf16 kernels hold a weight as
    two bf16 parts, off by 2^-16 in P V (2^-15 A covers the sum of both
    halves' rounding)."""
    n_rows, hq, d = b.q.shape
    q, k, v = b.q.double(), b.k.double(), b.v.double()
    out = torch.zeros(n_rows, hq, d, dtype=torch.float64)
    bound = torch.zeros_like(out)
    lo = 0.0 if b.q.dtype == torch.float32 else 2.0 ** -15
    for i, t in enumerate(b.lens.tolist()):
        q0, m = int(b.start[i]), b.nodes[i]
        if m == 0:
            continue
        blocks = b.tables[i, :-(-t // b.bs)].long()
        seen = torch.zeros(m, t, dtype=torch.bool)
        seen[:, :t - m] = True
        for j in range(m):
            seen[j, [t - m + a for a in path_of(b.par[i], j)]] = True
        for g in range(k.shape[1]):
            kk = k[blocks, g].reshape(-1, d)[:t]
            vv = v[blocks, g].reshape(-1, d)[:t]
            for h in range(g * b.group, (g + 1) * b.group):
                for j in range(m):
                    at = seen[j]
                    s = (kk[at] @ q[q0 + j, h]) * b.scale
                    p = torch.softmax(s, 0)
                    ds = (d + 4) * 2.0 ** -24 * abs(b.scale) * float(
                        (kk[at].abs() @ q[q0 + j, h].abs()).max())
                    out[q0 + j, h] = p @ vv[at]
                    a = p @ vv[at].abs()
                    bound[q0 + j, h] = a * (2 * ds + 2 * int(at.sum()) * 2.0 ** -24
                                            + 2.0 ** -19 + lo)
    return out, bound


def assert_tree_close(got, ref, bound, dtype, what=""):
    got = got.double().cpu()
    half = torch.finfo(dtype).eps / 2
    err = (got - ref).abs()
    bad = ~(err <= bound + half * (ref.abs() + bound))
    if bad.any():
        at = bad.nonzero()[:5].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())}/{bad.numel()} beyond the bound; worst "
                             f"{float((err / (bound + half * ref.abs())).nan_to_num(1e9).max()):.2f} "
                             f"of it; first {at}")


def accept_reference(b, leaf, k, v):
    """(new_lens, accepted_rows) and the caches moved in place (clones of b's)."""
    lens, rows = [], torch.full((b.total,), -1, dtype=torch.int32)
    for i, c in enumerate(b.ctx):
        q0 = int(b.start[i])
        path = path_of(b.par[i], leaf[i])
        lens.append(c + len(path))
        moved = []
        for j, a in enumerate(path):
            rows[q0 + j] = q0 + a
            sb, db = int(b.tables[i, (c + a) // b.bs]), int(b.tables[i, (c + j) // b.bs])
            moved.append((db, (c + j) % b.bs, k[sb, :, (c + a) % b.bs].clone(),
                          v[sb, :, (c + a) % b.bs].clone()))
        for db, off, kk, vv in moved:
            k[db, :, off], v[db, :, off] = kk, vv
    return torch.tensor(lens, dtype=torch.int32), rows


class PlanState:
    """Host state of a plan: a BlockPool with ``lens`` cached tokens and, per
    sequence, ``extra`` blocks held behind them."""

    def __init__(self, lens, extra, bs, num_blocks, width, seed):
        rng = np.random.default_rng(seed)
        self.pool = BlockPool(num_blocks, bs, rng.permutation(num_blocks).tolist())
        self.lens, self.bs, self.num_blocks = list(lens), bs, num_blocks
        n = len(self.lens)
        for i, t in enumerate(self.lens):
            self.pool.add(i, t)
        self.held = [len(self.pool.tables[i]) + e for i, e in enumerate(extra)]
        for i, e in enumerate(extra):
            self.pool.tables[i].extend(self.pool._take_fresh(e))
        self.tables = torch.tensor(self.pool.table_rows(range(n), width),
                                   dtype=torch.int32).view(n, width)
        self.free = list(self.pool.free_queue)


def plan_reference(st, new, head, max_tokens, front=()):
    """The plan's outputs from the pool's grow and slots; ``front`` are the
    queue entries before ``head``."""
    pool, n, bs = st.pool, len(st.lens), st.bs
    held, start, taken = list(st.held), [0], [0]
    slots, pos, seq = [], [], []
    for i, m in enumerate(new):
        before = len(pool.tables[i])
        # blocks held behind the length: grow takes what is missing
        need = pool.blocks_for(st.lens[i] + m)
        if need > before:
            pool.tables[i].extend(pool._take_fresh(need - before))
        pool.lengths[i] = st.lens[i] + m
        held[i] = len(pool.tables[i])
        slots += pool.slots(i, st.lens[i], m)
        pos += list(range(st.lens[i], st.lens[i] + m))
        seq += [i] * m
        start.append(start[-1] + m)
        taken.append(taken[-1] + held[i] - before)
    pad = [-1] * (max_tokens - len(slots))
    width = st.tables.shape[1]
    return dict(tables=pool.table_rows(range(n), width), seq_lens=[a + m for a, m in zip(st.lens, new)],
                blocks_held=held, free_head=[head + taken[-1]], query_start_loc=start,
                block_start=taken, slot_mapping=slots + pad, positions=pos + pad,
                seq_ids=seq + pad)
