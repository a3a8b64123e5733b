"""Plain 64-bit forms of pa_rope_write, pa_verify_tree, pa_release_blocks and
pa_fork_blocks, and random batches for their tests."""
import math
from fractions import Fraction

import numpy as np
import torch

from paged_kv_cache_109_gb300.block_pool import BlockPool
from tests._draft import random_parents

# 1 / (2 pi) to 60 digits
INV_TURN = Fraction(159154943091895335768883763372514362034459645740456448747667, 10 ** 60)


# ---- rope_write ------------------------------------------------------------------------

def axis_of_pair(half, sections, cyclic):
    if sections is None or len(sections) == 1:
        return [0] * half
    if not cyclic:
        return [a for a, m in enumerate(sections) for _ in range(m)]
    axes = len(sections)
    return [j % axes if j < axes * sections[j % axes] else 0 for j in range(half)]


def angles(positions, inv_freq, sections, cyclic):
    """[n, half] angles in (-pi, pi], whole turns taken off in exact arithmetic."""
    pos = positions.view(-1, positions.shape[-1]).tolist()
    inv = [Fraction(float(f)) * INV_TURN for f in inv_freq]
    axis = axis_of_pair(len(inv), sections, cyclic)
    out = torch.zeros(len(pos[0]), len(inv), dtype=torch.float64)
    for j, f in enumerate(inv):
        for t, p in enumerate(pos[axis[j]]):
            x = p * f
            x -= math.floor(x)
            out[t, j] = 2 * math.pi * float(x if x <= Fraction(1, 2) else x - 1)
    return out


def rope_reference(x, weight, eps, angle, neighbours, scale):
    """(rows, bound) of [n, heads, D] rows, in 64 bits.

    The kernel's sum of D squares is off by at most D 2^-24 of itself, the inverse
    root by half that and 2^-22 of its own; with the two products a normed value by
    (D / 2 + 8) 2^-24.  cos and sin: 2^-23 of the unit in their last place twice, the
    angle's conversion 2^-24 of at most pi / 4: 4 2^-24; two products and their sum
    3 2^-24, the factor on cos and sin another."""
    d, half = x.shape[-1], angle.shape[1]
    y = x.double()
    ey = 0.0
    if weight is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
        ey = (d / 2 + 8) * 2.0 ** -24
    out, bound = y.clone(), y.abs() * ey
    j = torch.arange(half)
    a, b = (2 * j, 2 * j + 1) if neighbours else (j, j + half)
    c, s = (scale * angle.cos())[:, None], (scale * angle.sin())[:, None]
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    size = abs(scale) * (y[..., a].abs() + y[..., b].abs()) * (ey + 8 * 2.0 ** -24)
    bound[..., a] = size
    bound[..., b] = size
    return out, bound


class RopeBatch:
    """Host tensors of one call; q, k and v are slices of one projection's rows."""

    def __init__(self, n, hq, hkv, d, bs, dtype, seed, rot=None, axes=1, sections=None,
                 cyclic=False, neighbours=False, norm=True, far=5000, scale=1.0, skip=(),
                 uncached=(), pad_row=0):
        g = torch.Generator().manual_seed(seed)
        rot = d if rot is None else rot
        self.args = dict(sections=sections, cyclic=cyclic, neighbours=neighbours, scale=scale,
                         eps=1e-5)
        width = (hq + 2 * hkv) * d + pad_row
        qkv = torch.randn(n, width, generator=g).to(dtype)
        self.qkv, self.cut = qkv, (hq * d, hkv * d, hkv * d)
        self.shape = (n, hq, hkv, d, bs)
        nb = -(-n // bs) + 3
        self.k_cache = torch.randn(nb, hkv, bs, d, generator=g).to(dtype)
        self.v_cache = torch.randn(nb, hkv, bs, d, generator=g).to(dtype)
        self.slots = torch.randperm(nb * bs, generator=g)[:n]
        self.slots[list(uncached)] = -1
        self.pos = torch.randint(0, far, (axes, n), generator=g).int()
        if skip:
            self.pos[0, list(skip)] = -1
        if axes == 1:
            self.pos = self.pos[0]
        self.inv = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float()
        self.qw = self.kw = None
        if norm:
            self.qw = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
            self.kw = (1 + 0.3 * torch.randn(d, generator=g)).to(dtype)
        self.out = torch.randn(n, hq, d, generator=g).to(dtype)

    def split(self, qkv):
        n, hq, hkv, d, _ = self.shape
        q, k, v = qkv[:, :sum(self.cut)].split(self.cut, 1)
        return q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d))

    def run(self, pa, dev, **kw):
        """(out, k_cache, v_cache) after the call, on the host."""
        q, k, v = self.split(self.qkv.to(dev))
        kc, vc, out = self.k_cache.to(dev), self.v_cache.to(dev), self.out.to(dev)
        move = lambda t: None if t is None else t.to(dev)
        got = pa.rope_write(q, k, v, self.pos.to(dev), self.inv.to(dev), self.slots.to(dev), kc, vc,
                            q_weight=move(self.qw), k_weight=move(self.kw), out=out, **self.args,
                            **kw)
        assert got is out
        return out.cpu(), kc.cpu(), vc.cpu()

    def check(self, out, kc, vc):
        n, hq, hkv, d, bs = self.shape
        q, k, v = self.split(self.qkv)
        a = self.args
        half = torch.finfo(self.out.dtype).eps / 2
        angle = angles(self.pos, self.inv, a["sections"], a["cyclic"])
        first = self.pos.view(-1, n)[0]
        want_k, want_v = self.k_cache.double(), self.v_cache.clone()
        bound_k = torch.zeros_like(want_k)
        ref, err = rope_reference(q, self.qw, a["eps"], angle, a["neighbours"], a["scale"])
        kref, kerr = rope_reference(k, self.kw, a["eps"], angle, a["neighbours"], a["scale"])
        for t in range(n):
            if first[t] < 0:
                assert torch.equal(out[t], self.out[t]), t
                continue
            tol = err[t] + half * (ref[t].abs() + err[t]) + 1e-37
            assert ((out[t].double() - ref[t]).abs() <= tol).all(), (
                t, float(((out[t].double() - ref[t]).abs() / tol).max()))
            s = int(self.slots[t])
            if 0 <= s < want_v.shape[0] * bs:
                want_k[s // bs, :, s % bs] = kref[t]
                bound_k[s // bs, :, s % bs] = kerr[t] + half * (kref[t].abs() + kerr[t]) + 1e-37
                want_v[s // bs, :, s % bs] = v[t]
        assert torch.equal(vc.view(torch.uint8), want_v.view(torch.uint8))
        assert ((kc.double() - want_k).abs() <= bound_k).all()


# ---- verify_tree -----------------------------------------------------------------------

class VerifyBatch:
    """Host tensors of one call: trees whose node 0 is the root."""

    def __init__(self, nodes, vocab, dtype, seed, kind="mixed", draft=True, temps=None, spread=2.0,
                 sure=0.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.nodes, self.vocab = list(nodes), vocab
        n = len(self.nodes)
        self.par = []
        for m in nodes:
            p = random_parents(rng, m, kind)
            self.par.append([-1 if j == 0 else (0 if x < 0 else x) for j, x in enumerate(p)])
        self.start = torch.tensor([0] + list(np.cumsum(nodes)), dtype=torch.int32)
        self.parents = torch.tensor([p for ps in self.par for p in ps], dtype=torch.int32)
        total = int(self.start[-1])
        x = spread * torch.randn(total, vocab, generator=g)
        self.logits = x.to(dtype)
        y = x + (1 - sure) * 0.7 * torch.randn(total, vocab, generator=g)
        self.draft = y.to(dtype) if draft else None
        self.temps = None if temps is None else torch.tensor(
            [temps[i % len(temps)] for i in range(n)], dtype=torch.float32)
        self.uniforms = torch.rand(total, generator=g)
        self.noise = torch.empty(n, vocab).exponential_(generator=g)
        self.tokens = torch.zeros(total, dtype=torch.int32)
        for i, ps in enumerate(self.par):
            heat = 1.0 if temps is None else max(float(self.temps[i]), 0.05)
            q0 = int(self.start[i])
            for j, p in enumerate(ps):
                if p >= 0:
                    e = torch.empty(vocab).exponential_(generator=g)
                    self.tokens[q0 + j] = int((y[q0 + p] / heat - e.log()).argmax())
        self.max_q = max(self.nodes, default=0)

    def run(self, pa, dev, **kw):
        move = lambda t: None if t is None else t.to(dev)
        leaf, token = pa.verify_tree(self.logits.to(dev), self.tokens.to(dev),
                                     self.parents.to(dev), self.start.to(dev),
                                     self.uniforms.to(dev), self.noise.to(dev), self.max_q,
                                     draft_logits=move(self.draft), temperature=move(self.temps),
                                     **kw)
        return leaf.cpu(), token.cpu()


def verify_reference(b):
    """Per sequence (leaf, token, close): by the definition in 64 bits.  close: a
    decision was nearer to its border than the kernel's roundings reach.  With
    logits whose distance from the largest is at most 64 (in powers of two of their
    weight) a weight is off by at most 64 2^-23 of itself, its exponential by 2^-22,
    the sums and products by less: 2^-16 covers them, of each term of a
    difference."""
    eps = 2.0 ** -16
    out = []
    for i, m in enumerate(b.nodes):
        if m == 0:
            out.append((-1, -1, False))
            continue
        q0, cur, close = int(b.start[i]), 0, False
        heat = 1.0 if b.temps is None else float(b.temps[i])
        while True:
            row = b.logits[q0 + cur].double()
            kids = [j for j in range(cur + 1, m) if b.par[i][j] == cur]
            if heat <= 0:
                best = int((row == row.max()).nonzero()[0, 0])
                took = [j for j in kids if int(b.tokens[q0 + j]) == best]
                if took:
                    cur = took[0]
                    continue
                out.append((cur, best, close))
                break
            p = torch.softmax(row / heat, 0)
            q = None if b.draft is None else torch.softmax(b.draft[q0 + cur].double() / heat, 0)
            left, size, c, share, took = p.clone(), p.clone(), 0.0, 1.0, -1
            for j in kids:
                t, u = int(b.tokens[q0 + j]), float(b.uniforms[q0 + j])
                if not 0 <= t < b.vocab:
                    continue
                ask = u * share * (1.0 if q is None else float(q[t]))
                # (weights that are zero, as of masked tokens, are so exactly)
                room = eps * (ask / max(share, 1e-300) + ask + float(size[t]))
                close |= room > 0 and abs(ask - float(left[t])) <= room
                if ask < float(left[t]):
                    took = j
                    break
                if q is None:
                    share -= float(left[t])
                    left[t] = size[t] = 0.0
                else:
                    c += share
                    left, size = (p - c * q).clamp(min=0), p + c * q
                    share = float(left.sum())
            if took >= 0:
                cur = took
                continue
            if not float(left.sum()) > 0:
                left = size = p
            e = b.noise[i].double()
            race, room = left / e, eps * size / e
            best = int(race.argmax())
            rival = race + room
            rival[best] = -1.0
            close |= float(rival.max()) >= float(race[best] - room[best])
            out.append((cur, best, close))
            break
    return out


def assert_verified(b, leaf, token, most_close=1):
    ref = verify_reference(b)
    near = 0
    for i, (x, t, close) in enumerate(ref):
        if close:
            near += 1
        else:
            assert (int(leaf[i]), int(token[i])) == (x, t), (i, int(leaf[i]), int(token[i]), x, t)
    assert near <= most_close, near
    return ref


# ---- release, fork -------------------------------------------------------------------------

class PoolState:
    """A BlockPool with sequences of ``lens`` tokens (``share``: (sequence, source,
    blocks) prefixes) as the device calls see it: rows, counts, and a queue of
    all blocks whose front is behind those in use."""

    def __init__(self, lens, bs, num_blocks, width, seed, share=(), spare=None):
        rng = np.random.default_rng(seed)
        self.pool = BlockPool(num_blocks, bs, rng.permutation(num_blocks).tolist())
        self.bs, self.num_blocks, self.width, self.lens = bs, num_blocks, width, list(lens)
        prefix = {i: (j, k) for i, j, k in share}
        for i, t in enumerate(lens):
            if i in prefix:
                j, k = prefix[i]
                self.pool.add(i, t, prefix_of=j, prefix_tokens=k * bs)
            else:
                self.pool.add(i, t)
        for i, e in enumerate(spare or []):
            self.pool.tables[i].extend(self.pool._take_fresh(e))
        n = len(self.lens)
        self.held = [len(self.pool.tables[i]) for i in range(n)]
        self.tables = torch.tensor(self.pool.table_rows(range(n), width),
                                   dtype=torch.int32).view(n, width)
        self.head = num_blocks - self.pool.num_free
        self.free = [-1] * self.head + list(self.pool.free_queue)

    def counts(self):
        return torch.tensor(self.pool.ref_cnt, dtype=torch.int32)


def i32(x, dev="cpu"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def release_reference(tables, held, keep, counts, free, head, num_blocks):
    """(blocks held, head) after; counts and free (lists) are updated.  A block's
    place is that of its last dropped entry."""
    drops = [int(tables[i][b]) for i in range(len(held)) for b in range(keep[i], held[i])]
    freed = []
    for at, b in enumerate(drops):
        if not 0 <= b < num_blocks:
            continue
        if counts is None:
            freed.append(b)
            continue
        counts[b] -= 1
        if counts[b] == 0:
            freed.append(b)
    head -= len(freed)
    free[head:head + len(freed)] = freed
    return [min(h, k) for h, k in zip(held, keep)], head
