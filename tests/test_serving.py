"""pa_rope_write, pa_verify_tree, pa_release_blocks and pa_fork_blocks on a GPU
against their plain 64-bit forms, at the sizes and values where they can go wrong,
and a serving loop of all of them."""
import math
import threading

import pytest
import torch

import paged_kv_cache_109_gb300 as pa
from tests._draft import path_of
from tests._serving import (PoolState, RopeBatch, VerifyBatch, assert_verified, i32,
                            release_reference, verify_reference)

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def clear_device_error(cuda_device):
    pa.last_device_error()
    yield


# ---- rope_write ------------------------------------------------------------------------

# tokens, query heads, kv heads, head dim, block size, dtype, what else
ROPE = [
    (1, 4, 1, 128, 16, BF, {}),
    (1, 32, 8, 128, 16, F32, dict(norm=False)),
    (7, 8, 8, 64, 8, BF, dict(neighbours=True)),
    (7, 6, 2, 96, 24, BF, dict(rot=48)),
    (5, 6, 3, 80, 5, F32, dict(rot=48, neighbours=True)),
    (5, 2, 1, 256, 16, BF, dict(rot=64)),
    (3, 2, 1, 256, 16, F32, dict(axes=3, sections=(32, 48, 48))),
    (9, 4, 2, 112, 16, BF, dict(axes=2, sections=(20, 36))),
    (9, 5, 1, 48, 16, F32, dict(axes=3, sections=(8, 8, 8), cyclic=True)),
    (9, 4, 4, 16, 4, BF, dict(axes=3, sections=(6, 1, 1), cyclic=True, neighbours=True)),
    (9, 4, 4, 16, 4, BF, dict(axes=3, sections=(0, 8, 0))),
    (6, 3, 1, 7, 3, F32, dict(rot=6)), (6, 3, 1, 7, 3, BF, dict(rot=4, neighbours=True)),
    (6, 3, 1, 255, 3, F32, dict(rot=254)), (6, 3, 1, 250, 3, BF, dict(rot=2)),
    (4, 3, 3, 1, 4, F32, dict(rot=0)), (4, 3, 3, 1, 4, BF, dict(rot=0)),
    (4, 2, 2, 36, 4, BF, dict(rot=20)), (4, 2, 2, 36, 4, F32, dict(rot=20)),
    (4, 2, 2, 36, 4, BF, dict(rot=18, neighbours=True)),
    (4, 8, 2, 128, 16, BF, dict(scale=1.3)), (4, 8, 2, 128, 16, BF, dict(scale=-0.5)),
    (33, 8, 2, 128, 16, BF, dict(skip=(0, 5, 32), uncached=(1, 5, 9))),
    (33, 8, 2, 128, 16, BF, dict(pad_row=1)), (33, 8, 2, 128, 16, BF, dict(pad_row=4)),
    (33, 8, 2, 128, 16, F32, dict(pad_row=2)), (33, 8, 2, 128, 16, F32, dict(pad_row=7)),
    (1025, 4, 1, 64, 16, BF, dict(skip=(1020, 1021, 1022, 1023, 1024))),
    (1027, 3, 1, 40, 16, F32, dict(axes=2, sections=(10, 10), uncached=(1026,))),
    (300, 1, 1, 128, 128, BF, {}), (40, 128, 1, 128, 16, BF, {}),
    (20, 4, 1, 128, 16, F32, dict(far=2 ** 31 - 1)), (20, 4, 1, 128, 16, BF, dict(far=10 ** 6)),
]


@pytest.mark.parametrize("n,hq,hkv,d,bs,dtype,kw", ROPE)
def test_rope_write(cuda_device, n, hq, hkv, d, bs, dtype, kw):
    b = RopeBatch(n, hq, hkv, d, bs, dtype, seed=n + d, **kw)
    b.check(*b.run(pa, cuda_device))
    assert pa.last_device_error() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_without_norm_and_rotation_it_is_the_cache_write(cuda_device, dtype):
    b = RopeBatch(50, 4, 2, 96, 16, dtype, seed=1, rot=0, norm=False, uncached=(3, 4))
    b.qkv[7] = float("inf")
    b.qkv[8, 5] = 1e-40
    out, kc, vc = b.run(pa, cuda_device)
    q, k, v = b.split(b.qkv)
    kd, vd = b.k_cache.to(cuda_device), b.v_cache.to(cuda_device)
    pa.write_kv(k.contiguous().to(cuda_device), v.contiguous().to(cuda_device),
                b.slots.to(cuda_device), kd, vd)
    assert torch.equal(out, q) and torch.equal(kc, kd.cpu()) and torch.equal(vc, vd.cpu())


def test_rope_largest_and_smallest_values(cuda_device):
    """Rows of zeros, of tiny and of large values: the norm's own range in 32 bits."""
    b = RopeBatch(4, 2, 1, 64, 8, F32, seed=2)
    b.qkv[0] = 0.0
    b.qkv[1] *= 1e-15
    b.qkv[2] *= 1e15
    b.check(*b.run(pa, cuda_device))
    b.qkv[3] = float("nan")
    out, kc, vc = b.run(pa, cuda_device)
    assert torch.isnan(out[3]).all() and torch.isfinite(out[:3]).all()


def test_rope_in_place_and_apart(cuda_device):
    b = RopeBatch(70, 8, 2, 128, 16, BF, seed=3, skip=(4,))
    q, k, v = (x.contiguous().to(cuda_device) for x in b.split(b.qkv))
    kc, vc = b.k_cache.to(cuda_device), b.v_cache.to(cuda_device)
    move = lambda t: t.to(cuda_device)
    args = (move(b.pos), move(b.inv), move(b.slots))
    kw = dict(q_weight=move(b.qw), k_weight=move(b.kw), **b.args)
    want = pa.rope_write(q, k, v, *args, kc.clone(), vc.clone(), out=q.clone(), **kw)
    got = pa.rope_write(q, k, v, *args, kc, vc, out=q, **kw)
    assert got is q and torch.equal(got.view(torch.int16), want.view(torch.int16))
    b.out = b.split(b.qkv)[0].contiguous()
    b.check(got.cpu(), kc.cpu(), vc.cpu())


def test_rope_slots_past_the_pool_and_bad_frequencies(cuda_device):
    b = RopeBatch(20, 4, 2, 64, 8, BF, seed=4)
    b.slots[3], b.slots[9] = b.k_cache.shape[0] * 8, 2 ** 40
    out, kc, vc = b.run(pa, cuda_device)
    assert pa.last_device_error() == pa.DEVERR_SLOT
    b.check(out, kc, vc)
    b = RopeBatch(20, 4, 2, 64, 8, F32, seed=4)
    b.inv[5], b.inv[6], b.inv[7] = math.inf, math.nan, 2.0 ** 32
    out, _, _ = b.run(pa, cuda_device)
    bad = torch.isnan(out).all(0).all(0)
    assert bad.nonzero()[:, 0].tolist() == [5, 6, 7, 37, 38, 39]
    assert torch.isfinite(out[..., ~bad]).all()


def test_rope_frequencies_of_every_size(cuda_device):
    """Tiny, large and negative frequencies at near and far positions."""
    b = RopeBatch(12, 1, 1, 64, 8, F32, seed=5, norm=False, far=2 ** 31 - 1)
    e = torch.linspace(-140, 31, 32)
    b.inv = (torch.pow(2.0, e.double()) * (1 + 0.37)).float() * torch.tensor([1.0, -1.0]).repeat(16)
    b.inv[0] = 0.0
    b.pos[:4] = torch.tensor([0, 1, 2, 2 ** 31 - 1], dtype=torch.int32)
    b.check(*b.run(pa, cuda_device))


def test_rope_pinned_arguments_and_another_stream(cuda_device):
    b = RopeBatch(37, 8, 2, 128, 16, BF, seed=6, axes=2, sections=(40, 24))
    want = b.run(pa, cuda_device)
    q, k, v = (x.contiguous().pin_memory() for x in b.split(b.qkv))
    kc, vc = b.k_cache.to(cuda_device), b.v_cache.to(cuda_device)
    pin = lambda t: t.pin_memory()
    out = b.out.clone().pin_memory()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pa.rope_write(q, k, v, pin(b.pos), pin(b.inv), pin(b.slots), kc, vc, q_weight=pin(b.qw),
                  k_weight=pin(b.kw), out=out, stream=s, **b.args)
    s.synchronize()
    for x, y in zip((out, kc.cpu(), vc.cpu()), want):
        assert torch.equal(x, y)


def test_rope_refusals(cuda_device):
    b = RopeBatch(4, 4, 2, 64, 8, BF, seed=7)
    q, k, v = (x.to(cuda_device) for x in b.split(b.qkv))
    kc, vc = b.k_cache.to(cuda_device), b.v_cache.to(cuda_device)
    pos, inv, slots = b.pos.to(cuda_device), b.inv.to(cuda_device), b.slots.to(cuda_device)
    run = lambda q=q, k=k, v=v, pos=pos, inv=inv, slots=slots, **kw: pa.rope_write(
        q, k, v, pos, inv, slots, kc, vc, **kw)
    for kw in (dict(q=q.float()), dict(k=k[:3]), dict(v=v[:, :1]), dict(q=q.transpose(0, 1)),
               dict(q=q[..., ::2]), dict(pos=pos.long()), dict(pos=pos[:3]), dict(slots=slots.int()),
               dict(inv=inv.double()), dict(sections=(8, 8, 8, 8)), dict(sections=(16, 16)),
               dict(q_weight=torch.ones(64, device=cuda_device)),
               dict(q_weight=torch.ones(32, device=cuda_device, dtype=BF)),
               dict(out=torch.empty(4, 4, 64, device=cuda_device)),
               dict(pos=pos.repeat(2).view(4, 2), sections=(16, 16))):
        with pytest.raises(ValueError):
            run(**kw)
    for kw in (dict(inv=torch.ones(33, device=cuda_device)), dict(eps=-1.0), dict(scale=math.inf),
               dict(pos=pos.repeat(2).view(2, 4), sections=(16, 15)),
               dict(out=kc.view(-1)[:4 * 4 * 64].view(4, 4, 64)),
               dict(slots=b.slots)):                    # pageable memory
        with pytest.raises(pa.PaError):
            run(**kw)


# ---- verify_tree -----------------------------------------------------------------------

# nodes, vocabulary, dtype, kind, draft, temperatures
VERIFY = [
    ([1], 50, F32, "chain", True, None), ([1, 1, 1], 4099, BF, "chain", False, [0.5, 1.0, 0.0]),
    ([6], 32000, BF, "chain", True, None), ([6], 32000, F32, "chain", False, [0.8]),
    ([3, 0, 5, 1, 8], 1000, F32, "chain", True, [1.0, 0.7]),
    ([0, 0], 64, F32, "chain", True, None),
    ([9, 4, 17, 2, 31, 1], 2003, F32, "mixed", True, [1.0, 0.0, 0.6]),
    ([9, 4, 17, 2, 31, 1], 2003, F32, "mixed", False, [1.0, 0.0, 0.6]),
    ([9, 4, 17, 2, 31, 1], 8192, BF, "mixed", True, None),
    ([9, 4, 17, 2, 31, 1], 8200, BF, "mixed", False, None),
    ([64, 40], 500, F32, "star", True, None), ([64, 40], 500, F32, "star", False, None),
    ([256, 200], 300, F32, "mixed", True, None), ([256], 300, F32, "chain", True, None),
    ([5] * 40, 5000, F32, "mixed", True, [0.9]), ([5] * 400, 333, F32, "mixed", True, None),
    ([4, 3], 1, F32, "mixed", True, None), ([4, 3], 2, F32, "mixed", False, None),
    ([4, 3], 7, BF, "mixed", True, [1.5]), ([3, 3], 100003, F32, "chain", True, None),
    ([2, 5, 3], 131072, BF, "mixed", True, None), ([2, 5, 3], 131075, BF, "mixed", True, None),
    ([4] * 20, 4096, F32, "mixed", True, [0.01, 100.0, -1.0]),
]


@pytest.mark.parametrize("nodes,vocab,dtype,kind,draft,temps", VERIFY)
def test_verify_tree(cuda_device, nodes, vocab, dtype, kind, draft, temps):
    for seed in (0, 1, 2):
        b = VerifyBatch(nodes, vocab, dtype, seed, kind=kind, draft=draft, temps=temps)
        leaf, token = b.run(pa, cuda_device)
        assert pa.last_device_error() == 0
        assert_verified(b, leaf, token, most_close=1 + len(nodes) // 100)


@pytest.mark.parametrize("draft", [True, False])
def test_close_drafts_hold_deep(cuda_device, draft):
    """A draft equal to the target holds whole chains; its rest after a failure is
    empty, so the sequences end in the plain rows."""
    b = VerifyBatch([12] * 16, 700, F32, seed=3, kind="chain", draft=draft, sure=1.0)
    leaf, token = b.run(pa, cuda_device)
    ref = assert_verified(b, leaf, token)
    if draft:
        assert all(x == 11 for x, _, _ in ref)


def test_masks_and_edges_of_the_logits(cuda_device):
    """-inf and the type's lowest value as masks, a single token left, equal
    largest logits."""
    for dtype in (F32, BF):
        low = torch.finfo(dtype).min
        for mask in (-math.inf, low):
            b = VerifyBatch([7, 5, 4, 6, 1], 900, dtype, seed=4, temps=[1.0, 0.8, 0.0])
            g = torch.Generator().manual_seed(9)
            hide = torch.rand(b.logits.shape, generator=g) < 0.6
            hide[:, 5] = False
            b.logits[hide] = mask
            b.draft[hide] = mask
            b.logits[0, 6:] = mask                  # few tokens left
            b.logits[0, :5] = mask
            leaf, token = b.run(pa, cuda_device)
            assert pa.last_device_error() == 0
            assert_verified(b, leaf, token)
        # one row all at the lowest value: every token alike
        b = VerifyBatch([1, 2], 40, dtype, seed=5)
        b.logits[:] = low
        leaf, token = b.run(pa, cuda_device)
        assert_verified(b, leaf, token)
        # greedy ties: the lowest index
        b = VerifyBatch([1, 1], 70000, dtype, seed=6, temps=[0.0])
        b.logits[:] = 0.0
        b.logits[0, [33333, 44444, 69999]] = 1.0
        leaf, token = b.run(pa, cuda_device)
        assert token.tolist() == [33333, 0]


@pytest.mark.parametrize("temps", [None, [0.0]])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows_that_give_no_token(cuda_device, dtype, temps):
    for bad, hit in ((math.nan, 17), (math.inf, 899), (-math.inf, slice(None))):
        b = VerifyBatch([3, 3, 3], 900, dtype, seed=7, kind="chain", temps=temps)
        clean = b.run(pa, cuda_device)
        b.logits[3, hit] = bad                      # the second sequence's root
        leaf, token = b.run(pa, cuda_device)
        assert pa.last_device_error() == pa.DEVERR_LOGITS
        assert leaf.tolist() == [int(clean[0][0]), -1, int(clean[0][2])]
        assert token.tolist() == [int(clean[1][0]), -1, int(clean[1][2])]
        # rows that the walk does not reach may hold anything
        b = VerifyBatch([2, 2], 900, dtype, seed=8, kind="chain", temps=temps)
        b.tokens[[1, 3]] = 0
        b.logits[[0, 2], 0] = -20.0
        b.logits[[1, 3], hit] = bad
        leaf, token = b.run(pa, cuda_device)
        assert leaf.tolist() == [0, 0] and pa.last_device_error() == 0


def test_bad_draft_rows_and_temperatures(cuda_device):
    for bad in (math.nan, math.inf):
        b = VerifyBatch([3, 1], 300, F32, seed=9, kind="chain")
        b.draft[0, 5] = bad
        b.draft[3] = bad                            # a leaf's: not read
        leaf, token = b.run(pa, cuda_device)
        assert pa.last_device_error() == pa.DEVERR_LOGITS
        assert leaf.tolist() == [-1, 0] and token[0] == -1
    heats = [math.nan, math.inf, 1e-39, 1e-44, 1.0, -math.inf]
    b = VerifyBatch([2] * 6, 300, F32, seed=9, temps=[1.0])
    b.temps = torch.tensor(heats)
    leaf, token = b.run(pa, cuda_device)
    assert pa.last_device_error() == pa.DEVERR_LOGITS
    assert [int(x) for x in leaf[:4]] == [-1] * 4
    ref = verify_reference(_only(b, [4, 5]))
    assert [(int(leaf[i]), int(token[i])) for i in (4, 5)] == [r[:2] for r in ref]


def _only(b, keep):
    """The batch of some of b's sequences."""
    c = VerifyBatch([b.nodes[i] for i in keep], b.vocab, b.logits.dtype, seed=0,
                    draft=b.draft is not None)
    rows = torch.cat([torch.arange(int(b.start[i]), int(b.start[i + 1])) for i in keep]).long()
    c.par = [b.par[i] for i in keep]
    c.parents, c.tokens, c.uniforms = b.parents[rows], b.tokens[rows], b.uniforms[rows]
    c.logits, c.noise = b.logits[rows], b.noise[keep]
    c.draft = None if b.draft is None else b.draft[rows]
    c.temps = None if b.temps is None else b.temps[keep]
    return c


def test_bad_trees(cuda_device):
    b = VerifyBatch([4, 3, 5, 2], 200, F32, seed=10, kind="chain")
    clean = b.run(pa, cuda_device)
    # rows out of range: that sequence only
    start = b.start.clone()
    start[4] = 1000
    b.start = start
    leaf, token = b.run(pa, cuda_device)
    assert pa.last_device_error() == pa.DEVERR_SEQ_LEN
    assert leaf.tolist() == clean[0].tolist()[:3] + [-1]
    # more nodes than the bound
    b = VerifyBatch([4, 3, 5, 2], 200, F32, seed=10, kind="chain")
    b.max_q = 4
    leaf, token = b.run(pa, cuda_device)
    assert pa.last_device_error() == pa.DEVERR_SEQ_LEN and int(leaf[2]) == int(token[2]) == -1
    assert leaf[[0, 1, 3]].tolist() == clean[0][[0, 1, 3]].tolist()
    # starts that descend
    b.max_q = 5
    b.start = i32([0, 4, 2, 12, 14])
    b.run(pa, cuda_device)
    assert pa.last_device_error() == pa.DEVERR_SEQ_LEN
    # a parent out of range is read as -1: the node is never reached
    b = VerifyBatch([4, 3], 200, F32, seed=11, kind="chain")
    b.parents[1], b.par[0] = 7, [-1, -1, 1, 2]
    b.parents[4], b.par[1] = 0, [-1, 0, 1]          # node 0's too
    leaf, token = b.run(pa, cuda_device)
    assert pa.last_device_error() == pa.DEVERR_TREE and int(leaf[0]) == 0
    assert_verified(b, leaf, token)
    # tokens outside the vocabulary are passed over
    for draft in (True, False):
        b = VerifyBatch([4, 4], 200, F32, seed=12, kind="star", draft=draft)
        b.tokens[1], b.tokens[6] = 200, -1
        leaf, token = b.run(pa, cuda_device)
        assert pa.last_device_error() == pa.DEVERR_TREE
        assert_verified(b, leaf, token)


def test_noise_at_its_edges(cuda_device):
    """Zeros win (the lowest index first); noise that leaves nothing is refused."""
    b = VerifyBatch([1] * 4, 5000, F32, seed=13)
    b.noise[0, [100, 4999]] = 0.0
    b.noise[1, :] = math.inf
    b.noise[2, :] = math.nan
    b.noise[3, 77] = math.nan
    leaf, token = b.run(pa, cuda_device)
    assert pa.last_device_error() == pa.DEVERR_LOGITS
    assert int(token[0]) == 100 and token[1:3].tolist() == [-1, -1] and leaf[1:3].tolist() == [-1, -1]
    b.noise[3, 77] = 1e30
    assert int(token[3]) == verify_reference(_only(b, [3]))[0][1]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("vocab,a,b", [(40, 5, 6), (3001, 8, 2900), (131072, 100, 131071),
                                       (131072, 70000, 70001), (100003, 50000, 99999)])
def test_near_ties_of_the_next_token(cuda_device, dtype, vocab, a, b):
    """Two tokens of one weight whose noise is equal, or differs in its last bits:
    the lower index, or the smaller noise."""
    for child in (False, True):
        c = VerifyBatch([1 + child] * 3, vocab, dtype, seed=18, kind="chain", spread=0.1)
        row = c.start[:-1].long()
        c.logits[row] = c.logits[row].clamp(max=0.5)
        c.logits[row[:, None], torch.tensor([a, b])] = 8.0
        c.noise[:, [a, b]] = 1e-3
        c.noise[1, b] = torch.nextafter(torch.tensor(1e-3), torch.tensor(0.0))
        c.noise[2, a] = torch.nextafter(torch.tensor(1e-3), torch.tensor(0.0))
        if child:
            # a draft that leaves both tokens their weights: it fails on another one
            c.draft[row] = -20.0
            c.draft[row, 20] = 8.0
            c.logits[row, 20] = -30.0
            c.tokens[row + 1], c.uniforms[row + 1] = 20, 0.9
        leaf, token = c.run(pa, cuda_device)
        p = torch.softmax(c.logits[row].double(), 1)
        if child:
            p = (p - torch.softmax(c.draft[row].double(), 1)).clamp(min=0)
        race = p / c.noise.double()
        first = [int((r == r.max()).nonzero()[0, 0]) for r in race]
        # (of 131072 tokens a third one may have noise small enough to win)
        assert sum(x == y for x, y in zip(first, (a, b, a))) >= 2
        assert leaf.tolist() == [0] * 3 and token.tolist() == first, child


@pytest.mark.parametrize("vocab", [50, 4100, 131072])
def test_a_rest_that_rounding_leaves_empty(cuda_device, vocab):
    """A draft equal to the target, all tries failed (uniforms of one): nothing is
    left of P, and the next token is drawn from P itself."""
    for dtype in (F32, BF):
        b = VerifyBatch([3, 4], vocab, dtype, seed=19, kind="star", sure=1.0)
        b.draft = b.logits.clone()
        b.uniforms[:] = 1.0
        leaf, token = b.run(pa, cuda_device)
        p = torch.softmax(b.logits[b.start[:-1].long()].double(), 1)
        assert leaf.tolist() == [0, 0] and token.tolist() == (p / b.noise.double()).argmax(1).tolist()


@pytest.mark.parametrize("draft", [True, False])
def test_tokens_are_distributed_as_the_targets(cuda_device, draft):
    """The first token behind the root over 40000 sequences, within five standard
    deviations of the target's probabilities."""
    vocab, reps = 12, 40000
    g = torch.Generator(device="cuda").manual_seed(3)
    row, drow = (torch.randn(vocab, device="cuda", generator=g) for _ in range(2))
    q = torch.softmax(drow.double(), 0)
    tokens = (torch.multinomial(q, 4 * reps, replacement=True, generator=g).int() if draft
              else i32([0, 3, 1, 3], "cuda").repeat(reps))
    logits = row.repeat(4 * reps, 1)
    par = i32([-1, 0, 0, 0], "cuda").repeat(reps)
    start = torch.arange(0, 4 * reps + 1, 4, device="cuda", dtype=torch.int32)
    leaf, token = pa.verify_tree(
        logits, tokens, par, start, torch.rand(4 * reps, device="cuda", generator=g),
        torch.empty(reps, vocab, device="cuda").exponential_(generator=g), 4,
        draft_logits=drow.repeat(4 * reps, 1) if draft else None)
    first = torch.where(leaf > 0, tokens[(start[:-1] + leaf).long()], token).long()
    count = torch.bincount(first, minlength=vocab).double().cpu()
    p = torch.softmax(row.double(), 0).cpu()
    assert ((count - reps * p).abs() <= 5 * (reps * p * (1 - p)).sqrt()).all(), (count / reps, p)
    assert 0.2 < float((leaf > 0).double().mean()) < 0.99


def test_logits_in_wider_rows_and_off_alignment(cuda_device):
    b = VerifyBatch([5, 9, 2], 5008, BF, seed=14)
    want = b.run(pa, cuda_device)
    total = b.logits.shape[0]
    dev = lambda t: t.to(cuda_device)
    for extra, off in ((8, 0), (8, 8), (3, 1), (5, 2)):
        wide, dwide = (torch.full((total, 5008 + extra + off), float("nan"), dtype=BF,
                                  device=cuda_device) for _ in range(2))
        nwide = torch.full((3, 5008 + extra + off), float("nan"), device=cuda_device)
        wide[:, off:off + 5008], dwide[:, off:off + 5008] = dev(b.logits), dev(b.draft)
        nwide[:, off:off + 5008] = dev(b.noise)
        cut = slice(off, off + 5008)
        got = pa.verify_tree(wide[:, cut], dev(b.tokens), dev(b.parents), dev(b.start),
                             dev(b.uniforms), nwide[:, cut], b.max_q, draft_logits=dwide[:, cut])
        assert [x.tolist() for x in got] == [x.tolist() for x in want], (extra, off)
    assert_verified(b, *want)


def test_verify_pinned_arguments_streams_and_replay(cuda_device):
    b = VerifyBatch([5, 9, 2, 14], 6000, F32, seed=15, temps=[1.0, 0.0])
    c = VerifyBatch([5, 9, 2, 14], 6000, F32, seed=16, temps=[0.7, 1.0])
    want, want_c = b.run(pa, cuda_device), c.run(pa, cuda_device)
    pin = lambda t: t.pin_memory()
    leaf, token = torch.empty(4, dtype=torch.int32).pin_memory(), torch.empty(4, dtype=torch.int32).pin_memory()
    pa.verify_tree(b.logits.to(cuda_device), pin(b.tokens), pin(b.parents), pin(b.start),
                   pin(b.uniforms), pin(b.noise), b.max_q, draft_logits=pin(b.draft),
                   temperature=pin(b.temps), leaf=leaf, next_tokens=token)
    torch.cuda.synchronize()
    assert torch.equal(leaf, want[0]) and torch.equal(token, want[1])
    # two streams at once
    names = ("logits", "tokens", "parents", "start", "uniforms", "noise", "draft", "temps")
    put = lambda x: [getattr(x, k).to(cuda_device) for k in names]
    call = lambda t, x, **kw: pa.verify_tree(*t[:6], x.max_q, draft_logits=t[6], temperature=t[7], **kw)
    tb, tc = put(b), put(c)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append((call(tb, b, stream=s1), call(tc, c, stream=s2)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0].cpu(), want[0]) and torch.equal(y[1].cpu(), want_c[1])
    # captured, replayed on other values
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        leaf, token = call(tb, b)
    for t, src in zip(tb, tc):
        if t.shape == src.shape:
            t.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(leaf.cpu(), want_c[0]) and torch.equal(token.cpu(), want_c[1])


def test_verify_refusals(cuda_device):
    b = VerifyBatch([3, 2], 64, F32, seed=17)
    names = ("logits", "tokens", "parents", "start", "uniforms", "noise")
    good = {k: getattr(b, k).to(cuda_device) for k in names}
    draft = b.draft.to(cuda_device)

    def run(draft_logits=draft, max_q=3, **kw):
        t = {**good, **kw}
        temps = t.pop("temperature", None)
        leaf, token = t.pop("leaf", None), t.pop("next_tokens", None)
        return pa.verify_tree(*t.values(), max_q, draft_logits=draft_logits, temperature=temps,
                              leaf=leaf, next_tokens=token)
    for kw in (dict(logits=good["logits"].half()), dict(logits=good["logits"][0]),
               dict(logits=good["logits"].T), dict(draft_logits=draft.bfloat16()),
               dict(draft_logits=draft[:4]), dict(tokens=good["tokens"].long()),
               dict(parents=good["parents"][:4]), dict(uniforms=good["uniforms"].double()),
               dict(noise=good["noise"][:1]), dict(noise=good["noise"].bfloat16()),
               dict(temperature=torch.ones(3, device=cuda_device)),
               dict(temperature=torch.ones(2, device=cuda_device, dtype=torch.float64)),
               dict(leaf=torch.empty(3, device=cuda_device, dtype=torch.int32)),
               dict(next_tokens=torch.empty(2, device=cuda_device))):
        with pytest.raises(ValueError):
            run(**kw)
    for kw in (dict(max_q=257), dict(max_q=-1), dict(leaf=good["start"][:2]),
               dict(tokens=b.tokens)):
        with pytest.raises(pa.PaError):
            run(**kw)


# ---- release, fork -------------------------------------------------------------------------

RELEASE = [
    # tokens, shared prefixes (row, source, blocks), spare blocks, tokens kept, block size
    ([9], [], [0], [0], 4), ([9], [], [2], [9], 4), ([0, 0], [], [0, 3], [0, 0], 4),
    ([9, 6, 12, 3], [(2, 0, 2)], [0, 2, 0, 1], [0, 6, 0, 3], 4),
    ([9, 6, 12, 3], [(2, 0, 2)], [0, 2, 0, 1], [0, 2, 12, 1], 4),
    ([9, 9, 9, 9], [(1, 0, 2), (2, 0, 2), (3, 1, 1)], None, [0, 0, 0, 0], 4),
    ([9, 9, 9, 9], [(1, 0, 2), (2, 0, 2), (3, 1, 1)], None, [9, 0, 8, 0], 4),
    ([4000, 17, 900, 2500], [(1, 0, 1), (3, 0, 200)], None, [0, 17, 0, 0], 8),
    ([7] * 300, [(i, i - 1, 1) for i in range(1, 300, 3)], None, [0, 7, 3] * 100, 3),
]


@pytest.mark.parametrize("lens,share,spare,keep,bs", RELEASE)
@pytest.mark.parametrize("counted", [True, False])
@pytest.mark.parametrize("in_place", [False, True])
def test_release(cuda_device, lens, share, spare, keep, bs, counted, in_place):
    share = share if counted else []
    nb = sum(-(-t // bs) + 4 for t in lens) + 5
    st = PoolState(lens, bs, nb, max(-(-t // bs) for t in lens) + 5, seed=1, share=share, spare=spare)
    blocks = [-(-t // bs) for t in keep]
    counts, free = (list(st.pool.ref_cnt) if counted else None), list(st.free)
    held, head = release_reference(st.tables, st.held, blocks, counts, free, st.head, nb)
    dev = lambda x: i32(x, cuda_device)
    tables, free_d, held_d, head_d = st.tables.to(cuda_device), dev(st.free), dev(st.held), dev([st.head])
    ref = st.counts().to(cuda_device) if counted else None
    got = pa.release_blocks(dev(keep), tables, held_d, free_d, head_d, nb, bs, ref_cnt=ref,
                            blocks_held_out=held_d if in_place else None,
                            free_head_out=head_d if in_place else None)
    assert pa.last_device_error() == 0
    assert got[0].tolist() == held and got[1].tolist() == [head]
    assert free_d.tolist() == free and torch.equal(tables.cpu(), st.tables)
    if counted:
        assert ref.tolist() == counts
    if not in_place:
        assert held_d.tolist() == st.held and head_d.tolist() == [st.head]


@pytest.mark.parametrize("counted", [True, False])
def test_release_of_many_sequences(cuda_device, counted):
    """More sequences than one round, some with many blocks."""
    g = torch.Generator().manual_seed(2)
    n, bs = 9001, 4
    lens = torch.randint(0, 30, (n,), generator=g).tolist()
    lens[4500], lens[9000], lens[4095] = 9000, 5000, 7000
    share = [(i, i - 1, min(lens[i], lens[i - 1]) // bs) for i in range(5000, 5400)] if counted else []
    nb = sum(-(-t // bs) for t in lens) + 9
    st = PoolState(lens, bs, nb, 9000 // bs + 1, seed=2, share=share)
    keep = [t if i % 5 else 0 for i, t in enumerate(lens)]
    keep[4500] = keep[9000] = keep[4095] = 0
    counts, free = (list(st.pool.ref_cnt) if counted else None), list(st.free)
    held, head = release_reference(st.tables, st.held, [-(-t // bs) for t in keep], counts, free,
                                   st.head, nb)
    free_d = i32(st.free, cuda_device)
    ref = st.counts().to(cuda_device) if counted else None
    got = pa.release_blocks(i32(keep, cuda_device), st.tables.to(cuda_device),
                            i32(st.held, cuda_device), free_d, i32([st.head], cuda_device), nb, bs,
                            ref_cnt=ref)
    assert pa.last_device_error() == 0
    assert got[0].tolist() == held and got[1].tolist() == [head] and free_d.tolist() == free
    if counted:
        assert ref.tolist() == counts


@pytest.mark.parametrize("counted", [True, False])
def test_release_refuses_as_a_whole(cuda_device, counted):
    st = PoolState([9, 6, 12], 4, 20, 6, seed=3, share=[(2, 0, 2)] if counted else [])
    dev = lambda x: i32(x, cuda_device)

    def run(keep=(0, 6, 0), held=None, head=None, free=None, counts=None, tables=None):
        held = st.held if held is None else held
        head = st.head if head is None else head
        free_d = dev(st.free if free is None else free)
        ref = dev(counts or st.pool.ref_cnt) if counted else None
        before = free_d.clone(), None if ref is None else ref.clone()
        got = pa.release_blocks(dev(list(keep)), (st.tables if tables is None else tables).to(cuda_device),
                                dev(held), free_d, dev([head]), 20, 4, ref_cnt=ref)
        err = pa.last_device_error()
        kept = torch.equal(free_d, before[0]) and (ref is None or torch.equal(ref, before[1]))
        return got[0].tolist() == list(held) and got[1].tolist() == [head] and kept, err
    for kw, bit in ((dict(keep=(-1, 6, 0)), pa.DEVERR_SEQ_LEN), (dict(keep=(0, 9, 0)), pa.DEVERR_SEQ_LEN),
                    (dict(held=[3, 7, 3], keep=(0, 30, 0)), pa.DEVERR_SEQ_LEN),
                    (dict(held=[3, -2, 3]), pa.DEVERR_SEQ_LEN), (dict(held=[3, 2, 7]), pa.DEVERR_SEQ_LEN),
                    (dict(head=2), pa.DEVERR_POOL), (dict(head=0), pa.DEVERR_POOL),
                    (dict(head=-3), pa.DEVERR_POOL), (dict(head=21), pa.DEVERR_POOL)):
        same, err = run(**kw)
        assert same and err == bit, kw
    if counted:
        # a count that would drop below zero: one row's block has none left
        counts = list(st.pool.ref_cnt)
        counts[int(st.tables[0, 2])] = 0
        assert run(counts=counts) == (True, pa.DEVERR_SHARED)
        counts = list(st.pool.ref_cnt)
        counts[int(st.tables[0, 0])] = 1                # two rows drop it
        assert run(counts=counts) == (True, pa.DEVERR_SHARED)


def test_release_passes_over_bad_entries(cuda_device):
    st = PoolState([12, 12], 4, 20, 4, seed=4)
    st.tables[0, 1], st.tables[1, 2] = -1, 20
    free = list(st.free)
    counts = list(st.pool.ref_cnt)
    held, head = release_reference(st.tables, st.held, [0, 0], counts, free, st.head, 20)
    for ref in (None, st.counts().to(cuda_device)):
        free_d = i32(st.free, cuda_device)
        got = pa.release_blocks(i32([0, 0], cuda_device), st.tables.to(cuda_device),
                                i32(st.held, cuda_device), free_d, i32([st.head], cuda_device), 20, 4,
                                ref_cnt=ref)
        assert pa.last_device_error() == pa.DEVERR_TABLE_ENTRY
        assert got[1].tolist() == [head] and free_d.tolist() == free and held == got[0].tolist()


def _fork_reference(st, src, k, v):
    """After the fork, on the host: the pool's fork and copy_on_write, row by row."""
    bs, tables, counts = st.bs, st.tables.clone(), st.counts()
    head, lens, held, pairs = st.head, list(st.lens), list(st.held), []
    for i, p in enumerate(src):
        pairs.append([-1, -1])
        if p < 0:
            continue
        t = st.lens[p]
        lens[i], held[i] = t, -(-t // bs)
        for b in range(t // bs):
            tables[i, b] = st.tables[p, b]
            counts[int(tables[i, b])] += 1
        if t % bs:
            old, new = int(st.tables[p, t // bs]), st.free[head]
            head += 1
            tables[i, t // bs], counts[new], pairs[-1] = new, 1, [old, new]
            for c in (k, v):
                c[..., new, :, :t % bs, :] = c[..., old, :, :t % bs, :]
    return tables, counts, head, lens, held, pairs


@pytest.mark.parametrize("lens,src,bs,hkv,d,dtype,layers", [
    ([9, 0, 0], [-1, 0, 0], 4, 2, 64, BF, 1), ([8, 0], [-1, 0], 4, 2, 64, BF, 3),
    ([0, 0], [-1, 0], 4, 1, 8, F32, 1), ([3, 0, 0, 0, 700], [-1, 4, 0, 4, -1], 16, 8, 128, BF, 17),
    ([5, 0, 0], [-1, 0, 0], 4, 3, 7, BF, 2), ([5, 0, 0], [-1, 0, 0], 4, 3, 7, F32, 2),
    ([5, 0, 0], [-1, -5, 0], 1, 1, 16, F32, 1), ([5, 6], [-1, -1], 4, 1, 16, F32, 1),
    ([1000, 0, 0, 33] * 30, [-1, 0, 3, -1] * 30, 8, 1, 16, BF, 2),
    ([130, 0], [-1, 0], 64, 1, 36, BF, 130),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(cuda_device, lens, src, bs, hkv, d, dtype, layers, in_place):
    nb = sum(-(-t // bs) for t in lens) + len(lens) + 3
    st = PoolState(lens, bs, nb, max(-(-t // bs) for t in lens) + 2, seed=5)
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(layers, nb, hkv, bs, d, generator=g).to(dtype) for _ in range(2))
    dev = lambda x: i32(x, cuda_device)
    kd, vd, tables, ref = k.to(cuda_device), v.to(cuda_device), st.tables.to(cuda_device), st.counts().to(cuda_device)
    lens_d, held_d, head_d = dev(lens), dev(st.held), dev([st.head])
    out = dict(seq_lens_out=lens_d, blocks_held_out=held_d, free_head_out=head_d) if in_place else {}
    if layers == 1:
        kd, vd = kd[0], vd[0]
    got = pa.fork_blocks(dev(src), lens_d, tables, held_d, ref, dev(st.free), head_d, kd, vd, **out)
    assert pa.last_device_error() == 0
    want = _fork_reference(st, src, k, v)
    assert torch.equal(tables.cpu(), want[0]) and torch.equal(ref.cpu(), want[1])
    assert got[2].tolist() == [want[2]] and got[0].tolist() == want[3] and got[1].tolist() == want[4]
    assert got[3].tolist() == want[5]
    assert torch.equal(kd.cpu().view(k.shape), k) and torch.equal(vd.cpu().view(v.shape), v)


def test_fork_of_many_rows(cuda_device):
    n, bs = 9000, 4
    lens = [(i * 7) % 23 if i % 3 == 0 else 0 for i in range(n)]
    lens[6000] = 20003
    src = [-1 if i % 3 == 0 else (6000 if i in (1, 8999) else (i * 31 % n) // 3 * 3) for i in range(n)]
    nb = sum(-(-t // bs) for t in lens) + n
    st = PoolState(lens, bs, nb, 20003 // bs + 1, seed=6)
    k, v = torch.randn(nb, 1, bs, 2), torch.randn(nb, 1, bs, 2)
    kd, vd, tables, ref = k.to(cuda_device), v.to(cuda_device), st.tables.to(cuda_device), st.counts().to(cuda_device)
    got = pa.fork_blocks(i32(src, cuda_device), i32(lens, cuda_device), tables, i32(st.held, cuda_device),
                         ref, i32(st.free, cuda_device), i32([st.head], cuda_device), kd, vd)
    assert pa.last_device_error() == 0
    want = _fork_reference(st, src, k, v)
    assert torch.equal(tables.cpu(), want[0]) and torch.equal(ref.cpu(), want[1])
    assert got[2].tolist() == [want[2]] and got[0].tolist() == want[3] and got[3].tolist() == want[5]
    assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)


def test_fork_refuses_as_a_whole(cuda_device):
    st = PoolState([9, 0, 0, 6], 4, 12, 4, seed=7)
    k, v = torch.randn(12, 1, 4, 8, device=cuda_device), torch.randn(12, 1, 4, 8, device=cuda_device)
    dev = lambda x: i32(x, cuda_device)

    def run(src=(-1, 0, 3, -1), lens=None, held=None, head=None):
        lens, held = lens or st.lens, held or st.held
        head = st.head if head is None else head
        tables, ref, kd, vd = st.tables.to(cuda_device), st.counts().to(cuda_device), k.clone(), v.clone()
        got = pa.fork_blocks(dev(list(src)), dev(lens), tables, dev(held), ref, dev(st.free), dev([head]),
                             kd, vd)
        err = pa.last_device_error()
        return (torch.equal(tables.cpu(), st.tables) and torch.equal(ref.cpu(), st.counts())
                and torch.equal(k, kd) and torch.equal(v, vd) and got[0].tolist() == lens
                and got[1].tolist() == held and got[2].tolist() == [head]
                and got[3].tolist() == [[-1, -1]] * 4), err
    for kw, bit in ((dict(src=(-1, 4, 3, -1)), pa.DEVERR_FORK),          # no such row
                    (dict(src=(-1, 2, 0, -1)), pa.DEVERR_FORK),          # a fork of a fork
                    (dict(src=(-1, 1, 0, -1)), pa.DEVERR_FORK),          # of itself
                    (dict(src=(3, 0, 0, -1)), pa.DEVERR_FORK),           # a row with blocks
                    (dict(held=[3, 1, 0, 2]), pa.DEVERR_FORK),
                    (dict(lens=[-9, 0, 0, 6]), pa.DEVERR_SEQ_LEN),
                    (dict(lens=[13, 0, 0, 6]), pa.DEVERR_SEQ_LEN),
                    (dict(held=[5, 0, 0, 2]), pa.DEVERR_SEQ_LEN),
                    (dict(head=11), pa.DEVERR_POOL), (dict(head=-1), pa.DEVERR_POOL)):
        same, err = run(**kw)
        assert same and err == bit, (kw, err)
    same, err = run()
    assert not same and err == 0


def test_fork_with_bad_entries(cuda_device):
    st = PoolState([9, 0, 6, 0, 10, 0], 4, 16, 4, seed=8)
    st.tables[0, 1], st.tables[2, 1] = 99, -1       # a shared entry, a tail
    st.free[st.head + 2] = 16                       # the third fresh block
    k = torch.randn(16, 1, 4, 8, device=cuda_device)
    v, k0 = k.clone(), k.clone()
    tables, ref = st.tables.to(cuda_device), st.counts().to(cuda_device)
    got = pa.fork_blocks(i32([-1, 0, -1, 2, -1, 4], cuda_device), i32(st.lens, cuda_device), tables,
                         i32(st.held, cuda_device), ref, i32(st.free, cuda_device),
                         i32([st.head], cuda_device), k, v)
    assert pa.last_device_error() == pa.DEVERR_TABLE_ENTRY
    f = st.free[st.head:st.head + 2]
    assert tables[1].tolist() == [int(st.tables[0, 0]), 99, f[0], -1]
    assert tables[3].tolist() == [int(st.tables[2, 0]), f[1], -1, -1]
    assert tables[5].tolist() == st.tables[4, :2].tolist() + [-1, -1]
    assert got[3].tolist() == [[-1, -1], [int(st.tables[0, 2]), f[0]]] + [[-1, -1]] * 4
    counts = st.counts()
    for b in [int(st.tables[0, 0]), int(st.tables[2, 0]), *st.tables[4, :2].tolist()]:
        counts[b] += 1
    counts[f] = 1
    assert torch.equal(ref.cpu(), counts)
    want = k0.clone()
    want[f[0], :, :1] = k0[int(st.tables[0, 2]), :, :1]
    assert torch.equal(k, want)


def test_pool_refusals(cuda_device):
    dev = lambda x: i32(x, cuda_device)
    t, k = dev([[0, 1], [2, -1]]), torch.zeros(4, 1, 4, 8, device=cuda_device)
    a, one = dev([0, 0]), dev([2])
    release = lambda lens=a, tables=t, held=dev([2, 1]), free=dev([0] * 4), head=one, **kw: \
        pa.release_blocks(lens, tables, held, free, head, 4, 4, **kw)
    fork = lambda src=dev([-1, -1]), lens=a, tables=t, held=dev([2, 1]), ref=dev([1] * 4), free=dev([0] * 4), \
        head=one, k=k, v=k.clone(), **kw: pa.fork_blocks(src, lens, tables, held, ref, free, head, k, v, **kw)
    for call, kw in ((release, dict(lens=a.long())), (release, dict(lens=dev([0]))),
                     (release, dict(held=dev([2]))), (release, dict(head=a)),
                     (release, dict(tables=t[0])), (release, dict(ref_cnt=a)),
                     (release, dict(blocks_held_out=one)), (release, dict(free_head_out=a)),
                     (release, dict(free=dev([0] * 8)[::2])),
                     (fork, dict(src=dev([-1]))), (fork, dict(ref=dev([1] * 3))),
                     (fork, dict(held=dev([2, 1]).long())), (fork, dict(v=k[:3].clone())),
                     (fork, dict(block_pairs=dev([0] * 4))), (fork, dict(seq_lens_out=one)),
                     (fork, dict(tables=t.T))):
        with pytest.raises(ValueError):
            call(**kw)
    held = dev([2, 1])
    for call, kw in ((release, dict(blocks_held_out=a)), (release, dict(free=a, lens=a)),
                     (release, dict(held=held, free_head_out=held[:1])), (fork, dict(k=k, v=k)),
                     (fork, dict(seq_lens_out=held, held=held)),
                     (release, dict(lens=torch.zeros(2, dtype=torch.int32)))):
        with pytest.raises(pa.PaError):
            call(**kw)


def test_a_fork_and_its_release_leave_the_pool_as_it_was(cuda_device):
    """Captured in a graph and replayed; another stream beside it on another pool."""
    def state(seed):
        st = PoolState([90, 0, 0, 64, 0, 7, 0], 16, 40, 8, seed=seed)
        d = dict(st=st, src=i32([-1, 0, 0, -1, 3, -1, 5], cuda_device), lens=i32(st.lens, cuda_device),
                 tables=st.tables.to(cuda_device), held=i32(st.held, cuda_device),
                 ref=st.counts().to(cuda_device), free=i32(st.free, cuda_device),
                 head=i32([st.head], cuda_device), k=torch.randn(3, 40, 2, 16, 32, device=cuda_device),
                 v=torch.randn(3, 40, 2, 16, 32, device=cuda_device))
        return d

    def cycle(d, stream=None):
        lens, held, head, pairs = pa.fork_blocks(d["src"], d["lens"], d["tables"], d["held"], d["ref"],
                                                 d["free"], d["head"], d["k"], d["v"], stream=stream)
        held2, head2 = pa.release_blocks(d["lens"], d["tables"], held, d["free"], head, 40, 16,
                                         ref_cnt=d["ref"], stream=stream)
        return lens, held, head, pairs, held2, head2

    def check(d, out):
        st = d["st"]
        assert out[4].tolist() == st.held and out[5].tolist() == [st.head]
        assert d["free"].tolist()[st.head:] == st.free[st.head:] and torch.equal(d["ref"].cpu(), st.counts())
        assert out[2].tolist() == [st.head + 3] and out[1].tolist() == [6, 6, 6, 4, 4, 1, 1]
    d = state(1)
    check(d, cycle(d))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cycle(d)
    for _ in range(3):
        graph.replay()
    check(d, out)
    x, y = state(2), state(3)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [(cycle(x, s1), cycle(y, s2)) for _ in range(5)]
    torch.cuda.synchronize()
    for a, b in outs:
        check(x, a)
        check(y, b)
    assert pa.last_device_error() == 0


# ---- the loop --------------------------------------------------------------------------------

class Toy:
    """A model of one layer: token embedding, projection, attention, logits."""

    def __init__(self, vocab, hq, hkv, d, seed):
        g = torch.Generator().manual_seed(seed)
        self.embed = torch.randn(vocab, 24, generator=g)
        self.proj = torch.randn(24, (hq + 2 * hkv) * d, generator=g) / 5
        self.head = torch.randn(hq * d, vocab, generator=g) / 3
        self.qw, self.kw = 1 + 0.2 * torch.randn(d, generator=g), 1 + 0.2 * torch.randn(d, generator=g)
        self.inv = (1000.0 ** (-torch.arange(0, d, 2) / d)).float()
        self.cut = (hq * d, hkv * d, hkv * d)


def test_a_serving_loop_of_all_calls(cuda_device):
    """Three steps of drafted decoding for five requests, one forked from another
    and one ended on the way: plan, projection rows to the cache, tree attention,
    verification, the accepted path, blocks back.  Against a loop in 64 bits over
    whole histories."""
    vocab, hq, hkv, d, bs, nb, width, most = 60, 4, 2, 32, 4, 64, 12, 40
    toy = Toy(vocab, hq, hkv, d, 1)
    dev = cuda_device
    on = lambda t: t.to(dev)
    g = torch.Generator().manual_seed(4)
    prompts = [torch.randint(0, vocab, (m,), generator=g).tolist() for m in (9, 5, 13, 8)] + [[]]
    n = 5
    kc, vc = torch.zeros(nb, hkv, bs, d, device=dev), torch.zeros(nb, hkv, bs, d, device=dev)
    tables = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    lens, held = torch.zeros(n, dtype=torch.int32, device=dev), torch.zeros(n, dtype=torch.int32, device=dev)
    free, head = torch.arange(nb, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    ref = torch.zeros(nb, dtype=torch.int32, device=dev)
    w = {k: on(getattr(toy, k)) for k in ("embed", "proj", "head", "qw", "kw", "inv")}

    def rows(tokens, plan, trees=()):
        """Projected rows of the step's tokens into the cache; the queries.  A
        drafted node's position counts its ancestors, not the nodes before it."""
        behind = [len(path_of(t, j)) - 1 - j for t in trees for j in range(len(t))]
        positions = torch.where(plan.positions < 0, plan.positions, plan.positions + padded(behind))
        x = w["embed"][tokens.long()] @ w["proj"]
        q, k, v = x.split(toy.cut, 1)
        return pa.rope_write(q.unflatten(1, (hq, d)), k.unflatten(1, (hkv, d)), v.unflatten(1, (hkv, d)),
                             positions, w["inv"], plan.slot_mapping, kc, vc, q_weight=w["qw"],
                             k_weight=w["kw"])

    def plan_of(counts):
        p = pa.plan_step(lens, i32(counts, dev), tables, held, free, head, nb, bs, max_tokens=most, ref_cnt=ref)
        held.copy_(p.blocks_held)
        head.copy_(p.free_head)
        return p

    def padded(tokens):
        return on(i32(tokens + [0] * (most - len(tokens))))

    # the prompts but for each one's last token, which is the first step's root
    first = [p[:-1] for p in prompts]
    plan = plan_of([len(p) for p in first])
    rows(padded(sum(first, [])), plan)
    lens.copy_(plan.seq_lens)
    history = [list(p) for p in prompts]            # cached tokens and the root

    def plain_logits(tokens):
        """[len, vocab] logits behind every token, in 64 bits."""
        x = toy.embed[torch.tensor(tokens)].double() @ toy.proj.double()
        q, k, v = (t.unflatten(1, (-1, d)) for t in x.split(toy.cut, 1))
        angle = torch.arange(len(tokens)).double()[:, None] * toy.inv.double()
        c, s = angle.cos()[:, None], angle.sin()[:, None]

        def turn(y, weight):
            y = y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
            a, b = y[..., :d // 2], y[..., d // 2:]
            return torch.cat([a * c - b * s, a * s + b * c], -1)
        q, k = turn(q, toy.qw), turn(k, toy.kw)
        k, v = (t.repeat_interleave(hq // hkv, 1) for t in (k, v))
        score = torch.einsum("qhd,khd->hqk", q, k) / math.sqrt(d)
        score.masked_fill_(torch.ones(len(tokens), len(tokens)).triu(1).bool(), -math.inf)
        return torch.einsum("hqk,khd->qhd", score.softmax(-1), v).flatten(1) @ toy.head.double()

    trees = [[-1, 0, 0, 1], [-1, 0], [-1, 0, 1, 1, 3], [-1], []]
    for step in range(3):
        if step == 1:
            # row 4 starts as a fork of row 2
            trees[4] = [-1, 0, 0]
            lens_f, held_f, head_f, pairs = pa.fork_blocks(i32([-1, -1, -1, -1, 2], dev), lens, tables,
                                                           held, ref, free, head, kc, vc)
            lens, held = lens_f, held_f
            head.copy_(head_f)
            history[4] = list(history[2])
        if step == 2:
            # row 0 ends: its blocks and those of rejected drafts go back
            trees[0] = []
            lens = lens * on(i32([0, 1, 1, 1, 1]))
            before = int(head)
            pa.release_blocks(lens, tables, held, free, head, nb, bs, ref_cnt=ref, blocks_held_out=held,
                              free_head_out=head)
            assert int(head) < before and int(held[0]) == 0
            history[0] = []
        tokens, q0 = [], [0]
        for i, t in enumerate(trees):
            tokens += history[i][-1:] * bool(t) + torch.randint(0, vocab, (max(len(t) - 1, 0),),
                                                                generator=g).tolist()
            q0.append(len(tokens))
        # likely drafts, so that some hold: the plain model's own choice
        for i, t in enumerate(trees):
            for j, p in enumerate(t):
                if p >= 0:
                    chain = history[i][:-1] + [tokens[q0[i] + a] for a in path_of(t, p)]
                    tokens[q0[i] + j] = int(plain_logits(chain)[-1].topk(j + 1).indices[-1 if j % 2 else 0])
        parents = sum(trees, [])
        plan = plan_of([len(t) for t in trees])
        q = rows(padded(tokens), plan, trees)
        par = padded(parents)
        out = pa.decode_tree(q, plan.query_start_loc, par, kc, vc, tables, plan.seq_lens, 5, width * bs)
        logits = out.flatten(1) @ w["head"]
        b = VerifyBatch([len(t) for t in trees], vocab, F32, seed=step, draft=False)
        uniforms, noise = torch.rand(most, generator=g), b.noise
        leaf, token = pa.verify_tree(logits, padded(tokens), par, plan.query_start_loc, on(uniforms),
                                     on(noise), 5)
        new_lens, _ = pa.accept_tree(leaf, par, plan.query_start_loc, plan.seq_lens, kc, vc, tables, 5)
        lens = new_lens
        assert pa.last_device_error() == 0
        # the same step in 64 bits
        b.par, b.parents, b.start = trees, i32(parents), i32(q0)
        b.tokens, b.uniforms = i32(tokens), uniforms
        b.logits = torch.zeros(len(tokens), vocab, dtype=torch.float64)
        for i, t in enumerate(trees):
            for j in range(len(t)):
                chain = history[i][:-1] + [tokens[q0[i] + a] for a in path_of(t, j)]
                b.logits[q0[i] + j] = plain_logits(chain)[-1]
        got = logits[:len(tokens)].double().cpu()
        assert float(((got - b.logits).abs() / (1 + b.logits.abs())).max()) <= 1e-3
        ref_out = verify_reference(b)
        for i, (x, t, close) in enumerate(ref_out):
            if trees[i]:
                assert not close
                assert (int(leaf[i]), int(token[i])) == (x, t), (step, i)
                history[i] = history[i][:-1] + [tokens[q0[i] + a] for a in path_of(trees[i], x)] + [t]
        assert lens.tolist() == [max(len(h) - 1, 0) for h in history]
    # every block is in the queue or counted, once
    counted = {i for i, c in enumerate(ref.tolist()) if c > 0}
    queue = free.tolist()[int(head):]
    assert len(set(queue)) == len(queue) and not counted & set(queue) and len(counted) + len(queue) == nb


# ---- the calls that fit nowhere above ---------------------------------------------------------

def test_empty_batches(cuda_device):
    e = lambda *shape, dtype=F32: torch.empty(shape, dtype=dtype, device=cuda_device)
    n32 = e(0, dtype=torch.int32)
    k = torch.zeros(4, 2, 4, 8, device=cuda_device)
    out = pa.rope_write(e(0, 4, 8), e(0, 2, 8), e(0, 2, 8), n32, e(4), e(0, dtype=torch.int64), k, k.clone())
    assert out.shape == (0, 4, 8)
    leaf, token = pa.verify_tree(e(0, 50), n32, n32, i32([0], cuda_device), e(0), e(0, 50), 0)
    assert leaf.numel() == token.numel() == 0
    free, head, counts = i32([3, 1], cuda_device), i32([1], cuda_device), i32([0] * 4, cuda_device)
    for ref in (None, counts):
        held, after = pa.release_blocks(n32, e(0, 5, dtype=torch.int32), n32, free, head, 4, 4, ref_cnt=ref)
        assert held.numel() == 0 and after.tolist() == [1]
    got = pa.fork_blocks(n32, n32, e(0, 5, dtype=torch.int32), n32, counts, free, head, k, k.clone())
    assert got[2].tolist() == [1] and pa.last_device_error() == 0
    # sequences, but none with nodes: no logits at all
    leaf, token = pa.verify_tree(e(0, 50), n32, n32, i32([0, 0, 0], cuda_device), e(0), torch.ones(2, 50, device=cuda_device), 0)
    assert leaf.tolist() == token.tolist() == [-1, -1]


def test_pinned_logits(cuda_device):
    for dtype, vocab in ((BF, 5003), (F32, 8192)):
        b = VerifyBatch([5, 9, 2], vocab, dtype, seed=20, temps=[1.0, 0.0])
        want = b.run(pa, cuda_device)
        leaf, token = torch.empty(3, dtype=torch.int32, device=cuda_device), torch.empty(3, dtype=torch.int32, device=cuda_device)
        pin = lambda t: t.pin_memory()
        lib, dev = pa.load_library(), lambda t: t.to(cuda_device)
        t = [pin(b.logits), pin(b.draft), dev(b.tokens), dev(b.parents), dev(b.start), dev(b.uniforms), dev(b.noise),
             dev(b.temps)]
        st = lib.pa_verify_tree(t[0].data_ptr(), t[1].data_ptr(), vocab, vocab, vocab,
                                pa.PA_F32 if dtype == F32 else pa.PA_BF16, *(x.data_ptr() for x in t[2:5]), 3, 16, 9,
                                t[5].data_ptr(), t[6].data_ptr(), vocab, t[7].data_ptr(), leaf.data_ptr(),
                                token.data_ptr(), None)
        torch.cuda.synchronize()
        assert st == pa.PA_OK and torch.equal(leaf.cpu(), want[0]) and torch.equal(token.cpu(), want[1])


def test_debug_checks(cuda_device, monkeypatch):
    """PA_DEBUG refuses what the kernels cannot see or would report later."""
    monkeypatch.setenv("PA_DEBUG", "1")
    dev = lambda x: i32(x, cuda_device)
    st = PoolState([9, 6], 4, 12, 4, seed=9)
    state = lambda: [dev([0, 6]), st.tables.to(cuda_device), dev(st.held), dev(st.free), dev([st.head]), 12, 4]
    assert pa.release_blocks(*state())[0].tolist() == [0, 2]
    twice, queued, outside = st.tables.clone(), st.tables.clone(), st.tables.clone()
    twice[0, 1], queued[0, 1], outside[0, 1] = twice[0, 0], st.free[-1], 12
    for tables in (twice, queued, outside):
        args = state()
        args[1] = tables.to(cuda_device)
        with pytest.raises(pa.PaError):
            pa.release_blocks(*args)
    with pytest.raises(pa.PaError):
        pa.release_blocks(*state(), ref_cnt=dev([0] * 12))
    k = torch.zeros(12, 1, 4, 8, device=cuda_device)
    fork = lambda src, held: pa.fork_blocks(dev(src), dev([9, 6, 0]), dev([[0, 1, 2], [3, 4, -1], [-1] * 3]), dev(held),
                                            dev([1] * 5 + [0] * 7), dev([-1] * 5 + [5, 6]), dev([5]), k, k.clone())
    assert fork([-1, -1, 0], [3, 2, 0])[1].tolist() == [3, 2, 3]
    for src, held in (([-1, 0, -1], [3, 2, 0]), ([-1, -1, 3], [3, 2, 0]), ([-1, -1, 2], [3, 2, 0])):
        with pytest.raises(pa.PaError):
            fork(src, held)
    b = RopeBatch(6, 2, 1, 16, 4, F32, seed=21)
    b.slots[3] = b.slots[1]
    with pytest.raises(pa.PaError):
        b.run(pa, cuda_device)
    v = VerifyBatch([3, 2], 30, F32, seed=22, kind="chain")
    v.parents[1] = 2
    with pytest.raises(pa.PaError):
        v.run(pa, cuda_device)


@pytest.mark.parametrize("n,heads,d,dtype", [(2433, 4, 128, BF), (5000, 3, 80, F32), (40000, 1, 32, BF)])
def test_rope_of_many_tokens(cuda_device, n, heads, d, dtype):
    """More tokens than warps fit at once, against a call for each part."""
    b = RopeBatch(n, heads, 1, d, 16, dtype, seed=23, far=100000, skip=tuple(range(0, n, 97)))
    q, k, v = (x.to(cuda_device) for x in b.split(b.qkv))
    kc, vc = b.k_cache.to(cuda_device), b.v_cache.to(cuda_device)
    kc2, vc2 = kc.clone(), vc.clone()
    move = lambda t: t.to(cuda_device)
    pos, inv, slots, kw = move(b.pos), move(b.inv), move(b.slots), dict(q_weight=move(b.qw), k_weight=move(b.kw), **b.args)
    out = pa.rope_write(q, k, v, pos, inv, slots, kc, vc, out=move(b.out), **kw)
    parts = move(b.out)
    for i in range(0, n, 501):
        c = slice(i, i + 501)
        pa.rope_write(q[c], k[c], v[c], pos[c], inv, slots[c], kc2, vc2, out=parts[c], **kw)
    assert torch.equal(out, parts) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
    assert pa.last_device_error() == 0


def test_rope_captured_and_replayed_on_other_tokens(cuda_device):
    b = RopeBatch(70, 8, 2, 128, 16, BF, seed=24, axes=2, sections=(24, 40), skip=(69,))
    c = RopeBatch(70, 8, 2, 128, 16, BF, seed=25, axes=2, sections=(24, 40), skip=(3, 68))
    dev = lambda t: t.to(cuda_device)
    qkv, pos, slots, out = dev(b.qkv), dev(b.pos), dev(b.slots), dev(b.out)
    kc, vc, inv, qw, kw = (dev(t) for t in (b.k_cache, b.v_cache, b.inv, b.qw, b.kw))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, k, v = b.split(qkv)
        pa.rope_write(q, k, v, pos, inv, slots, kc, vc, q_weight=qw, k_weight=kw, out=out, **b.args)
    for t, x in ((qkv, c.qkv), (pos, c.pos), (slots, c.slots), (out, c.out), (kc, c.k_cache), (vc, c.v_cache),
                 (qw, c.qw), (kw, c.kw)):
        t.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    c.check(out.cpu(), kc.cpu(), vc.cpu())


def test_calls_from_several_host_threads(cuda_device):
    """Shapes of different instances of the kernels, each thread on a stream of its
    own."""
    ropes = [RopeBatch(40, 4, 2, d, 8, t, seed=26 + i, **kw) for i, (d, t, kw) in enumerate(
        [(128, BF, {}), (80, F32, dict(neighbours=True)), (36, BF, dict(rot=20)), (256, F32, {})])]
    trees = [VerifyBatch([4, 7, 1], v, t, seed=30 + i, draft=d) for i, (v, t, d) in enumerate(
        [(5000, BF, True), (20000, F32, False), (333, F32, True), (40003, BF, False)])]
    want = [(r.run(pa, cuda_device), t.run(pa, cuda_device)) for r, t in zip(ropes, trees)]
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got = ropes[i].run(pa, cuda_device), trees[i].run(pa, cuda_device)
                    same = all(torch.equal(x.view(torch.uint8), y.view(torch.uint8))
                               for a, b in zip(got, want[i]) for x, y in zip(a, b))
                    if not same:
                        wrong.append(i)
        except Exception as e:                          # a thread's error must reach the test
            wrong.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and pa.last_device_error() == 0
