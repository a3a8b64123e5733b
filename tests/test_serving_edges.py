"""Calls around the attention that the documentation allows and that the other tests
do not make: the documented loop, one token in place, reports of a greedy walk, the
largest sizes, releases that do not fit in shared memory, first calls in a graph, what
PA_DEBUG refuses and what it does not."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import paged_kv_cache_109_gb300 as pa
from tests._serving import PoolState, RopeBatch, VerifyBatch, i32
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def clear_device_error(cuda_device):
    pa.last_device_error()
    yield


# ---- the documented loop -----------------------------------------------------------------

def _documented_step():
    """The drafted step as the documentation gives it."""
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    begin = text.index("# one drafted (speculative) step")
    return text[begin:text.index("```", begin)]


def test_the_documented_step_runs_as_a_loop(cuda_device):
    """The drafted step, run as it stands for several steps: a request that
    ends, a fork into its row, and at the end every block back in the queue."""
    dev = lambda x: i32(x, cuda_device)
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(*s, device=cuda_device, generator=g)
    n, hq, hkv, d, bs, blocks, width, vocab, most = 4, 4, 2, 32, 4, 48, 8, 50, 20
    lens, held = [9, 5, 6, 0], [3, 2, 2, 0]
    table = [[0, 1, 2] + [-1] * 5, [3, 4] + [-1] * 6, [5, 6] + [-1] * 6, [-1] * 8]
    s = dict(pa=pa, torch=torch, seq_lens=dev(lens), blocks_held=dev(held), block_tables=dev(table),
             free_blocks=dev([-1] * 7 + list(range(7, blocks))), free_head=dev([7]),
             ref_cnt=dev([1] * 7 + [0] * (blocks - 7)), num_blocks=blocks, block_size=bs, max_rows=most,
             inv_freq=(1000.0 ** (-torch.arange(0, d, 2) / d)).to(cuda_device),
             k_cache=rand(blocks, hkv, bs, d), v_cache=rand(blocks, hkv, bs, d), wq=rand(d), wk=rand(d),
             max_q_len=4, max_seq_len=width * bs)
    s["k_caches"], s["v_caches"] = s["k_cache"], s["v_cache"]
    step = compile(_documented_step(), "README.md", "exec")
    # nodes of each row's chain, rows that go on, sources of the rows that fork
    for nodes, running, src in (([4, 3, 4, 0], [1, 0, 1, 0], [-1, 0, -1, -1]),
                                ([3, 4, 1, 0], [1, 1, 1, 0], [-1, -1, -1, 1]),
                                ([2, 2, 4, 4], [1, 1, 0, 1], [-1, -1, -1, -1]),
                                ([0, 3, 0, 2], [0, 0, 0, 0], [-1, -1, -1, -1])):
        before = s["seq_lens"].tolist()
        parents = [j - 1 for m in nodes for j in range(m)]
        s.update(new_tokens=dev(nodes), parents=dev(parents + [-1] * (most - len(parents))),
                 q=rand(most, hq, d), k=rand(most, hkv, d), v=rand(most, hkv, d),
                 positions=dev([t % 7 for t in range(most)]), logits=rand(most, vocab),
                 draft_logits=rand(most, vocab), tokens=dev([t % vocab for t in range(most)]),
                 uniforms=torch.rand(most, device=cuda_device, generator=g),
                 noise=rand(n, vocab).exponential_(generator=g),
                 temperature=torch.ones(n, device=cuda_device), running=dev(running), src=dev(src))
        exec(step, s)
        assert pa.last_device_error() == 0
        leaf = s["leaf"].tolist()
        want = [(c + l + 1) * r for c, l, r in zip(before, leaf, running)]
        want = [want[p] if p >= 0 else t for t, p in zip(want, src)]
        assert s["seq_lens"].tolist() == want
        assert s["blocks_held"].tolist() == [-(-t // bs) for t in want]
        # each block is in the queue or counted, as often as rows hold it
        rows, count = s["block_tables"].tolist(), [0] * blocks
        for row, h in zip(rows, s["blocks_held"].tolist()):
            for b in row[:h]:
                count[b] += 1
        assert s["ref_cnt"].tolist() == count
        assert sorted(s["free_blocks"].tolist()[int(s["free_head"]):]) == [b for b in range(blocks) if not count[b]]
    assert int(s["free_head"]) == 0


# ---- rope_write ----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad_row", [0, 1, 24])
def test_one_token_of_a_projection_in_place(cuda_device, dtype, pad_row):
    """One token's heads follow one another, however wide the row that they were cut
    from: its queries may be rotated where they are."""
    b = RopeBatch(1, 8, 2, 64, 8, dtype, seed=1, pad_row=pad_row)
    q, k, v = b.split(b.qkv.to(cuda_device))
    kc, vc = b.k_cache.to(cuda_device), b.v_cache.to(cuda_device)
    move = lambda t: t.to(cuda_device)
    got = pa.rope_write(q, k, v, move(b.pos), move(b.inv), move(b.slots), kc, vc, q_weight=move(b.qw),
                        k_weight=move(b.kw), out=q, **b.args)
    assert got is q
    b.check(q.cpu(), kc.cpu(), vc.cpu())
    # cut from all heads at once, so that torch's stride is the projection's
    heads = b.qkv.to(cuda_device)[:, :12 * 64].view(1, 12, 64)
    q2, kc, vc = heads[:, :8], b.k_cache.to(cuda_device), b.v_cache.to(cuda_device)
    assert q2.stride(0) == 12 * 64
    got = pa.rope_write(q2, heads[:, 8:10], heads[:, 10:], move(b.pos), move(b.inv), move(b.slots), kc, vc,
                        q_weight=move(b.qw), k_weight=move(b.kw), out=q2, **b.args)
    assert torch.equal(q2, q)
    b.check(q2.cpu(), kc.cpu(), vc.cpu())
    # the C call with the row's own stride
    q2, k2, v2 = b.split(b.qkv.to(cuda_device))
    kc, vc = b.k_cache.to(cuda_device), b.v_cache.to(cuda_device)
    pos, inv, slots, qw, kw = (move(t) for t in (b.pos, b.inv, b.slots, b.qw, b.kw))
    desc = pa.CacheDesc(kc.shape[0], 8, 2, 64, pa.PA_BF16 if dtype is BF else pa.PA_F32)
    rope = pa.RopeDesc(64, 1, (pa.ctypes.c_int32 * 3)(), 0, 0, 1.0, 1e-5)
    width = b.qkv.shape[1]
    st = pa.load_library().pa_rope_write(
        q2.data_ptr(), k2.data_ptr(), v2.data_ptr(), width, width, width, 1, 8, pos.data_ptr(), inv.data_ptr(),
        qw.data_ptr(), kw.data_ptr(), pa.ctypes.byref(rope), slots.data_ptr(), q2.data_ptr(), kc.data_ptr(),
        vc.data_ptr(), pa.ctypes.byref(desc), None)
    torch.cuda.synchronize()
    assert st == pa.PA_OK and torch.equal(q2.cpu(), q.cpu())


def test_sections_that_change_between_calls(cuda_device):
    """What a call does follows from the values of its sections, not from the objects
    that hold them."""
    sections = [torch.tensor(8), torch.tensor(24)]
    for first in (8, 20):
        sections[0].fill_(first)
        sections[1].fill_(32 - first)
        b = RopeBatch(5, 2, 1, 64, 8, F32, seed=2, axes=2, sections=(first, 32 - first))
        b.args["sections"] = sections
        out = b.run(pa, cuda_device)
        b.args["sections"] = (first, 32 - first)
        b.check(*out)


# ---- verify_tree ---------------------------------------------------------------------------

@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_greedy_walks_report_tokens_outside_the_vocabulary(cuda_device, draft, dtype):
    b = VerifyBatch([4, 4, 4, 4], 300, dtype, seed=3, kind="star", draft=draft, temps=[0.0])
    best = b.logits[b.start[:-1].long()].float().argmax(1).tolist()
    # met before the child that holds, met without one, behind the one that holds
    b.tokens[:] = i32([0, 300, best[0], 1, 0, -1, 2 ** 31 - 1, -(2 ** 31), 0, best[2], 300, 1, 0, best[3], 0, 0])
    want = ([2, 0, 1, 1], [0, 1])
    for keep, bit in (([0, 1, 2, 3], pa.DEVERR_TREE), ([2, 3], 0)):
        rows = torch.cat([torch.arange(4 * i, 4 * i + 4) for i in keep])
        c = VerifyBatch([4] * len(keep), 300, dtype, seed=3, kind="star", draft=draft, temps=[0.0])
        c.tokens, c.logits, c.parents = b.tokens[rows], b.logits[rows], b.parents[rows]
        c.draft = b.draft[rows] if draft else None
        leaf, token = c.run(pa, cuda_device)
        assert pa.last_device_error() == bit
        assert leaf.tolist() == [want[0][i] for i in keep]
        assert int(token[keep.index(2)]) == int(b.logits[9].float().argmax())


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("vocab", [1, 2, 300, 4099, 20000])
def test_a_token_of_all_the_probability_holds(cuda_device, vocab, dtype, draft):
    """P(t) is one, then a power of two (equal tokens): the largest uniform below P(t) / q(t)
    holds, P(t) / q(t) itself does not."""
    below = 1 - 2.0 ** -24
    for rest in (-float("inf"), -300.0, torch.finfo(dtype).min):
        for alike in (1, 2, 4):
            if alike > vocab or (draft and alike > 1):
                continue
            b = VerifyBatch([2, 2], vocab, dtype, seed=4, kind="chain", draft=draft)
            b.logits[:] = rest
            b.logits[:, vocab - alike:] = 3.0
            if draft:
                b.draft[:] = b.logits
            b.tokens[:] = vocab - 1
            b.uniforms[:] = below / alike
            b.uniforms[3] = 1.0 / alike
            leaf, _ = b.run(pa, cuda_device)
            assert pa.last_device_error() == 0
            assert leaf.tolist() == [1, 0], (rest, alike)


# ---- release, fork ---------------------------------------------------------------------------

def _wide_pool(n, width, seed, counted):
    """Rows of random lengths up to ``width`` blocks over a pool of all their blocks;
    with counts, each third row starts with the leading blocks of the row before it."""
    rng = np.random.default_rng(seed)
    held = rng.integers(width // 2, width + 1, n).astype(np.int32)
    total = int(held.sum())
    perm = rng.permutation(total).astype(np.int32)
    tables = np.full((n, width), -1, np.int32)
    tables[np.arange(width) < held[:, None]] = perm
    if counted:
        for i in range(3, n, 3):
            k = int(min(held[i], held[i - 1])) // 2
            tables[i, :k] = tables[i - 1, :k]
    counts = np.bincount(tables[tables >= 0], minlength=total).astype(np.int32)
    idle = np.flatnonzero(counts == 0).astype(np.int32)       # blocks of no row: the queue
    head = total - len(idle)
    free = np.full(total, -1, np.int32)
    free[head:] = idle
    return held, tables, counts, free, head


def _wide_release(held, keep, tables, counts, free, head):
    """The release on the host: counts, queue, front after it."""
    col = np.arange(tables.shape[1])
    drops = tables[(col >= keep[:, None]) & (col < held[:, None])]
    drops = drops[(drops >= 0) & (drops < len(free))]
    if counts is None:
        freed = drops
    else:
        counts = counts - np.bincount(drops, minlength=len(free)).astype(np.int32)
        _, last = np.unique(drops[::-1], return_index=True)
        last = np.sort(len(drops) - 1 - last)
        freed = drops[last]
        freed = freed[counts[freed] == 0]
    free, head = free.copy(), head - len(freed)
    free[head:head + len(freed)] = freed
    return counts, free, head


@pytest.mark.parametrize("n,width", [(260, 6100), (5003, 300)])
@pytest.mark.parametrize("counted", [True, False])
def test_release_of_more_entries_than_shared_memory_keeps(cuda_device, n, width, counted):
    """Some 1.1 million entries, in one round of sequences and in two: each pass reads
    the tables again.  As a whole, and refused as a whole."""
    bs = 4
    held, tables, counts, free, head = _wide_pool(n, width, seed=n, counted=counted)
    keep = np.where(np.arange(n) % 17 == 5, held // 2, 0).astype(np.int32)
    tables[7, 3], tables[n - 2, 5] = -1, len(free)            # passed over
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(cuda_device)
    args = lambda head, free_d: (dev(keep * bs), dev(tables), dev(held), free_d, i32([head], cuda_device),
                                 len(free), bs)
    assert int((held - keep).sum()) > 16 * 40960

    def run(head, counts):
        free_d, ref = dev(free), dev(counts) if counted else None
        got = pa.release_blocks(*args(head, free_d), ref_cnt=ref)
        return got[0].cpu().numpy(), int(got[1]), free_d.cpu().numpy(), ref.cpu().numpy() if counted else None
    want_counts, want_free, want_head = _wide_release(held, keep, tables, counts if counted else None, free, head)
    got = run(head, counts)
    assert pa.last_device_error() == pa.DEVERR_TABLE_ENTRY
    assert (got[0] == keep).all() and got[1] == want_head and (got[2] == want_free).all()
    if counted:
        assert (got[3] == want_counts).all()
    # no room in front of the queue for the last block
    short = head - want_head - 1
    got = run(short, counts)
    assert pa.last_device_error() & pa.DEVERR_POOL
    assert (got[0] == held).all() and got[1] == short and (got[2] == free).all()
    assert not counted or (got[3] == counts).all()
    if counted:
        less = counts.copy()
        less[tables[n - 1, held[n - 1] - 1]] -= 1               # dropped once more than held
        got = run(head, less)
        assert pa.last_device_error() & pa.DEVERR_SHARED
        assert (got[0] == held).all() and got[1] == head and (got[2] == free).all() and (got[3] == less).all()


def test_fork_outputs_over_a_cache_are_refused(cuda_device):
    dev = lambda x: i32(x, cuda_device)
    st = PoolState([9, 0], 4, 12, 4, seed=4)
    k, v = torch.zeros(12, 1, 4, 8, device=cuda_device), torch.zeros(12, 1, 4, 8, device=cuda_device)
    tables, lens, held, ref = st.tables.to(cuda_device), dev(st.lens), dev(st.held), st.counts().to(cuda_device)
    free, head = dev(st.free), dev([st.head])
    inside = lambda c, m: c.view(-1).view(torch.int32)[-m:]
    call = lambda k=k, v=v, tables=tables, **kw: pa.fork_blocks(
        dev([-1, 0]), lens, tables, held, ref, free, head, k, v, **kw)
    for kw in (dict(seq_lens_out=inside(k, 2)), dict(blocks_held_out=inside(v, 2)), dict(free_head_out=inside(v, 1)),
               dict(block_pairs=inside(k, 8).view(torch.int64).view(2, 2)), dict(tables=inside(v, 8).view(2, 4))):
        with pytest.raises(pa.PaError) as e:
            call(**kw)
        assert e.value.status == pa.PA_ERR_INVALID_ARG
    assert call()[1].tolist() == [3, 3] and pa.last_device_error() == 0


# ---- the error word ----------------------------------------------------------------------------

def test_every_reported_bit_is_read_once(cuda_device):
    """The kernels of both source files have a word of their own; a read takes and clears
    both."""
    k = torch.zeros(4, 1, 4, 8, device=cuda_device)
    rows, past = torch.zeros(1, 1, 8, device=cuda_device), torch.tensor([16], device=cuda_device)
    write = lambda: pa.write_kv(rows, rows, past, k, k.clone())
    one, zero = i32([1], cuda_device), i32([0], cuda_device)
    release = lambda: pa.release_blocks(zero, i32([[2]], cuda_device), one, i32([0, 0], cuda_device), zero, 4, 4)
    for calls, bits in (((write,), pa.DEVERR_SLOT), ((release,), pa.DEVERR_POOL),
                        ((write, release), pa.DEVERR_SLOT | pa.DEVERR_POOL), ((), 0)):
        for call in calls:
            call()
        assert pa.last_device_error() == bits
        assert pa.last_device_error() == 0


# ---- PA_DEBUG --------------------------------------------------------------------------------

def test_debug_passes_tokens_that_are_skipped(cuda_device, monkeypatch):
    """A token with a negative position writes nothing: its slot is not looked at."""
    monkeypatch.setenv("PA_DEBUG", "1")
    for axes, sections in ((1, None), (2, (20, 12))):
        b = RopeBatch(6, 2, 1, 64, 4, F32, seed=5, skip=(1, 4, 5), axes=axes, sections=sections)
        b.slots[1], b.slots[4], b.slots[5] = b.slots[0], b.slots[0], 2 ** 40
        b.check(*b.run(pa, cuda_device))
        assert pa.last_device_error() == 0
        b.pos.view(axes, -1)[0, 4] = 0
        with pytest.raises(pa.PaError):
            b.run(pa, cuda_device)


def test_debug_refuses_forks_of_blocks_without_counts(cuda_device, monkeypatch):
    """A shared block's count says who holds it: one that no row counts would be freed
    by the fork's release, under its source."""
    monkeypatch.setenv("PA_DEBUG", "1")
    dev = lambda x: i32(x, cuda_device)
    st = PoolState([9, 0], 4, 12, 4, seed=6)
    k, v = torch.zeros(12, 1, 4, 8, device=cuda_device), torch.zeros(12, 1, 4, 8, device=cuda_device)

    def fork(counts):
        return pa.fork_blocks(dev([-1, 0]), dev(st.lens), st.tables.to(cuda_device), dev(st.held), counts, dev(st.free),
                              dev([st.head]), k, v)
    assert fork(st.counts().to(cuda_device))[1].tolist() == [3, 3]
    for b in st.tables[0, :3].tolist():
        counts = st.counts()
        counts[b] = 0
        with pytest.raises(pa.PaError):
            fork(counts.to(cuda_device))


# ---- sizes past 32 bits ------------------------------------------------------------------------

def test_rows_and_blocks_past_32_bits(cuda_device):
    """Slots, tails and strides behind 2^31 elements."""
    nb, hkv, bs, d = 33000, 8, 64, 128                  # 2.2e9 elements, 4.3 GB a cache
    b = RopeBatch(5, 16, hkv, d, bs, BF, seed=7)
    kc, vc = (torch.zeros(nb, hkv, bs, d, dtype=BF, device=cuda_device) for _ in range(2))
    last = [nb - 1, nb - 2, 1]
    b.slots[:] = torch.tensor([last[0] * bs + 3, last[0] * bs + 63, last[1] * bs, last[2] * bs + 5, 0])
    width, far = b.qkv.shape[1], 550_000_000            # tokens 1.1 GB apart
    wide = torch.empty(4 * far + width, dtype=BF, device=cuda_device)
    rows = wide.as_strided((5, width), (far, 1))
    rows.copy_(b.qkv)
    move = lambda t: t.to(cuda_device)
    out = pa.rope_write(*b.split(rows), move(b.pos), move(b.inv), move(b.slots), kc, vc, q_weight=move(b.qw),
                        k_weight=move(b.kw), out=move(b.out), **b.args)
    # the same rows into a cache of the four blocks alone
    near = RopeBatch(5, 16, hkv, d, bs, BF, seed=7)
    near.k_cache, near.v_cache = torch.zeros(4, hkv, bs, d, dtype=BF), torch.zeros(4, hkv, bs, d, dtype=BF)
    near.slots[:] = torch.tensor([3 * bs + 3, 3 * bs + 63, 2 * bs, bs + 5, 0])
    want = near.run(pa, cuda_device)
    near.check(*want)
    at = [0, 1, nb - 2, nb - 1]
    assert torch.equal(out.cpu(), want[0]) and torch.equal(kc[at].cpu(), want[1]) and torch.equal(vc[at].cpu(), want[2])
    assert int(kc.view(torch.int16).count_nonzero()) == int(want[1].view(torch.int16).count_nonzero())
    del wide, rows
    # a fork's tail between the last blocks
    got = pa.fork_blocks(i32([-1, 0], cuda_device), i32([bs + 1, 0], cuda_device),
                         i32([[5, nb - 2], [-1, -1]], cuda_device), i32([2, 0], cuda_device),
                         torch.ones(nb, dtype=torch.int32, device=cuda_device), i32([nb - 3], cuda_device),
                         i32([0], cuda_device), kc, vc)
    assert got[3].tolist() == [[-1, -1], [nb - 2, nb - 3]] and pa.last_device_error() == 0
    assert torch.equal(kc[nb - 3, :, 0], kc[nb - 2, :, 0]) and torch.equal(vc[nb - 3, :, 0], vc[nb - 2, :, 0])
    assert int(kc[nb - 3, :, 1:].count_nonzero()) == 0 and int(kc[nb - 3].count_nonzero()) > 0


def test_tables_past_32_bits(cuda_device):
    """The last rows of a table of 2^31 entries and more."""
    n, width, bs, nb = 65535, 33000, 4, 1000
    tables = torch.full((n, width), -1, dtype=torch.int32, device=cuda_device)
    lens, held = torch.zeros(n, dtype=torch.int32), torch.zeros(n, dtype=torch.int32)
    lens[n - 1], held[n - 1], held[40000] = 9, 3, 2
    tables[n - 1, :3], tables[40000, :2] = i32([10, 11, 12], cuda_device), i32([20, 21], cuda_device)
    src = torch.full((n,), -1, dtype=torch.int32)
    src[n - 2] = n - 1
    counts = torch.zeros(nb, dtype=torch.int32, device=cuda_device)
    counts[[10, 11, 12, 20, 21]] = 1
    free, head = torch.arange(nb, dtype=torch.int32, device=cuda_device), i32([30], cuda_device)
    k, v = torch.randn(nb, 1, bs, 8, device=cuda_device), torch.randn(nb, 1, bs, 8, device=cuda_device)
    dev = lambda t: t.to(cuda_device)
    lens2, held2, head2, pairs = pa.fork_blocks(dev(src), dev(lens), tables, dev(held), counts, free, head, k, v)
    assert pa.last_device_error() == 0
    assert tables[n - 2, :4].tolist() == [10, 11, 30, -1] and pairs[n - 2].tolist() == [12, 30] and head2.tolist() == [31]
    assert counts[[10, 11, 12, 30]].tolist() == [2, 2, 1, 1] and torch.equal(k[30, :, :1], k[12, :, :1])
    held3, head3 = pa.release_blocks(dev(lens), tables, held2, free, head2, nb, bs, ref_cnt=counts)
    assert pa.last_device_error() == 0
    assert head3.tolist() == [28] and free[28:31].tolist() == [20, 21, 30]
    assert counts.sum() == 3 and held3[[40000, n - 2, n - 1]].tolist() == [0, 0, 3]


def test_logits_past_32_bits(cuda_device):
    """Rows of logits, draft and noise behind 2^31 elements, and a far stride."""
    n, vocab = 3, 5003
    for dtype, draft in ((BF, True), (F32, False)):
        b = VerifyBatch([4, 5, 3], vocab, dtype, seed=8, draft=draft, temps=[1.0, 0.0, 0.7])
        want = b.run(pa, cuda_device)
        total, far = b.logits.shape[0], 250_000_000     # 12 rows: 2.75e9 elements
        dev = lambda t: t.to(cuda_device)

        def apart(t, step):
            big = torch.empty((t.shape[0] - 1) * step + t.shape[1], dtype=t.dtype, device=cuda_device)
            rows = big.as_strided(t.shape, (step, 1))
            rows.copy_(t)
            return rows
        got = pa.verify_tree(apart(b.logits, far), dev(b.tokens), dev(b.parents), dev(b.start), dev(b.uniforms),
                             apart(b.noise, 1_200_000_000), b.max_q,
                             draft_logits=apart(b.draft, far + 1) if draft else None, temperature=dev(b.temps))
        assert pa.last_device_error() == 0
        assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
        del got
        torch.cuda.empty_cache()


@pytest.mark.parametrize("vocab", [1 << 30, (1 << 30) - 5])
def test_the_largest_vocabulary(cuda_device, vocab):
    """One row of 2^30 tokens: greedy, sampled, and a drafted token of half the weight."""
    g = torch.Generator(device="cuda").manual_seed(9)
    logits = torch.full((2, vocab), -30.0, dtype=BF, device=cuda_device)
    spots = [0, 7, vocab // 2 + 1, vocab - 2, vocab - 1]
    logits[0, spots] = torch.tensor([1.0, 0.0, 2.0, 4.0, 3.0], dtype=BF, device=cuda_device)
    logits[1, spots[2]] = 9.0
    noise = torch.full((1, vocab), 1.0, device=cuda_device)
    noise[0, spots] = torch.rand(5, device=cuda_device, generator=g) * 0.2 + 0.1
    child, start, par = i32([0, vocab - 2], cuda_device), i32([0, 2], cuda_device), i32([-1, 0], cuda_device)
    call = lambda u, heat: [int(x) for x in pa.verify_tree(
        logits, child, par, start, torch.tensor([0.0, u], device=cuda_device), noise, 2,
        temperature=torch.tensor([heat], device=cuda_device))]
    assert call(0.5, 0.0) == [1, spots[2]]
    # 2^30 weights of e^-34 are 1.8e-6 of the largest
    p = torch.softmax(torch.tensor([1.0, 0.0, 2.0, 4.0, 3.0]).double(), 0)
    assert call(float(p[3]) - 1e-4, 1.0) == [1, spots[2]]
    race = p / noise[0, spots].cpu().double()
    race[3] = 0.0
    assert call(float(p[3]) + 1e-4, 1.0) == [0, spots[int(race.argmax())]]
    assert pa.last_device_error() == 0


# ---- the first calls of a process ----------------------------------------------------------------

FIRST = """
import torch
import paged_kv_cache_109_gb300 as pa
dev = torch.device("cuda:0")
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
kc, vc = (torch.zeros(16, 2, 4, 64, device=dev) for _ in range(2))
q, k, v = (torch.randn(3, h, 64, device=dev) for h in (4, 2, 2))
pos, inv, slots = i32([0, 1, 2]), torch.ones(32, device=dev), torch.arange(3, device=dev)
logits, noise, u = torch.randn(4, 50, device=dev), torch.rand(2, 50, device=dev) + 0.1, torch.rand(4, device=dev)
tokens, parents, start = i32([0, 1, 0, 2]), i32([-1, 0, -1, 0]), i32([0, 2, 4])
src, lens, held = i32([-1, 0]), i32([6, 0]), i32([2, 0])
table, counts, free, head = i32([[0, 1], [-1, -1]]), i32([1, 1] + [0] * 14), i32(range(16)), i32([2])
def step():
    out = pa.rope_write(q, k, v, pos, inv, slots, kc, vc)
    leaf, token = pa.verify_tree(logits, tokens, parents, start, u, noise, 2, draft_logits=logits)
    _, held2, head2, pairs = pa.fork_blocks(src, lens, table, held, counts, free, head, kc, vc)
    held3, head3 = pa.release_blocks(lens, table, held2, free, head2, 16, 4, ref_cnt=counts)
    return [out, leaf, token, pairs, held3, head3]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
assert pa.last_device_error() == 0 and got[3].tolist() == [[-1, -1], [1, 2]] and got[5].tolist() == [2]
for x, y in zip(got, step()):
    assert torch.equal(x, y)
print("same")
"""


def test_the_first_calls_of_a_process_may_be_captured(cuda_device):
    done = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.split() == ["same"], done.stderr[-2000:]
