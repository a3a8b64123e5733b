"""The drafted (speculative) step on the GPU: pa_plan_step against the host
block pool, pa_decode_tree against attention in 64 bits, pa_accept_tree bit
for bit, and the three together in a captured step."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_109_gb300 as pa
from tests._draft import (Batch, PlanState, accept_reference, assert_tree_close, path_of,
                          plan_reference, random_parents, tree_reference)

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def clear_device_error(cuda_device):
    pa.last_device_error()
    yield


# ---- pa_plan_step --------------------------------------------------------------------

def _plan(dev, st, new, head=0, max_tokens=None, extra_free=0, in_place=False, ref_cnt=None,
          free=None):
    """Runs the plan on device copies; returns every output as lists."""
    front = [0] * head
    free = torch.tensor(front + (st.free if free is None else free), dtype=torch.int32, device=dev)
    lens = torch.tensor(st.lens, dtype=torch.int32, device=dev)
    held = torch.tensor(st.held, dtype=torch.int32, device=dev)
    hd = torch.tensor([head], dtype=torch.int32, device=dev)
    tables = st.tables.to(dev)
    tokens = sum(new) if max_tokens is None else max_tokens
    plan = pa.StepPlan.empty(len(st.lens), tokens, dev)
    if in_place:
        plan.seq_lens, plan.blocks_held, plan.free_head = lens, held, hd
    got = pa.plan_step(lens, torch.tensor(new, dtype=torch.int32, device=dev), tables, held, free,
                       hd, st.num_blocks, st.bs, plan, ref_cnt=ref_cnt)
    torch.cuda.synchronize()
    assert got is plan
    out = {k: getattr(plan, k).tolist() for k in pa.StepPlan.__slots__}
    out["tables"] = tables.tolist()
    return out


@pytest.mark.parametrize("n,bs,new_hi,head,in_place", [
    (1, 16, 1, 0, False), (1, 16, 0, 0, True), (3, 1, 5, 2, True), (31, 8, 64, 0, False),
    (33, 16, 1, 7, True), (256, 16, 1, 0, False), (257, 4, 40, 3, True),
    (1023, 24, 9, 0, False), (1025, 64, 130, 1, True), (2500, 16, 17, 5, False),
])
def test_plan_matches_the_pool(cuda_device, n, bs, new_hi, head, in_place):
    rng = np.random.default_rng(n * bs + new_hi)
    lens = rng.integers(0, 5 * bs + 3, n).tolist()
    extra = rng.integers(0, 3, n).tolist()
    new = rng.integers(0, new_hi + 1, n).tolist()
    if n > 2:
        lens[1], new[1] = 0, 0
    width = max(-(-(a + new_hi) // bs) for a in lens) + 4
    blocks = sum(-(-(a + new_hi) // bs) + 3 for a in lens)
    st = PlanState(lens, extra, bs, blocks, width, seed=n)
    max_tokens = sum(new) + int(rng.integers(0, 300))
    got = _plan(cuda_device, st, new, head, max_tokens, in_place=in_place)
    assert pa.last_device_error() == 0
    ref = plan_reference(st, new, head, max_tokens)
    for k in ref:
        assert got[k] == [list(r) if isinstance(r, tuple) else r for r in ref[k]], k


def test_plan_prompts_of_many_tiles(cuda_device):
    """Long chunks: tokens and fresh blocks past one tile of the fill."""
    rng = np.random.default_rng(3)
    lens, new = [0, 5000, 31], [70001, 0, 4097]
    st = PlanState(lens, [0, 1, 0], 16, 6000, 4500, seed=1)
    got = _plan(cuda_device, st, new, 0, sum(new) + 5)
    assert pa.last_device_error() == 0
    ref = plan_reference(st, new, 0, sum(new) + 5)
    for k in ref:
        assert got[k] == ref[k], k
    assert rng is not None


@pytest.mark.parametrize("n,new", [
    (1, {0: 9001}), (2, {1: 8999}), (33, {0: 5000, 32: 4003}),
    # runs of sequences without tokens at the front, inside and at the end
    (1025, {1024: 3}), (1057, {0: 1, 512: 2, 513: 300}), (2500, {700: 1, 1500: 140, 1501: 1}),
    (1500, {i: 1 for i in range(0, 1500, 7)}), (1030, {}),
])
def test_plan_of_few_sequences_with_tokens(cuda_device, n, new):
    """Plans past the one-launch form: a warp's tokens of one sequence, of many,
    and of sequences that others without tokens lie between."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 60, n).tolist()
    counts = [new.get(i, 0) for i in range(n)]
    width = max(-(-(a + c) // 16) for a, c in zip(lens, counts)) + 2
    blocks = sum(-(-(a + c) // 16) for a, c in zip(lens, counts)) + n + 3
    st = PlanState(lens, rng.integers(0, 2, n).tolist(), 16, blocks, width, seed=n)
    max_tokens = max(sum(counts) + 7, 1)
    got = _plan(cuda_device, st, counts, 0, max_tokens)
    assert pa.last_device_error() == 0
    ref = plan_reference(st, counts, 0, max_tokens)
    for k in ref:
        assert got[k] == [list(r) if isinstance(r, tuple) else r for r in ref[k]], k


def _unplanned(st, got, head, max_tokens):
    n = len(st.lens)
    assert got["tables"] == st.tables.tolist()
    assert got["seq_lens"] == st.lens and got["blocks_held"] == st.held
    assert got["free_head"] == [head]
    assert got["query_start_loc"] == [0] * (n + 1) == got["block_start"]
    for k in ("slot_mapping", "positions", "seq_ids"):
        assert got[k] == [-1] * max_tokens


@pytest.mark.parametrize("why", ["pool", "tokens", "table", "negative", "held", "shared"])
@pytest.mark.parametrize("n", [3, 1500])
def test_plan_that_does_not_fit_plans_nothing(cuda_device, why, n):
    bs, lens, new = 4, [6, 8, 1] + [3] * (n - 3), [4, 3, 2] + [1] * (n - 3)
    st = PlanState(lens, [0] * n, bs, 4 * n + 8, 4, seed=5)
    tokens, bit, ref_cnt, free = sum(new), pa.DEVERR_SEQ_LEN, None, None
    if why == "pool":
        free, bit = st.free[:1], pa.DEVERR_POOL      # 10 and 11 tokens: one block more each
    elif why == "tokens":
        tokens -= 1
    elif why == "table":
        new[2] = 17                                    # 18 tokens, 4 blocks of 4 in a row
        tokens = sum(new)
    elif why == "negative":
        new[1], tokens = -1, sum(new) + 8
    elif why == "held":
        st.held[0] = 1                                 # 6 tokens need 2 blocks
    elif why == "shared":
        ref_cnt = torch.tensor(st.pool.ref_cnt, dtype=torch.int32, device=cuda_device)
        ref_cnt[int(st.tables[0, 1])] = 2              # the first sequence's tail
        bit = pa.DEVERR_SHARED
    before = None if ref_cnt is None else ref_cnt.clone()
    got = _plan(cuda_device, st, new, 0, tokens, ref_cnt=ref_cnt, free=free)
    assert pa.last_device_error() == bit
    _unplanned(st, got, 0, tokens)
    if ref_cnt is not None:
        assert torch.equal(ref_cnt, before)


def test_plan_counts_taken_blocks_and_ignores_a_full_shared_tail(cuda_device):
    st = PlanState([8, 3], [0, 0], 4, 12, 5, seed=2)
    ref = torch.tensor(st.pool.ref_cnt, dtype=torch.int32, device=cuda_device)
    ref[int(st.tables[0, 1])] = 2                      # full: nothing is appended into it
    got = _plan(cuda_device, st, [5, 1], 0, ref_cnt=ref)
    assert pa.last_device_error() == 0
    assert got["blocks_held"] == [4, 1]
    want = list(st.pool.ref_cnt)
    want[int(st.tables[0, 1])] = 2
    for b in st.free[:2]:
        want[b] = 1
    assert ref.tolist() == want


def test_plan_bad_ids_lose_their_tokens_only(cuda_device):
    st = PlanState([2, 2, 2], [0, 0, 0], 4, 12, 3, seed=4)
    st.tables[1, 0] = 99                               # an existing block outside the pool
    free = list(st.free)
    free[0] = -5                                       # the first sequence's fresh block
    got = _plan(cuda_device, st, [4, 1, 1], 0, free=free)
    assert pa.last_device_error() == pa.DEVERR_TABLE_ENTRY
    b = int(st.tables[0, 0])
    assert got["slot_mapping"] == [b * 4 + 2, b * 4 + 3, -1, -1, -1, int(st.tables[2, 0]) * 4 + 2]
    assert got["tables"][0][1] == -1


def test_plan_without_sequences(cuda_device):
    st = PlanState([], [], 4, 6, 2, seed=1)
    st.tables = torch.zeros(0, 2, dtype=torch.int32)
    got = _plan(cuda_device, st, [], 3, max_tokens=5)
    assert pa.last_device_error() == 0
    assert got["free_head"] == [3] and got["query_start_loc"] == [0] == got["block_start"]
    assert got["slot_mapping"] == got["positions"] == got["seq_ids"] == [-1] * 5


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("n,most", [(5, 40), (3000, 30000)])
def test_plan_into_unaligned_buffers_of_odd_sizes(cuda_device, offset, n, most):
    """Token buffers that start off a 16-byte boundary, positions and ids left
    out, and neighbours of the buffers untouched."""
    rng = np.random.default_rng(n + offset)
    lens, new = rng.integers(0, 50, n).tolist(), rng.integers(0, 9, n).tolist()
    st = PlanState(lens, [0] * n, 8, 10 * n, 9, seed=n)
    tokens = most + offset
    plan = pa.StepPlan.empty(n, tokens, cuda_device)
    slots = torch.full((tokens + 8,), 77, dtype=torch.int64, device=cuda_device)
    plan.slot_mapping, plan.positions, plan.seq_ids = slots[offset:offset + tokens], None, None
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    tables = st.tables.to(cuda_device)
    pa.plan_step(dev(lens), dev(new), tables, dev(st.held), dev(st.free), dev([0]), st.num_blocks, 8,
                 plan)
    torch.cuda.synchronize()
    assert pa.last_device_error() == 0
    ref = plan_reference(st, new, 0, tokens)
    assert plan.slot_mapping.tolist() == ref["slot_mapping"] and tables.tolist() == ref["tables"]
    assert (slots[:offset] == 77).all() and (slots[offset + tokens:] == 77).all()


@pytest.mark.parametrize("n", [4096, 4097, 20000, 65535])
def test_plan_of_many_sequences(cuda_device, n):
    """Past one round of the scan: sums against torch's."""
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 60, (n,), generator=g, dtype=torch.int32)
    new = torch.randint(0, 4, (n,), generator=g, dtype=torch.int32)
    held = (lens + 7) // 8
    need = torch.maximum(held, (lens + new + 7) // 8)
    blocks = int(need.sum())
    tables = torch.full((n, 9), -1, dtype=torch.int32)
    perm = torch.randperm(blocks, generator=g).int()
    used = torch.arange(9) < held[:, None]
    tables[used] = perm[:int(held.sum())]
    free = perm[int(held.sum()):].contiguous()
    dev = [x.to(cuda_device) for x in (lens, new, tables, held, free)]
    plan = pa.plan_step(*dev, torch.zeros(1, dtype=torch.int32, device=cuda_device), blocks, 8,
                        max_tokens=int(new.sum()))
    torch.cuda.synchronize()
    assert pa.last_device_error() == 0
    start = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
    assert torch.equal(plan.query_start_loc.cpu().long(), start)
    assert int(plan.free_head) == free.numel()
    fresh = (torch.arange(9) >= held[:, None]) & (torch.arange(9) < need[:, None])
    tables[fresh] = free
    assert torch.equal(dev[2].cpu(), tables)
    seq = torch.repeat_interleave(torch.arange(n), new.long())
    pos = lens[seq] + torch.arange(seq.numel()) - start[seq]
    slot = tables[seq, pos // 8].long() * 8 + pos % 8
    assert torch.equal(plan.slot_mapping.cpu(), slot)
    assert torch.equal(plan.positions.cpu().long(), pos) and torch.equal(plan.seq_ids.cpu().long(), seq)


# ---- pa_decode_tree ----------------------------------------------------------------------

# kv heads, group, head dim, block size, dtype
SHAPES = [
    (2, 4, 128, 16, BF), (1, 8, 128, 32, BF), (4, 1, 64, 16, BF), (2, 5, 96, 24, BF),
    (2, 2, 80, 8, BF), (1, 16, 64, 64, BF), (2, 3, 112, 40, BF), (1, 4, 16, 16, BF),
    (1, 7, 48, 8, BF), (1, 33, 128, 16, BF), (1, 128, 64, 16, BF), (1, 200, 64, 16, BF),
    (1, 4, 128, 48, BF), (1, 2, 64, 96, BF), (1, 3, 128, 256, BF), (1, 2, 64, 512, BF),
    (2, 2, 256, 16, BF), (1, 1, 144, 16, BF), (1, 20, 256, 16, BF), (1, 9, 128, 4, BF),
    (1, 2, 8, 16, BF), (1, 40, 72, 16, BF), (2, 2, 64, 4, BF), (1, 3, 32, 5, BF),
    (1, 3, 20, 5, BF), (1, 2, 72, 16, BF),
    (2, 4, 128, 16, F32), (1, 3, 64, 24, F32), (1, 1, 256, 16, F32), (2, 2, 20, 5, F32),
    (1, 2, 7, 3, F32), (1, 70, 36, 16, F32), (1, 20, 16, 8, F32), (1, 9, 200, 16, F32),
    (1, 12, 128, 1, F32),
]


@pytest.mark.parametrize("hkv,group,d,bs,dtype", SHAPES)
def test_tree_matches_64_bits(cuda_device, hkv, group, d, bs, dtype):
    ctx = [0, 0, 1, bs, 127, 128, 129, 300, 65, 2 * bs - 1]
    nodes = [1, 7, 1, 3, 2, 33, 5, 1, 0, 16]
    if group * hkv > 64:
        ctx, nodes = [0, 130, 61], [3, 5, 2]
    b = Batch(ctx, nodes, hkv, group, d, bs, dtype, seed=hkv * d + bs + group)
    got = b.run(pa, cuda_device)
    torch.cuda.synchronize()
    assert pa.last_device_error() == 0
    ref, bound = tree_reference(b)
    assert_tree_close(got, ref, bound, dtype)


@pytest.mark.parametrize("kind", ["chain", "star", "forest", "mixed"])
@pytest.mark.parametrize("nodes", [64, 129, 200, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_shapes_up_to_the_largest(cuda_device, kind, nodes, dtype):
    b = Batch([0, 77, 190], [nodes, 1, max(1, nodes - 3)], 1, 2, 64, 16, dtype, seed=nodes,
              kind=kind)
    got = b.run(pa, cuda_device)
    torch.cuda.synchronize()
    assert pa.last_device_error() == 0
    ref, bound = tree_reference(b)
    assert_tree_close(got, ref, bound, dtype, kind)


@pytest.mark.parametrize("dtype,d,bs", [(BF, 128, 16), (BF, 64, 8), (BF, 256, 16), (F32, 64, 16)])
def test_long_contexts_in_one_batch_with_short_ones(cuda_device, dtype, d, bs):
    """Work of one sequence split over the GPU next to sequences of a few keys."""
    b = Batch([9000, 0, 3, 2500, 129], [3, 2, 1, 9, 4], 2, 2, d, bs, dtype, seed=d)
    got = b.run(pa, cuda_device)
    again = b.run(pa, cuda_device)
    torch.cuda.synchronize()
    assert pa.last_device_error() == 0
    ref, bound = tree_reference(b)
    assert_tree_close(got, ref, bound, dtype)
    assert torch.equal(got.view(torch.uint8), again.view(torch.uint8))


def test_many_short_sequences(cuda_device):
    rng = np.random.default_rng(0)
    b = Batch(rng.integers(0, 40, 700).tolist(), rng.integers(0, 4, 700).tolist(), 2, 2, 64, 16,
              BF, seed=9)
    got = b.run(pa, cuda_device)
    torch.cuda.synchronize()
    ref, bound = tree_reference(b)
    assert_tree_close(got, ref, bound, BF)


@pytest.mark.parametrize("dtype,d,bs", [(BF, 128, 16), (BF, 256, 16), (F32, 64, 16), (F32, 20, 5)])
def test_chain_is_prefill_and_single_node_is_decode(cuda_device, dtype, d, bs):
    b = Batch([0, 50, 400], [9, 1, 30], 2, 4, d, bs, dtype, seed=1, kind="chain")
    q, start, parents, k, v, tables, lens = b.to(cuda_device)
    got = b.run(pa, cuda_device)
    pre = pa.prefill(q, start, k, v, tables, lens, b.max_q, b.max_len, b.scale)
    ref, bound = tree_reference(b)
    assert_tree_close(got, ref, bound, dtype)
    assert_tree_close(pre, ref, bound, dtype)
    one = Batch([0, 50, 400], [1, 1, 1], 2, 4, d, bs, dtype, seed=2)
    q, start, parents, k, v, tables, lens = one.to(cuda_device)
    ref, bound = tree_reference(one)
    assert_tree_close(one.run(pa, cuda_device), ref, bound, dtype)
    assert_tree_close(pa.decode(q, k, v, tables, lens, one.max_len, one.scale), ref, bound, dtype)
    assert pa.last_device_error() == 0


@pytest.mark.parametrize("hkv,group,d,bs,dtype", [(1, 4, 128, 16, BF), (1, 1, 64, 8, BF),
                                                  (1, 2, 256, 16, BF), (1, 2, 64, 16, F32),
                                                  (1, 2, 20, 5, F32), (1, 64, 128, 16, BF)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_keys_a_node_does_not_see_leave_no_trace(cuda_device, hkv, group, d, bs, dtype, bad):
    """One node's K and V hold NaN, infinities or the type's largest values:
    the rows that see it have the formula's value, the others do not change."""
    for hit in ("v", "k"):
        b = Batch([37, 200], [8, 40], hkv, group, d, bs, dtype, seed=11)
        node = [3, 17]
        for i in range(2):
            p = b.ctx[i] + node[i]
            blk, off = int(b.tables[i, p // bs]), p % bs
            if hit == "v":
                b.v[blk, :, off, 1::3] = bad
            else:
                b.k[blk, :, off] = bad
        got = b.run(pa, cuda_device).double().cpu()
        torch.cuda.synchronize()
        ref, bound = tree_reference(b)
        for i in range(2):
            for j in range(b.nodes[i]):
                r = int(b.start[i]) + j
                sees = node[i] in path_of(b.par[i], j)
                if not sees:
                    assert torch.isfinite(got[r]).all(), (hit, r)
                    assert_tree_close(got[r], ref[r], bound[r], dtype, f"{hit} {r}")
                elif hit == "v" and not math.isfinite(bad):
                    # visible: NaN and infinities where the formula has them
                    assert torch.equal(torch.isnan(got[r]), torch.isnan(ref[r]))
                    assert torch.equal(torch.isinf(got[r]), torch.isinf(ref[r]))
                    fine = torch.isfinite(ref[r])
                    assert_tree_close(got[r][fine], ref[r][fine], bound[r][fine], dtype)


def test_visible_infinities_of_both_signs_are_nan(cuda_device):
    b = Batch([20], [4], 1, 2, 128, 16, BF, seed=3, kind="chain")
    for j, x in ((0, float("inf")), (2, -float("inf"))):
        p = 20 + j
        b.v[int(b.tables[0, p // 16]), :, p % 16, 5] = x
    got = b.run(pa, cuda_device).float().cpu()
    assert torch.isinf(got[:2, :, 5]).all() and (got[:2, :, 5] > 0).all()
    assert torch.isnan(got[2:, :, 5]).all()
    keep = [c for c in range(128) if c != 5]
    assert torch.isfinite(got[..., keep]).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.5])
@pytest.mark.parametrize("dtype,d", [(BF, 64), (F32, 64), (F32, 20)])
def test_scales(cuda_device, scale, dtype, d):
    b = Batch([50, 200], [5, 12], 1, 3, d, 16 if d == 64 else 5, dtype, seed=8, scale=scale)
    got = b.run(pa, cuda_device)
    ref, bound = tree_reference(b)
    assert_tree_close(got, ref, bound, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_behind_and_refused_sequences_are_left_untouched(cuda_device, dtype):
    b = Batch([30, 10, 20], [4, 6, 3], 1, 2, 64, 16, dtype, seed=6)
    q, start, parents, k, v, tables, lens = b.to(cuda_device)
    ref, bound = tree_reference(b)
    pad = 9
    q = torch.cat([q, torch.full_like(q[:pad], float("nan"))])
    parents = torch.cat([parents, torch.full((pad,), 1000, dtype=torch.int32, device=cuda_device)])

    def run(start, lens, max_q=6, max_len=34):
        out = torch.full_like(q, 7.0)
        pa.decode_tree(q, start, parents, k, v, tables, lens, max_q, max_len, b.scale, out=out)
        torch.cuda.synchronize()
        return out.double().cpu()

    def expect(out, seqs):
        for i in range(3):
            rows = slice(int(b.start[i]), int(b.start[i + 1]))
            if i in seqs:
                assert_tree_close(out[rows], ref[rows], bound[rows], dtype)
            else:
                assert (out[rows] == 7.0).all()
        assert (out[b.total:] == 7.0).all()

    expect(run(start, lens), (0, 1, 2))
    assert pa.last_device_error() == 0
    expect(run(start, lens, max_q=5), (0, 2))                  # six nodes, bound five
    assert pa.last_device_error() == pa.DEVERR_SEQ_LEN
    bad = lens.clone()
    bad[1] = 5                                                  # fewer keys than nodes
    expect(run(start, bad), (0, 2))
    assert pa.last_device_error() == pa.DEVERR_SEQ_LEN
    bad[1] = 35                                                 # past max_seq_len
    expect(run(start, bad), (0, 2))
    assert pa.last_device_error() == pa.DEVERR_SEQ_LEN
    bad[1] = -1
    expect(run(start, bad), (0, 2))
    assert pa.last_device_error() == pa.DEVERR_SEQ_LEN
    late = start.clone()
    late[3] = b.total + pad + 1                                 # rows past total_q
    expect(run(late, lens, max_q=20), (0, 1))
    assert pa.last_device_error() == pa.DEVERR_SEQ_LEN


@pytest.mark.parametrize("dtype,d,bs", [(BF, 64, 16), (BF, 256, 16), (F32, 64, 16), (F32, 20, 5)])
def test_bad_parents_and_table_entries_are_reported(cuda_device, dtype, d, bs):
    b = Batch([30, 150], [6, 7], 1, 2, d, bs, dtype, seed=6, kind="chain")
    for wrong in (4, 9, -2):
        c = b.parents.clone()
        c[3] = wrong if wrong != 4 else 3                       # itself, past it, below -1
        q, start, _, k, v, tables, lens = b.to(cuda_device)
        got = pa.decode_tree(q, start, c.to(cuda_device), k, v, tables, lens, b.max_q, b.max_len,
                             b.scale)
        assert pa.last_device_error() == pa.DEVERR_TREE
        keep, b.par[0][3] = b.par[0][3], -1
        ref, bound = tree_reference(b)
        assert_tree_close(got, ref, bound, dtype)
        b.par[0][3] = keep
    ref, bound = tree_reference(b)
    for entry in (-1, b.k.shape[0]):
        bad = b.tables.clone()
        bad[0, 0] = entry
        q, start, parents, k, v, _, lens = b.to(cuda_device)
        got = pa.decode_tree(q, start, parents, k, v, bad.to(cuda_device), lens, b.max_q,
                             b.max_len, b.scale)
        assert pa.last_device_error() == pa.DEVERR_TABLE_ENTRY
        assert_tree_close(got[6:], ref[6:], bound[6:], dtype)


def test_pinned_arguments_and_unaligned_queries(cuda_device):
    b = Batch([40, 3], [5, 2], 2, 2, 64, 16, BF, seed=12)
    ref, bound = tree_reference(b)
    k, v = b.k.to(cuda_device), b.v.to(cuda_device)
    pin = [x.pin_memory() for x in (b.q, b.start, b.parents, b.tables, b.lens)]
    out = torch.empty(b.q.shape, dtype=BF).pin_memory()
    pa.decode_tree(pin[0], pin[1], pin[2], k, v, pin[3], pin[4], b.max_q, b.max_len, b.scale,
                   out=out)
    torch.cuda.synchronize()
    assert_tree_close(out, ref, bound, BF)
    store = torch.empty(b.q.numel() + 1, dtype=BF, device=cuda_device)
    q = store[1:].view(b.q.shape)                               # 2-byte aligned
    q.copy_(b.q)
    got = pa.decode_tree(q, *b.to(cuda_device)[1:], b.max_q, b.max_len, b.scale)
    assert_tree_close(got, ref, bound, BF)
    store = torch.empty(b.k.numel() + 1, dtype=BF, device=cuda_device)
    k = store[1:].view(b.k.shape)
    k.copy_(b.k)
    args = b.to(cuda_device)
    args[3] = k
    assert_tree_close(pa.decode_tree(*args, b.max_q, b.max_len, b.scale), ref, bound, BF)


@pytest.mark.parametrize("n,d,dtype", [(129, 64, BF), (20000, 64, BF), (20000, 20, F32),
                                       (65535, 16, BF)])
def test_batches_of_many_sequences(cuda_device, n, d, dtype):
    """Every sequence one node on one cached token: a mean of two value rows
    weighted by two scores."""
    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.randn(n, 1, 8, d, generator=g, device=cuda_device).to(dtype)
    v = torch.randn(n, 1, 8, d, generator=g, device=cuda_device).to(dtype)
    q = torch.randn(n, 1, d, generator=g, device=cuda_device).to(dtype)
    i32 = lambda *a: torch.arange(*a, dtype=torch.int32, device=cuda_device)  # noqa: E731
    lens = torch.full((n,), 2, dtype=torch.int32, device=cuda_device)
    got = pa.decode_tree(q, i32(n + 1), torch.full_like(lens, -1), k, v, i32(n)[:, None].contiguous(),
                         lens, 1, 8)
    torch.cuda.synchronize()
    assert pa.last_device_error() == 0
    kk, vv, qq = k[:, 0, :2].double(), v[:, 0, :2].double(), q.double()
    s = (qq @ kk.transpose(1, 2)) / math.sqrt(d)
    p = torch.softmax(s, 2)
    ref = p @ vv
    # as tree_reference's bound, with one ds for all rows
    ds = (d + 4) * 2.0 ** -24 / math.sqrt(d) * float((qq.abs() @ kk.abs().transpose(1, 2)).max())
    bound = (p @ vv.abs()) * (2 * ds + 4 * 2.0 ** -24 + 2.0 ** -19 + (2.0 ** -15 if dtype == BF else 0))
    assert_tree_close(got, ref.cpu(), bound.cpu(), dtype)


def test_positions_of_one_block_shared_by_a_long_table(cuda_device):
    """A table whose rows all name one block: 400,000 positions over 16 rows of
    keys give the softmax over those 16, whatever the split."""
    d, bs, blocks = 64, 16, 25000
    g = torch.Generator().manual_seed(5)
    k = torch.randn(2, 1, bs, d, generator=g).to(BF)
    v = torch.randn(2, 1, bs, d, generator=g).to(BF)
    q = torch.randn(1, 2, d, generator=g).to(BF)
    tables = torch.zeros(1, blocks + 1, dtype=torch.int32)
    tables[0, -1] = 1
    lens = torch.tensor([blocks * bs + 1], dtype=torch.int32)
    dev = [x.to(cuda_device) for x in (q, torch.tensor([0, 1], dtype=torch.int32),
                                       torch.tensor([-1], dtype=torch.int32), k, v, tables, lens)]
    got = pa.decode_tree(*dev, 1, int(lens[0])).double().cpu()
    s = torch.cat([k[0, 0].double(), k[1, 0, :1].double()]) @ q[0].double().T / math.sqrt(d)
    w = torch.exp(s) * torch.tensor([float(blocks)] * bs + [1.0], dtype=torch.float64)[:, None]
    vv = torch.cat([v[0, 0].double(), v[1, 0, :1].double()])
    p = w / w.sum(0)
    ds = (d + 4) * 2.0 ** -24 / 8 * float((k[0, 0].double().abs() @ q[0].double().abs().T).max())
    # 400,001 keys: sums of 128 a block, the rest as that many rounded additions
    n = int(lens[0]) / 128 + 128
    bound = (p.T @ vv.abs()) * (2 * ds + 2 * n * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** -15)
    assert_tree_close(got[0], p.T @ vv, bound, BF)


def test_unaligned_outputs_of_cut_units(cuda_device):
    b = Batch([5000, 40], [5, 2], 1, 2, 64, 16, BF, seed=12)
    ref, bound = tree_reference(b)
    store = torch.full((b.q.numel() + 2,), 7.0, dtype=BF, device=cuda_device)
    out = store[1:-1].view(b.q.shape)                           # 2-byte aligned
    pa.decode_tree(*b.to(cuda_device), b.max_q, b.max_len, b.scale, out=out)
    torch.cuda.synchronize()
    assert_tree_close(out, ref, bound, BF)
    assert float(store[0]) == 7.0 == float(store[-1])


def test_side_streams_own_what_a_call_allocates(cuda_device):
    """Calls on a stream that is not the current one, their workspaces dropped
    at once while the current stream allocates."""
    b = Batch([6000, 900], [6, 9], 2, 4, 128, 16, BF, seed=4)
    ref, bound = tree_reference(b)
    args = b.to(cuda_device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for s in (side, side.cuda_stream, side):
        outs.append(pa.decode_tree(*args, b.max_q, b.max_len, b.scale, stream=s))
        torch.full((64 << 20,), float("nan"), device=cuda_device)
    leaf = torch.tensor([5, 8], dtype=torch.int32, device=cuda_device)
    side.wait_stream(torch.cuda.current_stream())
    lens, rows = pa.accept_tree(leaf, args[2], args[1], args[6], args[3], args[4], args[5], b.max_q,
                                stream=side)
    torch.cuda.synchronize()
    for out in outs:
        assert_tree_close(out, ref, bound, BF)
    want = accept_reference(b, [5, 8], b.k, b.v)
    assert torch.equal(lens.cpu(), want[0]) and torch.equal(rows.cpu(), want[1])


def test_two_calls_at_once_with_their_own_workspaces(cuda_device):
    bs = [Batch([3000, 100], [6, 9], 2, 4, 128, 16, BF, seed=s) for s in (1, 2)]
    refs = [tree_reference(b) for b in bs]
    args = [b.to(cuda_device) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    ws = [torch.empty(max(1, pa.decode_tree_workspace_bytes(
        2, b.total, 8, b.max_q, b.max_len, b.k)), dtype=torch.uint8, device=cuda_device)
        for b in bs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        outs = [pa.decode_tree(*a, b.max_q, b.max_len, b.scale, workspace=w, stream=s)
                for a, b, w, s in zip(args, bs, ws, streams)]
    torch.cuda.synchronize()
    for out, (ref, bound) in zip(outs, refs):
        assert_tree_close(out, ref, bound, BF)


# ---- pa_accept_tree ------------------------------------------------------------------------

@pytest.mark.parametrize("hkv,d,bs,dtype,layers", [
    (8, 128, 16, BF, 1), (2, 64, 8, BF, 3), (3, 80, 24, F32, 2), (1, 7, 3, F32, 1),
    (1, 5, 4, BF, 2), (1, 1, 1, BF, 1), (2, 20, 5, BF, 130),
])
@pytest.mark.parametrize("kind", ["mixed", "chain", "star"])
def test_accept_moves_the_path(cuda_device, hkv, d, bs, dtype, layers, kind):
    ctx, nodes = [0, 5, 31, 64, 100, 7], [1, 9, 64, 256, 0, 30]
    b = Batch(ctx, nodes, hkv, 1, d, bs, dtype, seed=d + layers, kind=kind)
    rng = np.random.default_rng(1)
    leaf = [0, 8, 63, 255, -1, int(rng.integers(0, 30))]
    g = torch.Generator().manual_seed(4)
    ks = [torch.randn(b.k.shape, generator=g).to(dtype) for _ in range(layers)]
    vs = [torch.randn(b.k.shape, generator=g).to(dtype) for _ in range(layers)]
    _, start, parents, _, _, tables, lens = b.to(cuda_device)
    kd, vd = [x.to(cuda_device) for x in ks], [x.to(cuda_device) for x in vs]
    got = pa.accept_tree(torch.tensor(leaf, dtype=torch.int32, device=cuda_device), parents, start,
                         lens, kd, vd, tables, b.max_q)
    torch.cuda.synchronize()
    assert pa.last_device_error() == 0
    for k, v, kk, vv in zip(ks, vs, kd, vd):
        ref = accept_reference(b, leaf, k, v)
        assert torch.equal(kk.cpu().view(torch.uint8), k.view(torch.uint8))
        assert torch.equal(vv.cpu().view(torch.uint8), v.view(torch.uint8))
    assert torch.equal(got[0].cpu(), ref[0]) and torch.equal(got[1].cpu(), ref[1])


def test_accept_stacked_layers_and_unaligned_caches(cuda_device):
    b = Batch([10, 3], [12, 6], 2, 1, 64, 8, BF, seed=2)
    leaf = [11, 4]
    store = torch.randn(2, b.k.numel() * 3 + 1).to(BF)
    _, start, parents, _, _, tables, lens = b.to(cuda_device)
    for off in (0, 1):
        k = store[0, off:off + b.k.numel() * 3].view(3, *b.k.shape).clone()
        v = store[1, off:off + b.k.numel() * 3].view(3, *b.k.shape).clone()
        dev = store.to(cuda_device)
        kd = dev[0, off:off + b.k.numel() * 3].view(k.shape)
        vd = dev[1, off:off + b.k.numel() * 3].view(k.shape)
        pa.accept_tree(torch.tensor(leaf, dtype=torch.int32, device=cuda_device), parents, start,
                       lens, kd, vd, tables, b.max_q)
        torch.cuda.synchronize()
        for l in range(3):
            accept_reference(b, leaf, k[l], v[l])
        assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)


def test_accept_reports_and_skips(cuda_device):
    b = Batch([10, 3, 8], [5, 6, 4], 2, 1, 64, 8, BF, seed=2, kind="chain")
    _, start, parents, k, v, tables, lens = b.to(cuda_device)
    k0, v0 = k.clone(), v.clone()

    def run(leaf, parents=parents, lens=lens, tables=tables, max_q=6):
        got = pa.accept_tree(torch.tensor(leaf, dtype=torch.int32, device=cuda_device), parents,
                             start, lens, k, v, tables, max_q)
        torch.cuda.synchronize()
        return got[0].tolist(), got[1].tolist(), pa.last_device_error()

    same = lambda: torch.equal(k.view(torch.uint8), k0.view(torch.uint8)) and torch.equal(  # noqa: E731
        v.view(torch.uint8), v0.view(torch.uint8))
    new, rows, err = run([5, 6, -2])                            # all outside their trees
    assert (new, err) == ([10, 3, 8], pa.DEVERR_TREE) and rows == [-1] * 15 and same()
    new, rows, err = run([4, 5, 3])                             # whole chains: nothing moves
    assert (new, err) == ([15, 9, 12], 0) and rows == list(range(15)) and same()
    bad = parents.clone()
    bad[7] = 2                                                  # node 2 continues itself
    new, rows, err = run([4, 5, 3], parents=bad)
    assert (new, err) == ([15, 3, 12], pa.DEVERR_TREE) and rows[5:11] == [-1] * 6 and same()
    short = lens.clone()
    short[1] = 4
    new, rows, err = run([0, 0, 0], lens=short)
    assert (new[0], new[1], new[2], err) == (11, 4, 9, pa.DEVERR_SEQ_LEN) and same()
    new, rows, err = run([0, 0, 0], max_q=5)
    assert (new[0], new[1], new[2], err) == (11, 9, 9, pa.DEVERR_SEQ_LEN) and same()
    star = torch.full_like(parents, -1)
    gone = tables.clone()
    gone[1, 0] = 99                                             # positions 0..7 of sequence 1
    new, rows, err = run([0, 5, 0], parents=star, tables=gone)  # position 8 -> 3: no block
    assert (new, err) == ([11, 4, 9], pa.DEVERR_TABLE_ENTRY) and same()


# ---- the step as a whole ----------------------------------------------------------------------

def _verify(rng, nodes, parents):
    """A made-up verification: the deepest accepted node of each tree."""
    return [int(rng.integers(-1, m)) for m in nodes]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("hkv,group,d,bs,dtype", [(2, 4, 64, 16, BF), (1, 2, 20, 5, F32)])
def test_draft_steps_follow_the_host(cuda_device, captured, hkv, group, d, bs, dtype):
    """Several verify steps of a batch: plan, cache write, tree attention,
    accept, lengths and blocks staying on the device; eagerly and as one
    captured graph replayed.  A contiguous host history gives the attention,
    and every block stays with one sequence."""
    dev, n, layers, most, pool = cuda_device, 5, 2, 12, 220
    width, cap = 24, 24 * bs
    rng = np.random.default_rng(7)
    g = torch.Generator().manual_seed(7)
    scale = 1 / math.sqrt(d)
    kc = torch.full((layers, pool, hkv, bs, d), float("nan"), dtype=dtype, device=dev)
    vc = kc.clone()
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    lens, held, head, new = i32(n), i32(n), i32(1), i32(n)
    tables = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    free = torch.tensor(rng.permutation(pool), dtype=torch.int32, device=dev)
    tokens = n * most
    plan = pa.StepPlan.empty(n, tokens, dev)
    plan.blocks_held, plan.free_head = held, head             # in place
    parents, leaf = i32(tokens), i32(n)
    q = torch.zeros(layers, tokens, hkv * group, d, dtype=dtype, device=dev)
    kn = torch.zeros(layers, tokens, hkv, d, dtype=dtype, device=dev)
    vn = torch.zeros_like(kn)
    out = torch.zeros_like(q)
    ws = torch.empty(max(1, pa.decode_tree_workspace_bytes(n, tokens, hkv * group, most, cap,
                                                           kc[0])), dtype=torch.uint8, device=dev)

    def step():
        pa.plan_step(lens, new, tables, held, free, head, pool, bs, plan)
        for l in range(layers):
            pa.write_kv(kn[l], vn[l], plan.slot_mapping, kc[l], vc[l])
            pa.decode_tree(q[l], plan.query_start_loc, parents, kc[l], vc[l], tables,
                           plan.seq_lens, most, cap, scale, out=out[l], workspace=ws)
        pa.accept_tree(leaf, parents, plan.query_start_loc, plan.seq_lens, kc, vc, tables, most,
                       new_lens=lens, accepted_rows=plan.positions)

    graph = None
    if captured:
        new.zero_()                                           # warm-up: nothing to plan
        leaf.fill_(-1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        torch.cuda.synchronize()
        assert lens.tolist() == [0] * n
    hist_k = [[torch.zeros(0, hkv, d, dtype=dtype) for _ in range(n)] for _ in range(layers)]
    hist_v = [[torch.zeros(0, hkv, d, dtype=dtype) for _ in range(n)] for _ in range(layers)]
    for s in range(6):
        nodes = [int(x) for x in rng.integers(0 if s else 1, most + 1, n)]
        par = [random_parents(rng, m, "mixed") if m else [] for m in nodes]
        leafs = _verify(rng, nodes, par)
        flat = [p for ps in par for p in ps]
        start = np.concatenate([[0], np.cumsum(nodes)])
        total = int(start[-1])
        vals = [torch.randn(layers, total, hkv * (group if x == 0 else 1), d, generator=g).to(dtype)
                for x in range(3)]
        for buf, x in zip((q, kn, vn), vals):
            buf[:, :total] = x.to(dev)
        new.copy_(torch.tensor(nodes, dtype=torch.int32))
        leaf.copy_(torch.tensor(leafs, dtype=torch.int32))
        parents[:total] = torch.tensor(flat, dtype=torch.int32, device=dev)
        out.fill_(7.0)
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        assert pa.last_device_error() == 0
        got = out.cpu()
        assert (got[:, total:] == 7.0).all()
        for l in range(layers):
            # one batch over contiguous host rows: a table of blocks in order
            b = Batch([len(h) for h in hist_k[l]], nodes, hkv, group, d, bs, dtype, seed=s)
            b.par, b.scale, b.q = par, scale, vals[0][l]
            for i in range(n):
                rows = slice(int(start[i]), int(start[i + 1]))
                for cache, hist, fresh in ((b.k, hist_k, vals[1]), (b.v, hist_v, vals[2])):
                    for p, x in enumerate(torch.cat([hist[l][i], fresh[l, rows]])):
                        cache[int(b.tables[i, p // bs]), :, p % bs] = x
                path = [int(start[i]) + a for a in path_of(par[i], leafs[i])]
                hist_k[l][i] = torch.cat([hist_k[l][i], vals[1][l, path]])
                hist_v[l][i] = torch.cat([hist_v[l][i], vals[2][l, path]])
            ref, bound = tree_reference(b)
            assert_tree_close(got[l, :total], ref, bound, dtype, f"step {s} layer {l}")
        assert lens.tolist() == [len(h) for h in hist_k[0]]
        rows = [int(start[i]) + a for i in range(n) for a in path_of(par[i], leafs[i])]
        assert [r for r in plan.positions[:total].tolist() if r >= 0] == rows
    # every block belongs to one sequence
    used = [tables[i, :held[i]].tolist() for i in range(n)]
    flat = [x for u in used for x in u]
    assert len(flat) == len(set(flat)) == int(head)
    assert sorted(flat) == sorted(free[:int(head)].tolist())


# ---- refusals on the host -----------------------------------------------------------------------

def test_refusals(cuda_device):
    b = Batch([10, 3], [12, 6], 2, 2, 64, 8, BF, seed=2)
    q, start, parents, k, v, tables, lens = b.to(cuda_device)
    with pytest.raises(pa.PaError) as e:
        pa.decode_tree(q, start, parents, k, v, tables, lens, 257, 1000)   # past the table too
    assert e.value.status == pa.PA_ERR_INVALID_ARG
    wide = torch.cat([tables] * 40, 1).contiguous()
    with pytest.raises(pa.PaError) as e:
        pa.decode_tree(q, start, parents, k, v, wide, lens, 257, 1000)
    assert e.value.status == pa.PA_ERR_UNSUPPORTED
    with pytest.raises(pa.PaError) as e:
        pa.decode_tree(q[:, :3].contiguous(), start, parents, k, v, tables, lens, 12, 22)
    assert e.value.status == pa.PA_ERR_INVALID_ARG             # 3 heads over 2 kv heads
    with pytest.raises(ValueError):
        pa.decode_tree(q, start, parents.long(), k, v, tables, lens, 12, 22)
    with pytest.raises(ValueError):
        pa.decode_tree(q, start, parents[:-1], k, v, tables, lens, 12, 22)
    with pytest.raises(ValueError):
        pa.decode_tree(q.float(), start, parents, k, v, tables, lens, 12, 22)
    with pytest.raises(ValueError):
        pa.decode_tree(q, start, parents, k, v, tables, lens, 12, 22, out=q[:3])
    leaf = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    for bad in ([k, k], [k, v]):                               # one memory twice
        with pytest.raises(pa.PaError) as e:
            pa.accept_tree(leaf, parents, start, lens, bad, [v, k.clone()], tables, 12)
        assert e.value.status == pa.PA_ERR_INVALID_ARG
    with pytest.raises(pa.PaError) as e:
        pa.accept_tree(leaf, parents, start, lens, k, v, tables, 12, new_lens=lens)
    assert e.value.status == pa.PA_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        pa.accept_tree(leaf, parents, start, lens, [k, k], [v], tables, 12)
    one = torch.ones(2, dtype=torch.int32, device=cuda_device)
    free = torch.arange(8, dtype=torch.int32, device=cuda_device)
    zero = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    plan = pa.StepPlan.empty(2, 4, cuda_device)
    plan.query_start_loc = torch.empty(6, dtype=torch.int32, device=cuda_device)[:3]
    plan.block_start = plan.query_start_loc
    with pytest.raises(pa.PaError) as e:
        pa.plan_step(lens, one, tables, one, free, zero, 20, 8, plan)
    assert e.value.status == pa.PA_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        pa.plan_step(lens, one, tables, one, free, zero, 20, 8)
    with pytest.raises(ValueError):
        pa.plan_step(lens, one[:1], tables, one, free, zero, 20, 8, max_tokens=4)
    assert pa.last_device_error() == 0


def test_debug_pass(cuda_device, monkeypatch):
    b = Batch([10, 3], [12, 6], 2, 2, 64, 8, BF, seed=2)
    q, start, parents, k, v, tables, lens = b.to(cuda_device)
    monkeypatch.setenv("PA_DEBUG", "1")
    ref, bound = tree_reference(b)
    assert_tree_close(b.run(pa, cuda_device), ref, bound, BF)
    bad = parents.clone()
    bad[4] = 4
    leaf = torch.tensor([0, 6], dtype=torch.int32, device=cuda_device)
    one = torch.ones(2, dtype=torch.int32, device=cuda_device)
    zero = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    twice = torch.tensor([1, 2, 1], dtype=torch.int32, device=cuda_device)
    for call in (lambda: pa.decode_tree(q, start, bad, k, v, tables, lens, 12, 22),
                 lambda: pa.accept_tree(leaf, parents, start, lens, k, v, tables, 12),
                 lambda: pa.plan_step(lens, one, tables, one, twice, zero, 20, 8, max_tokens=4)):
        with pytest.raises(pa.PaError) as e:
            call()
        assert e.value.status == pa.PA_ERR_INVALID_ARG
    assert pa.last_device_error() == 0
