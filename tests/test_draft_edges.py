"""The drafted step at its edges: values at the type's ends, infinities in the
caches, sequences that are refused, workspaces kept for calls of other sizes, calls
from several host threads."""
import ctypes
import math
import threading

import pytest
import torch

import paged_kv_cache_109_gb300 as pa
from tests._draft import (Batch, PlanState, assert_tree_close, path_of, plan_reference,
                          tree_reference)

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def clear_device_error(cuda_device):
    pa.last_device_error()
    yield


def _place(b, i, p):
    """Block and row of position ``p`` of sequence ``i``."""
    return int(b.tables[i, p // b.bs]), p % b.bs


# ---- values at the type's ends, infinities ---------------------------------------------

# kv heads, group, head dim, block size, dtype, cached tokens, nodes
ENDS = [
    (1, 4, 128, 16, F32, [37, 200], [8, 40]), (1, 2, 64, 16, F32, [37, 200], [8, 40]),
    (1, 1, 64, 8, F32, [37, 5], [8, 9]), (1, 2, 128, 16, F32, [37, 60], [8, 9]),
    (1, 1, 256, 16, F32, [37, 200], [8, 40]), (1, 2, 36, 16, F32, [37, 200], [8, 40]),
    (2, 1, 64, 16, F32, [5000, 3], [9, 4]), (1, 2, 7, 3, F32, [37, 20], [8, 5]),
    (1, 4, 128, 16, BF, [37, 200], [8, 40]), (1, 1, 64, 8, BF, [37, 200], [8, 40]),
    (1, 2, 256, 16, BF, [37, 200], [8, 40]), (1, 2, 72, 16, BF, [37, 200], [8, 40]),
    (1, 64, 128, 16, BF, [37, 200], [8, 40]),
]


def _largest(dtype):
    # the largest value, and in fp32 the least one that 11 bits round up to 2^128
    top = torch.finfo(dtype).max
    least = torch.tensor(0x7F7FF000, dtype=torch.int32).view(F32).item()
    return [top, -top] + ([least, -least] if dtype == F32 else [])


@pytest.mark.parametrize("hkv,group,d,bs,dtype,ctx,nodes", ENDS)
@pytest.mark.parametrize("which", range(4))
def test_a_hidden_nodes_largest_values_leave_no_trace(cuda_device, hkv, group, d, bs, dtype, ctx,
                                                      nodes, which):
    bads = _largest(dtype)
    if which >= len(bads):
        pytest.skip("two values of this type")
    for hit in ("v", "k"):
        b = Batch(ctx, nodes, hkv, group, d, bs, dtype, seed=11)
        node = [3, nodes[1] // 2]
        for i in range(2):
            blk, off = _place(b, i, ctx[i] + node[i])
            if hit == "v":
                b.v[blk, :, off, 1::3] = bads[which]
            else:
                b.k[blk, :, off] = bads[which]
        got = b.run(pa, cuda_device).double().cpu()
        torch.cuda.synchronize()
        ref, bound = tree_reference(b)
        for i in range(2):
            for j in range(nodes[i]):
                r = int(b.start[i]) + j
                sees = node[i] in path_of(b.par[i], j)
                if not sees or (hit == "v" and dtype == F32):
                    # (fp32: one such value under a weight of at most one is
                    # finite, and the bound is in terms of sum p |v|)
                    assert torch.isfinite(got[r]).all(), (hit, r)
                    assert_tree_close(got[r], ref[r], bound[r], dtype, f"{hit} {r}")


FP32 = [x for x in ENDS if x[4] == F32]


@pytest.mark.parametrize("hkv,group,d,bs,dtype,ctx,nodes", FP32)
@pytest.mark.parametrize("bad", ["max", "least", "inf", "-inf", "both"])
def test_cached_values_at_the_ends_fp32(cuda_device, hkv, group, d, bs, dtype, ctx, nodes, bad):
    """A cached token's V holds the type's largest value or an infinity: the
    formula's value, in every row of the sequence."""
    b = Batch(ctx, nodes, hkv, group, d, bs, dtype, seed=5)
    top = _largest(F32)
    for i, p in ((0, ctx[0] // 2), (1, 1)):
        blk, off = _place(b, i, p)
        b.v[blk, :, off, 2::5] = {"max": top[0], "least": -top[2], "inf": math.inf,
                                  "-inf": -math.inf, "both": math.inf}[bad]
        if bad == "both":
            blk, off = _place(b, i, p + 1)
            b.v[blk, :, off, 2::5] = -math.inf
    got = b.run(pa, cuda_device).double().cpu()
    assert pa.last_device_error() == 0
    ref, bound = tree_reference(b)
    if bad in ("max", "least"):
        assert torch.isfinite(got).all()
        assert_tree_close(got, ref, bound, dtype)
        return
    assert torch.isfinite(got).logical_not()[..., 2::5].all()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    fine = torch.isfinite(ref)
    assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)])
    assert_tree_close(got[fine], ref[fine], bound[fine], dtype)


@pytest.mark.parametrize("hkv,group,d,bs,dtype,ctx,nodes", FP32)
@pytest.mark.parametrize("bad", ["max", "least", "inf"])
def test_cached_keys_at_the_ends_fp32(cuda_device, hkv, group, d, bs, dtype, ctx, nodes, bad):
    """One element of a cached K holds the largest value or an infinity, q half
    of one against it with either sign: weight one, weight zero, or (an
    infinite score) NaN."""
    b = Batch(ctx, nodes, hkv, group, d, bs, dtype, seed=6)
    top = _largest(F32)
    x = {"max": top[0], "least": top[2], "inf": math.inf}[bad]
    g = torch.Generator().manual_seed(1)
    b.q[..., 1] = torch.where(torch.rand(b.q.shape[:2], generator=g) < 0.5, 0.5, -0.5)
    at = [(0, ctx[0] // 2), (1, 1)]
    # rows with q < 0: the formula without that key
    clean = Batch(ctx, nodes, hkv, group, d, bs, dtype, seed=6)
    clean.q = b.q
    for i, p in at:
        blk, off = _place(clean, i, p)
        clean.k[blk, :, off] = 0.0
        clean.k[blk, :, off, 1] = 1e6              # a weight of exp(-0.5e6 scale) = 0
    drop, _ = tree_reference(clean)
    for i, p in at:
        blk, off = _place(b, i, p)
        b.k[blk, :, off, 1] = x
    got = b.run(pa, cuda_device).double().cpu()
    assert pa.last_device_error() == 0
    # (tree_reference's bound, with products of q and k below 64 and |v| below 6)
    ds = (d + 4) * 2.0 ** -24 * b.scale * 64 * d
    for i, (_, p) in enumerate(at):
        blk, off = _place(b, i, p)
        for r in range(int(b.start[i]), int(b.start[i + 1])):
            for h in range(hkv * group):
                if b.q[r, h, 1] < 0:
                    share = 2 * ds + 2 * (ctx[i] + nodes[i]) * 2.0 ** -24 + 2.0 ** -19
                    tol = share * 6 + 2.0 ** -24 * drop[r, h].abs()
                    assert ((got[r, h] - drop[r, h]).abs() <= tol).all(), (r, h)
                elif bad == "inf":
                    assert torch.isnan(got[r, h]).all(), (r, h)
                else:
                    want = b.v[blk, h // group, off].double()
                    assert ((got[r, h] - want).abs() <= 2.0 ** -22 * want.abs()).all(), (r, h)


@pytest.mark.parametrize("hkv,group,d,bs,dtype,ctx,nodes", FP32)
def test_queries_at_the_ends_fp32(cuda_device, hkv, group, d, bs, dtype, ctx, nodes):
    """A row's q holds the largest value where every key holds zero, another's
    NaN: the first is the formula's, the second NaN, the others do not change."""
    b = Batch(ctx, nodes, hkv, group, d, bs, dtype, seed=7)
    b.k[..., 1] = torch.where(torch.isnan(b.k[..., 1]), b.k[..., 1], torch.zeros(()))
    b.q[1, :, 1] = torch.finfo(F32).max
    ref, bound = tree_reference(b)
    # (q k is zero there: its share of the bound too)
    b.q[2, :, 3] = math.nan
    got = b.run(pa, cuda_device).double().cpu()
    assert torch.isnan(got[2]).all()
    keep = [r for r in range(b.total) if r != 2]
    assert_tree_close(got[keep], ref[keep], bound[keep], dtype)


# ---- refused sequences -------------------------------------------------------------------

def test_accept_gives_a_refused_sequences_rows_as_none(cuda_device):
    b = Batch([10, 3, 8], [5, 6, 4], 2, 1, 64, 8, BF, seed=2, kind="chain")
    _, start, parents, k, v, tables, lens = b.to(cuda_device)
    k0, v0 = k.clone(), v.clone()

    def run(start=start, lens=lens, max_q=6):
        rows = torch.full((b.total,), 12345, dtype=torch.int32, device=cuda_device)
        got = pa.accept_tree(torch.zeros(3, dtype=torch.int32, device=cuda_device), parents, start,
                             lens, k, v, tables, max_q, accepted_rows=rows)
        torch.cuda.synchronize()
        assert torch.equal(k.view(torch.uint8), k0.view(torch.uint8))
        assert torch.equal(v.view(torch.uint8), v0.view(torch.uint8))
        return got[0].tolist(), rows.tolist(), pa.last_device_error()

    kept = [0, -1, -1, -1, -1], [11, -1, -1, -1]
    for short in (4, -1, 10 ** 6):                               # lengths out of range
        bad = lens.clone()
        bad[1] = short
        new, rows, err = run(lens=bad)
        assert (new, err) == ([11, short, 9], pa.DEVERR_SEQ_LEN)
        assert rows == kept[0] + [-1] * 6 + kept[1]
    new, rows, err = run(max_q=5)                               # six nodes, bound five
    assert (new, err) == ([11, 9, 9], pa.DEVERR_SEQ_LEN)
    assert rows == kept[0] + [-1] * 6 + kept[1]
    late = start.clone()
    late[3] = b.total + 1000                                    # rows past total_q
    new, rows, err = run(start=late)
    assert (new, err) == ([11, 4, 12], pa.DEVERR_SEQ_LEN)
    assert rows == kept[0] + [5] + [-1] * 5 + [-1] * 4
    early = start.clone()
    early[0] = -2147483648                                      # rows before the first
    new, rows, err = run(start=early)
    assert (new, err) == ([15, 4, 9], pa.DEVERR_SEQ_LEN)
    assert rows == [-1] * 5 + [5] + [-1] * 5 + kept[1]
    back = start.clone()
    back[1], back[2] = 20, 11                                   # 0..20 and 20..11 refused
    for _ in range(20):
        new, rows, err = run(start=back)
        assert (new, err) == ([15, 9, 9], pa.DEVERR_SEQ_LEN)
        assert rows == [12345] * 11 + kept[1]                   # the third's own stay


TREES = [(64, 16, BF), (144, 16, BF), (72, 16, BF), (64, 16, F32), (7, 3, F32), (20, 5, BF)]


@pytest.mark.parametrize("d,bs,dtype", TREES)
def test_refused_sequences_without_rows_are_reported(cuda_device, d, bs, dtype):
    b = Batch([30, 10, 20], [4, 0, 3], 1, 2, d, bs, dtype, seed=6)
    q, start, parents, k, v, tables, lens = b.to(cuda_device)
    ref, bound = tree_reference(b)

    def run(lens):
        out = pa.decode_tree(q, start, parents, k, v, tables, lens, b.max_q, b.max_len, b.scale)
        torch.cuda.synchronize()
        assert_tree_close(out, ref, bound, dtype)
        return pa.last_device_error()

    assert run(lens) == 0
    for bad in (-1, b.max_len + 1):
        wrong = lens.clone()
        wrong[1] = bad
        assert run(wrong) == pa.DEVERR_SEQ_LEN


@pytest.mark.parametrize("d,bs,dtype", TREES)
@pytest.mark.parametrize("head", [[4], [0, 9], [-3], [0, 0, 2, 9, 7]])
def test_rows_of_a_sequence_behind_refused_ones(cuda_device, d, bs, dtype, head):
    """Starts that do not ascend: the sequences that they break are refused, and
    one whose own rows are in range has its value."""
    b = Batch([30], [3], 1, 2, d, bs, dtype, seed=6)
    q, _, parents, k, v, tables, lens = b.to(cuda_device)
    ref, bound = tree_reference(b)
    n = len(head) + 1
    rows = torch.full((8, 2, d), 1.0, dtype=dtype, device=cuda_device)
    rows[2:5] = q
    par = torch.full((8,), -1, dtype=torch.int32, device=cuda_device)
    par[2:5] = parents
    start = torch.tensor(head + [2, 5], dtype=torch.int32, device=cuda_device)
    out = torch.full_like(rows, 7.0)
    every = lens.repeat(n)
    every[:-1] = 2                              # (two keys: sequences of two rows and none fit)
    pa.decode_tree(rows, start, par, k, v, tables.repeat(n, 1).contiguous(), every, 4, 33, b.scale,
                   out=out)
    torch.cuda.synchronize()
    assert pa.last_device_error() == pa.DEVERR_SEQ_LEN
    got = out.double().cpu()
    assert_tree_close(got[2:5], ref, bound, dtype)
    assert (got[5:] == 7.0).all()


# ---- workspaces and plans kept for calls of other sizes ----------------------------------

@pytest.mark.parametrize("hkv,group,d,bs,dtype", [
    (8, 4, 128, 16, F32), (8, 1, 256, 16, F32), (8, 4, 128, 4, BF), (8, 2, 256, 16, BF),
    (8, 4, 72, 16, BF), (8, 3, 200, 8, BF), (8, 4, 128, 16, BF), (8, 5, 96, 24, BF),
    (2, 40, 64, 16, BF), (3, 7, 64, 16, F32),
])
def test_a_workspace_serves_every_smaller_call(cuda_device, hkv, group, d, bs, dtype):
    desc = pa.CacheDesc(4096, bs, hkv, d, pa.PA_BF16 if dtype == BF else pa.PA_F32)
    hq = hkv * group

    def size(n, nodes, keys):
        return pa.decode_tree_workspace_bytes(n, n * nodes, hq, nodes, keys, desc)

    steps = [1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 64, 65, 129, 256]
    for keys in (300, 4000, 131072):
        for n in (1, 7, 64):
            sizes = [size(n, x, keys) for x in steps]
            assert sizes == sorted(sizes), (n, keys)
            assert size(n, 8, keys) <= size(n + 9, 8, keys + 5000)
    # a batch that fills the GPU, its workspace made for 64 nodes
    b = Batch([700] * 24, [3] * 24, hkv, group, d, bs, dtype, seed=3)
    ref, bound = tree_reference(b)
    ws = torch.empty(max(1, size(24, 64, 4000)), dtype=torch.uint8, device=cuda_device)
    args = b.to(cuda_device)
    args[5] = torch.cat([args[5], torch.full((24, -(-4000 // bs)), -1, dtype=torch.int32,
                                             device=cuda_device)], 1).contiguous()
    got = pa.decode_tree(*args, 3, 4000, b.scale, workspace=ws)
    assert_tree_close(got, ref, bound, dtype)


# ---- two host threads -----------------------------------------------------------------------

@pytest.mark.parametrize("dtype,dims,bs", [(F32, (128, 96), 16), (BF, (256, 192), 16),
                                           (BF, (232, 200), 16), (BF, (128, 112), 4)])
def test_host_threads_with_two_head_dims(cuda_device, dtype, dims, bs):
    """Calls at once that share a kernel and need different shared memory."""
    bs_ = [Batch([60] * 2, [16] * 2, 1, 4, d, bs, dtype, seed=d) for d in dims]
    lib, refs = pa.load_library(), [tree_reference(b) for b in bs_]
    work = []
    for x in range(4):
        b = bs_[x % 2]
        q, start, parents, k, v, tables, lens = b.to(cuda_device)
        out, stream = torch.zeros_like(q), torch.cuda.Stream()
        desc = pa.CacheDesc(k.shape[0], bs, 1, k.shape[3], pa.PA_F32 if dtype == F32 else pa.PA_BF16)
        p = [ctypes.c_void_p(t.data_ptr()) for t in (q, start, parents, k, v, tables, lens, out)]
        args = (p[0], p[1], p[2], b.total, b.max_q, p[3], p[4], p[5], tables.shape[1], p[6], 2,
                b.max_len, 4, b.scale, p[7], None, 0, ctypes.byref(desc),
                ctypes.c_void_p(stream.cuda_stream))
        work.append((args, out, stream, desc, (q, start, parents, k, v, tables, lens)))
    torch.cuda.synchronize()
    go, failed = threading.Barrier(len(work)), []

    def run(args):
        torch.cuda.set_device(cuda_device)
        go.wait()
        failed.append(sum(lib.pa_decode_tree(*args) != pa.PA_OK for _ in range(4000)))

    threads = [threading.Thread(target=run, args=(w[0],)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(work)
    assert pa.last_device_error() == 0
    for x, w in enumerate(work):
        assert_tree_close(w[1], *refs[x % 2], dtype)


# ---- a plan's shared blocks ---------------------------------------------------------------

@pytest.mark.parametrize("n", [3, 1500])
@pytest.mark.parametrize("lens0,new0,extra,shared,bit", [
    (8, 1, 1, 2, "shared"),       # a full tail, the block behind it shared
    (6, 3, 1, 2, "shared"),       # the tail the sequence's own, the next block not
    (6, 7, 2, 3, "shared"),       # the last of the blocks that tokens go into
    (6, 6, 2, 3, 0),              # tokens end before it
    (6, 0, 2, 2, 0),              # no tokens
    (8, 3, 1, 1, 0),              # a full tail: nothing goes into it
])
def test_plan_never_writes_into_shared_blocks(cuda_device, n, lens0, new0, extra, shared, bit):
    """Blocks held behind the cached tokens whose count is above one (a fork's)
    are refused like a shared tail, where new tokens would go into them."""
    lens, new = [lens0] + [3] * (n - 1), [new0] + [1] * (n - 1)
    st = PlanState(lens, [extra] + [0] * (n - 1), 4, 3 * n + 12, 5, seed=n)
    ref_cnt = torch.tensor(st.pool.ref_cnt, dtype=torch.int32, device=cuda_device)
    ref_cnt[int(st.tables[0, shared])] = 2
    before = ref_cnt.clone()
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    tables = st.tables.to(cuda_device)
    plan = pa.plan_step(dev(lens), dev(new), tables, dev(st.held), dev(st.free), dev([0]),
                        st.num_blocks, 4, max_tokens=sum(new), ref_cnt=ref_cnt)
    torch.cuda.synchronize()
    if bit:
        assert pa.last_device_error() == pa.DEVERR_SHARED
        assert torch.equal(tables.cpu(), st.tables) and torch.equal(ref_cnt, before)
        assert plan.seq_lens.tolist() == lens and plan.blocks_held.tolist() == st.held
        assert plan.free_head.tolist() == [0] and plan.slot_mapping.tolist() == [-1] * sum(new)
    else:
        assert pa.last_device_error() == 0
        want = plan_reference(st, new, 0, sum(new))
        assert plan.slot_mapping.tolist() == want["slot_mapping"]
        assert plan.seq_lens.tolist() == want["seq_lens"] and tables.tolist() == want["tables"]


@pytest.mark.parametrize("n", [1, 3, 1500])
def test_a_plan_of_views_serves_a_smaller_batch(cuda_device, n):
    """A loop's plan for its largest batch, its first entries for a smaller one."""
    big = pa.StepPlan.empty(n + 5, 4 * n + 9, cuda_device)
    plan = pa.StepPlan(big.seq_lens[:n], big.blocks_held[:n], big.free_head,
                       big.query_start_loc[:n + 1], big.block_start[:n + 1], big.slot_mapping,
                       big.positions, big.seq_ids)
    st = PlanState([3] * n, [0] * n, 4, 3 * n + 2, 4, seed=n)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    tables = st.tables.to(cuda_device)
    args = (dev(st.lens), dev([2] * n), tables, dev(st.held), dev(st.free), dev([0]), st.num_blocks,
            4)
    with pytest.raises(ValueError):
        pa.plan_step(*args, big)
    pa.plan_step(*args, plan)
    torch.cuda.synchronize()
    assert pa.last_device_error() == 0
    ref = plan_reference(st, [2] * n, 0, 4 * n + 9)
    for k in pa.StepPlan.__slots__:
        assert getattr(plan, k).tolist() == ref[k], k
    assert tables.tolist() == ref["tables"]
