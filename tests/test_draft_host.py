"""Host side of the drafted step's calls: argument checks that come before
any device work (CPU only)."""
import ctypes

import pytest
import torch

import paged_kv_cache_109_gb300 as pa
from paged_kv_cache_109_gb300 import _build
from tests._draft import Batch, PlanState, accept_reference, path_of, plan_reference, tree_reference


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load_library()


def _desc(**kw):
    d = dict(nb=64, bs=16, hkv=8, dim=128, dtype=pa.PA_BF16)
    d.update(kw)
    return ctypes.byref(pa.CacheDesc(d["nb"], d["bs"], d["hkv"], d["dim"], d["dtype"]))


def test_empty_batches_are_no_ops(lib):
    # (a plan without sequences still has outputs to write)
    assert lib.pa_plan_step(None, None, None, 0, None, 0, None, None, 8, 16, None, 4, None, None,
                            None, None, None, None, None, None, 0, None) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_decode_tree(None, None, None, 0, 0, None, None, None, 4, None, 0, 0, 32, 1.0,
                              None, None, 0, _desc(), None) == pa.PA_OK
    assert lib.pa_decode_tree(None, None, None, 7, 0, None, None, None, 4, None, 3, 9, 32, 1.0,
                              None, None, 0, _desc(), None) == pa.PA_OK
    assert lib.pa_accept_tree(None, None, None, None, 0, 0, 0, None, 4, None, None, 1, None, None,
                              _desc(), None) == pa.PA_OK


@pytest.mark.parametrize("hq,max_q,max_len,width,dim,status", [
    (32, 4, 100, 4, 128, 1),        # 100 tokens need 7 blocks of a 4-entry row
    (30, 4, 60, 4, 128, 1),         # 30 query heads over 8 kv heads
    (32, 70, 60, 4, 128, 1),        # more nodes than tokens
    (32, -1, 60, 4, 128, 1), (32, 4, -1, 4, 128, 1),
    (32, 257, 300, 40, 128, 2),     # past PA_MAX_TREE_NODES
    (32, 4, 2 ** 31 - 1, 2 ** 28, 128, 2),   # positions past 32 bits
    (32, 4, 60, 4, 264, 2),         # past the largest head dim
])
def test_tree_argument_errors(lib, hq, max_q, max_len, width, dim, status):
    p = ctypes.c_void_p(4096)       # never read: every case fails before
    st = lib.pa_decode_tree(p, p, p, 5, max_q, p, p, p, width, p, 2, max_len, hq, 1.0, p, None, 0,
                            _desc(dim=dim), None)
    assert st == status


def test_null_and_range_errors(lib):
    p = ctypes.c_void_p(4096)
    ptrs = (ctypes.c_void_p * 1)(4096)
    assert lib.pa_decode_tree(None, p, p, 5, 4, p, p, p, 4, p, 2, 60, 32, 1.0, p, None, 0,
                              _desc(), None) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_accept_tree(p, p, p, p, 2, 5, 257, p, 4, ptrs, ptrs, 1, p, None, _desc(),
                              None) == pa.PA_ERR_UNSUPPORTED
    assert lib.pa_accept_tree(p, p, p, p, 2, 5, 4, p, 4, ptrs, ptrs, 0, p, None, _desc(),
                              None) == pa.PA_ERR_INVALID_ARG
    args = [p, p, p, 2, p, 8, p, None, 8, 16, p, 4, p, p, p, p, p, p, p, p, 5, None]
    for at, value, status in ((0, None, 1), (3, 65536, 2), (3, -1, 1), (8, 0, 1), (9, 0, 1),
                              (20, -1, 1), (20, 2 ** 31 - 1, 2), (15, None, 1)):
        a = list(args)
        a[at] = value
        assert lib.pa_plan_step(*a) == status, (at, value)


def test_cpu_tensors_are_refused(lib):
    b = Batch([4], [2], 1, 1, 8, 4, torch.float32, seed=0)
    with pytest.raises(ValueError):
        pa.decode_tree(b.q, b.start, b.parents, b.k, b.v, b.tables, b.lens, 2, 6)
    with pytest.raises(ValueError):
        pa.accept_tree(b.lens, b.parents, b.start, b.lens, b.k, b.v, b.tables, 2)
    with pytest.raises(ValueError):
        pa.plan_step(b.lens, b.lens, b.tables, b.lens, b.lens, b.lens, 4, 4, max_tokens=3)


# the plain forms the GPU tests compare with

def test_plain_tree_of_a_chain_is_causal_attention():
    b = Batch([3], [4], 1, 1, 8, 2, torch.float32, seed=1, kind="chain")
    out, bound = tree_reference(b)
    rows = b.tables[0, :4].long()
    k, v = b.k[rows, 0].reshape(-1, 8)[:7].double(), b.v[rows, 0].reshape(-1, 8)[:7].double()
    s = b.q[:, 0].double() @ k.T * b.scale
    s = s.masked_fill(torch.ones(4, 7).tril(3) == 0, float("-inf"))
    assert torch.allclose(out[:, 0], torch.softmax(s, 1) @ v, rtol=0, atol=1e-14)
    assert (bound > 0).all()


def test_plain_accept_moves_a_path_up():
    b = Batch([2], [5], 1, 1, 1, 4, torch.float32, seed=1)
    b.par = [[-1, 0, 0, 2, 1]]
    pos = torch.arange(7, dtype=torch.float32)
    k = torch.zeros_like(b.k)
    for p in range(7):
        k[int(b.tables[0, p // 4]), :, p % 4] = pos[p]
    lens, rows = accept_reference(b, [3], k, k.clone())
    assert path_of(b.par[0], 3) == [0, 2, 3] and lens.tolist() == [5]
    assert rows.tolist() == [0, 2, 3, -1, -1]
    got = [float(k[int(b.tables[0, p // 4]), 0, p % 4, 0]) for p in range(7)]
    assert got == [0, 1, 2, 4, 5, 5, 6]


def test_plain_plan_is_grow():
    st = PlanState([5, 0, 8], [0, 1, 0], 4, 12, 6, seed=3)
    free = list(st.free)
    ref = plan_reference(st, [4, 3, 1], 2, 10)
    # 9 tokens need 3 blocks (2 held), 3 need 1 (held), 9 need 3 (2 held)
    assert ref["blocks_held"] == [3, 1, 3] and ref["block_start"] == [0, 1, 1, 2]
    assert ref["tables"][0][2] == free[0] and ref["tables"][2][2] == free[1]
    assert ref["free_head"] == [4] and ref["query_start_loc"] == [0, 4, 7, 8]
    assert ref["slot_mapping"][-2:] == [-1, -1] and ref["slot_mapping"][7] == free[1] * 4
