"""Host side of pa_rope_write, pa_verify_tree, pa_release_blocks and
pa_fork_blocks: argument checks that come before any device work, and the plain
forms the GPU tests compare with (CPU only)."""
import ctypes
import math

import pytest
import torch

import paged_kv_cache_109_gb300 as pa
from paged_kv_cache_109_gb300 import _build
from paged_kv_cache_109_gb300.block_pool import BlockPool
from tests._serving import (PoolState, VerifyBatch, angles, axis_of_pair, release_reference,
                            rope_reference, verify_reference)

P = ctypes.c_void_p(4096)               # never read: every case fails before
BAD, UNSUPPORTED = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load_library()


def _desc(**kw):
    d = dict(nb=64, bs=16, hkv=8, dim=128, dtype=pa.PA_BF16)
    d.update(kw)
    return ctypes.byref(pa.CacheDesc(d["nb"], d["bs"], d["hkv"], d["dim"], d["dtype"]))


def _rope(lib, n=4, hq=32, dim=128, at=(), strides=(6144, 6144, 6144), **kw):
    r = dict(rot_dim=128, num_axes=1, sections=(0, 0, 0), cyclic=0, neighbours=0, scale=1.0, eps=1e-6)
    r.update(kw)
    rope = pa.RopeDesc(r["rot_dim"], r["num_axes"], (ctypes.c_int32 * 3)(*r["sections"]), r["cyclic"],
                       r["neighbours"], r["scale"], r["eps"])
    # arrays far apart, so that only what `at` changes can be wrong
    p = [ctypes.c_void_p((i + 1) << 30) for i in range(11)]
    args = [p[0], p[1], p[2], *strides, n, hq, p[3], p[4], p[5], p[6], ctypes.byref(rope), p[7], p[8],
            p[9], p[10], _desc(dim=dim), None]
    for i, value in at:
        args[i] = value
    return lib.pa_rope_write(*args)


@pytest.mark.parametrize("kw,status", [
    (dict(hq=30), BAD), (dict(hq=0), BAD), (dict(n=-1), BAD), (dict(rot_dim=127), BAD),
    (dict(rot_dim=130), BAD), (dict(rot_dim=-2), BAD), (dict(num_axes=0), BAD),
    (dict(num_axes=4), BAD), (dict(num_axes=2, sections=(32, 31, 0)), BAD),
    (dict(num_axes=3, sections=(70, -3, -3)), BAD),
    (dict(num_axes=3, sections=(8, 28, 28), cyclic=1), BAD),      # pair 1 + 3 * 27 of 64
    (dict(eps=-1.0), BAD), (dict(eps=math.inf), BAD), (dict(eps=math.nan), BAD),
    (dict(scale=math.inf), BAD), (dict(scale=math.nan), BAD),
    (dict(strides=(4095, 6144, 6144)), BAD), (dict(strides=(6144, 1023, 6144)), BAD),
    (dict(strides=(6144, 6144, 1 << 62)), BAD),
    (dict(dim=264, rot_dim=128, strides=(9000, 9000, 9000)), UNSUPPORTED),
    (dict(at=[(0, None)]), BAD), (dict(at=[(8, None)]), BAD), (dict(at=[(9, None)]), BAD),
    (dict(at=[(13, None)]), BAD), (dict(at=[(14, None)]), BAD), (dict(at=[(16, None)]), BAD),
    (dict(at=[(13, ctypes.c_void_p((8 << 30) + 4))]), BAD),       # slots off their 8 bytes
    (dict(at=[(0, ctypes.c_void_p((1 << 30) + 1))]), BAD),
    (dict(at=[(14, ctypes.c_void_p(2 << 30))]), BAD),             # out over k
    (dict(at=[(14, ctypes.c_void_p(1 << 30))]), BAD),             # in place, rows apart
    (dict(at=[(16, ctypes.c_void_p(10 << 30))]), BAD),            # one cache for both
    (dict(n=0), pa.PA_OK),
])
def test_rope_argument_errors(lib, kw, status):
    assert _rope(lib, **kw) == status


def test_pointers_that_no_kernel_may_touch_are_refused(lib):
    # (without a GPU no pointer is device memory)
    if torch.cuda.is_available():
        pytest.skip("a GPU is there")
    assert _rope(lib) == BAD


def _verify_args():
    p = [ctypes.c_void_p((i + 1) << 30) for i in range(10)]
    return [p[0], p[1], 1000, 1000, 1000, pa.PA_F32, p[2], p[3], p[4], 2, 6, 4, p[5], p[6], 1000, p[7],
            p[8], p[9], None]


@pytest.mark.parametrize("at,value,status", [
    (4, 0, BAD), (4, -5, BAD), (4, (1 << 30) + 1, UNSUPPORTED), (5, 7, BAD), (9, -1, BAD),
    (9, 65536, UNSUPPORTED), (10, -1, BAD), (11, -1, BAD), (11, 257, UNSUPPORTED),
    (2, 999, BAD), (3, 999, BAD), (14, 999, BAD), (14, 1 << 62, BAD), (0, None, BAD),
    (6, None, BAD), (7, None, BAD), (8, None, BAD), (12, None, BAD), (13, None, BAD),
    (16, None, BAD), (17, None, BAD), (16, ctypes.c_void_p(10 << 30), BAD),
    (17, ctypes.c_void_p(7 << 30), BAD), (6, ctypes.c_void_p(4098), BAD), (9, 0, pa.PA_OK),
])
def test_verify_argument_errors(lib, at, value, status):
    args = _verify_args()
    args[at] = value
    assert lib.pa_verify_tree(*args) == status


def test_release_argument_errors(lib):
    p = [ctypes.c_void_p((i + 1) << 30) for i in range(9)]
    good = [p[0], p[1], 8, p[2], 4, p[3], 64, p[4], p[5], 64, 16, p[6], p[7], None]
    for at, value, status in [
            (4, -1, BAD), (4, 65536, UNSUPPORTED), (6, -1, BAD), (6, 2 ** 31 - 1, UNSUPPORTED),
            (9, 0, BAD), (10, 0, BAD), (2, -1, BAD), (0, None, BAD), (1, None, BAD), (3, None, BAD),
            (5, None, BAD), (7, None, BAD), (11, None, BAD), (12, None, BAD),
            (11, p[0], BAD),                    # over the lengths
            (12, p[2], BAD), (12, p[6], BAD),   # over what is held, over the other output
            (8, p[3], BAD), (0, ctypes.c_void_p(4097), BAD)]:
        args = list(good)
        args[at] = value
        assert lib.pa_release_blocks(*args) == status, (at, value)


def test_fork_argument_errors(lib):
    p = [ctypes.c_void_p((i + 1) << 30) for i in range(11)]
    one = (ctypes.c_void_p * 1)(4096)
    good = [p[0], p[1], p[2], 8, p[3], 4, p[4], p[5], 64, p[6], one, one, 1, p[7], p[8], p[9], p[10],
            _desc(), None]
    for at, value, status in [
            (5, -1, BAD), (5, 65536, UNSUPPORTED), (8, -1, BAD), (8, 2 ** 31 - 1, UNSUPPORTED),
            (3, -1, BAD), (12, 0, BAD), (12, 1025, UNSUPPORTED), (17, _desc(nb=0), BAD),
            (0, None, BAD), (1, None, BAD), (2, None, BAD), (4, None, BAD), (6, None, BAD),
            (7, None, BAD), (9, None, BAD), (10, None, BAD), (11, None, BAD), (13, None, BAD),
            (14, None, BAD), (15, None, BAD), (16, None, BAD),
            (13, p[3], BAD), (16, p[2], BAD), (16, ctypes.c_void_p((11 << 30) + 4), BAD)]:
        args = list(good)
        args[at] = value
        assert lib.pa_fork_blocks(*args) == status, (at, value)


def test_cpu_tensors_are_refused(lib):
    x = torch.zeros(2, 1, 8)
    c = torch.zeros(4, 1, 4, 8)
    t = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.rope_write(x, x, x, t, torch.ones(4), t.long(), c, c.clone())
    with pytest.raises(ValueError):
        pa.verify_tree(torch.zeros(2, 5), t, t, t, torch.zeros(2), torch.zeros(1, 5), 1)
    with pytest.raises(ValueError):
        pa.release_blocks(t, t.view(2, 1), t, t, t[:1], 4, 4)
    with pytest.raises(ValueError):
        pa.fork_blocks(t, t, t.view(2, 1), t, torch.zeros(4, dtype=torch.int32), t, t[:1], c,
                       c.clone())


# ---- the plain forms -------------------------------------------------------------------

def test_plain_rotation():
    # one pair, a quarter turn: (1, 2) -> (-2, 1)
    x = torch.tensor([[[1.0, 2.0, 5.0]]])
    angle = torch.tensor([[math.pi / 2]], dtype=torch.float64)
    for neighbours in (False, True):
        out, _ = rope_reference(x, None, 0.0, angle, neighbours, 1.0)
        assert torch.allclose(out[0, 0], torch.tensor([-2.0, 1.0, 5.0], dtype=torch.float64))
    # angles of far positions: 2^30 turns by 1 rad, against 2^30 mod 2 pi in 64 bits
    a = angles(torch.tensor([[1 << 30]]), torch.tensor([1.0]), None, False)
    assert abs(math.remainder(float(a) - math.remainder(2.0 ** 30, 2 * math.pi), 2 * math.pi)) < 1e-6
    assert axis_of_pair(6, (2, 3, 1), False) == [0, 0, 1, 1, 1, 2]
    assert axis_of_pair(7, (3, 2, 2), True) == [0, 1, 2, 0, 1, 2, 0]
    assert axis_of_pair(7, (5, 1, 1), True) == [0, 1, 2, 0, 0, 0, 0]


def test_plain_norm():
    x = torch.tensor([[[3.0, 4.0]]])
    w = torch.tensor([1.0, 2.0])
    out, bound = rope_reference(x, w, 0.0, torch.zeros(1, 0, dtype=torch.float64), False, 1.0)
    r = math.sqrt(12.5)
    assert torch.allclose(out[0, 0], torch.tensor([3 / r, 8 / r], dtype=torch.float64))
    assert (bound > 0).all()


@pytest.mark.parametrize("draft", [True, False])
def test_plain_verification_gives_the_targets_distribution(draft):
    """The first token behind the root (held child or next) over many draws,
    against the target's probabilities: within five standard deviations."""
    vocab, reps = 5, 4000
    g = torch.Generator().manual_seed(1)
    row, drow = torch.randn(vocab, generator=g), torch.randn(vocab, generator=g)
    b = VerifyBatch([4] * reps, vocab, torch.float32, seed=2, kind="star", draft=draft)
    b.par = [[-1, 0, 0, 0]] * reps
    b.parents = torch.tensor([p for ps in b.par for p in ps], dtype=torch.int32)
    first = b.start[:-1].long()
    b.logits[first] = row
    q = torch.softmax(drow.double(), 0)
    for i in range(reps):
        q0 = 4 * i
        b.tokens[q0 + 1:q0 + 4] = (torch.multinomial(q, 3, replacement=True, generator=g).int()
                                   if draft else torch.tensor([3, 1, 3], dtype=torch.int32))
    if draft:
        b.draft[first] = drow
    count = torch.zeros(vocab)
    for i, (leaf, token, _) in enumerate(verify_reference(b)):
        # a held child is a leaf of the tree, but the token counts, not what follows
        count[int(b.tokens[4 * i + leaf]) if leaf > 0 else token] += 1
    p = torch.softmax(row.double(), 0)
    sigma = (reps * p * (1 - p)).sqrt()
    assert ((count - reps * p).abs() <= 5 * sigma).all(), (count / reps, p)


def test_plain_release_is_the_pools():
    st = PoolState([9, 6, 12, 3], 4, 30, 6, seed=3, share=[(2, 0, 2)], spare=[0, 2, 0, 1])
    pool = st.pool
    counts, free = list(pool.ref_cnt), list(st.free)
    held, head = release_reference(st.tables, st.held, [0, 2, 0, 1], counts, free, st.head, 30)
    want = BlockPool.release(pool, 0)                   # shared blocks stay
    spare = pool.tables[1][2:]
    pool.tables[1] = pool.tables[1][:2]
    for b in spare:
        pool.ref_cnt[b] = 0
    want = want + spare + BlockPool.release(pool, 2)
    spare = pool.tables[3][1:]
    pool.ref_cnt[spare[0]] = 0
    want = want + spare
    assert held == [0, 2, 0, 1] and free[head:st.head] == want and counts == pool.ref_cnt
