"""Paged-attention decode for GB300: Python binding of libpa.so.

Every function here marshals tensors into the C ABI declared in
``include/pa.h``; all computation runs in the library's CUDA kernels.  There
is no CPU path: every call raises ``ImportError`` when ``libpa.so`` has not
been built, and the calls only accept CUDA tensors.

    import paged_kv_cache_109_gb300 as pa
    pa.write_kv(k, v, slot_mapping, k_cache, v_cache)
    out = pa.decode(q, k_cache, v_cache, block_tables, seq_lens, max_seq_len)
"""
from __future__ import annotations

import ctypes
import functools
import math
import operator
import os

import torch

from ._build import LIB as LIBRARY_PATH
from ._build import build
from .block_pool import BlockPool, SharedTailWrite

__all__ = ["write_kv", "write_kv_positions", "copy_blocks", "decode", "decode_append",
           "decode_shared_prefix", "prefix_groups", "PrefixGroups", "decode_shared_prefix_workspace_bytes",
           "decode_shared_prefix_mode", "prefill",
           "plan_step", "StepPlan", "decode_tree", "decode_tree_workspace_bytes", "accept_tree",
           "MAX_TREE_NODES",
           "rope_write", "verify_tree", "release_blocks", "fork_blocks",
           "decode_workspace_bytes", "decode_partition_tokens",
           "decode_path", "last_device_error", "PaError", "build", "BlockPool",
           "SharedTailWrite", "LIBRARY_PATH", "load_library", "CacheDesc"]

PA_OK, PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_ERR_CUDA = range(5)
PA_F32, PA_BF16 = 0, 1
DEVERR_TABLE_ENTRY, DEVERR_SEQ_LEN, DEVERR_SLOT, DEVERR_TIMEOUT, DEVERR_BLOCK_PAIR = 1, 2, 4, 8, 16
DEVERR_GROUP, DEVERR_POOL, DEVERR_SHARED, DEVERR_TREE = 32, 64, 128, 256
DEVERR_LOGITS, DEVERR_FORK = 512, 1024
MAX_TREE_NODES = 256
SHARED_AUTO, SHARED_ONCE, SHARED_PLAIN = 0, 1, 2


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("num_axes", ctypes.c_int32),
                ("sections", ctypes.c_int32 * 3), ("cyclic", ctypes.c_int32),
                ("neighbours", ctypes.c_int32), ("scale", ctypes.c_float),
                ("eps", ctypes.c_float)]


class PaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_status_str(status)} (status {status})")


_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libpa.so (built in-tree by ``build()``); raises if it is absent."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    target = path or LIBRARY_PATH
    if not os.path.exists(target):
        raise ImportError(f"{target} is not built; run paged_kv_cache_109_gb300.build()")
    lib = ctypes.CDLL(target)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    DP = ctypes.POINTER(CacheDesc)
    lib.pa_write_kv.argtypes = [P, P, P, I32, P, P, DP, P]
    lib.pa_write_kv.restype = ctypes.c_int
    lib.pa_write_kv_positions.argtypes = [P, P, P, P, I32, P, I32, I32, P, P, DP, P]
    lib.pa_write_kv_positions.restype = ctypes.c_int
    lib.pa_copy_blocks.argtypes = [P, P, I32, P, P, I32, P, I32, DP, P]
    lib.pa_copy_blocks.restype = ctypes.c_int
    lib.pa_prefill.argtypes = [P, P, I32, I32, P, P, P, I32, P, I32, I32, I32, ctypes.c_float,
                               P, DP, P]
    lib.pa_prefill.restype = ctypes.c_int
    lib.pa_decode_partition_tokens.argtypes = [I32, I32, I32, DP]
    lib.pa_decode_partition_tokens.restype = I32
    lib.pa_decode_workspace_bytes.argtypes = [I32, I32, I32, I32, DP]
    lib.pa_decode_workspace_bytes.restype = SZ
    lib.pa_decode.argtypes = [P, P, P, P, I32, P, I32, I32, I32, ctypes.c_float, I32, P, P, SZ,
                              DP, P]
    lib.pa_decode.restype = ctypes.c_int
    lib.pa_decode_append.argtypes = [P, P, P, P, P, P, I32, P, I32, I32, I32, ctypes.c_float,
                                     I32, P, P, SZ, DP, P]
    lib.pa_decode_append.restype = ctypes.c_int
    lib.pa_decode_shared_prefix_workspace_bytes.argtypes = [I32, I32, I32, I32, I32, DP]
    lib.pa_decode_shared_prefix_workspace_bytes.restype = SZ
    lib.pa_decode_shared_prefix.argtypes = [P, P, P, P, I32, P, I32, I32, I32, ctypes.c_float,
                                            I32, P, P, P, P, I32, I32, I32, I32, P, P, SZ, DP,
                                            P]
    lib.pa_decode_shared_prefix_mode.argtypes = [I32, I32, I32, DP]
    lib.pa_decode_shared_prefix_mode.restype = I32
    lib.pa_decode_shared_prefix.restype = ctypes.c_int
    lib.pa_plan_step.argtypes = [P, P, P, I32, P, I32, P, P, I32, I32, P, I32, P, P, P, P, P, P,
                                 P, P, I32, P]
    lib.pa_plan_step.restype = ctypes.c_int
    lib.pa_decode_tree_workspace_bytes.argtypes = [I32, I32, I32, I32, I32, DP]
    lib.pa_decode_tree_workspace_bytes.restype = SZ
    lib.pa_decode_tree.argtypes = [P, P, P, I32, I32, P, P, P, I32, P, I32, I32, I32,
                                   ctypes.c_float, P, P, SZ, DP, P]
    lib.pa_decode_tree.restype = ctypes.c_int
    lib.pa_accept_tree.argtypes = [P, P, P, P, I32, I32, I32, P, I32, P, P, I32, P, P, DP, P]
    lib.pa_accept_tree.restype = ctypes.c_int
    lib.pa_rope_write.argtypes = [P, P, P, I64, I64, I64, I32, I32, P, P, P, P,
                                  ctypes.POINTER(RopeDesc), P, P, P, P, DP, P]
    lib.pa_rope_write.restype = ctypes.c_int
    lib.pa_verify_tree.argtypes = [P, P, I64, I64, I32, I32, P, P, P, I32, I32, I32, P, P, I64, P,
                                   P, P, P]
    lib.pa_verify_tree.restype = ctypes.c_int
    lib.pa_release_blocks.argtypes = [P, P, I32, P, I32, P, I32, P, P, I32, I32, P, P, P]
    lib.pa_release_blocks.restype = ctypes.c_int
    lib.pa_fork_blocks.argtypes = [P, P, P, I32, P, I32, P, P, I32, P, P, P, I32, P, P, P, P, DP,
                                   P]
    lib.pa_fork_blocks.restype = ctypes.c_int
    lib.pa_decode_path.argtypes = [I32, DP]
    lib.pa_decode_path.restype = I32
    lib.pa_status_str.argtypes = [ctypes.c_int]
    lib.pa_status_str.restype = ctypes.c_char_p
    lib.pa_last_device_error.argtypes = []
    lib.pa_last_device_error.restype = I32
    lib.pa_check_wait_timeout.argtypes = [I32, I32, ctypes.c_int64, P]
    lib.pa_check_wait_timeout.restype = ctypes.c_int
    if path is None:
        _lib = lib
    return lib


def _status_str(status: int) -> str:
    try:
        return load_library().pa_status_str(status).decode()
    except ImportError:
        return "unknown"


# ---- marshalling helpers ----------------------------------------------------

_DTYPES = {torch.float32: PA_F32, torch.bfloat16: PA_BF16}


def cache_desc(k_cache: torch.Tensor) -> CacheDesc:
    if k_cache.dim() != 4:
        raise ValueError("caches are [num_blocks, num_kv_heads, block_size, head_dim]")
    if k_cache.dtype not in _DTYPES:
        raise ValueError(f"unsupported cache dtype {k_cache.dtype}")
    nb, hkv, bs, d = k_cache.shape
    return CacheDesc(nb, bs, hkv, d, _DTYPES[k_cache.dtype])


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _dev(*ts: torch.Tensor) -> None:
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _dev_or_pinned(*ts: torch.Tensor) -> None:
    for t in ts:
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError("tensors must be on a CUDA device or in page-locked host memory")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, where: str) -> None:
    if status != PA_OK:
        raise PaError(status, where)


# ---- public calls -------------------------------------------------------------

def write_kv(k, v, slot_mapping, k_cache, v_cache, stream=None) -> None:
    """Scatter k, v [n_tok, Hkv, D] into the caches at slot_mapping [n_tok] (int64).
    k, v and slot_mapping may be page-locked host tensors: the kernel reads them
    over the host link."""
    _dev(k_cache, v_cache)
    _dev_or_pinned(k, v, slot_mapping)
    if slot_mapping.dtype != torch.int64:
        raise ValueError("slot_mapping must be int64")
    if k.dtype != k_cache.dtype or v.dtype != k_cache.dtype or v_cache.dtype != k_cache.dtype:
        raise ValueError("k, v and caches must share one dtype")
    desc = cache_desc(k_cache)
    if tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache and v_cache shapes differ")
    n = slot_mapping.numel()
    if k.shape != (n, desc.num_kv_heads, desc.head_dim) or v.shape != k.shape:
        raise ValueError(f"k, v must be [{n}, {desc.num_kv_heads}, {desc.head_dim}]")
    st = load_library().pa_write_kv(_ptr(k), _ptr(v), _ptr(slot_mapping), n, _ptr(k_cache),
                                    _ptr(v_cache), ctypes.byref(desc), _stream(stream))
    _check(st, "pa_write_kv")


def write_kv_positions(k, v, seq_ids, positions, block_tables, k_cache, v_cache,
                       stream=None) -> None:
    """Scatter k, v [n_tok, Hkv, D] to the slots of (seq_ids[j], positions[j])
    through block_tables [N, max_blocks]; slots are computed on the device.
    Everything but the caches may be page-locked host memory."""
    _dev(k_cache, v_cache)
    _dev_or_pinned(k, v, seq_ids, positions, block_tables)
    for t in (seq_ids, positions, block_tables):
        if t.dtype != torch.int32:
            raise ValueError("seq_ids, positions and block_tables must be int32")
    if k.dtype != k_cache.dtype or v.dtype != k_cache.dtype or v_cache.dtype != k_cache.dtype:
        raise ValueError("k, v and caches must share one dtype")
    desc = cache_desc(k_cache)
    n = seq_ids.numel()
    if positions.numel() != n or k.shape != (n, desc.num_kv_heads, desc.head_dim) \
            or v.shape != k.shape:
        raise ValueError("k, v, seq_ids and positions disagree on the token count")
    st = load_library().pa_write_kv_positions(
        _ptr(k), _ptr(v), _ptr(seq_ids), _ptr(positions), n, _ptr(block_tables),
        block_tables.shape[0], block_tables.shape[1], _ptr(k_cache), _ptr(v_cache),
        ctypes.byref(desc), _stream(stream))
    _check(st, "pa_write_kv_positions")


def copy_blocks(src_k, src_v, dst_k, dst_v, pairs, stream=None) -> None:
    """Copy whole blocks src -> dst for each row (src, dst) of ``pairs``
    (int64 [n, 2]).  Caches may be device tensors or pinned host tensors
    (swap space); the destination may be the source (copy-on-write)."""
    _dev_or_pinned(src_k, src_v, dst_k, dst_v, pairs)
    if pairs.dtype != torch.int64 or pairs.dim() != 2 or pairs.shape[1] != 2:
        raise ValueError("pairs must be int64 [n, 2]")
    if tuple(src_k.shape[1:]) != tuple(dst_k.shape[1:]) or src_k.dtype != dst_k.dtype:
        raise ValueError("source and destination caches differ in block geometry")
    desc = cache_desc(src_k)
    st = load_library().pa_copy_blocks(
        _ptr(src_k), _ptr(src_v), src_k.shape[0], _ptr(dst_k), _ptr(dst_v), dst_k.shape[0],
        _ptr(pairs), pairs.shape[0], ctypes.byref(desc), _stream(stream))
    _check(st, "pa_copy_blocks")


def decode_partition_tokens(num_seqs: int, num_q_heads: int, max_seq_len: int,
                            k_cache) -> int:
    desc = k_cache if isinstance(k_cache, CacheDesc) else cache_desc(k_cache)
    return int(load_library().pa_decode_partition_tokens(num_seqs, num_q_heads, max_seq_len,
                                                         ctypes.byref(desc)))


def decode_workspace_bytes(num_seqs: int, num_q_heads: int, max_seq_len: int, k_cache,
                           partition_tokens: int = 0) -> int:
    desc = k_cache if isinstance(k_cache, CacheDesc) else cache_desc(k_cache)
    return int(load_library().pa_decode_workspace_bytes(num_seqs, num_q_heads, max_seq_len,
                                                        partition_tokens, ctypes.byref(desc)))


def decode_path(num_q_heads: int, k_cache) -> int:
    desc = k_cache if isinstance(k_cache, CacheDesc) else cache_desc(k_cache)
    return int(load_library().pa_decode_path(num_q_heads, ctypes.byref(desc)))


def decode(q, k_cache, v_cache, block_tables, seq_lens, max_seq_len: int,
           scale: float | None = None, out=None, workspace=None, partition_tokens: int = 0,
           stream=None) -> torch.Tensor:
    """Single-query paged attention; returns out [N, Hq, D] in the cache dtype.

    ``max_seq_len`` is a host-side upper bound of ``seq_lens`` (no device
    read-back).  ``workspace`` (uint8, device) is allocated if not given and
    split-K needs one.  q, block_tables, seq_lens and out may be page-locked
    host tensors, read and written by the kernels over the host link; a
    missing ``out`` is allocated on the caches' device.
    """
    _dev(k_cache, v_cache)
    _dev_or_pinned(q, block_tables, seq_lens)
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("block_tables and seq_lens must be int32")
    desc = cache_desc(k_cache)
    n, hq, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q, device=k_cache.device)
    _dev_or_pinned(out)
    need = decode_workspace_bytes(n, hq, max_seq_len, desc, partition_tokens)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=k_cache.device)
    if workspace is not None:
        _dev(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().pa_decode(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
        _ptr(seq_lens), n, max_seq_len, hq, float(scale), partition_tokens, _ptr(out),
        _ptr(workspace), ws_bytes, ctypes.byref(desc), _stream(stream))
    _check(st, "pa_decode")
    return out


def decode_append(q, k_new, v_new, k_cache, v_cache, block_tables, seq_lens,
                  max_seq_len: int, scale: float | None = None, out=None, workspace=None,
                  partition_tokens: int = 0, stream=None) -> torch.Tensor:
    """One decode step in one call: sequence i's newest token, at position
    seq_lens[i] - 1, takes the rows k_new[i], v_new[i] ([N, Hkv, D]) in both
    caches, then the decode runs as ``decode`` does.  Caches and output equal
    ``write_kv_positions`` (positions seq_lens - 1) followed by ``decode``,
    bit for bit; on the TMA decode kernel the write is fused into it."""
    _dev(k_cache, v_cache)
    _dev_or_pinned(q, k_new, v_new, block_tables, seq_lens)
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("block_tables and seq_lens must be int32")
    if k_new.dtype != k_cache.dtype or v_new.dtype != k_cache.dtype \
            or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_new, v_new and caches must share one dtype")
    desc = cache_desc(k_cache)
    n, hq, d = q.shape
    if k_new.shape != (n, desc.num_kv_heads, desc.head_dim) or v_new.shape != k_new.shape:
        raise ValueError(f"k_new, v_new must be [{n}, {desc.num_kv_heads}, {desc.head_dim}]")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q, device=k_cache.device)
    _dev_or_pinned(out)
    need = decode_workspace_bytes(n, hq, max_seq_len, desc, partition_tokens)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=k_cache.device)
    if workspace is not None:
        _dev(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().pa_decode_append(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), n, max_seq_len, hq, float(scale),
        partition_tokens, _ptr(out), _ptr(workspace), ws_bytes, ctypes.byref(desc),
        _stream(stream))
    _check(st, "pa_decode_append")
    return out


class PrefixGroups:
    """The groups of a shared-prefix decode as the C ABI takes them: int32
    tensors ``seq_group`` [num_seqs] (group of each sequence, -1 for none),
    ``member_start`` [num_groups + 1], ``members`` and ``prefix_blocks``
    [num_groups], with the host bounds ``max_group_size`` and
    ``max_prefix_blocks``."""

    def __init__(self, seq_group, member_start, members, prefix_blocks, max_group_size: int,
                 max_prefix_blocks: int):
        self.seq_group = seq_group
        self.member_start = member_start
        self.members = members
        self.prefix_blocks = prefix_blocks
        self.max_group_size = int(max_group_size)
        self.max_prefix_blocks = int(max_prefix_blocks)

    @property
    def num_groups(self) -> int:
        return int(self.prefix_blocks.numel())

    def to(self, device) -> "PrefixGroups":
        return PrefixGroups(self.seq_group.to(device), self.member_start.to(device),
                            self.members.to(device), self.prefix_blocks.to(device),
                            self.max_group_size, self.max_prefix_blocks)


def prefix_groups(groups, num_seqs: int, device=None) -> PrefixGroups:
    """PrefixGroups from a list of (member sequence ids, shared leading
    blocks), e.g. ``BlockPool.shared_prefix_groups``; groups of fewer than
    two members are dropped."""
    groups = [(list(map(int, m)), int(b)) for m, b in groups if len(m) >= 2]
    seq_group = [-1] * num_seqs
    starts, members, blocks = [0], [], []
    for k, (mem, b) in enumerate(groups):
        for i in mem:
            seq_group[i] = k
        members += mem
        starts.append(len(members))
        blocks.append(b)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=device)

    return PrefixGroups(i32(seq_group), i32(starts), i32(members), i32(blocks),
                        max((len(m) for m, _ in groups), default=0),
                        max(blocks, default=0))


def decode_shared_prefix_workspace_bytes(num_seqs: int, num_q_heads: int, max_seq_len: int,
                                         max_prefix_blocks: int, k_cache,
                                         partition_tokens: int = 0) -> int:
    desc = k_cache if isinstance(k_cache, CacheDesc) else cache_desc(k_cache)
    return int(load_library().pa_decode_shared_prefix_workspace_bytes(
        num_seqs, num_q_heads, max_seq_len, max_prefix_blocks, partition_tokens,
        ctypes.byref(desc)))


def decode_shared_prefix_mode(num_q_heads: int, max_prefix_blocks: int, k_cache,
                              mode: int = SHARED_AUTO) -> int:
    """1 when decode_shared_prefix reads the shared blocks once per row tile
    for these arguments, 0 when it runs the plain decode."""
    desc = k_cache if isinstance(k_cache, CacheDesc) else cache_desc(k_cache)
    return int(load_library().pa_decode_shared_prefix_mode(num_q_heads, max_prefix_blocks,
                                                           mode, ctypes.byref(desc)))


def decode_shared_prefix(q, k_cache, v_cache, block_tables, seq_lens, max_seq_len: int,
                         groups: PrefixGroups, scale: float | None = None, out=None,
                         workspace=None, partition_tokens: int = 0, mode: int = SHARED_AUTO,
                         stream=None) -> torch.Tensor:
    """``decode`` for a batch whose ``groups`` of sequences share leading
    blocks: the same result, with each group's shared blocks read once per
    kv head and row tile instead of once per member (``mode``: SHARED_ONCE,
    SHARED_PLAIN, or SHARED_AUTO to choose by the expected saving)."""
    _dev(k_cache, v_cache)
    _dev_or_pinned(q, block_tables, seq_lens, groups.seq_group, groups.member_start,
                   groups.members, groups.prefix_blocks)
    for t in (block_tables, seq_lens, groups.seq_group, groups.member_start, groups.members,
              groups.prefix_blocks):
        if t.dtype != torch.int32:
            raise ValueError("tables, lengths and group arrays must be int32")
    desc = cache_desc(k_cache)
    n, hq, d = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q, device=k_cache.device)
    _dev_or_pinned(out)
    need = decode_shared_prefix_workspace_bytes(n, hq, max_seq_len, groups.max_prefix_blocks,
                                                desc, partition_tokens)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=k_cache.device)
    if workspace is not None:
        _dev(workspace)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = load_library().pa_decode_shared_prefix(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), block_tables.shape[1],
        _ptr(seq_lens), n, max_seq_len, hq, float(scale), partition_tokens,
        _ptr(groups.seq_group), _ptr(groups.member_start), _ptr(groups.members),
        _ptr(groups.prefix_blocks), groups.num_groups, groups.max_group_size,
        groups.max_prefix_blocks, mode, _ptr(out), _ptr(workspace), ws_bytes,
        ctypes.byref(desc), _stream(stream))
    _check(st, "pa_decode_shared_prefix")
    return out


def last_device_error() -> int:
    """PA_DEVERR_* bits raised since the last call (synchronises the device)."""
    return int(load_library().pa_last_device_error())


def check_wait_timeout(expected: int, arrivals: int, limit_cycles: int, stream=None) -> None:
    """Runs the bounded-wait check: an mbarrier needing `expected` arrivals
    gets `arrivals`, and one CTA waits for it for at most `limit_cycles`
    clocks (PA_DEVERR_TIMEOUT when it gives up; read last_device_error())."""
    st = load_library().pa_check_wait_timeout(expected, arrivals, limit_cycles,
                                              _stream(stream))
    _check(st, "pa_check_wait_timeout")


def prefill(q, query_start_loc, k_cache, v_cache, block_tables, seq_lens, max_q_len: int,
            max_seq_len: int, scale: float | None = None, out=None, stream=None):
    """Causal multi-query attention over the paged cache: sequence i's packed
    rows query_start_loc[i]..query_start_loc[i+1] are its last positions.
    Returns out [total_q, Hq, D] in the cache dtype.  Everything but the
    caches may be page-locked host memory (read and written over the host
    link); a missing ``out`` is allocated on the caches' device."""
    _dev(k_cache, v_cache)
    _dev_or_pinned(q, query_start_loc, block_tables, seq_lens)
    for t in (query_start_loc, block_tables, seq_lens):
        if t.dtype != torch.int32:
            raise ValueError("query_start_loc, block_tables and seq_lens must be int32")
    desc = cache_desc(k_cache)
    total, hq, d = q.shape
    if query_start_loc.numel() != seq_lens.numel() + 1:
        raise ValueError("query_start_loc must have num_seqs + 1 entries")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q, device=k_cache.device)
    _dev_or_pinned(out)
    st = load_library().pa_prefill(
        _ptr(q), _ptr(query_start_loc), total, max_q_len, _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), seq_lens.numel(), max_seq_len,
        hq, float(scale), _ptr(out), ctypes.byref(desc), _stream(stream))
    _check(st, "pa_prefill")
    return out


# ---- drafted (speculative) steps ------------------------------------------------
#
# These calls run once a layer or a step with little work on the GPU, so their
# checks here are few: what would be read wrongly (dtype, strides, sizes).  Where
# the memory is, the library checks (PaError for another device's or pageable
# memory).

def _contiguous(*ts) -> None:
    for t in ts:
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def _int32(*ts) -> None:
    i32 = torch.int32
    for t in ts:
        if t.dtype is not i32:
            raise ValueError("lengths, tables, rows and indices must be int32")


def _current(t) -> int:
    """Index of ``t``'s device, which must be the current one."""
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    device = t.get_device()
    if device != torch.cuda.current_device():
        raise ValueError(f"tensors live on device {device}, which is not the current one")
    return device


def _raw_stream(stream, device: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return _stream(stream)


def _empty(shape, dtype, device: int, stream):
    """A tensor for a call on ``stream``, from that stream's memory: what the
    call leaves behind is only reused by work ordered after it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class StepPlan:
    """What ``plan_step`` writes, all int32 but slot_mapping (int64):
    ``seq_lens`` and ``blocks_held`` [N] after the step, ``free_head`` [1],
    ``query_start_loc`` and ``block_start`` [N + 1], and per packed token
    ``slot_mapping``, ``positions`` and ``seq_ids`` [max_tokens] (the last two
    may be None).  A loop keeps one plan and passes it every step."""

    __slots__ = ("seq_lens", "blocks_held", "free_head", "query_start_loc", "block_start",
                 "slot_mapping", "positions", "seq_ids")

    def __init__(self, seq_lens, blocks_held, free_head, query_start_loc, block_start,
                 slot_mapping, positions=None, seq_ids=None):
        self.seq_lens = seq_lens
        self.blocks_held = blocks_held
        self.free_head = free_head
        self.query_start_loc = query_start_loc
        self.block_start = block_start
        self.slot_mapping = slot_mapping
        self.positions = positions
        self.seq_ids = seq_ids

    @classmethod
    def empty(cls, num_seqs: int, max_tokens: int, device="cuda") -> "StepPlan":
        """Buffers for a step of num_seqs sequences, no fewer, and up to
        max_tokens tokens.  (Views of their first entries make the plan of a
        smaller batch: [:n] of seq_lens and blocks_held, [:n + 1] of
        query_start_loc and block_start.)"""
        def i32(n):
            return torch.empty(n, dtype=torch.int32, device=device)

        return cls(i32(num_seqs), i32(num_seqs), i32(1), i32(num_seqs + 1), i32(num_seqs + 1),
                   torch.empty(max_tokens, dtype=torch.int64, device=device), i32(max_tokens),
                   i32(max_tokens))


def plan_step(seq_lens, new_tokens, block_tables, blocks_held, free_blocks, free_head,
              num_blocks: int, block_size: int, plan: StepPlan | None = None,
              max_tokens: int | None = None, ref_cnt=None, stream=None) -> StepPlan:
    """Block tables and slot mapping of a step from the requests' lengths, on
    the device: ``BlockPool.grow`` for every sequence in order.

    Sequence i has seq_lens[i] cached tokens, gets new_tokens[i] more and
    holds the first blocks_held[i] entries of its row of ``block_tables``
    [N, max_blocks] (updated in place); blocks come from the front of
    ``free_blocks`` (int32, from index free_head[0]).  Writes ``plan`` (or a
    new one for ``max_tokens`` tokens) and returns it; its seq_lens,
    blocks_held and free_head may be the input tensors.  A step that does not
    fit plans nothing and raises a bit of ``last_device_error``
    (DEVERR_POOL, DEVERR_SHARED, DEVERR_SEQ_LEN).  ``ref_cnt`` (int32
    [num_blocks]) adds the check for shared blocks and the counts of taken ones."""
    device = _current(block_tables)
    n = seq_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != n or new_tokens.numel() != n \
            or blocks_held.numel() != n or free_head.numel() != 1:
        raise ValueError("seq_lens, new_tokens, blocks_held and block_tables disagree on the "
                         "sequence count")
    if plan is None:
        if max_tokens is None:
            raise ValueError("pass a plan or max_tokens")
        i32 = torch.int32
        plan = StepPlan(*(_empty(k, i32, device, stream) for k in (n, n, 1, n + 1, n + 1)),
                        _empty(max_tokens, torch.int64, device, stream),
                        _empty(max_tokens, i32, device, stream),
                        _empty(max_tokens, i32, device, stream))
    lens_out, held_out, head_out = plan.seq_lens, plan.blocks_held, plan.free_head
    start, taken, slots = plan.query_start_loc, plan.block_start, plan.slot_mapping
    positions, seq_ids = plan.positions, plan.seq_ids
    tokens = slots.numel()
    if lens_out.numel() != n or held_out.numel() != n or head_out.numel() != 1 \
            or start.numel() != n + 1 or taken.numel() != n + 1 \
            or (positions is not None and positions.numel() != tokens) \
            or (seq_ids is not None and seq_ids.numel() != tokens) \
            or (max_tokens is not None and max_tokens != tokens):
        raise ValueError("the plan's buffers do not fit the step")
    ints = (seq_lens, new_tokens, blocks_held, free_blocks, free_head, block_tables, lens_out,
            held_out, head_out, start, taken)
    if positions is not None:
        ints += (positions,)
    if seq_ids is not None:
        ints += (seq_ids,)
    if ref_cnt is not None:
        ints += (ref_cnt,)
        if ref_cnt.numel() != num_blocks:
            raise ValueError("ref_cnt must have num_blocks entries")
    if slots.dtype is not torch.int64:
        raise ValueError("slot_mapping must be int64")
    _int32(*ints)
    _contiguous(slots, *ints)
    st = load_library().pa_plan_step(
        seq_lens.data_ptr(), new_tokens.data_ptr(), blocks_held.data_ptr(), n,
        free_blocks.data_ptr(), free_blocks.numel(), free_head.data_ptr(), _ptr(ref_cnt),
        num_blocks, block_size, block_tables.data_ptr(), block_tables.shape[1],
        lens_out.data_ptr(), held_out.data_ptr(), head_out.data_ptr(), start.data_ptr(),
        taken.data_ptr(), slots.data_ptr(), _ptr(positions), _ptr(seq_ids), tokens,
        _raw_stream(stream, device))
    if st != PA_OK:
        raise PaError(st, "pa_plan_step")
    return plan


def decode_tree_workspace_bytes(num_seqs: int, total_q: int, num_q_heads: int, max_q_len: int,
                                max_seq_len: int, k_cache) -> int:
    desc = k_cache if isinstance(k_cache, CacheDesc) else cache_desc(k_cache)
    return int(load_library().pa_decode_tree_workspace_bytes(
        num_seqs, total_q, num_q_heads, max_q_len, max_seq_len, ctypes.byref(desc)))


def decode_tree(q, query_start_loc, parents, k_cache, v_cache, block_tables, seq_lens,
                max_q_len: int, max_seq_len: int, scale: float | None = None, out=None,
                workspace=None, stream=None) -> torch.Tensor:
    """Attention of trees of drafted tokens over the paged cache: sequence i's
    packed rows query_start_loc[i]..query_start_loc[i+1] are its tree's nodes,
    already in the cache at its last positions.  A node sees the cached
    tokens, its ancestors (``parents`` [total_q]: the node it continues,
    within its sequence, -1 for the cached tokens) and itself.  Returns out
    [total_q, Hq, D] in the cache dtype; rows behind the last sequence are
    left as they were (a missing ``out`` is allocated, not cleared)."""
    device = _current(k_cache)
    shape, q_shape, dtype = k_cache.shape, q.shape, k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache are [num_blocks, num_kv_heads, block_size, "
                         "head_dim], of one shape")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported cache dtype {dtype}")
    blocks, heads, block, d = shape
    desc = CacheDesc(blocks, block, heads, d, _DTYPES[dtype])
    if len(q_shape) != 3 or q_shape[2] != d:
        raise ValueError(f"q must be [total_q, num_q_heads, {d}]")
    total, hq, _ = q_shape
    n = seq_lens.numel()
    if q.dtype is not dtype or v_cache.dtype is not dtype:
        raise ValueError("q and caches must share one dtype")
    _int32(query_start_loc, parents, block_tables, seq_lens)
    if query_start_loc.numel() != n + 1 or parents.numel() != total \
            or block_tables.dim() != 2 or block_tables.shape[0] != n:
        raise ValueError("query_start_loc, parents, block_tables and seq_lens disagree on the "
                         "sequence or row count")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty(q_shape, dtype, device, stream)
    elif out.shape != q_shape or out.dtype is not dtype:
        raise ValueError("out must have q's shape and dtype")
    lib = load_library()
    ref = ctypes.byref(desc)
    if workspace is None:
        ws_bytes = lib.pa_decode_tree_workspace_bytes(n, total, hq, max_q_len, max_seq_len, ref)
        if ws_bytes:
            workspace = _empty(ws_bytes, torch.uint8, device, stream)
    else:
        _contiguous(workspace)
        ws_bytes = workspace.numel() * workspace.element_size()
    _contiguous(k_cache, v_cache, q, query_start_loc, parents, block_tables, seq_lens, out)
    st = lib.pa_decode_tree(
        q.data_ptr(), query_start_loc.data_ptr(), parents.data_ptr(), total, max_q_len,
        k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
        seq_lens.data_ptr(), n, max_seq_len, hq, scale, out.data_ptr(), _ptr(workspace),
        ws_bytes, ref, _raw_stream(stream, device))
    if st != PA_OK:
        raise PaError(st, "pa_decode_tree")
    return out


def _layer_caches(caches):
    """(one layer's shape, dtype, device, addresses of all layers) of one
    cache, a stack of them, or a sequence."""
    if isinstance(caches, torch.Tensor):
        shape = caches.shape
        if not (caches.is_cuda and caches.is_contiguous()):
            raise ValueError("caches must be contiguous CUDA tensors")
        base = caches.data_ptr()
        if len(shape) == 4:
            return shape, caches.dtype, caches.get_device(), (base,)
        if len(shape) != 5 or shape[0] < 1:
            raise ValueError("caches are [num_blocks, num_kv_heads, block_size, head_dim], with "
                             "a leading dimension of layers or in a sequence")
        step = caches.stride(0) * caches.element_size()
        return shape[1:], caches.dtype, caches.get_device(), range(base, base + step * shape[0],
                                                                   step)
    caches = list(caches)
    if not caches or caches[0].dim() != 4:
        raise ValueError("caches are [num_blocks, num_kv_heads, block_size, head_dim], with "
                         "a leading dimension of layers or in a sequence")
    first = caches[0]
    for c in caches:
        if c.shape != first.shape or c.dtype is not first.dtype or c.device != first.device \
                or not (c.is_cuda and c.is_contiguous()):
            raise ValueError("the caches must share one shape, dtype and CUDA device, and be "
                             "contiguous")
    return first.shape, first.dtype, first.get_device(), [c.data_ptr() for c in caches]


def accept_tree(leaf, parents, query_start_loc, seq_lens, k_caches, v_caches, block_tables,
                max_q_len: int, new_lens=None, accepted_rows=None, stream=None):
    """Keeps each tree's accepted path: leaf[i] is its deepest accepted node
    (-1: none); the K/V rows of that node and its ancestors move to the
    positions right behind the cached tokens, in every layer.  ``k_caches``
    and ``v_caches`` are one cache each, a [layers, num_blocks, Hkv, B, D]
    tensor, or a sequence of caches.  Returns (new_lens [N], accepted_rows
    [total_q]): the lengths with the path, and per sequence the packed rows
    of its path from its first row on, then -1 (a refused sequence's are all
    -1; rows behind the last sequence are left as they were)."""
    shape, dtype, device, keys = _layer_caches(k_caches)
    v_shape, v_dtype, v_device, values = _layer_caches(v_caches)
    if device != torch.cuda.current_device():
        raise ValueError(f"tensors live on device {device}, which is not the current one")
    if len(keys) != len(values) or v_shape != shape or v_dtype is not dtype \
            or v_device != device:
        raise ValueError("k_caches and v_caches must have the same layers, shape and dtype")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported cache dtype {dtype}")
    n, total = seq_lens.numel(), parents.numel()
    if leaf.numel() != n or query_start_loc.numel() != n + 1 or block_tables.dim() != 2 \
            or block_tables.shape[0] != n:
        raise ValueError("leaf, query_start_loc, block_tables and seq_lens disagree on the "
                         "sequence count")
    if new_lens is None:
        new_lens = _empty(n, torch.int32, device, stream)
    if accepted_rows is None:
        accepted_rows = _empty(total, torch.int32, device, stream)
    if new_lens.numel() != n or accepted_rows.numel() != total:
        raise ValueError("new_lens must have N and accepted_rows total_q entries")
    ints = (leaf, parents, query_start_loc, seq_lens, block_tables, new_lens, accepted_rows)
    _int32(*ints)
    _contiguous(*ints)
    ptrs = ctypes.c_void_p * len(keys)
    desc = CacheDesc(shape[0], shape[2], shape[1], shape[3], _DTYPES[dtype])
    st = load_library().pa_accept_tree(
        leaf.data_ptr(), parents.data_ptr(), query_start_loc.data_ptr(), seq_lens.data_ptr(), n,
        total, max_q_len, block_tables.data_ptr(), block_tables.shape[1], ptrs(*keys),
        ptrs(*values), len(keys), new_lens.data_ptr(), accepted_rows.data_ptr(),
        ctypes.byref(desc), _raw_stream(stream, device))
    if st != PA_OK:
        raise PaError(st, "pa_accept_tree")
    return new_lens, accepted_rows


# ---- around the attention -----------------------------------------------------------

@functools.lru_cache(maxsize=256)
def _descriptors(cache: tuple, rope: tuple, sections: tuple):
    """The C structs of a cache's and a rotation's plain values (a model's layers
    pass the same ones every step)."""
    return (ctypes.byref(CacheDesc(*cache)),
            ctypes.byref(RopeDesc(rope[0], rope[1], (ctypes.c_int32 * 3)(*sections), *rope[2:])))


def _token_rows(t, d: int, what: str):
    """(tokens, heads, elements from token to token) of [n, heads, D] rows whose
    heads follow one another; tokens may be apart (slices of a projection)."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[2] != d:
        raise ValueError(f"{what} must be [num_tokens, heads, {d}]")
    n, heads, _ = shape
    if n > 1 and stride[2] == 1 and stride[1] == d and stride[0] >= heads * d:
        return n, heads, stride[0]
    if (d > 1 and stride[2] != 1) or (heads > 1 and stride[1] != d) \
            or (n > 1 and stride[0] < heads * d):
        raise ValueError(f"the heads of {what} must follow one another, tokens without overlap")
    return n, heads, stride[0] if n > 1 else heads * d


def rope_write(q, k, v, positions, inv_freq, slot_mapping, k_cache, v_cache, q_weight=None,
               k_weight=None, eps: float = 1e-6, sections=None, cyclic: bool = False,
               neighbours: bool = False, scale: float = 1.0, out=None, stream=None):
    """A layer's projected rows to its attention in one pass: each head of q
    [n, Hq, D] and k [n, Hkv, D] is normed (``q_weight``, ``k_weight`` [D]; None:
    not normed) and its first 2 * len(``inv_freq``) dimensions rotated by the
    token's position; the keys and v [n, Hkv, D] go to the caches at
    ``slot_mapping``.  Returns the queries, ``out`` [n, Hq, D].

    ``positions`` is int32 [n], or [axes, n] with ``sections``, the pairs of each of
    2 or 3 axes (in order; ``cyclic``: the axes alternate).  Pair j is (j, j +
    len(inv_freq)), with ``neighbours`` (2 j, 2 j + 1).  ``scale`` multiplies cos and
    sin.  q, k and v may be slices of one projection's rows (tokens apart, heads
    together).  A token with a negative (first) position is skipped, its row of
    ``out`` left as it was; one with a negative slot is not cached.  ``out`` may be
    q itself where its tokens follow one another."""
    device = _current(k_cache)
    shape, dtype = k_cache.shape, k_cache.dtype
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache are [num_blocks, num_kv_heads, block_size, "
                         "head_dim], of one shape")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported cache dtype {dtype}")
    blocks, heads, block, d = shape
    n, hq, q_stride = _token_rows(q, d, "q")
    kn, k_heads, k_stride = _token_rows(k, d, "k")
    vn, v_heads, v_stride = _token_rows(v, d, "v")
    if kn != n or vn != n or k_heads != heads or v_heads != heads:
        raise ValueError(f"k, v must be [{n}, {heads}, {d}]")
    if q.dtype is not dtype or k.dtype is not dtype or v.dtype is not dtype \
            or v_cache.dtype is not dtype:
        raise ValueError("q, k, v and caches must share one dtype")
    for w in (q_weight, k_weight):
        if w is not None:
            if w.dtype is not dtype or w.numel() != d:
                raise ValueError(f"norm weights must be [{d}], of the caches' dtype")
            _contiguous(w)
    axes = 1 if sections is None else len(sections)
    if not 1 <= axes <= 3:
        raise ValueError("sections are the pairs of 1 to 3 axes")
    if positions.numel() != axes * n or slot_mapping.numel() != n \
            or (positions.dim() == 2 and positions.shape[0] != axes):
        raise ValueError("positions ([n], or [axes, n] with sections) and slot_mapping [n] must "
                         "have an entry per token")
    if slot_mapping.dtype is not torch.int64 or inv_freq.dtype is not torch.float32:
        raise ValueError("slot_mapping must be int64 and inv_freq float32")
    _int32(positions)
    if out is None:
        out = _empty((n, hq, d), dtype, device, stream)
    elif out.shape != q.shape or out.dtype is not dtype:
        raise ValueError("out must have q's shape and dtype")
    _contiguous(k_cache, v_cache, positions, inv_freq, slot_mapping, out)
    desc, rope = _descriptors((blocks, block, heads, d, _DTYPES[dtype]),
                              (2 * inv_freq.numel(), axes, bool(cyclic), bool(neighbours),
                               float(scale), float(eps)),
                              () if sections is None else tuple(map(operator.index, sections)))
    st = load_library().pa_rope_write(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), q_stride, k_stride, v_stride, n, hq,
        positions.data_ptr(), inv_freq.data_ptr(), _ptr(q_weight), _ptr(k_weight),
        rope, slot_mapping.data_ptr(), out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), desc,
        _raw_stream(stream, device))
    if st != PA_OK:
        raise PaError(st, "pa_rope_write")
    return out


def _rows(t, what: str) -> int:
    """Elements from row to row of a matrix whose rows' elements follow one another."""
    if t.dim() != 2:
        raise ValueError(f"{what} must have two dimensions")
    width, (step, one) = t.shape[1], t.stride()
    if (width > 1 and one != 1) or (t.shape[0] > 1 and step < width):
        raise ValueError(f"the elements of a row of {what} must follow one another, rows without "
                         "overlap")
    return step if t.shape[0] > 1 else width


def verify_tree(logits, tokens, parents, query_start_loc, uniforms, noise, max_q_len: int,
                draft_logits=None, temperature=None, leaf=None, next_tokens=None, stream=None):
    """Which drafted tokens hold against the target's probabilities, and the token
    that follows, from given random numbers.  Returns (leaf, next_tokens), int32
    [N]: each tree's deepest node that holds (what ``accept_tree`` takes) and the
    token drawn behind it.

    Sequence i's nodes are the rows query_start_loc[i]..query_start_loc[i+1]; node 0
    is its last sampled token, whose drafted continuations are the nodes below it
    (``parents`` as in ``decode_tree``, ``tokens`` [total_q]).  ``logits``
    [total_q, V] are the target's behind each node, ``draft_logits`` the draft's
    that the node's children were drawn from (None: the children were chosen, not
    drawn).  ``uniforms`` [total_q] in [0, 1) decide each drafted token, exponential
    ``noise`` [N, V] the next one; ``temperature`` [N] divides both logits (0:
    greedy; None: 1).  With one node a sequence it samples plainly."""
    device = _current(logits)
    dtype = logits.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported logits dtype {dtype}")
    step = _rows(logits, "logits")
    noise_step = _rows(noise, "noise")
    total, vocab = logits.shape
    n = query_start_loc.numel() - 1
    draft_step = 0
    if draft_logits is not None:
        draft_step = _rows(draft_logits, "draft_logits")
        if draft_logits.shape != logits.shape or draft_logits.dtype is not dtype:
            raise ValueError("draft_logits must have the shape and dtype of logits")
    if n < 0 or tokens.numel() != total or parents.numel() != total \
            or uniforms.numel() != total or tuple(noise.shape) != (n, vocab):
        raise ValueError("logits, tokens, parents and uniforms must have a row per node, noise "
                         "[N, V] one per sequence")
    f32 = torch.float32
    if uniforms.dtype is not f32 or noise.dtype is not f32 \
            or (temperature is not None and temperature.dtype is not f32):
        raise ValueError("uniforms, noise and temperature must be float32")
    if temperature is not None:
        if temperature.numel() != n:
            raise ValueError("temperature must have an entry per sequence")
        _contiguous(temperature)
    if leaf is None:
        leaf = _empty(n, torch.int32, device, stream)
    if next_tokens is None:
        next_tokens = _empty(n, torch.int32, device, stream)
    if leaf.numel() != n or next_tokens.numel() != n:
        raise ValueError("leaf and next_tokens must have an entry per sequence")
    _int32(tokens, parents, query_start_loc, leaf, next_tokens)
    _contiguous(tokens, parents, query_start_loc, uniforms, leaf, next_tokens)
    st = load_library().pa_verify_tree(
        logits.data_ptr(), _ptr(draft_logits), step, draft_step, vocab, _DTYPES[dtype],
        tokens.data_ptr(), parents.data_ptr(), query_start_loc.data_ptr(), n, total, max_q_len,
        uniforms.data_ptr(), noise.data_ptr(), noise_step, _ptr(temperature), leaf.data_ptr(),
        next_tokens.data_ptr(), _raw_stream(stream, device))
    if st != PA_OK:
        raise PaError(st, "pa_verify_tree")
    return leaf, next_tokens


def release_blocks(seq_lens, block_tables, blocks_held, free_blocks, free_head, num_blocks: int,
                   block_size: int, ref_cnt=None, blocks_held_out=None, free_head_out=None,
                   stream=None):
    """Blocks that sequences no longer need go back to the free queue of
    ``plan_step``, on the device (``BlockPool.release``).  Sequence i keeps the
    blocks of its first seq_lens[i] tokens (0 for a finished request); the others
    of its blocks_held[i] lose a reference in ``ref_cnt`` (int32 [num_blocks]; None:
    no block is shared), and those at none are put in front of the queue, in the
    order of sequences and table entries.  The counts are those that ``plan_step`` and
    ``fork_blocks`` were given; a finished request's length is 0 for the next
    ``plan_step`` too.  Returns (blocks_held, free_head) after it, new tensors or the given ones, which may be the inputs.  All or nothing,
    with a bit of ``last_device_error`` (DEVERR_SEQ_LEN, DEVERR_POOL,
    DEVERR_SHARED)."""
    device = _current(block_tables)
    n = seq_lens.numel()
    if block_tables.dim() != 2 or block_tables.shape[0] != n or blocks_held.numel() != n \
            or free_head.numel() != 1:
        raise ValueError("seq_lens, blocks_held and block_tables disagree on the sequence count")
    if blocks_held_out is None:
        blocks_held_out = _empty(n, torch.int32, device, stream)
    if free_head_out is None:
        free_head_out = _empty(1, torch.int32, device, stream)
    if blocks_held_out.numel() != n or free_head_out.numel() != 1:
        raise ValueError("blocks_held_out must have N entries, free_head_out one")
    ints = (seq_lens, block_tables, blocks_held, free_blocks, free_head, blocks_held_out,
            free_head_out)
    if ref_cnt is not None:
        ints += (ref_cnt,)
        if ref_cnt.numel() != num_blocks:
            raise ValueError("ref_cnt must have num_blocks entries")
    _int32(*ints)
    _contiguous(*ints)
    st = load_library().pa_release_blocks(
        seq_lens.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
        blocks_held.data_ptr(), n, free_blocks.data_ptr(), free_blocks.numel(),
        free_head.data_ptr(), _ptr(ref_cnt), num_blocks, block_size, blocks_held_out.data_ptr(),
        free_head_out.data_ptr(), _raw_stream(stream, device))
    if st != PA_OK:
        raise PaError(st, "pa_release_blocks")
    return blocks_held_out, free_head_out


def fork_blocks(src, seq_lens, block_tables, blocks_held, ref_cnt, free_blocks, free_head,
                k_caches, v_caches, seq_lens_out=None, blocks_held_out=None, free_head_out=None,
                block_pairs=None, stream=None):
    """Sequences that start as copies of others, on the device
    (``BlockPool.fork``): row i with src[i] >= 0, which holds no blocks, shares the
    full blocks of sequence src[i] (``ref_cnt`` int32 [num_blocks] counts them: the
    same that ``plan_step`` counts the blocks it takes in) and
    gets a fresh block of the queue with a copy of its partly filled one, in every
    layer of ``k_caches`` and ``v_caches`` (as in ``accept_tree``).  Rows of
    ``block_tables`` are written in place.  Returns (seq_lens, blocks_held,
    free_head, block_pairs) after it, new tensors or the given ones, the first
    three of which may be the inputs; block_pairs int64 [N, 2] are the copied blocks
    (source, fresh), -1 where none was.  All or nothing, with a bit of
    ``last_device_error`` (DEVERR_FORK, DEVERR_SEQ_LEN, DEVERR_POOL)."""
    shape, dtype, device, keys = _layer_caches(k_caches)
    v_shape, v_dtype, v_device, values = _layer_caches(v_caches)
    if device != torch.cuda.current_device():
        raise ValueError(f"tensors live on device {device}, which is not the current one")
    if len(keys) != len(values) or v_shape != shape or v_dtype is not dtype \
            or v_device != device:
        raise ValueError("k_caches and v_caches must have the same layers, shape and dtype")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported cache dtype {dtype}")
    n = seq_lens.numel()
    if src.numel() != n or blocks_held.numel() != n or block_tables.dim() != 2 \
            or block_tables.shape[0] != n or free_head.numel() != 1:
        raise ValueError("src, seq_lens, blocks_held and block_tables disagree on the sequence "
                         "count")
    if ref_cnt.numel() != shape[0]:
        raise ValueError("ref_cnt must have num_blocks entries")
    i32 = torch.int32
    if seq_lens_out is None:
        seq_lens_out = _empty(n, i32, device, stream)
    if blocks_held_out is None:
        blocks_held_out = _empty(n, i32, device, stream)
    if free_head_out is None:
        free_head_out = _empty(1, i32, device, stream)
    if block_pairs is None:
        block_pairs = _empty((n, 2), torch.int64, device, stream)
    if seq_lens_out.numel() != n or blocks_held_out.numel() != n or free_head_out.numel() != 1 \
            or block_pairs.numel() != 2 * n or block_pairs.dtype is not torch.int64:
        raise ValueError("seq_lens_out and blocks_held_out must have N entries, free_head_out one, "
                         "block_pairs int64 [N, 2]")
    ints = (src, seq_lens, block_tables, blocks_held, ref_cnt, free_blocks, free_head,
            seq_lens_out, blocks_held_out, free_head_out)
    _int32(*ints)
    _contiguous(block_pairs, *ints)
    ptrs = ctypes.c_void_p * len(keys)
    desc = CacheDesc(shape[0], shape[2], shape[1], shape[3], _DTYPES[dtype])
    st = load_library().pa_fork_blocks(
        src.data_ptr(), seq_lens.data_ptr(), block_tables.data_ptr(), block_tables.shape[1],
        blocks_held.data_ptr(), n, ref_cnt.data_ptr(), free_blocks.data_ptr(),
        free_blocks.numel(), free_head.data_ptr(), ptrs(*keys), ptrs(*values), len(keys),
        seq_lens_out.data_ptr(), blocks_held_out.data_ptr(), free_head_out.data_ptr(),
        block_pairs.data_ptr(), ctypes.byref(desc), _raw_stream(stream, device))
    if st != PA_OK:
        raise PaError(st, "pa_fork_blocks")
    return seq_lens_out, blocks_held_out, free_head_out, block_pairs
