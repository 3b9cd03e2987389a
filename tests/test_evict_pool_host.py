"""Eviction inside one pool: which arrays two caches may share (arguments only, no GPU)."""
from __future__ import annotations

import ctypes

from block_sparse_gqa_min_b200 import sba
from tests.test_small_cache_host import ARG, c4, c16

CUDA = sba.SBA_ERR_CUDA     # past the checks: the launch finds no GPU here


def test_one_pool_shares_its_arrays():
    import torch

    if torch.cuda.is_available():
        return                                                # (addresses are made up)
    lib, e = sba.load(), ctypes.byref(sba.evict_params(64))
    acc, new, kept = 0x50000, 0x600000, 0x700000

    def four(src, dst, acc_dst):
        return lib.sba_evict_kv4(c4(**src), acc, e, c4(**dst), acc_dst, new, kept, None)

    def bf16(src, dst, acc_dst):
        return lib.sba_evict(c16(**src), acc, e, c16(**dst), acc_dst, new, kept, None)

    a, b = dict(block_table=0x800000), dict(block_table=0x900000)
    for call in (four, bf16):
        # two tables, or a table on one side only: the pages can be apart
        assert call(a, b, acc) == CUDA and call(a, {}, acc) == CUDA and call({}, b, acc) == CUDA
        assert call(a, b, None) == CUDA
        assert call({}, {}, acc) == ARG and call({}, {}, None) == ARG
    # weights of two pools are two arrays, and arrays that overlap are refused
    pool = dict(kv=0x10000000, desc=None)
    size = 64 * 2 * 64 * 4
    assert four(a, {**b, **pool}, acc) == ARG and four({}, pool, acc) == ARG
    assert four({}, pool, acc + size) == CUDA and four({}, pool, acc + size - 16) == ARG
    assert four(a, b, acc + 16) == ARG
    assert bf16(a, {**b, "v": 0x20000000}, acc) == ARG
    # a destination that begins at a later page of the pool: its weights at that page, or apart
    page4, page16, cells = 2 * 2 * 4608, 2 * 64 * 256, 2 * 64 * 4
    part = dict(block_table=0x900000, desc=None)
    for pages in (1, 40, -3):
        later = dict(**part, kv=0x1000 + pages * page4)
        assert four(a, later, acc + pages * cells) == CUDA and four(a, later, acc + (pages + 1) * cells) == ARG
        assert four(a, later, acc) == ARG and four(a, later, acc + 2 * size) == CUDA
        both = dict(**part, k=0x1000 + pages * page16, v=0x2000 + pages * page16)
        assert bf16(a, both, acc + pages * cells) == CUDA and bf16(a, {**both, "v": 0x2000}, acc + pages * cells) == ARG
    assert four(a, dict(**part, kv=0x1000 + 16), acc) == ARG
    # descriptors of another pool are another array, unless its own table keeps the pages apart
    assert four({}, dict(kv=0x10000000), None) == ARG and four(a, dict(kv=0x10000000), None) == ARG
