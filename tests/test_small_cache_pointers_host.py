"""Pointers of the smaller cache's calls that a kernel could not read or write as they are: refused on the host."""
from __future__ import annotations

import ctypes

import pytest
import torch

from block_sparse_gqa_min_b200 import sba
from tests.test_small_cache_host import ARG, c4, c16

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses are made up: nothing may run")
ODD = 0x6002


def test_words_have_to_be_aligned():
    lib, p = sba.load(), ctypes.byref(sba.evict_params(64))
    other = c4(kv=0x100000, desc=None)
    assert lib.sba_append_kv4(c4(), 0x8000, 0x9000, ODD, 1, None) == ARG
    assert lib.sba_read_kv4(c4(), ODD, 1, 0x8000, 0x9000, None) == ARG
    for idx, cnt, lse in ((ODD, 0x7000, None), (0x7000, ODD, None), (0x7000, 0x8000, ODD)):
        assert lib.sba_decode_kv4(c4(), 0x5000, 1, idx, cnt, 4, 0.1, 0x6000, 0, lse, 0x8000, 1 << 30, None) == ARG
    for idx, cnt, bias in ((ODD, 0x7000, None), (0x7000, ODD, None), (0x7000, 0x8000, ODD)):
        assert lib.sba_accumulate_weights(c16(), 0x5000, 1, idx, cnt, bias, 4, 0.1, 0xa000, 0xb000, 0xb000, None) == ARG
    for acc_dst, new, kept in ((ODD, 0x7000, 0x8000), (None, ODD, 0x8000), (None, 0x7000, ODD)):
        assert lib.sba_evict_kv4(c4(), 0x5000, p, other, acc_dst, new, kept, None) == ARG
    for bad in (dict(seq_lens=ODD), dict(block_table=ODD), dict(status=ODD)):
        assert lib.sba_append_kv4(c4(**bad), 0x8000, 0x9000, 0x7000, 1, None) == ARG
        assert lib.sba_evict(c16(**bad), 0x5000, p, c16(k=0x100000, v=0x200000, desc=None), None, 0x7000, 0x8000, None) == ARG
        assert lib.sba_accumulate_weights(c16(**bad), 0x5000, 1, None, None, None, 0, 0.1, 0xa000, 0xb000, 0xb000, None) == ARG


def test_sums_in_place_or_apart():
    lib, size = sba.load(), 64 * 2 * 64 * 4
    a = 0x100000
    for o in (a + 4, a - 4, a + size - 4, a - size + 4):
        assert lib.sba_accumulate_weights(c16(), 0x5000, 1, None, None, None, 0, 0.1, 0xa000, a, o, None) == ARG
        assert lib.sba_accumulate_weights_kv4(c4(), 0x5000, 1, None, None, 0, 0.1, 0xa000, a, o, None) == ARG
    for o in (a, a + size, a - size):       # past the checks: no GPU to launch on
        assert lib.sba_accumulate_weights(c16(), 0x5000, 1, None, None, None, 0, 0.1, 0xa000, a, o, None) == sba.SBA_ERR_CUDA
        assert lib.sba_accumulate_weights_kv4(c4(), 0x5000, 1, None, None, 0, 0.1, 0xa000, a, o, None) == sba.SBA_ERR_CUDA
