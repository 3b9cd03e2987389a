"""The binding of the smaller cache's calls without a GPU: shapes that it refuses and values that it takes."""
from __future__ import annotations

import pytest
import torch

from block_sparse_gqa_min_b200 import sba


class Calls:
    """Stands in for the library: every call is noted, none is made."""

    def __init__(self):
        self.made = []

    def __getattr__(self, name):
        def call(*args):
            self.made.append((name, args))
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    """CPU tensors taken for ones of the current device, -1."""
    got = Calls()
    monkeypatch.setattr(sba, "load", lambda: got)
    monkeypatch.setattr(sba, "_current", lambda device, stream: 0)
    monkeypatch.setattr(sba, "_opened", lambda c: (c, c, -1))
    return got


@pytest.fixture
def c4():
    return sba.sba_cache4(B=2, H_q=8, H_kv=2, d=128, b=64, max_blocks=4, num_pages=8, max_len=256)


def test_rows_of_a_window_have_one_shape(calls, c4):
    pos = torch.zeros(2, dtype=torch.int32)

    def rows(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16)

    good = rows(2, 5, 2, 128)
    sba.sba_append_kv4(c4, good, good, pos)
    sba.sba_read_kv4(c4, pos, good, good.clone())
    assert [(n, a[4] if n == "sba_append_kv4" else a[2]) for n, a in calls.made] == [("sba_append_kv4", 5), ("sba_read_kv4", 5)]
    # heads before tokens, another number of heads or tokens, too many rows, flat rows: none has enough of a
    # shape to be taken for what it is not
    for bad in (rows(2, 2, 5, 128), rows(2, 5, 8, 128), rows(2, 6, 2, 128), rows(4, 5, 2, 128), rows(2, 5, 256),
                rows(2 * 5 * 2 * 128), rows(2, 5, 2, 64)):
        for k, v in ((good, bad), (bad, good)):
            with pytest.raises(ValueError, match="must be bf16"):
                sba.sba_append_kv4(c4, k, v, pos)
            with pytest.raises(ValueError, match="must be bf16"):
                sba.sba_read_kv4(c4, pos, k, v)
    assert len(calls.made) == 2


def test_the_scale_may_be_any_number(calls, c4):
    """As in the library's other calls: a numpy number, a tensor of one element."""
    import numpy as np

    q, out = (torch.zeros((2, 8, 128), dtype=torch.bfloat16) for _ in range(2))
    lse, acc, ws = torch.zeros((2, 8)), torch.zeros((8, 2, 64)), torch.zeros(64, dtype=torch.uint8)
    for scale in (np.float32(0.5), torch.tensor(0.5), 1, 0.5):
        sba.sba_decode_kv4(c4, q, scale, out, ws)
        sba.sba_accumulate_weights(c4, q, lse, scale, acc, acc)
        sba.sba_accumulate_weights_kv4(c4, q, lse, scale, acc, acc)
    assert len(calls.made) == 12
    for name, args in calls.made:
        got = [x for x in args if type(x) is float]
        assert len(got) == 1 and got[0] in (0.5, 1.0), (name, args)


def test_caches_can_be_copied():
    """A cache that has been used (and so holds its C struct) is copied like any dataclass of tensors."""
    import copy
    import pickle

    lens = torch.zeros(1, dtype=torch.int32)
    k = torch.zeros((4, 2, 64, 128), dtype=torch.bfloat16)
    for c, st in ((sba.Cache4(kv=torch.zeros((4, 2, 2, 4608), dtype=torch.uint8), seq_lens=lens, H_q=4, max_blocks=4,
                              max_len=256), sba.sba_cache4()),
                  (sba.Cache(k=k, v=k, seq_lens=lens, H_q=4, max_blocks=4, max_len=256), sba.sba_cache())):
        c.__dict__["_struct"] = st
        for other in (copy.copy(c), copy.deepcopy(c), pickle.loads(pickle.dumps(c))):
            assert other.max_len == 256 and torch.equal(other.seq_lens, lens) and "_struct" not in other.__dict__
        assert copy.copy(c).seq_lens is lens and c.__dict__["_struct"] is st
