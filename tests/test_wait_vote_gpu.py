"""A warp's bounded wait ends with one verdict for all lanes, even where the limit runs out for some of them
and the phase completes before the others' does."""
from __future__ import annotations

import pytest
import torch

from block_sparse_gqa_min_b200 import sba

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def test_a_warp_gives_up_as_one():
    dev = torch.device("cuda")
    status = torch.full((1,), sba.SBA_DEV_BAD_PAGE, dtype=torch.int32, device=dev)
    verdicts = torch.full((32,), 9, dtype=torch.int32, device=dev)
    sba.sba_selftest_wait_vote(status, verdicts, 5_000_000)             # 5 ms
    torch.cuda.synchronize()
    assert verdicts.tolist() == [0] * 32
    assert int(status.item()) == sba.SBA_DEV_BAD_PAGE | sba.SBA_DEV_TIMEOUT
