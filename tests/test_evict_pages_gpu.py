"""Eviction: pages that the block table gets wrong."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_sparse_gqa_min_b200 import sba
from oracle import small_cache as SC
from tests.kv4_helpers import cache4, layout
from tests.test_kv4_gpu import i32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = torch.device("cuda")


@pytest.mark.parametrize("H,n,max_len,bad", [
    (80, 70000, None, 69000),        # more heads than clusters: the slice passes what shared memory holds
    (80, 70000, None, 100),
    (1, 5000, 300, 4000),            # an understated max_len holds fewer weights
    (2, 9000, 0, 4000),              # ... or none
])
def test_a_bad_page_is_reported_wherever_its_weights_are(H, n, max_len, bad):
    """Tokens of a bad page rank last, and SBA_DEV_BAD_PAGE says so, whether their weights would be held in
    shared memory or read again in every pass."""
    b, keep = 64, 300
    lay, dlay = layout([n], b, False, 1, slack=0), layout([keep], b, False, 2, slack=0)
    g = torch.Generator(device="cuda").manual_seed(3)
    src = cache4(lay, torch.zeros((lay.pages, H, b // 32, 4608), dtype=torch.uint8, device=DEV), H_q=H, desc=False,
                 max_len=max_len)
    table = torch.arange(lay.max_blocks, dtype=torch.int32, device=DEV)[None].contiguous()
    src.block_table = table
    dst = cache4(dlay, torch.zeros((dlay.pages, H, b // 32, 4608), dtype=torch.uint8), H)
    acc = torch.rand((lay.pages, H, b), generator=g, device=DEV)
    new_lens, kept = i32([0]), torch.zeros((1, H, keep), dtype=torch.int32, device=DEV)
    p = sba.evict_params(keep, 3, 20)
    sba.sba_evict_kv4(src, acc, p, dst, new_lens, kept)
    assert int(src.status.item()) == 0
    table[0, bad // b] = lay.pages
    sba.sba_evict_kv4(src, acc, p, dst, new_lens, kept)
    assert int(src.status.item()) == sba.SBA_DEV_BAD_PAGE and int(dst.status.item()) == 0
    a = acc.cpu().numpy()
    a[bad // b] = np.nan
    for h in {0, H // 2, H - 1}:
        assert np.array_equal(kept[0, h].cpu().numpy(), SC.keep(SC.gather(a, None, 0, lay.max_blocks, h, n), keep, 3, 20))
