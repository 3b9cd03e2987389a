"""Accumulated weights of gated rows whose biases are the type's lowest value, or -inf."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_sparse_gqa_min_b200 import sba
from oracle import small_cache as SC
from tests.kv4_helpers import SCALE, cache16, f64, layout, logit_bound, rand_bf16
from tests.test_kv4_gpu import i32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = torch.device("cuda")
LOW = float(np.finfo(np.float32).min)


@pytest.mark.parametrize("lens,H,G", [([200], 2, 4), ([40000, 64, 130], 8, 3)])
def test_biases_of_the_lowest_value(lens, H, G):
    """Heads by turns: every selected block at the lowest value (lse is that value too, and the weights follow from
    what is left: exp(logit + (bias - lse))), one block at it (its tokens add 0), one at -inf (0), all at -inf
    (lse -inf: the row adds nothing), ordinary ones."""
    b, B = 64, len(lens)
    lay = layout(lens, b, True, 3)
    k = rand_bf16((lay.pages, H, b, 128), 1)
    c = cache16(lay, k, k, H * G, desc=False)
    q = rand_bf16((B, 1, H * G, 128), 2, 0)
    n_sel = max(-(-x // b) for x in lens)
    idx = torch.arange(n_sel, dtype=torch.int32, device=DEV).expand(B, H, -1).contiguous()
    cnt = i32([[-(-x // b)] * H for x in lens])
    g = torch.Generator().manual_seed(4)
    bias = -4 * torch.rand((B, H * G, n_sel), generator=g)
    lse = 2 + torch.rand((B, 1, H * G), generator=g)
    for r in range(H * G):
        if r % 5 == 0:
            bias[:, r], lse[:, 0, r] = LOW, LOW
        elif r % 5 == 1:
            bias[:, r, 0] = LOW
        elif r % 5 == 2:
            bias[:, r, 0] = -torch.inf
        elif r % 5 == 3:
            bias[:, r], lse[:, 0, r] = -torch.inf, -torch.inf
    acc = torch.zeros((lay.pages, H, b), device=DEV)
    sba.sba_accumulate_weights(c, q.to(DEV), lse.to(DEV), SCALE, acc, acc, sel_idx=idx, sel_cnt=cnt, gate_bias=bias.to(DEV))
    assert int(c.status.item()) == 0
    K = f64(k)
    for s, n in enumerate(lens):
        for h in range(H):
            rows = slice(h * G, (h + 1) * G)
            kk = SC.gather(K, lay.table, s, lay.max_blocks, h, n)
            qg = f64(q)[s, :, rows]
            x = SC.logits(qg, kk, np.arange(n), n, SCALE)[0]
            lg = f64(lse)[s, 0, rows]
            with np.errstate(invalid="ignore"):
                off = f64(bias)[s, rows][:, np.arange(n) // b] - lg[:, None]
                w = np.where((lg == -np.inf)[:, None], 0.0, np.exp(x + off)).sum(0)
            rel = np.expm1(logit_bound(qg, kk)) + 6 * 2.0 ** -24 * (np.abs(x).max() + 8) + 2.0 ** -21 + G * 2.0 ** -24
            got = SC.gather(f64(acc), lay.table, s, lay.max_blocks, h, n)
            assert (np.abs(got - w) <= rel * w + 1e-37).all(), (s, h)
