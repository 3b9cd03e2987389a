"""Four-bit attention over launches whose CTAs take equal shares of all units, with so many strips a warp that
fp32 sums leave the accumulators many times: 8 and 16 rows a tile, both output types, whole caches and
selections, and maxima that grow along the sequence, so that sums already moved out are scaled again.  Against
the definition in fp64."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_sparse_gqa_min_b200 import sba
from oracle import small_cache as SC
from tests.kv4_helpers import SCALE, cache4, layout, page, rand_bf16, selection

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = torch.device("cuda")
SMS, WARPS, STRIP = 148, 8, 32


def shared_strips(lens, b, H, G, M, n_sel):
    """Strips a warp of a launch with equal shares, 0 where a CTA works on one unit (the rule of the launch)."""
    rows = M * G
    tile = 8 if rows <= 8 else 16
    fit = (2 if tile == 8 else 1) * SMS
    groups = -(-rows // tile)
    units = len(lens) * H * groups
    per = (n_sel or -(-max(lens) // b)) * (b // STRIP)
    if units <= fit and units * per <= fit * WARPS * 4:
        return 0
    strips = sum(min(n_sel or 1 << 30, -(-x // b)) * (b // STRIP) for x in lens) * H * groups
    return strips // fit // WARPS


def tiles(pages, H, b, seed):
    """Random codes, scales from 2^-2 to below 2^0."""
    g = torch.Generator().manual_seed(seed)
    kv = torch.randint(0, 256, (pages, H, b // STRIP, 4608), generator=g, dtype=torch.uint8)
    kv[..., 4096:] = torch.randint(13 * 8, 15 * 8, (pages, H, b // STRIP, 512), generator=g, dtype=torch.uint8)
    return kv


def rows(kv, which):
    """fp64 rows [...][32][128] of strips on the GPU."""
    table = torch.tensor(SC.CODES, device=DEV)
    scales = torch.tensor(np.nan_to_num(SC.SCALES), device=DEV)
    by = kv[..., 2048 * which:2048 * (which + 1)].reshape(*kv.shape[:-1], 32, 64)
    code = torch.stack((by & 15, by >> 4), -1).flatten(-2).long()
    sc = kv[..., 4096 + 256 * which:4096 + 256 * (which + 1)].reshape(*kv.shape[:-1], 32, 8).long()
    x = table[code & 7] * scales[sc].repeat_interleave(16, -1)
    return torch.where(code >= 8, -x, x)


CASES = [
    # b, lens, H, G, M, n_sel, f32, grow, strips a warp at least
    (64, [120000], 4, 8, 2, 0, True, False, 12),
    (64, [120000], 4, 8, 2, 0, False, False, 12),
    (64, [150000, 3], 4, 8, 1, 0, False, False, 7),
    (64, [300000], 5, 8, 1, 0, True, False, 17),
    (128, [200000, 90000], 4, 5, 1, 0, True, True, 14),
    (64, [120000], 4, 5, 3, 0, True, True, 12),
    (64, [150000], 4, 4, 1, 0, False, True, 7),
    (64, [30000, 26000], 8, 4, 1, 400, True, False, 4),
    (64, [30000, 26000], 8, 4, 3, 400, False, True, 9),
    (64, [50000, 41000], 2, 8, 5, 0, True, False, 12),        # 40 rows: three row groups
]


@pytest.mark.parametrize("b,lens,H,G,M,n_sel,f32,grow,strips", CASES)
def test_long_shares(b, lens, H, G, M, n_sel, f32, grow, strips):
    assert shared_strips(lens, b, H, G, M, n_sel) >= strips
    lay = layout(lens, b, True, seed=G)
    B = len(lens)
    kv = tiles(lay.pages, H, b, G + M)
    if grow:        # key scales from 2^-5 in the first block to 2^0 in the last
        for s, x in enumerate(lens):
            N = -(-x // b)
            for j in range(N):
                kv[page(lay, s, j), ..., 4096:4352] = 8 * (10 + 6 * j // N)
    q = rand_bf16((B, M, H * G, 128), 3, 0)
    c = cache4(lay, kv, H_q=H * G, desc=False)
    kw, sel = {}, None
    if n_sel:
        sel = selection(lay, b, H, n_sel, 5)
        kw = dict(sel_idx=torch.from_numpy(sel[0]).to(DEV), sel_cnt=torch.from_numpy(sel[1]).to(DEV))
    out = torch.empty((B, M, H * G, 128), dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    lse = torch.empty((B, M, H * G), device=DEV)
    ws = torch.zeros(sba.sba_decode_kv4_workspace_size(c, M, n_sel), dtype=torch.uint8, device=DEV)
    sba.sba_decode_kv4(c, q.to(DEV), SCALE, out, ws, lse_out=lse, **kw)
    first = out.clone()
    sba.sba_decode_kv4(c, q.to(DEV), SCALE, out, ws, lse_out=lse, **kw)
    assert torch.equal(first, out) and int(c.status.item()) == 0
    qd = q.to(DEV).double()
    for s in range(B):
        n = lens[s]
        pages = torch.from_numpy(lay.table[s, :-(-n // b)]).long().to(DEV)
        for h in range(H):
            blocks = torch.arange(len(pages), device=DEV) if sel is None else kw["sel_idx"][s, h, :int(sel[1][s, h])].long()
            t = (blocks[:, None] * b + torch.arange(b, device=DEV)).flatten()
            tile = c.kv[pages[blocks], h]
            k, v = (rows(tile, i).reshape(-1, 128)[t < n] for i in range(2))
            t = t[t < n]
            qq = qd[s, :, h * G:(h + 1) * G]
            x = torch.einsum("mgd,td->mgt", qq, k) * SCALE
            hidden = t[None] > (n - M + torch.arange(M, device=DEV))[:, None]
            x = x.masked_fill(hidden[:, None], -torch.inf)
            z = torch.logsumexp(x, -1)
            o = torch.exp(x - z[..., None]) @ v
            # the bounds of the shorter calls' test: logits in two chains of MMAs, weights, sums, roundings
            mass = float((qq.abs().flatten(0, 1) @ k.abs().T).max())
            low = float(qq.abs().max() * k.abs().sum(-1).max()) * 2.0 ** -25
            big = float(x[x > -torch.inf].abs().max())
            eps = (mass * (4 * 18 + 2) * 2.0 ** -23 + low) * SCALE + 3 * 2.0 ** -24 * (big + 8)
            T = len(t)
            rel = 2 * np.expm1(eps) + 2.0 ** -20 + (T / 32 + 64) * 2.0 ** -24 * 2 + 2.0 ** -22
            tol = rel * float(v.abs().max()) + (2.0 ** -23 if f32 else 2.0 ** -8) * o.abs()
            got = out[s, :, h * G:(h + 1) * G].double()
            assert ((got - o).abs() <= tol).all(), (s, h, float(((got - o).abs() - tol).max()), rel)
            zt = eps + 2.0 ** -20 + (T / 32 + 64) * 2.0 ** -24 + 2.0 ** -23 * z.abs()
            assert ((lse[s, :, h * G:(h + 1) * G].double() - z).abs() <= zt).all(), (s, h)
