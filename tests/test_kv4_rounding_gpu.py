"""Roundings of the four-bit attention: a bf16 output is the fp32 result rounded once, whatever type is
asked for (sba_decode_kv4)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_sparse_gqa_min_b200 import sba
from oracle import small_cache as SC
from tests.kv4_helpers import cache4, f64, layout, packed, rand_bf16

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = torch.device("cuda")


def rounded(x: np.ndarray) -> np.ndarray:
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("b,G,M,T", [(64, 4, 1, 33), (64, 8, 1, 64), (128, 16, 1, 64), (64, 5, 3, 61)])
def test_bf16_outputs_are_the_fp32_result_rounded_once(b, G, M, T):
    """Queries with one channel make every logit exact (one product; the codes and scales have few bits), so
    what is left is small and known, and a bf16 output has to lie between the roundings of o - tol and o + tol:

    a weight: its argument (s - m) * scale * log2(e) + 8 carries at most three roundings of 2^-24 (log2(e),
    its product with the scale, the fma) of values up to |x| * 1.45 + 8, times ln 2; ex2.approx 2^-22; the two
    f16 parts of P leave 2^-22.  Once for the product, once for the sum.
    products: a warp's 32 tokens are two MMA steps of 16 tokens for each of P's two parts, and a step drops at
    most 18 times 2^-23 of the largest term or sum, none of which passes the sum of p |v|; merging the warps
    and dividing add at most 16 roundings of 2^-24."""
    H, scale = 2, 1.0
    lay = layout([T], b, False, 0)
    k, v = rand_bf16((lay.pages, H, b, 128), 1), rand_bf16((lay.pages, H, b, 128), 2)
    kv = packed(k, v)
    c = cache4(lay, kv, H_q=H * G, desc=False)
    rng = np.random.default_rng(G)
    q = torch.zeros((1, M, H * G, 128))
    for i in range(M):
        for r in range(H * G):
            q[0, i, r, rng.integers(128)] = 1.0
    q = q.to(torch.bfloat16)
    out = torch.full((1, M, H * G, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(sba.sba_decode_kv4_workspace_size(c, M, 0), dtype=torch.uint8, device=DEV)
    sba.sba_decode_kv4(c, q.to(DEV), scale, out, ws)
    K, V = SC.unpack_tile(kv.numpy())
    got = f64(out)
    for h in range(H):
        kk, vv = SC.gather(K, None, 0, lay.max_blocks, h, T), SC.gather(V, None, 0, lay.max_blocks, h, T)
        x = SC.logits(f64(q)[0, :, h * G:(h + 1) * G], kk, np.arange(T), T, scale)
        o, z = SC.attend(x, vv)
        p = np.exp(x - z[..., None])
        mass = p @ np.abs(vv)
        big = np.abs(x[np.isfinite(x)]).max()
        weight = np.log(2) * 3 * 2.0 ** -24 * (2 * big * 1.45 + 8) + 2.0 ** -22 + 2.0 ** -22
        tol = mass * (2 * weight + 4 * 18 * 2.0 ** -23 + 16 * 2.0 ** -24)
        g = got[0, :, h * G:(h + 1) * G]
        lo, hi = rounded(o - tol), rounded(o + tol)
        assert ((lo <= g) & (g <= hi)).all(), (h, int(((g < lo) | (g > hi)).sum()), g.size)
    assert int(c.status.item()) == 0
