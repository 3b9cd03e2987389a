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


@pytest.mark.parametrize("H,G", [(8, 1), (4, 16)])
def test_fp32_sums_over_many_strips_are_rounded_not_cut(H, G):
    """Equal weights (a query of zeros: P is 2^8 and the sum of 2048 of them a power of two, all exact) and
    values of 7168 and of 1 or 3 times u = 2^-6, in every eighth strip only: one warp has them all, eight
    strips, and every other warp adds zeros.  16 tokens (an MMA step) hold nine large values and seven small
    ones, so two strips add up to less than 2^24 u: exact in an accumulator.  The sums of two strips are then
    added by rounding, to values below 2^25 u, 1.5 * 2^25 u and 2^26 u: at most 1 + 2 + 2 u off.  An
    accumulator that runs through all eight strips passes 2^24 u after the second, and every step (an odd
    number of u) is cut by 1 u or more: 4 steps in strips 3 and 4, 8 in strips 5 to 8, at least 12 u."""
    b, B, T = 64, 37, 2048                                    # a unit a CTA: 296 of 8 rows, 148 of 16
    lay = layout([T] * B, b, False, 0, slack=0)
    g = torch.Generator().manual_seed(G)
    kv = torch.zeros((lay.pages, H, b // 32, 4608), dtype=torch.uint8)
    sums = np.zeros((B, H, 128))
    big = torch.zeros(16, dtype=torch.bool)
    big[[0, 1, 3, 5, 6, 8, 10, 11, 15]] = True
    for x in range(8):
        page, strip = 8 * x // 2, 8 * x % 2                   # strip 8x of every sequence
        three = torch.randint(0, 2, (B, H, 32, 128), generator=g).bool()
        large = big.repeat(2)[:, None].expand(B, H, 32, 128)
        code = torch.where(large, 6, torch.where(three, 5, 2)).to(torch.uint8)       # 4, 3, 1
        scale = torch.where(large[..., ::16], 206, 72).to(torch.uint8)               # 1792, 2^-6
        at = torch.arange(B) * (T // b) + page
        kv[at, :, strip, 2048:4096] = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(B, H, 2048)
        kv[at, :, strip, 4352:4608] = scale.reshape(B, H, 256)
        sums += torch.where(large, 7168.0, torch.where(three, 3.0, 1.0) / 64).double().sum(2).numpy()
    c = cache4(lay, kv, H_q=H * G, desc=False)
    q = torch.zeros((B, H * G, 128), dtype=torch.bfloat16, device=DEV)
    out = torch.empty((B, H * G, 128), dtype=torch.float32, device=DEV)
    ws = torch.zeros(sba.sba_decode_kv4_workspace_size(c, 1, 0), dtype=torch.uint8, device=DEV)
    sba.sba_decode_kv4(c, q, 1.0, out, ws)
    off = np.abs(f64(out).reshape(B, H, G, 128) * T - sums[:, :, None]) * 64
    assert off.max() <= 5, off.max()
    assert int(c.status.item()) == 0
