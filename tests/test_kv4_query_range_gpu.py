"""Four-bit attention and weights for queries and scales at the ends of their ranges: a power of two moved from
the scale to the query changes no bit, and rows whose logits vanish weigh all tokens alike."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_sparse_gqa_min_b200 import sba
from oracle import small_cache as SC
from tests.kv4_helpers import SCALE, cache4, f64, layout, packed, rand_bf16
from tests.test_kv4_gpu import i32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = torch.device("cuda")


def run(c, q, scale):
    B, M, HQ, _ = q.shape
    out, lse = torch.empty(q.shape, device=DEV), torch.empty((B, M, HQ), device=DEV)
    ws = torch.zeros(sba.sba_decode_kv4_workspace_size(c, M, 0), dtype=torch.uint8, device=DEV)
    sba.sba_decode_kv4(c, q.to(DEV), scale, out, ws, lse_out=lse)
    acc = torch.zeros((c.num_pages, c.H_kv, c.b), device=DEV)
    sba.sba_accumulate_weights_kv4(c, q.to(DEV), lse, scale, acc, acc)
    return out, lse, acc


def cache(lens, H, G):
    lay = layout(lens, 64, False, 0)
    k, v = rand_bf16((lay.pages, H, 64, 128), 1), rand_bf16((lay.pages, H, 64, 128), 2)
    kv = packed(k, v)
    return lay, kv, cache4(lay, kv, H_q=H * G, desc=False)


@pytest.mark.parametrize("G,M", [(4, 1), (8, 4)])              # 4 rows, and 32: the register and the tensor-memory weights
@pytest.mark.parametrize("e", [124, 110, -110])
def test_a_power_of_two_of_the_query_is_one_of_the_scale(G, M, e):
    lay, kv, c = cache([1000, 70], 2, G)
    q = rand_bf16((2, M, 2 * G, 128), 3, 0)
    moved = (q.double() * 2.0 ** e).to(torch.bfloat16)
    assert torch.equal(moved.double() * 2.0 ** -e, q.double())
    want, got = run(c, q, SCALE), run(c, moved, SCALE * 2.0 ** -e)
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("G,M", [(4, 1), (8, 4)])
@pytest.mark.parametrize("size,scale", [(0.0, SCALE), (0.0, 1e-20), (0.0, 2.0 ** -126), (2.0 ** -120, 2.0 ** -100)])
def test_rows_without_logits_weigh_all_tokens_alike(G, M, size, scale):
    """Logits of 0, or below 2^-180: a row's output is the mean of the values it sees (P and its sum are exact, so
    the sum of the values, cut by 2^-23 of it at most 18 times in each MMA step, is what is off), its lse the
    logarithm of their number, and its weights 1 over it."""
    n, H = 200, 2
    lay, kv, c = cache([n], H, G)
    q = (rand_bf16((1, M, H * G, 128), 3, 0).double() * size).to(torch.bfloat16)
    out, lse, acc = run(c, q, scale)
    V = SC.unpack_tile(kv.numpy())[1]
    for h in range(H):
        v = SC.gather(V, None, 0, lay.max_blocks, h, n)
        w = np.zeros(n)
        for i in range(M):
            seen = n - M + i + 1
            o, mass = v[:seen].mean(0), np.abs(v[:seen]).mean(0)
            assert (np.abs(f64(out)[0, i, h * G:(h + 1) * G] - o) <= mass * 2.0 ** -16).all()
            assert np.abs(f64(lse)[0, i, h * G:(h + 1) * G] - np.log(seen)).max() <= 2.0 ** -20
            w[:seen] += G / seen
        assert np.abs(SC.gather(f64(acc), None, 0, lay.max_blocks, h, n) / w - 1).max() <= 2.0 ** -18
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("token", [1, 40, 150, 260, 3000])
def test_a_nan_value_is_seen_however_small_its_weight(token):
    """One token takes all the weight (the others' underflow); a NaN among a seen token's values is in the output
    all the same, wherever the token's strip was worked on, and nothing else changes."""
    n, H, G = 4000, 1, 4
    lay, kv, c = cache([n], H, G)
    q = torch.zeros((1, 1, H * G, 128), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    top = 20
    for j in range(lay.max_blocks):                            # channel 0 of the keys: 6 in one token, -6 in all others
        kv[j, 0, :, 0:2048:64] = (kv[j, 0, :, 0:2048:64] & 0xF0) | 0xF
        kv[j, 0, :, 4096:4352:8] = 15 * 8
    kv[top // 64, 0, top % 64 // 32, top % 32 * 64] &= 0xF7
    c.kv.copy_(kv)
    clean = run(c, q, 1e6)[0]
    V = SC.unpack_tile(kv.numpy())[1]
    assert np.array_equal(f64(clean)[0, 0, 0], V[0, 0, top])
    kv[token // 64, 0, token % 64 // 32, 4352 + token % 32 * 8 + 2] = 255
    c.kv.copy_(kv)
    got = run(c, q, 1e6)[0]
    assert torch.isnan(got[..., 32:48]).all()
    assert torch.equal(got[..., :32], clean[..., :32]) and torch.equal(got[..., 48:], clean[..., 48:])


@pytest.mark.parametrize("byte", [248, 249, 254, 255])
def test_scales_that_are_no_numbers_stay_with_the_rows_that_see_them(byte):
    """Any byte whose exponent bits are all ones, in a token that the first of several query tokens do not see:
    their rows do not change by a bit, the others' 16 channels are NaN."""
    n, H, G, M, t = 200, 1, 2, 4, 198                          # tokens 196 .. 199 ask; 198 is hidden from two
    lay, kv, c = cache([n], H, G)
    q = rand_bf16((1, M, H * G, 128), 3, 0)
    clean, clean_lse, _ = run(c, q, SCALE)
    kv[t // 64, 0, t % 64 // 32, 4352 + t % 32 * 8 + 5] = byte
    c.kv.copy_(kv)
    out, lse, _ = run(c, q, SCALE)
    assert torch.equal(out[:, :2], clean[:, :2]) and torch.equal(lse, clean_lse)
    assert torch.isnan(out[:, 2:, :, 80:96]).all()
    assert torch.equal(out[:, 2:, :, :80], clean[:, 2:, :, :80]) and torch.equal(out[:, 2:, :, 96:], clean[:, 2:, :, 96:])
