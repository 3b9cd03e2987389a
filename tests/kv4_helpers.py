"""Seeded layouts and caches for the tests of the smaller cache (four-bit rows, weights, eviction)."""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

from oracle import small_cache as SC

SCALE = 1.0 / math.sqrt(128)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


@dataclass
class Layout:
    lens: list
    max_blocks: int
    pages: int
    table: Optional[np.ndarray]      # int32 [B][max_blocks]


def layout(lens, b, paged, seed, slack=1) -> Layout:
    """Pages of sequences with room for `slack` more blocks each; paged: a seeded permutation of a
    pool that is larger than needed, table entries past a sequence's blocks invalid."""
    B = len(lens)
    mb = max(1, max(-(-x // b) for x in lens) + slack)
    if not paged:
        return Layout(list(lens), mb, B * mb, None)
    rng = np.random.default_rng(seed)
    pages = B * mb + 3
    perm = rng.permutation(pages)
    table = np.full((B, mb), -1, dtype=np.int32)
    at = 0
    for s, x in enumerate(lens):
        n = min(mb, -(-x // b) + slack)
        table[s, :n] = perm[at:at + n]
        at += n
    return Layout(list(lens), mb, pages, table)


def rand_bf16(shape, seed, channel_sigma=0.5) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if channel_sigma:
        x = x * torch.exp(channel_sigma * torch.randn(shape[-1:], generator=g))
    return x.to(torch.bfloat16)


def packed(k: torch.Tensor, v: torch.Tensor) -> torch.Tensor:
    """bf16 [pages][H][b][128] keys and values -> four-bit tiles (oracle)."""
    kk, vv = f64(k), f64(v)
    P, H, b, _ = kk.shape
    out = np.zeros((P, H, b // 32, SC.STRIP_BYTES), dtype=np.uint8)
    for p in range(P):
        for h in range(H):
            out[p, h] = SC.pack_tile(kk[p, h], vv[p, h])
    return torch.from_numpy(out)


def cache4(lay: Layout, kv: torch.Tensor, H_q, desc=True, max_len=None, lens=None):
    from block_sparse_gqa_min_b200 import sba

    dev = torch.device("cuda")
    kv = kv.to(dev)
    return sba.Cache4(
        kv=kv, seq_lens=torch.tensor(lens if lens is not None else lay.lens, dtype=torch.int32, device=dev), H_q=H_q,
        max_blocks=lay.max_blocks, max_len=max(lay.lens) if max_len is None else max_len,
        block_table=None if lay.table is None else torch.from_numpy(lay.table).to(dev),
        desc=torch.zeros((kv.shape[0], kv.shape[1], 2, 128), dtype=torch.bfloat16, device=dev) if desc else None,
        status=torch.zeros(1, dtype=torch.int32, device=dev))


def cache16(lay: Layout, k: torch.Tensor, v: torch.Tensor, H_q, desc=True):
    from block_sparse_gqa_min_b200 import sba

    dev = torch.device("cuda")
    return sba.Cache(
        k=k.to(dev), v=v.to(dev), seq_lens=torch.tensor(lay.lens, dtype=torch.int32, device=dev), H_q=H_q,
        max_blocks=lay.max_blocks, max_len=max(lay.lens),
        block_table=None if lay.table is None else torch.from_numpy(lay.table).to(dev),
        desc=torch.zeros((k.shape[0], k.shape[1], 2, 128), dtype=torch.bfloat16, device=dev) if desc else None,
        status=torch.zeros(1, dtype=torch.int32, device=dev))


def page(lay: Layout, s: int, j: int) -> int:
    return int(lay.table[s, j]) if lay.table is not None else s * lay.max_blocks + j


def selection(lay: Layout, b, H, n_max, seed):
    """Random ascending block lists [B][H][n_max] that hold the last block, and their counts."""
    rng = np.random.default_rng(seed)
    B = len(lay.lens)
    idx = np.full((B, H, n_max), -7, dtype=np.int32)
    cnt = np.zeros((B, H), dtype=np.int32)
    for s in range(B):
        N = -(-lay.lens[s] // b)
        for h in range(H):
            k = min(N, n_max)
            if k:
                idx[s, h, :k] = np.sort(np.append(rng.permutation(N - 1)[:k - 1], N - 1))
            cnt[s, h] = k
    return idx, cnt


def logit_bound(q: np.ndarray, k: np.ndarray) -> float:
    """How far an fp32 logit q.k * SCALE may be off: products are exact, 128 terms are added in two
    chains of four MMAs of 16 terms (each MMA aligns its 16 products and the accumulator to the
    largest and drops what is below 2^-23 of it, so at most 18 drops a step: 4 steps and the final
    sum), plus q's f16 rounding (2^-25 of its largest channel) and the scaling (two roundings)."""
    if k.shape[0] == 0:
        return 0.0
    aq, ak = np.abs(q).reshape(-1, q.shape[-1]), np.abs(k)
    mass = float((aq @ ak.T).max())
    low = float(aq.max() * ak.sum(-1).max()) * 2.0 ** -25
    return (mass * (4 * 18 + 2) * 2.0 ** -23 + low) * SCALE
