"""Eviction: pages that the block table gets wrong, and pages of one pool."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_sparse_gqa_min_b200 import sba
from oracle import small_cache as SC
from tests.kv4_helpers import (SCALE, cache4, cache16, f64, layout, packed, rand_bf16)
from tests.test_kv4_gpu import check_decode, i32, run_decode

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


def tables(B, blocks, seed):
    """Two block tables [B][blocks] over one pool, without a page in common, and the pool's pages."""
    pages = 2 * B * blocks + 3
    perm = np.random.default_rng(seed).permutation(pages).astype(np.int32)
    return perm[:B * blocks].reshape(B, blocks), perm[B * blocks:2 * B * blocks].reshape(B, blocks), pages


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("b,lens,H,keep", [(64, [1000, 130, 0, 700], 2, 300), (128, [9000], 4, 129)])
def test_evict_inside_one_pool(four, b, lens, H, keep):
    """The same pool, descriptors and weights under another block table: what two pools give, and the source's
    pages stay as they were."""
    B, blocks = len(lens), -(-max(lens) // b)
    ta, tb, pages = tables(B, blocks, 5)
    lay, dlay = layout(lens, b, False, 0, slack=0), layout(lens, b, False, 0, slack=0)
    lay.table, lay.pages, dlay.table, dlay.pages = ta, pages, tb, pages
    g = torch.Generator().manual_seed(3)
    acc = torch.exp(2 * torch.randn((pages, H, b), generator=g)).to(DEV)
    p = sba.evict_params(keep, 4, 30)
    k, v = rand_bf16((pages, H, b, 128), 1), rand_bf16((pages, H, b, 128), 2)
    rows = (packed(k, v),) if four else (k, v)
    make, call = (cache4, sba.sba_evict_kv4) if four else (cache16, sba.sba_evict)
    field = ("kv",) if four else ("k", "v")

    def run(one):
        src, dst = make(lay, *rows, H), make(dlay, *rows, H)
        src.desc.copy_(torch.randn(src.desc.shape, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16))
        dst.desc.copy_(src.desc)
        a = acc.clone()
        to = a if one else acc.clone()
        if one:
            dst.desc = src.desc
            for f in field:
                setattr(dst, f, getattr(src, f))
        new, kept = i32([0] * B), torch.zeros((B, H, keep), dtype=torch.int32, device=DEV)
        call(src, a, p, dst, new, kept, acc_dst=to)
        assert int(src.status.item()) == 0 and int(dst.status.item()) == 0
        return [getattr(dst, f) for f in field] + [dst.desc, to, new, kept]

    for x, y in zip(run(False), run(True)):
        assert torch.equal(x, y)


def test_loop_inside_one_pool_and_reused_pages():
    """A four-bit sequence that moves between two halves of one pool: tokens are appended (their weights set to
    0), attended to and weighed, and every eviction goes back into pages that held others before."""
    b, H, G, B, keep, blocks = 64, 2, 4, 2, 150, 5
    ta, tb, pages = tables(B, blocks, 6)
    lay = [layout([blocks * b] * B, b, False, 0, slack=0) for _ in range(2)]
    for x, t in zip(lay, (ta, tb)):
        x.table, x.pages = t, pages
    pool = torch.randint(0, 256, (pages, H, b // 32, 4608), dtype=torch.uint8)      # earlier tokens' rows and weights
    c = [cache4(x, pool, H_q=H * G, lens=[0] * B) for x in lay]
    c[1].kv, c[1].desc, c[1].status = c[0].kv, c[0].desc, c[0].status
    acc = torch.full((pages, H, b), 50.0, device=DEV)
    at, length = 0, 0
    total = [[np.zeros(0) for _ in range(H)] for _ in range(B)]
    for step, n in enumerate((200, 40, 60, 1, 100)):
        cc, L = c[at], lay[at]
        kn, vn, q = (rand_bf16((B, m, x, 128), 10 * step + i) for i, (m, x) in enumerate(((n, H), (n, H), (1, H * G))))
        cc.seq_lens.fill_(length + n)
        sba.sba_append_kv4(cc, kn.to(DEV), vn.to(DEV), i32([length] * B))
        t = torch.arange(length, length + n, device=DEV)
        for s in range(B):
            acc[cc.block_table[s].long()[t // b], :, t % b] = 0
        length += n
        out, lse, _ = run_decode(cc, q, None, True)
        sba.sba_accumulate_weights_kv4(cc, q.to(DEV), lse, SCALE, acc, acc)
        now = layout([length] * B, b, False, 0, slack=0)
        now.table, now.max_blocks, now.pages = L.table, L.max_blocks, pages
        kv = cc.kv.cpu().numpy()
        check_decode(cc, kv, now, q, None, out, lse, b, G, True)
        K = SC.unpack_tile(kv)[0]
        for s in range(B):
            for h in range(H):
                kk = SC.gather(K, L.table, s, L.max_blocks, h, length)
                x = SC.logits(f64(q)[s, :, h * G:(h + 1) * G], kk, np.arange(length), length, SCALE)
                total[s][h] = np.append(total[s][h], np.zeros(n)) + SC.weights(x, SC.attend(x, kk)[1])
                assert np.allclose(SC.gather(f64(acc), L.table, s, L.max_blocks, h, length), total[s][h], rtol=1e-4, atol=1e-6)
        if length > keep:
            new, kept = i32([0] * B), torch.zeros((B, H, keep), dtype=torch.int32, device=DEV)
            before = acc.clone()
            sba.sba_evict_kv4(cc, acc, sba.evict_params(keep, 4, 16), c[1 - at], new, kept, acc_dst=acc)
            assert new.tolist() == [keep] * B
            for s in range(B):
                for h in range(H):
                    w = SC.gather(f64(before), L.table, s, L.max_blocks, h, length)
                    t = kept[s, h].cpu().numpy()
                    assert np.array_equal(t, SC.keep(w, keep, 4, 16))
                    assert np.array_equal(SC.gather(f64(acc), lay[1 - at].table, s, blocks, h, keep), w[t])
                    total[s][h] = w[t]
            at, length = 1 - at, keep
    assert int(c[0].status.item()) == 0
