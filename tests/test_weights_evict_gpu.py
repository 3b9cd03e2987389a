"""Accumulated attention weights, and eviction by them, on the GPU against the fp64 oracle
(oracle.small_cache); and a decode loop that uses both on a four-bit cache."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_sparse_gqa_min_b200 import sba
from oracle import small_cache as SC
from tests.kv4_helpers import (SCALE, cache4, cache16, f64, layout, logit_bound, packed, page, rand_bf16, selection)
from tests.test_kv4_gpu import check_decode, i32, run_decode

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = torch.device("cuda")


def per_page(lay, b, H, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.rand((lay.pages, H, b), generator=g)


def check_weights(lay, b, G, K, q, lse, sel, bias, acc_in, acc_out, untouched):
    """acc_out against the oracle; entries of tokens outside the selection keep `untouched`."""
    B, M, H_q, _ = q.shape
    H = H_q // G
    want, bound = untouched.astype(np.float64), np.zeros(untouched.shape)
    qq, ll = f64(q), f64(lse)
    for s in range(B):
        n = lay.lens[s]
        for h in range(H):
            k = SC.gather(K, lay.table, s, lay.max_blocks, h, n)
            blocks = None if sel is None else sel[0][s, h, :sel[1][s, h]]
            tok = SC.tokens_of(n, b, blocks)
            if not len(tok):
                continue
            bb = None
            if bias is not None:
                pos = np.repeat(np.arange(len(blocks)), b)[:len(tok)]   # the last block is the partial one
                bb = bias[s, h * G:(h + 1) * G][:, pos][None]
            qg, lg = qq[s, :, h * G:(h + 1) * G], ll[s, :, h * G:(h + 1) * G]
            x = SC.logits(qg, k, tok, n, SCALE, bb)
            w = SC.weights(x, lg)
            big = max(np.abs(x[np.abs(x) < 1e30]).max(initial=0.0), np.abs(lg[np.isfinite(lg)]).max(initial=0.0))
            eps = logit_bound(qg, k[tok]) + 6 * 2.0 ** -24 * (2 * big + 1)
            rel = np.expm1(eps) + 2.0 ** -21 + M * G * 2.0 ** -24
            p = np.array([page(lay, s, j) for j in range(-(-n // b))])[tok // b]
            want[p, h, tok % b] = f64(acc_in)[p, h, tok % b] + w
            bound[p, h, tok % b] = rel * w + 2.0 ** -24 * want[p, h, tok % b]
    got = f64(acc_out)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    err = np.abs(got - want)[ok] - bound[ok]
    assert (err <= 0).all(), float(err.max())


WEIGHTS = [
    # four, b, lens, H, G, paged, M, n_sel, bias
    (True, 64, [1], 1, 1, False, 1, 0, False),
    (False, 64, [1, 0, 17], 1, 4, True, 1, 0, False),
    (True, 64, [64, 65, 2000], 2, 4, True, 1, 0, False),
    (False, 128, [129, 1500], 2, 7, False, 1, 0, False),
    (True, 128, [3000], 2, 7, True, 16, 0, False),       # 112 rows
    (False, 64, [700, 9], 1, 16, True, 10, 0, False),    # 160 rows: staged twice; a sequence shorter than M
    (True, 64, [4096, 100], 2, 5, True, 1, 16, False),
    (False, 64, [4096, 100], 2, 5, True, 1, 16, True),
    (False, 128, [5000], 2, 16, False, 1, 7, True),
    (True, 64, [600], 1, 3, False, 5, 4, False),
    (True, 64, [900, 5], 1, 16, True, 20, 0, False),     # 320 rows
    (True, 64, [3000, 70], 2, 6, True, 4, 9, False),     # 24 rows over an odd number of blocks
    (True, 128, [4000], 1, 11, False, 7, 5, False),      # 77 rows
    (False, 64, [3000, 70], 2, 6, True, 4, 9, False),
    (False, 128, [2222, 64], 1, 11, True, 7, 0, False),
    (False, 64, [40000, 100, 2500], 8, 2, True, 1, 0, False),   # long: shares that span sequences
    (True, 64, [40000, 100, 2500], 8, 2, True, 1, 0, False),
]


@pytest.mark.parametrize("four,b,lens,H,G,paged,M,n_sel,with_bias", WEIGHTS)
def test_weights_match_oracle(four, b, lens, H, G, paged, M, n_sel, with_bias):
    lay = layout(lens, b, paged, seed=G)
    B = len(lens)
    k = rand_bf16((lay.pages, H, b, 128), 1)
    for s, x in enumerate(lens):                            # garbage past the last token
        for r in range(x, -(-x // b) * b):
            k[page(lay, s, r // b), :, r % b] = float("nan")
    sel = selection(lay, b, H, n_sel, 3) if n_sel else None
    q = rand_bf16((B, M, H * G, 128), 4, 0)
    bias = None
    if with_bias:
        bias = -8 * np.random.default_rng(1).random((B, H * G, n_sel)).astype(np.float32)
        bias[0, 0, 0], bias[0, 1 % (H * G), 0] = -np.inf, np.finfo(np.float32).min
    kv = packed(k, k) if four else None
    K = SC.unpack_tile(kv.numpy())[0] if four else f64(k)
    # lse of the same attention, rounded to fp32
    lse = np.full((B, M, H * G), -np.inf)
    for s in range(B):
        for h in range(H):
            kk = SC.gather(K, lay.table, s, lay.max_blocks, h, lens[s])
            blocks = None if sel is None else sel[0][s, h, :sel[1][s, h]]
            tok = SC.tokens_of(lens[s], b, blocks)
            if len(tok):
                bb = None
                if bias is not None:
                    bb = bias[s, h * G:(h + 1) * G][:, np.repeat(np.arange(len(blocks)), b)[:len(tok)]][None]
                x = SC.logits(f64(q)[s, :, h * G:(h + 1) * G], kk, tok, lens[s], SCALE, bb)
                lse[s, :, h * G:(h + 1) * G] = SC.attend(x, kk[tok] * 0)[1]
    lse = torch.from_numpy(lse.astype(np.float32))
    acc = per_page(lay, b, H, 5)
    start = torch.full_like(acc, 3.0)
    c = cache4(lay, kv, H_q=H * G, desc=False) if four else cache16(lay, k, k, H * G, desc=False)
    call = sba.sba_accumulate_weights_kv4 if four else sba.sba_accumulate_weights
    kw = {} if sel is None else dict(sel_idx=torch.from_numpy(sel[0]).to(DEV), sel_cnt=torch.from_numpy(sel[1]).to(DEV))
    if bias is not None:
        kw["gate_bias"] = torch.from_numpy(bias).to(DEV)
    out, a_in = start.to(DEV), acc.to(DEV)
    call(c, q.to(DEV), lse.to(DEV), SCALE, a_in, out, **kw)
    check_weights(lay, b, G, K, q, lse, sel, bias, acc, out, f64(start))
    assert torch.equal(a_in.cpu(), acc) and int(c.status.item()) == 0
    call(c, q.to(DEV), lse.to(DEV), SCALE, a_in, a_in, **kw)            # in place, the same bits
    inside = out != 3.0
    assert torch.equal(a_in[inside], out[inside]) and torch.equal(a_in[~inside].cpu(), acc[~inside.cpu()])


def test_weights_of_a_step_sum_to_the_rows():
    """Every query row's weights sum to 1, whatever the split into pages: a step over all blocks adds
    the number of its rows, per KV head."""
    lay, b, H, G = layout([1777], 64, True, 2), 64, 2, 4
    k, v = rand_bf16((lay.pages, H, b, 128), 1), rand_bf16((lay.pages, H, b, 128), 2)
    c = cache4(lay, packed(k, v), H_q=H * G, desc=False)
    q = rand_bf16((1, 1, H * G, 128), 3, 0)
    _, lse, _ = run_decode(c, q, None, False)
    acc = torch.zeros((lay.pages, H, b), device=DEV)
    for step in range(1, 4):
        sba.sba_accumulate_weights_kv4(c, q.to(DEV), lse, SCALE, acc, acc)
        assert np.allclose(f64(acc).sum((0, 2)), step * G, rtol=1e-5)


def test_weights_refuse_a_block_listed_twice():
    lay, b, H, G = layout([640], 64, True, 2), 64, 1, 2
    k = rand_bf16((lay.pages, H, b, 128), 1)
    c = cache16(lay, k, k, H * G, desc=False)
    q = rand_bf16((1, 1, H * G, 128), 3, 0)
    lse = torch.full((1, 1, H * G), 9.0)
    acc = torch.zeros((lay.pages, H, b), device=DEV)
    idx, cnt = np.array([[[2, 5, 5, 4, 77]]], dtype=np.int32), np.array([[5]], dtype=np.int32)
    sba.sba_accumulate_weights(c, q.to(DEV), lse.to(DEV), SCALE, acc, acc, sel_idx=torch.from_numpy(idx).to(DEV),
                               sel_cnt=torch.from_numpy(cnt).to(DEV))
    assert int(c.status.item()) == sba.SBA_DEV_BAD_SELECTION
    got = acc.cpu().numpy()
    once = np.array([[[2, 5]]], dtype=np.int32)
    check_weights(lay, b, G, f64(k), q, lse, (once, np.array([[2]])), None, torch.zeros(got.shape), acc.cpu(),
                  np.zeros(got.shape))


# ---------------------------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------------------------

EVICTS = [
    # four, b, lens, H, paged, keep, sink, recent
    (False, 64, [1], 1, False, 1, 0, 0),
    (False, 64, [200, 64, 0, 65], 2, True, 64, 2, 7),
    (True, 64, [200, 64, 0, 65], 2, True, 65, 0, 0),
    (True, 128, [1000, 130], 2, True, 300, 4, 100),
    (False, 128, [1000], 3, False, 129, 129, 0),         # only the first ones
    (False, 64, [1000], 1, True, 100, 40, 60),           # nothing ranked
    (True, 64, [5000, 4097, 300], 1, True, 1000, 4, 32),
    (False, 64, [70000], 1, True, 3333, 4, 128),         # a cluster of eight
    (True, 128, [70000, 9000], 4, False, 2500, 0, 1),
    (False, 64, [500, 20], 1, True, 600, 4, 16),         # nothing to evict
]


@pytest.mark.parametrize("four,b,lens,H,paged,n_keep,n_sink,n_recent", EVICTS)
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict_matches_oracle(four, b, lens, H, paged, n_keep, n_sink, n_recent, kind):
    lay, dlay = layout(lens, b, paged, 1), layout([n_keep] * len(lens), b, paged, 2, slack=0)
    B = len(lens)
    g = torch.Generator().manual_seed(3)
    acc = torch.exp(2 * torch.randn((lay.pages, H, b), generator=g))
    if kind == "ties":
        acc = torch.round(acc)                              # many equal weights, most of them 0 or 1
    if kind == "odd":                                       # negative, both zeros, infinities, NaN, tiny
        vals = torch.tensor([-1.0, -0.0, 0.0, float("inf"), -float("inf"), float("nan"), 1e-42, 2.5])
        pick = torch.randint(0, 8, acc.shape, generator=g)
        acc = torch.where(torch.rand(acc.shape, generator=g) < 0.5, vals[pick], acc)
    if four:
        kv = torch.randint(0, 256, (lay.pages, H, b // 32, 4608), generator=g, dtype=torch.uint8)
        kv[..., 4096:] %= 227                               # finite scales
        src = cache4(lay, kv, H_q=H, desc=False)
        start = torch.randint(0, 256, (dlay.pages, H, b // 32, 4608), generator=g, dtype=torch.uint8)
        dst = cache4(dlay, start, H_q=H)
        keys = SC.unpack_tile(kv.numpy())[0]
    else:
        k, v = rand_bf16((lay.pages, H, b, 128), 4), rand_bf16((lay.pages, H, b, 128), 5)
        src = cache16(lay, k, v, H, desc=False)
        start_k, start_v = rand_bf16((dlay.pages, H, b, 128), 6), rand_bf16((dlay.pages, H, b, 128), 7)
        dst = cache16(dlay, start_k, start_v, H)
        keys = f64(k)
    acc_dst = torch.full((dlay.pages, H, b), -5.0, device=DEV)
    new_lens = torch.full((B,), -1, dtype=torch.int32, device=DEV)
    kept = torch.full((B, H, n_keep), -9, dtype=torch.int32, device=DEV)
    dst.seq_lens = new_lens
    call = sba.sba_evict_kv4 if four else sba.sba_evict
    call(src, acc.to(DEV), sba.evict_params(n_keep, n_sink, n_recent), dst, new_lens, kept, acc_dst=acc_dst)
    assert int(src.status.item()) == 0 and int(dst.status.item()) == 0
    want_new = [min(x, n_keep) for x in lens]
    assert new_lens.tolist() == want_new
    want_acc, want_desc = np.full(acc_dst.shape, -5.0), np.zeros((dlay.pages, H, 2, 128))
    if four:
        want_kv = start.numpy().copy()
    else:
        want_k, want_v = f64(start_k), f64(start_v)
    a = acc.numpy()
    for s in range(B):
        for h in range(H):
            w = SC.gather(a, lay.table, s, lay.max_blocks, h, lens[s])
            want = SC.keep(w, n_keep, n_sink, n_recent)
            got = kept[s, h].cpu().numpy()
            assert np.array_equal(got[:want_new[s]], want), (s, h)
            assert (got[want_new[s]:] == -9).all()
            for i, t in enumerate(want):
                p, r, dp, dr = page(lay, s, t // b), t % b, page(dlay, s, i // b), i % b
                want_acc[dp, h, dr] = a[p, h, r]
                if four:
                    for base, width in ((0, 64), (2048, 64), (4096, 8), (4352, 8)):
                        d, f = base + dr % 32 * width, base + r % 32 * width
                        want_kv[dp, h, dr // 32, d:d + width] = kv[p, h, r // 32, f:f + width].numpy()
                else:
                    want_k[dp, h, dr], want_v[dp, h, dr] = f64(k[p, h, r]), f64(v[p, h, r])
                x = keys[p, h, r]
                if dr == 0:
                    want_desc[dp, h, 0], want_desc[dp, h, 1] = x, x
                else:
                    want_desc[dp, h, 0] = np.minimum(want_desc[dp, h, 0], x)
                    want_desc[dp, h, 1] = np.maximum(want_desc[dp, h, 1], x)
    assert np.array_equal(f64(acc_dst), want_acc, equal_nan=True)
    assert np.array_equal(f64(dst.desc), want_desc)
    if four:
        assert np.array_equal(dst.kv.cpu().numpy(), want_kv)
    else:
        assert np.array_equal(f64(dst.k), want_k) and np.array_equal(f64(dst.v), want_v)


def test_evict_slices_longer_than_shared_memory():
    """More heads than the GPU holds clusters, each with more tokens than one CTA keeps in shared memory."""
    b, H, n, keep = 64, 80, 70000, 700
    lay, dlay = layout([n], b, False, 1, slack=0), layout([keep], b, False, 2, slack=0)
    g = torch.Generator(device="cuda").manual_seed(3)
    kv = torch.randint(0, 256, (lay.pages, H, b // 32, 4608), generator=g, dtype=torch.uint8, device=DEV)
    kv[..., 4096:] %= 227
    src, dst = cache4(lay, kv, H_q=H, desc=False), cache4(dlay, torch.zeros((dlay.pages, H, b // 32, 4608), dtype=torch.uint8), H)
    acc = torch.round(torch.exp(2 * torch.randn((lay.pages, H, b), generator=g, device=DEV)))
    new_lens, kept = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros((1, H, keep), dtype=torch.int32, device=DEV)
    sba.sba_evict_kv4(src, acc, sba.evict_params(keep, 5, 40), dst, new_lens, kept)
    assert new_lens.tolist() == [keep] and int(src.status.item()) == 0
    a, got = acc.cpu().numpy(), kept.cpu().numpy()
    for h in (0, 41, 79):
        assert np.array_equal(got[0, h], SC.keep(SC.gather(a, None, 0, lay.max_blocks, h, n), keep, 5, 40))
        t = torch.from_numpy(got[0, h]).long().to(DEV)
        rows = src.kv[t // b, h, (t % b) // 32, :2048].reshape(keep, 32, 64)[torch.arange(keep), t % 32]
        i = torch.arange(keep, device=DEV)
        moved = dst.kv[i // b, h, (i % b) // 32, :2048].reshape(keep, 32, 64)[torch.arange(keep), i % 32]
        assert torch.equal(rows, moved)


@pytest.mark.parametrize("H,n", [(1, 70000), (2, 9000), (80, 70000)])
@pytest.mark.parametrize("near", [1, 1023, 1024, 1025, 6000])
def test_evict_tokens_that_share_the_thresholds_upper_bits(H, n, near):
    """Around 1024 weights whose upper 16 bits are the threshold's; slices held in shared memory and longer ones."""
    b, sink, recent, more = 64, 3, 7, 50
    keep = sink + recent + more + (near + 1) // 2
    lay, dlay = layout([n], b, False, 1, slack=0), layout([keep], b, False, 2, slack=0)
    g = torch.Generator(device="cuda").manual_seed(near)
    acc = 0.5 * torch.rand((H, n), generator=g, device=DEV)
    for h in range(H):
        at = sink + torch.randperm(n - sink - recent, generator=g, device=DEV)[:near + more]
        low = torch.randint(0, 1 << (16 if h % 2 == 0 else 3), (near,), generator=g, device=DEV)  # distinct, or ties
        acc[h, at[:near]] = (0x3f800000 + low).to(torch.int32).view(torch.float32)
        acc[h, at[near:]] = 2 + torch.rand(more, generator=g, device=DEV)
    padded = torch.zeros((H, lay.pages * b), device=DEV)
    padded[:, :n] = acc
    pool = padded.reshape(H, lay.pages, b).transpose(0, 1).contiguous()
    kv = torch.zeros((lay.pages, H, b // 32, 4608), dtype=torch.uint8, device=DEV)
    src, dst = cache4(lay, kv, H_q=H, desc=False), cache4(dlay, torch.zeros((dlay.pages, H, b // 32, 4608), dtype=torch.uint8), H)
    new_lens, kept = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros((1, H, keep), dtype=torch.int32, device=DEV)
    sba.sba_evict_kv4(src, pool, sba.evict_params(keep, sink, recent), dst, new_lens, kept)
    assert new_lens.tolist() == [keep] and int(src.status.item()) == 0
    w, got = acc.cpu().numpy(), kept.cpu().numpy()
    for h in {0, 1, H - 1} & set(range(H)):
        assert np.array_equal(got[0, h], SC.keep(w[h], keep, sink, recent))


def test_weights_past_four_gigabytes_and_understated_selection():
    """Key pages whose byte offsets do not fit 32 bits (bf16 and four bits, few rows and many), and selections
    shorter than their row."""
    b, H, G = 128, 4, 8
    for four, M in ((False, 1), (False, 9), (True, 1), (True, 9)):
        lay = layout([700], b, True, 1)
        per = H * b // 32 * 4608 if four else H * b * 256
        pages = (5 << 30) // per
        lay.table[0, :6] = np.arange(pages - 9, pages - 3)[::-1]
        k = rand_bf16((6, H, b, 128), 3)
        small = layout([700], b, False, 1, slack=0)
        if four:
            big = torch.zeros((pages, H, b // 32, 4608), dtype=torch.uint8, device=DEV)
            rows = packed(k, k)
            big[torch.from_numpy(lay.table[0, :6]).long().to(DEV)] = rows.to(DEV)
            K = SC.unpack_tile(rows.numpy())[0]
            lay.pages = pages
            c = cache4(lay, big, H_q=H * G, desc=False)
        else:
            big = torch.zeros((pages, H, b, 128), dtype=torch.bfloat16, device=DEV)
            big[torch.from_numpy(lay.table[0, :6]).long().to(DEV)] = k.to(DEV)
            K = f64(k)
            lay.pages = pages
            c = cache16(lay, big, big, H_q=H * G, desc=False)
        q = rand_bf16((1, M, H * G, 128), 5, 0)
        lse = torch.full((1, M, H * G), 5.0)
        idx = torch.tensor([[[0, 2, 5, 900]] * H], dtype=torch.int32, device=DEV)     # the last entry does not count
        cnt = torch.full((1, H), 3, dtype=torch.int32, device=DEV)
        acc = torch.zeros((pages, H, b), device=DEV)
        call = sba.sba_accumulate_weights_kv4 if four else sba.sba_accumulate_weights
        call(c, q.to(DEV), lse.to(DEV), SCALE, acc, acc, sel_idx=idx, sel_cnt=cnt)
        assert int(c.status.item()) == 0
        got = acc[torch.from_numpy(lay.table[0, :6]).long().to(DEV)].cpu()
        sel = (np.array([[[0, 2, 5]] * H]), np.full((1, H), 3))
        check_weights(small, b, G, K, q, lse, sel, None, torch.zeros(got.shape), got, np.zeros(got.shape))
        del big, acc, c


def test_evict_bad_pages_are_skipped_and_reported():
    b, H = 64, 1
    lay, dlay = layout([640], b, True, 1), layout([128], b, True, 2, slack=0)
    k = rand_bf16((lay.pages, H, b, 128), 1)
    src, dst = cache16(lay, k, k, H, desc=False), cache16(dlay, torch.zeros((dlay.pages, H, b, 128), dtype=torch.bfloat16),
                                                          torch.zeros((dlay.pages, H, b, 128), dtype=torch.bfloat16), H)
    acc = per_page(lay, b, H, 3).to(DEV)
    new_lens, kept = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros((1, H, 128), dtype=torch.int32, device=DEV)
    src.block_table[0, 3] = lay.pages                       # its tokens rank last
    dst.block_table[0, 1] = -2                              # its rows are not written
    sba.sba_evict(src, acc, sba.evict_params(128), dst, new_lens, kept)
    assert int(src.status.item()) == sba.SBA_DEV_BAD_PAGE and int(dst.status.item()) == sba.SBA_DEV_BAD_PAGE
    t = kept[0, 0].cpu().numpy()
    assert (t // b != 3).all() and (np.diff(t) > 0).all()
    got = f64(dst.k)[page(dlay, 0, 0), 0]
    assert np.array_equal(got, np.stack([f64(k)[page(lay, 0, x // b), 0, x % b] for x in t[:b]]))
    assert (f64(dst.k)[[p for p in range(dlay.pages) if p != page(dlay, 0, 0)]] == 0).all()


# ---------------------------------------------------------------------------------------------
# all of them together
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("sparse", [False, True])
def test_decode_loop_with_eviction(sparse):
    """A prompt is written in four bits; steps append a token, (select,) attend and accumulate; every
    few steps the cache is cut and goes on in other pages.  Checked against the oracle at every step."""
    b, H, G, B, keep, prompt = 64, 2, 4, 2, 160, 300
    lay = [layout([prompt + 40] * B, b, True, 1), layout([keep + 40] * B, b, True, 2)]
    dev_kv = [torch.zeros((x.pages, H, b // 32, 4608), dtype=torch.uint8) for x in lay]
    c = [cache4(x, kv, H_q=H * G, lens=[prompt] * B) for x, kv in zip(lay, dev_kv)]
    acc = [torch.zeros((x.pages, H, b), device=DEV) for x in lay]
    kn, vn = rand_bf16((B, prompt, H, 128), 3), rand_bf16((B, prompt, H, 128), 4)
    sba.sba_append_kv4(c[0], kn.to(DEV), vn.to(DEV), i32([0] * B))
    keys = [[f for f in SC.held(f64(kn)).transpose(0, 2, 1, 3)[s]] for s in range(B)]       # [s][h] -> [len][128]
    vals = [[f for f in SC.held(f64(vn)).transpose(0, 2, 1, 3)[s]] for s in range(B)]
    total = [[np.zeros(prompt) for _ in range(H)] for _ in range(B)]
    at, length = 0, prompt
    p = sba.select_params(3, 1, 0)
    for step in range(14):
        cc, L = c[at], lay[at]
        k1, v1, q = (rand_bf16((B, 1, n, 128), 100 + 3 * step + i) for i, n in enumerate((H, H, H * G)))
        cc.seq_lens += 1
        sba.sba_append_kv4(cc, k1.to(DEV), v1.to(DEV), i32([length] * B))
        for s in range(B):
            for h in range(H):
                keys[s][h] = np.concatenate((keys[s][h], SC.held(f64(k1))[s, :, h]))
                vals[s][h] = np.concatenate((vals[s][h], SC.held(f64(v1))[s, :, h]))
                total[s][h] = np.append(total[s][h], 0.0)
                for p0, d in ((0, acc[at]),):
                    d[page(L, s, length // b), h, length % b] = 0
        length += 1
        sel, kw = None, {}
        if sparse:
            ws = torch.zeros(sba.sba_score_select_kv4_workspace_size(cc, p), dtype=torch.uint8, device=DEV)
            si, sc = torch.zeros((B, H, 3), dtype=torch.int32, device=DEV), torch.zeros((B, H), dtype=torch.int32, device=DEV)
            sba.sba_score_select_kv4(cc, q.to(DEV), p, si, sc, ws)
            sel, kw = (si.cpu().numpy(), sc.cpu().numpy()), dict(sel_idx=si, sel_cnt=sc)
        out, lse, _ = run_decode(cc, q, sel, True)
        sba.sba_accumulate_weights_kv4(cc, q.to(DEV), lse, SCALE, acc[at], acc[at], **kw)
        now = layout([length] * B, b, True, 0)
        now.table, now.max_blocks, now.pages = L.table, L.max_blocks, L.pages
        check_decode(cc, cc.kv.cpu().numpy(), now, q, sel, out, lse, b, G, True)
        for s in range(B):
            for h in range(H):
                blocks = None if sel is None else sel[0][s, h, :sel[1][s, h]]
                tok = SC.tokens_of(length, b, blocks)
                x = SC.logits(f64(q)[s, :, h * G:(h + 1) * G], keys[s][h], tok, length, SCALE)
                total[s][h][tok] += SC.weights(x, SC.attend(x, vals[s][h][tok])[1])
                got = SC.gather(f64(acc[at]), L.table, s, L.max_blocks, h, length)
                assert np.allclose(got, total[s][h], rtol=1e-4, atol=1e-6)
        if step % 5 == 4:
            new_lens = torch.zeros(B, dtype=torch.int32, device=DEV)
            kept = torch.zeros((B, H, keep), dtype=torch.int32, device=DEV)
            to = 1 - at
            sba.sba_evict_kv4(cc, acc[at], sba.evict_params(keep, 4, 16), c[to], new_lens, kept, acc_dst=acc[to])
            for s in range(B):
                for h in range(H):
                    t = kept[s, h].cpu().numpy()
                    w = SC.gather(f64(acc[at]), L.table, s, L.max_blocks, h, length)   # what the GPU ranked by
                    assert np.array_equal(t, SC.keep(w, keep, 4, 16))
                    keys[s][h], vals[s][h], total[s][h] = keys[s][h][t], vals[s][h][t], w[t]
            c[to].seq_lens.copy_(new_lens)
            at, length = to, keep
    assert all(int(x.status.item()) == 0 for x in c)


def test_calls_in_a_graph():
    """Accumulate and evict captured together and replayed on new inputs."""
    b, H, G = 64, 2, 4
    lay, dlay = layout([5000, 900], b, True, 1), layout([512] * 2, b, True, 2, slack=0)
    kv = packed(rand_bf16((lay.pages, H, b, 128), 1), rand_bf16((lay.pages, H, b, 128), 2))
    c, dst = cache4(lay, kv, H_q=H * G, desc=False), cache4(dlay, torch.zeros((dlay.pages, H, b // 32, 4608), dtype=torch.uint8), H * G)
    q = rand_bf16((2, 1, H * G, 128), 3, 0).to(DEV)
    lse = torch.empty((2, 1, H * G), device=DEV)
    out = torch.empty((2, 1, H * G, 128), dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(sba.sba_decode_kv4_workspace_size(c, 1, 0), dtype=torch.uint8, device=DEV)
    acc0 = per_page(lay, b, H, 4).to(DEV)

    def steps(acc, new_lens, kept):
        sba.sba_decode_kv4(c, q, SCALE, out, ws, lse_out=lse)
        sba.sba_accumulate_weights_kv4(c, q, lse, SCALE, acc0, acc)
        sba.sba_evict_kv4(c, acc, sba.evict_params(512, 4, 64), dst, new_lens, kept)

    bufs = [(acc0.clone(), torch.zeros(2, dtype=torch.int32, device=DEV),
             torch.zeros((2, H, 512), dtype=torch.int32, device=DEV)) for _ in range(2)]
    steps(*bufs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps(*bufs[1])
    for seed in (10, 11):
        q.copy_(rand_bf16((2, 1, H * G, 128), seed, 0))
        graph.replay()
        moved = dst.kv.clone()
        dst.kv.zero_()
        steps(*bufs[0])
        torch.cuda.synchronize()
        for x, y in zip(*bufs):
            assert torch.equal(x, y)
        assert torch.equal(moved, dst.kv)
