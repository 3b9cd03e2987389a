"""The bf16 loop as a program runs it: one-launch decode steps (Quest, and the gate at each of its places),
the selected tokens' weights accumulated, evictions into other pages, descriptors, and on."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_sparse_gqa_min_b200 import sba
from oracle import small_cache as SC
from tests.helpers import ATOL_OUT
from tests.kv4_helpers import SCALE, cache16, f64, layout, logit_bound, rand_bf16
from tests.test_kv4_gpu import i32

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = torch.device("cuda")
PLACES = {"off": sba.SBA_LOG_GATE_OFF, "inner": sba.SBA_LOG_GATE_INNER, "outer": sba.SBA_LOG_GATE_OUTER}


@pytest.mark.parametrize("place", ["quest", "off", "inner", "outer"])
def test_decode_weigh_evict_and_on(place):
    b, H, G, B, keep, start, n_max = 64, 2, 4, 2, 330, 600, 4
    gated = place != "quest"
    p = sba.select_params(n_max, 1, 0, 0, 0, sba.SBA_SCORER_GATE if gated else sba.SBA_SCORER_QUEST,
                          PLACES[place] if gated else 0)
    g = torch.Generator().manual_seed(1)
    W = [torch.randn(s, generator=g).to(DEV) * 0.1 for s in ((128, 128), (128, 384))] if gated else []
    A = None
    if gated:
        A = torch.empty((128, 384), device=DEV)
        sba.sba_fold_gate(*W, A)

    def cache(lay, k, v, n):
        c = cache16(lay, k, v, H * G, desc=not gated)
        c.seq_lens.fill_(n)
        c.kg = torch.zeros((lay.pages, H, 128), device=DEV) if gated else None
        return c

    lay = [layout([start + 10] * B, b, True, 1), layout([keep + 10] * B, b, True, 2)]
    k0, v0 = rand_bf16((lay[0].pages, H, b, 128), 1), rand_bf16((lay[0].pages, H, b, 128), 2)
    empty = torch.zeros((lay[1].pages, H, b, 128), dtype=torch.bfloat16)
    c = [cache(lay[0], k0, v0, start), cache(lay[1], empty, empty.clone(), 0)]
    acc = [torch.zeros((x.pages, H, b), device=DEV) for x in lay]
    sba.sba_update_descriptors(c[0], i32([0] * B), start, *W)
    at, length = 0, start
    si, sc = torch.zeros((B, H, n_max), dtype=torch.int32, device=DEV), torch.zeros((B, H), dtype=torch.int32, device=DEV)
    gb = torch.zeros((B, H * G, n_max), device=DEV) if gated else None
    out, lse = torch.empty((B, H * G, 128), device=DEV), torch.empty((B, H * G), device=DEV)
    for step in range(9):
        cc, L = c[at], lay[at]
        k1, v1, q = (rand_bf16((B, 1, n, 128), 50 + 3 * step + i, 0) for i, n in enumerate((H, H, H * G)))
        cc.seq_lens += 1
        for s in range(B):                                    # an appended token has received nothing yet
            acc[at][int(L.table[s, length // b]), :, length % b] = 0
        sba.sba_decode_step(cc, q[:, 0].contiguous().to(DEV), p, SCALE, out, lse, k_new=k1.to(DEV), v_new=v1.to(DEV),
                            pos_start=i32([length] * B), gate_A=A, sel_idx=si, sel_cnt=sc, gate_bias=gb)
        length += 1
        before = acc[at].clone()
        sba.sba_accumulate_weights(cc, q.to(DEV), lse, SCALE, acc[at], acc[at], sel_idx=si, sel_cnt=sc,
                                   gate_bias=gb if place in ("inner", "outer") else None)
        K, V, bias = f64(cc.k), f64(cc.v), None if gb is None else f64(gb)
        for s in range(B):
            for h in range(H):
                kk, vv = (SC.gather(x, L.table, s, L.max_blocks, h, length) for x in (K, V))
                assert np.array_equal(kk[-1], f64(k1)[s, 0, h])
                blocks = si[s, h, :int(sc[s, h])].cpu().numpy()
                assert len(blocks) == n_max and blocks[-1] == (length - 1) // b
                tok = SC.tokens_of(length, b, blocks)
                qg = f64(q)[s, :, h * G:(h + 1) * G]
                per_token = 0.0 if bias is None else bias[s, h * G:(h + 1) * G][:, np.repeat(np.arange(n_max), b)[:len(tok)]]
                x = SC.logits(qg, kk, tok, length, SCALE, per_token[None] if place == "inner" else None)
                z = SC.attend(x, vv[tok])[1]
                w = np.exp(x - z[..., None])[0]               # [G][tokens]: what each value enters the output with
                if place == "outer":
                    w = w * np.exp(per_token)
                assert np.abs(f64(out)[s, h * G:(h + 1) * G] - w @ vv[tok]).max() <= ATOL_OUT
                rel = 2 * np.expm1(logit_bound(qg, kk[tok])) + 2.0 ** -16
                was, now = (SC.gather(f64(a), L.table, s, L.max_blocks, h, length) for a in (before, acc[at]))
                want = was.copy()
                want[tok] += w.sum(0)
                assert (np.abs(now - want) <= rel * (want - was) + 2.0 ** -24 * np.abs(want)).all()
        if step % 4 == 3:
            new, kept = i32([0] * B), torch.zeros((B, H, keep), dtype=torch.int32, device=DEV)
            to = 1 - at
            sba.sba_evict(cc, acc[at], sba.evict_params(keep, 4, 70), c[to], new, kept, acc_dst=acc[to])
            assert new.tolist() == [keep] * B
            c[to].seq_lens.copy_(new)
            moved = None if gated else c[to].desc.clone()
            if gated:
                sba.sba_update_descriptors(c[to], i32([0] * B), keep, *W)
            # a cache built of the kept rows alone goes on with the same bits
            dl = lay[to]
            fresh = cache(dl, torch.zeros_like(c[to].k), torch.zeros_like(c[to].v), keep)
            for s in range(B):
                for h in range(H):
                    t = kept[s, h].cpu().numpy()
                    assert np.array_equal(t, SC.keep(SC.gather(f64(acc[at]), L.table, s, L.max_blocks, h, length), keep, 4, 70))
                    i = np.arange(keep)
                    for x, y in ((fresh.k, cc.k), (fresh.v, cc.v)):
                        x[torch.from_numpy(dl.table[s, i // b]).long(), h, torch.from_numpy(i % b)] = \
                            y[torch.from_numpy(L.table[s, t // b]).long(), h, torch.from_numpy(t % b)]
            sba.sba_update_descriptors(fresh, i32([0] * B), keep, *W)
            if not gated:
                pages = torch.from_numpy(np.unique(dl.table[:, :-(-keep // b)])).long().to(DEV)
                assert torch.equal(moved[pages], fresh.desc[pages])
            got = []
            for x in (c[to], fresh):
                o, l, i1, n1 = torch.empty_like(out), torch.empty_like(lse), torch.zeros_like(si), torch.zeros_like(sc)
                sba.sba_decode_step(x, q[:, 0].contiguous().to(DEV), p, SCALE, o, l, gate_A=A, sel_idx=i1, sel_cnt=n1)
                got.append((o, l, i1, n1))
            for x, y in zip(*got):
                assert torch.equal(x, y)
            at, length = to, keep
    assert all(int(x.status.item()) == 0 for x in c)
