"""The four-bit cache on the GPU against the fp64 oracle (oracle.small_cache): rows written and read
back exactly, Quest descriptors exactly, attention within a bound derived from its roundings."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block_sparse_gqa_min_b200 import sba
from oracle import small_cache as SC
from tests.kv4_helpers import (SCALE, cache4, f64, layout, logit_bound, packed, page, rand_bf16, selection)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

DEV = torch.device("cuda")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def same(got: np.ndarray, want: np.ndarray):
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(got[ok], want[ok])


# ---------------------------------------------------------------------------------------------
# rows
# ---------------------------------------------------------------------------------------------

WRITES = [
    # b, lens (after the write), H_kv, paged, n_new
    (64, [1], 1, False, 1),
    (64, [64, 65, 200], 2, True, 1),
    (64, [130, 97], 3, True, 33),
    (128, [128], 1, False, 128),
    (128, [129, 400, 131], 2, True, 130),
    (64, [1000, 700], 4, False, 700),
    (128, [300], 8, True, 299),
]


@pytest.mark.parametrize("b,lens,H,paged,n", WRITES)
def test_rows_written_read_back_and_described(b, lens, H, paged, n):
    lens = [max(x, n) for x in lens]
    lay = layout(lens, b, paged, seed=n)
    B = len(lens)
    old_k, old_v = rand_bf16((lay.pages, H, b, 128), 1), rand_bf16((lay.pages, H, b, 128), 2)
    kv0 = packed(old_k, old_v)
    c = cache4(lay, kv0, H_q=H)
    kn, vn = rand_bf16((B, n, H, 128), 3), rand_bf16((B, n, H, 128), 4)
    pos = [x - n for x in lens]
    sba.sba_append_kv4(c, kn.to(DEV), vn.to(DEV), i32(pos))
    # the pages hold exactly what the oracle packs (the sign of a zero is not kept)
    want = np.array(kv0.numpy())
    for s in range(B):
        for h in range(H):
            for x in range(n):
                t = pos[s] + x
                p, r = page(lay, s, t // b), t % b
                tile = want[p, h]
                for i, src in enumerate((kn, vn)):
                    codes, scales = SC.quantise(f64(src[s, x, h]))
                    tile[r // 32, 2048 * i + (r % 32) * 64:2048 * i + (r % 32) * 64 + 64] = codes[0::2] | (codes[1::2] << 4)
                    tile[r // 32, 4096 + 256 * i + (r % 32) * 8:4096 + 256 * i + (r % 32) * 8 + 8] = scales
    got = c.kv.cpu().numpy()
    for g, w in zip(SC.unpack_tile(got), SC.unpack_tile(want)):
        same(g, w)
    # rows that were not written keep their bytes
    touched = np.zeros(want.shape[:3] + (32,), dtype=bool)
    for s in range(B):
        for x in range(n):
            t = pos[s] + x
            touched[page(lay, s, t // b), :, (t % b) // 32, t % 32] = True
    for base, width in ((0, 64), (2048, 64), (4096, 8), (4352, 8)):
        part = got[..., base:base + 32 * width].reshape(*got.shape[:3], 32, width)
        was = kv0.numpy()[..., base:base + 32 * width].reshape(*got.shape[:3], 32, width)
        assert np.array_equal(part[~touched], was[~touched])
    # descriptors of the touched blocks, from all valid keys; the others untouched
    keys = SC.unpack_tile(want)[0]
    desc = np.zeros((lay.pages, H, 2, 128))
    for s in range(B):
        for j in range(pos[s] // b, (lens[s] - 1) // b + 1):
            valid = min(b, lens[s] - j * b)
            desc[page(lay, s, j), :, 0] = keys[page(lay, s, j), :, :valid].min(1)
            desc[page(lay, s, j), :, 1] = keys[page(lay, s, j), :, :valid].max(1)
    assert np.array_equal(f64(c.desc), desc)
    # read back
    ko, vo = (torch.full((B, n, H, 128), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sba.sba_read_kv4(c, i32(pos), ko, vo)
    assert np.array_equal(f64(ko), SC.held(f64(kn)))
    assert np.array_equal(f64(vo), SC.held(f64(vn)))
    assert int(c.status.item()) == 0


def test_every_kind_of_value():
    """Groups of random bit patterns over all exponents, ties, the largest and smallest scales, zeros,
    infinities and NaN: the held value of every element is the oracle's."""
    rng = np.random.default_rng(0)
    n, H, b = 4096, 1, 64
    bits = rng.integers(0, 1 << 16, size=(n, 8, 16), dtype=np.uint32)
    e = rng.integers(0, 255, size=(n, 8, 1))               # exponents near a common one, so that all codes occur
    near = ((np.clip(e - rng.integers(0, 5, size=bits.shape), 0, 254) << 7) | (bits & 0x807f)).astype(np.uint32)
    bits = np.where(rng.random((n, 8, 1)) < 0.9, near, bits)
    # exact ties: tie point * scale, with 6 * scale in the group
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for i in range(512):
        s = SC.SCALES[1 + i % 226]
        x = (np.tile(ties, 2) * s).astype(np.float32)
        bits[i, i % 8] = x.view(np.uint32) >> 16
    bits[600:604] = 0
    bits[604, 2] = 0x8000                                   # negative zeros
    bits[605, 3, 5] = 0x7f80                                # infinities and NaN poison their group only
    bits[606, 4, 0] = 0xff80
    bits[607, 5, 15] = 0x7fc0
    bits[608, 6] = 0x0001                                   # subnormals
    bits[609, 7] = 0x7f7f                                   # the largest bf16: held as 61440
    x = torch.from_numpy(bits.reshape(1, n, H, 128).astype(np.uint16).view(np.int16)).view(torch.bfloat16)
    lay = layout([n], b, False, 0)
    c = cache4(lay, torch.zeros((lay.pages, H, b // 32, 4608), dtype=torch.uint8), H_q=1)
    ko, vo = (torch.zeros((1, n, H, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sba.sba_append_kv4(c, x.to(DEV), x.flip(1).to(DEV), i32([0]))
    sba.sba_read_kv4(c, i32([0]), ko, vo)
    same(f64(ko), SC.held(f64(x)))
    same(f64(vo), SC.held(f64(x.flip(1))))
    same(SC.unpack_tile(c.kv.cpu().numpy())[0].reshape(-1, 128)[:n], SC.held(f64(x))[0, :, 0])


def test_rows_past_the_length_and_bad_places():
    b, H = 64, 2
    lay = layout([100, 50], b, True, seed=5)
    kv0 = packed(rand_bf16((lay.pages, H, b, 128), 1), rand_bf16((lay.pages, H, b, 128), 2))
    c = cache4(lay, kv0, H_q=H, lens=[90, 50])
    # positions 80..99 of a sequence of 90: written, but only 80..89 count in the descriptor
    kn, vn = rand_bf16((2, 20, H, 128), 3), rand_bf16((2, 20, H, 128), 4)
    sba.sba_append_kv4(c, kn.to(DEV), vn.to(DEV), i32([80, 30]))
    keys = SC.unpack_tile(c.kv.cpu().numpy())[0]
    assert np.array_equal(keys[page(lay, 0, 1), :, 16:36].transpose(1, 0, 2), SC.held(f64(kn[0])))
    assert np.array_equal(f64(c.desc)[page(lay, 0, 1), :, 1], keys[page(lay, 0, 1), :, :90 - 64].max(1))
    # reading 85..104: rows from 90 on are left
    ko, vo = (torch.full((2, 20, H, 128), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sba.sba_read_kv4(c, i32([85, 40]), ko, vo)
    assert np.array_equal(f64(ko)[0, :5], SC.held(f64(kn[0, 5:10])))
    assert (f64(ko)[0, 5:] == 9).all() and (f64(vo)[1, 10:] == 9).all() and not (f64(vo)[1, :10] == 9).all()
    assert int(c.status.item()) == 0
    # a sequence whose positions leave its table is left alone, the other one is written
    before = c.kv.clone()
    sba.sba_append_kv4(c, kn.to(DEV), vn.to(DEV), i32([lay.max_blocks * b - 19, 30]))
    assert int(c.status.item()) == sba.SBA_DEV_BAD_POSITION
    assert torch.equal(before, c.kv)                        # sequence 1 got the same rows again
    c.status.zero_()
    sba.sba_append_kv4(c, kn.to(DEV), vn.to(DEV), i32([-1, 30]))
    sba.sba_read_kv4(c, i32([-5, 40]), ko, vo)
    assert int(c.status.item()) == sba.SBA_DEV_BAD_POSITION and torch.equal(before, c.kv)
    # bad pages are skipped
    c.status.zero_()
    c.block_table[0, 1] = lay.pages
    c.block_table[1, 0] = -3
    sba.sba_append_kv4(c, kn.to(DEV), vn.to(DEV), i32([80, 30]))
    assert int(c.status.item()) == sba.SBA_DEV_BAD_PAGE and torch.equal(before, c.kv)


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------

def check_decode(c, kv, lay, q, sel, out, lse, b, G, f32, places=None):
    """Every row against the oracle; the bound follows the roundings of the kernel."""
    B, M, H_q, _ = q.shape
    K, V = SC.unpack_tile(kv)
    qq, oo, ll = f64(q), f64(out).reshape(q.shape), f64(lse).reshape(q.shape[:3])
    for s in range(B):
        for h in range(H_q // G):
            length = lay.lens[s]
            k = SC.gather(K, lay.table, s, lay.max_blocks, h, length)
            v = SC.gather(V, lay.table, s, lay.max_blocks, h, length)
            blocks = None if sel is None else sel[0][s, h, :sel[1][s, h]]
            tok = SC.tokens_of(length, b, blocks)
            qg = qq[s, :, h * G:(h + 1) * G]
            x = SC.logits(qg, k, tok, length, SCALE)
            o, z = SC.attend(x, v[tok])
            got_o, got_z = oo[s, :, h * G:(h + 1) * G], ll[s, :, h * G:(h + 1) * G]
            same(np.isneginf(got_z).astype(float), np.isneginf(z).astype(float))
            seen = np.isfinite(z)
            big = np.abs(x[np.isfinite(x)]).max(initial=0.0)
            eps = logit_bound(qg, k[tok]) + 3 * 2.0 ** -24 * (big + 8)
            # weights: the logit's error twice (weight and sum), exp2 and its argument, sums of T terms in
            # pairs and lanes (32 tokens a lane step, 8 warps, splits), P's f16 rounding
            T = len(tok)
            rel = 2 * np.expm1(eps) + 2.0 ** -20 + (T / 32 + 64) * 2.0 ** -24 * 2 + (2.0 ** -22 if f32 else 2.0 ** -11)
            vmax = np.abs(v[tok]).max(initial=0.0)
            tol = rel * vmax + (2.0 ** -23 if f32 else 2.0 ** -8) * np.abs(o)
            err = np.abs(got_o - o)
            assert (err <= tol)[seen].all(), (s, h, float((err - tol)[seen].max()), float(rel))
            assert (got_o[~seen] == 0).all()
            zt = eps + 2.0 ** -20 + (T / 32 + 64) * 2.0 ** -24 + 2.0 ** -23 * np.abs(z[seen])
            assert (np.abs(got_z[seen] - z[seen]) <= zt).all(), (s, h)


def decode_case(b, lens, H, G, paged, M, n_sel, f32, seed=0, qscale=1.0, sigma=0.5):
    lay = layout(lens, b, paged, seed)
    B = len(lens)
    kv = packed(rand_bf16((lay.pages, H, b, 128), seed + 1, sigma), rand_bf16((lay.pages, H, b, 128), seed + 2, sigma))
    # what lies past a sequence's last token is garbage: NaN scales
    for s, x in enumerate(lens):
        for r in range(x, -(-max(x, 1) // b) * b):
            p = page(lay, s, r // b)
            if p >= 0:
                kv[p, :, (r % b) // 32, 4096 + (r % 32) * 8:4096 + (r % 32) * 8 + 8] = 255
                kv[p, :, (r % b) // 32, 4352 + (r % 32) * 8:4352 + (r % 32) * 8 + 8] = 255
    q = (rand_bf16((B, M, H * G, 128), seed + 3, 0).float() * qscale).to(torch.bfloat16)
    c = cache4(lay, kv, H_q=H * G, desc=False)
    sel = selection(lay, b, H, n_sel, seed) if n_sel else None
    return lay, kv, q, c, sel


def run_decode(c, q, sel, f32, ws=None):
    n_max = 0 if sel is None else sel[0].shape[-1]
    M = q.shape[1]
    if ws is None:
        ws = torch.zeros(max(16, sba.sba_decode_kv4_workspace_size(c, M, n_max)), dtype=torch.uint8, device=DEV)
    out = torch.full(q.shape, 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, dtype=torch.float32, device=DEV)
    si = sc = None
    if sel is not None:
        si, sc = torch.from_numpy(sel[0]).to(DEV), torch.from_numpy(sel[1]).to(DEV)
    sba.sba_decode_kv4(c, q.to(DEV), SCALE, out, ws, lse_out=lse, sel_idx=si, sel_cnt=sc)
    return out, lse, ws


DECODES = [
    # b, lens, H_kv, G, paged, M, n_sel, f32
    (64, [1], 1, 1, False, 1, 0, True),
    (64, [31], 1, 8, False, 1, 0, True),
    (64, [32, 33], 2, 4, True, 1, 0, True),
    (64, [64, 65, 1, 0], 1, 3, True, 1, 0, False),
    (128, [127, 128, 129], 2, 7, True, 1, 0, True),
    (64, [5000, 777, 2049], 2, 4, True, 1, 0, True),
    (128, [9000], 1, 16, False, 1, 0, True),
    (64, [4096], 2, 9, False, 1, 0, False),
    (64, [4096, 100], 2, 4, True, 1, 16, True),
    (128, [20000], 2, 7, False, 1, 40, False),
    (64, [3000, 64], 1, 5, True, 1, 1, True),
    (64, [700, 3, 64], 2, 4, True, 4, 0, True),       # M = 4: 16 rows; a sequence shorter than M
    (64, [2000], 2, 5, False, 3, 8, False),
    (128, [1500, 129], 1, 8, True, 5, 6, True),       # 40 rows: three row groups
    (64, [513], 1, 16, False, 8, 0, True),
]


@pytest.mark.parametrize("b,lens,H,G,paged,M,n_sel,f32", DECODES)
def test_decode_matches_oracle(b, lens, H, G, paged, M, n_sel, f32):
    lay, kv, q, c, sel = decode_case(b, lens, H, G, paged, M, n_sel, f32, seed=len(lens) * 10 + G)
    out, lse, ws = run_decode(c, q, sel, f32)
    check_decode(c, kv.numpy(), lay, q, sel, out, lse, b, G, f32)
    assert int(c.status.item()) == 0
    again = run_decode(c, q, sel, f32, ws)                 # the workspace is reused as it was left
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("qscale,sigma", [(1e-30, 0.5), (2.0 ** 60, 0.5), (12.0, 0.5), (0.0, 0.5), (40.0, 1.5)])
def test_decode_small_large_and_peaked_queries(qscale, sigma):
    """Logits from none at all to thousands: rows scaled by powers of two, weights far below the maximum."""
    lay, kv, q, c, sel = decode_case(64, [2500, 300], 2, 4, True, 1, 0, True, seed=9, qscale=qscale, sigma=sigma)
    if qscale == 2.0 ** 60:                                 # one token takes everything; lse near 2^63
        out, lse, _ = run_decode(c, q, sel, True)
        K, V = SC.unpack_tile(kv.numpy())
        for s in range(2):
            for h in range(2):
                k = SC.gather(K, lay.table, s, lay.max_blocks, h, lay.lens[s])
                v = SC.gather(V, lay.table, s, lay.max_blocks, h, lay.lens[s])
                x = f64(q)[s, 0, h * 4:h * 4 + 4] @ k.T
                for g in range(4):
                    assert np.array_equal(f64(out)[s, 0, h * 4 + g], v[x[g].argmax()])
                    assert abs(f64(lse)[s, 0, h * 4 + g] / (x[g].max() * SCALE) - 1) <= 2.0 ** -16
        return
    out, lse, _ = run_decode(c, q, sel, True)
    check_decode(c, kv.numpy(), lay, q, sel, out, lse, 64, 4, True)


def test_decode_nan_reaches_only_the_rows_that_see_it():
    """A NaN value group of a token reaches its 16 channels of the rows that see the token; a NaN in the
    keys reaches whole rows; later rows' tokens reach no earlier row."""
    b, G, M = 64, 2, 4
    lay, kv, q, c, _ = decode_case(b, [200], 1, G, False, M, 0, True, seed=3)
    clean, clean_lse, _ = run_decode(c, q, None, True)
    t = 198                                                 # seen by tokens 2 and 3 of 196..199
    kv2 = kv.clone()
    kv2[page(lay, 0, t // b), 0, (t % b) // 32, 4352 + (t % 32) * 8 + 5] = 255
    c.kv.copy_(kv2)
    out, lse, _ = run_decode(c, q, None, True)
    assert torch.equal(out[:, :2], clean[:, :2]) and torch.equal(lse, clean_lse)
    assert torch.isnan(out[:, 2:, :, 80:96]).all()
    rest = torch.cat((out[:, 2:, :, :80], out[:, 2:, :, 96:]), -1)
    assert torch.equal(rest, torch.cat((clean[:, 2:, :, :80], clean[:, 2:, :, 96:]), -1))
    # a token every row sees
    kv2 = kv.clone()
    kv2[page(lay, 0, 0), 0, 0, 4352 + 3 * 8] = 255
    c.kv.copy_(kv2)
    out, lse, _ = run_decode(c, q, None, True)
    assert torch.isnan(out[..., :16]).all() and torch.equal(out[..., 16:], clean[..., 16:])
    # a NaN key
    kv2 = kv.clone()
    kv2[page(lay, 0, t // b), 0, (t % b) // 32, 4096 + (t % 32) * 8] = 255
    c.kv.copy_(kv2)
    out, lse, _ = run_decode(c, q, None, True)
    assert torch.equal(out[:, :2], clean[:, :2]) and torch.equal(lse[:, :2], clean_lse[:, :2])
    assert torch.isnan(out[:, 2:]).all() and torch.isnan(lse[:, 2:]).all()
    # a NaN query reaches its own row
    c.kv.copy_(kv)
    q2 = q.clone()
    q2[0, 1, 1, 7] = float("nan")
    out, lse, _ = run_decode(c, q2, None, True)
    assert torch.isnan(out[0, 1, 1]).all() and torch.isnan(lse[0, 1, 1])
    mask = torch.ones(M, G, dtype=torch.bool)
    mask[1, 1] = False
    assert torch.equal(out[0][mask], clean[0][mask])


def test_decode_bad_selection_and_pages():
    lay, kv, q, c, sel = decode_case(64, [1000], 1, 4, True, 1, 8, True, seed=4)
    idx, cnt = sel[0].copy(), sel[1].copy()
    good = (idx[:, :, 1:].copy(), cnt - 1)
    bad = idx.copy()
    bad[0, 0, 0] = 900                                      # a block that does not exist is skipped
    out, lse, _ = run_decode(c, q, (bad, cnt), True)
    assert int(c.status.item()) == sba.SBA_DEV_BAD_SELECTION
    check_decode(c, kv.numpy(), lay, q, good, out, lse, 64, 4, True)
    c.status.zero_()
    out, lse, _ = run_decode(c, q, (idx, cnt + 5), True)    # a count past the row is cut to it
    assert int(c.status.item()) == sba.SBA_DEV_BAD_SELECTION
    check_decode(c, kv.numpy(), lay, q, sel, out, lse, 64, 4, True)
    c.status.zero_()
    out, lse, _ = run_decode(c, q, (idx, cnt * 0), True)    # nothing selected
    assert int(c.status.item()) == 0 and (out == 0).all() and torch.isneginf(lse).all()
    c.block_table[0, int(idx[0, 0, 0])] = 10 ** 6
    out, lse, _ = run_decode(c, q, sel, True)
    assert int(c.status.item()) == sba.SBA_DEV_BAD_PAGE
    check_decode(c, kv.numpy(), lay, q, good, out, lse, 64, 4, True)


def test_decode_in_a_graph_and_on_another_stream():
    lay, kv, q, c, sel = decode_case(64, [3000, 500], 2, 4, True, 1, 0, True, seed=6)
    qd = q.to(DEV)
    out, lse, _ = run_decode(c, q, None, True)
    size = sba.sba_decode_kv4_workspace_size(c, 1, 0)
    ws = [torch.zeros(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [torch.empty_like(out) for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            sba.sba_decode_kv4(c, qd, SCALE, outs[0], ws[0])
    side = torch.cuda.Stream()
    for step in range(3):                                   # a graph and eager calls beside it, a workspace each
        q2 = rand_bf16(tuple(q.shape), 50 + step, 0)
        qd.copy_(q2)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            for _ in range(4):
                sba.sba_decode_kv4(c, qd, SCALE, outs[1], ws[1])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
        got, l2, _ = run_decode(c, q2, None, True)
        assert torch.equal(outs[0], got)
        check_decode(c, kv.numpy(), lay, q2, None, got, l2, 64, 4, True)


def test_decode_one_workspace_for_all_shapes():
    """A workspace of the largest size, zeroed once, serves calls of other shapes in any order: short and long
    caches (one unit a CTA; shares that span units), one and several tokens, selections."""
    cases = [decode_case(64, [700, 90], 2, 4, True, 1, 0, True, seed=21),
             decode_case(64, [40000, 333, 0, 9000], 2, 2, True, 1, 0, True, seed=22),
             decode_case(128, [300], 1, 8, False, 4, 0, True, seed=23),
             decode_case(64, [2000, 64], 2, 4, True, 1, 9, True, seed=24)]
    sizes = [sba.sba_decode_kv4_workspace_size(c, q.shape[1], 0 if sel is None else 9) for _, _, q, c, sel in cases]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device=DEV)
    own = [run_decode(c, q, sel, True)[:2] for _, _, q, c, sel in cases]
    for i in (0, 1, 2, 3, 1, 0, 3, 2, 2, 1):
        lay, kv, q, c, sel = cases[i]
        out, lse, _ = run_decode(c, q, sel, True, ws)
        assert torch.equal(out, own[i][0]) and torch.equal(lse, own[i][1])
    lay, kv, q, c, sel = cases[1]
    check_decode(c, kv.numpy(), lay, q, sel, *own[1], 64, 2, True)
    lay, kv, q, c, sel = cases[2]
    check_decode(c, kv.numpy(), lay, q, sel, *own[2], 128, 8, True)


@pytest.mark.parametrize("lens,H,G,M,f32", [([50000, 20000, 7, 33000], 4, 4, 1, True), ([60000], 2, 8, 2, False),
                                            ([9000] * 12, 4, 2, 1, True)])
def test_decode_long_launches(lens, H, G, M, f32):
    """Launches whose CTAs take equal shares of all sequences: units split over many CTAs, units within one,
    several units in one CTA."""
    lay, kv, q, c, sel = decode_case(64, lens, H, G, True, M, 0, f32, seed=31)
    out, lse, ws = run_decode(c, q, sel, f32)
    check_decode(c, kv.numpy(), lay, q, sel, out, lse, 64, G, f32)
    again = run_decode(c, q, sel, f32, ws)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and int(c.status.item()) == 0


def test_decode_pages_past_four_gigabytes():
    """Pages whose byte offsets do not fit 32 bits."""
    b, H, G = 128, 4, 4
    lens = [600]
    lay = layout(lens, b, True, 1)
    pages = (5 << 30) // (H * b // 32 * 4608)
    rng = np.random.default_rng(2)
    lay.table[0, :5] = rng.permutation(np.arange(pages - 40, pages))[:5]
    kv = torch.zeros((pages, H, b // 32, 4608), dtype=torch.uint8, device=DEV)
    c = cache4(lay, kv, H_q=H * G, desc=False)
    kn, vn = rand_bf16((1, 600, H, 128), 3), rand_bf16((1, 600, H, 128), 4)
    sba.sba_append_kv4(c, kn.to(DEV), vn.to(DEV), i32([0]))
    ko, vo = (torch.zeros((1, 600, H, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    sba.sba_read_kv4(c, i32([0]), ko, vo)
    assert np.array_equal(f64(ko), SC.held(f64(kn))) and np.array_equal(f64(vo), SC.held(f64(vn)))
    q = rand_bf16((1, 1, H * G, 128), 5, 0)
    out, lse, _ = run_decode(c, q, None, True)
    small = layout(lens, b, False, 1)
    tiles = c.kv[torch.from_numpy(lay.table[0, :5]).long().to(DEV)].cpu().numpy()
    check_decode(c, np.concatenate((tiles, tiles[:1])), small, q, None, out, lse, b, G, True)
    assert int(c.status.item()) == 0


def test_scoring_a_four_bit_cache():
    """sba_score_select_kv4 is the Quest selection on the descriptors of the held keys: the one
    sba_score_select makes on a bf16 cache of the read-back rows."""
    b, H, G, M = 64, 2, 4, 2
    lay = layout([4000, 900], b, True, 8)
    kv = torch.zeros((lay.pages, H, b // 32, 4608), dtype=torch.uint8)
    c = cache4(lay, kv, H_q=H * G)
    n = 4000
    kn, vn = rand_bf16((2, n, H, 128), 3), rand_bf16((2, n, H, 128), 4)
    for s, x in enumerate(lay.lens):                        # one call a sequence (the other's rows stay where they are)
        one = sba.Cache4(kv=c.kv, seq_lens=c.seq_lens[s:s + 1].clone(), H_q=H * G, max_blocks=lay.max_blocks,
                         max_len=x, block_table=c.block_table[s:s + 1].clone(), desc=c.desc, status=c.status)
        sba.sba_append_kv4(one, kn[s:s + 1, :x].contiguous().to(DEV), vn[s:s + 1, :x].contiguous().to(DEV), i32([0]))
    k16 = torch.zeros((lay.pages, H, b, 128), dtype=torch.bfloat16, device=DEV)
    k16.copy_(torch.from_numpy(SC.unpack_tile(c.kv.cpu().numpy())[0]))
    c16 = sba.Cache(k=k16, v=k16, seq_lens=c.seq_lens, H_q=H * G, max_blocks=lay.max_blocks, max_len=4000,
                    block_table=c.block_table, desc=torch.zeros_like(c.desc), status=c.status)
    sba.sba_update_descriptors(c16, i32([0, 0]), 4000)
    p = sba.select_params(12, 2, 4)
    q = rand_bf16((2, M, H * G, 128), 5, 0).to(DEV)
    ws = torch.zeros(sba.sba_score_select_kv4_workspace_size(c, p), dtype=torch.uint8, device=DEV)
    got = [torch.full((2, H, 12), -1, dtype=torch.int32, device=DEV) for _ in range(2)]
    cnt = [torch.zeros((2, H), dtype=torch.int32, device=DEV) for _ in range(2)]
    sba.sba_score_select_kv4(c, q, p, got[0], cnt[0], ws)
    sba.sba_score_select_multi(c16, q, p, got[1], cnt[1], ws)
    assert torch.equal(got[0], got[1]) and torch.equal(cnt[0], cnt[1]) and (cnt[0] == 12).all()
