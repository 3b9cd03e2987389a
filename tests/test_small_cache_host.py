"""The smaller cache without a GPU: the oracle's four-bit form pinned to hand values, and arguments
that the library or its binding reject before anything is enqueued."""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from block_sparse_gqa_min_b200 import sba
from oracle import small_cache as SC

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ARG, UNS, WS = sba.SBA_ERR_INVALID_ARG, sba.SBA_ERR_UNSUPPORTED, sba.SBA_ERR_WORKSPACE


def test_exports_every_declared_symbol_with_digits():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "sba.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(sba_[a-z0-9_]+)\s*\(", text))
    assert {"sba_append_kv4", "sba_read_kv4", "sba_decode_kv4", "sba_accumulate_weights_kv4", "sba_evict_kv4"} <= names
    for n in names:
        assert hasattr(sba.load(), n) and (n in sba._SIGS), n


# ---- the oracle's form ----

def row(*head):
    x = np.zeros(128)
    x[:len(head)] = head
    return x


def test_codes_are_the_nearest_and_ties_even():
    # max 6 -> scale 1: the codes themselves, their ties and their signs
    x = row(6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.26, -0.74, 1.24, 1.76, 2.51, -3.51, 5.01, -6)
    assert SC.held(x)[:16].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -0.5, -0.5, 1, 2, 3, -4, 6, -6]
    # the scale is the smallest that is at least max/6: 6.01 needs 1.125
    assert SC.held(row(6.01))[0] == 6.75
    assert SC.quantise(row(6.01))[1][0] == (15 << 3 | 1)
    # a group of its own every 16 channels
    y = row(*([0.0] * 16 + [12.0, 1.0]))
    assert SC.held(y)[16:18].tolist() == [12.0, 1.0] and SC.quantise(y)[1].tolist() == [0, 16 << 3, 0, 0, 0, 0, 0, 0]


def test_range_of_the_scales():
    assert SC.SCALES[1] == 2.0 ** -17 and SC.SCALES[8] == 2.0 ** -14 and SC.SCALES[226] == 10240
    assert SC.held(row(1e30, -1e30))[:2].tolist() == [61440, -61440]
    assert SC.held(row(2.0 ** -18))[0] == 2.0 ** -18 and SC.held(row(2.0 ** -18 * 0.5, 2.0 ** -17))[0] == 0
    assert np.isnan(SC.held(row(1.0, np.inf))[:16]).all() and not np.isnan(SC.held(row(1.0, np.inf))[16:]).any()
    assert np.isnan(SC.held(row(np.nan))[:16]).all()


def test_held_values_are_exact_in_f16_and_bf16_and_stay():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4096, 128)) * np.exp(3 * rng.standard_normal((4096, 1)))
    h = SC.held(x)
    t = torch.from_numpy(h)
    assert torch.equal(t, t.half().double()) and torch.equal(t, t.bfloat16().double())
    # inside the scales' range, relative to the group's largest, the error is at most half the widest code step (2 of 6) or the scale's 1/8
    g, e = np.abs(x).reshape(4096, 8, 16), np.abs(h - x).reshape(4096, 8, 16)
    big = (g.max(-1) > 6 * SC.SCALES[8]) & (g.max(-1) <= 61440)
    assert (e[big] <= (g.max(-1, keepdims=True) * 9 / 8 / 6)[big]).all()


def test_tiles_unpack_to_what_they_hold():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((128, 128)), rng.standard_normal((128, 128))
    a, b = SC.unpack_tile(SC.pack_tile(k, v))
    assert np.array_equal(a, SC.held(k)) and np.array_equal(b, SC.held(v))
    tile = SC.pack_tile(k, v)
    codes, scales = SC.quantise(k[37])
    assert tile[1, 5 * 64 + 3] == codes[6] | codes[7] << 4 and tile[1, 4096 + 5 * 8 + 2] == scales[2]


def test_attention_and_weights_of_the_oracle():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((2, 3, 128)), rng.standard_normal((50, 128)), rng.standard_normal((50, 128))
    x = SC.logits(q, k, SC.tokens_of(50, 64, None), 50, 0.1)
    o, lse = SC.attend(x, v)
    for i in range(2):
        n = 50 - 2 + i + 1
        s = torch.from_numpy(q[i] @ k[:n].T * 0.1)
        assert np.allclose(o[i], torch.softmax(s, -1).numpy() @ v[:n]) and np.allclose(lse[i], torch.logsumexp(s, -1))
    w = SC.weights(x, lse)
    assert np.isclose(w.sum(), 6) and np.isclose(w[49], np.exp(x[1, :, 49] - lse[1]).sum())


def test_eviction_rule_of_the_oracle():
    acc = np.array([0.0, 5, 1, 3, 3, np.nan, 3, 0, 2, -0.0])
    assert SC.keep(acc, 4, 0, 0).tolist() == [1, 3, 4, 6]
    assert SC.keep(acc, 4, 1, 1).tolist() == [0, 1, 3, 9]
    assert SC.keep(acc, 9, 0, 0).tolist() == [0, 1, 2, 3, 4, 6, 7, 8, 9]      # the NaN goes first
    assert SC.keep(acc, 7, 0, 0).tolist() == [0, 1, 2, 3, 4, 6, 8]            # 0 == -0: the first stays
    assert SC.keep(acc, 20, 3, 3).tolist() == list(range(10))


# ---- refusals ----

def c4(**kw):
    base = dict(kv=0x1000, block_table=None, seq_lens=0x3000, B=1, H_q=8, H_kv=2, d=128, b=64, max_blocks=64,
                num_pages=64, max_len=4096, desc=0x4000, status=None)
    base.update(kw)
    return ctypes.byref(sba.sba_cache4(**base))


def c16(**kw):
    base = dict(k=0x1000, v=0x2000, block_table=None, seq_lens=0x3000, B=1, H_q=8, H_kv=2, d=128, b=64, max_blocks=64,
                num_pages=64, max_len=4096, desc=0x4000, kg=None, status=None)
    base.update(kw)
    return ctypes.byref(sba.sba_cache(**base))


BAD_CACHES = [(dict(kv=None), ARG), (dict(kv=0x1008), ARG), (dict(seq_lens=None), ARG), (dict(B=0), ARG),
              (dict(H_q=7), ARG), (dict(d=64), UNS), (dict(b=32), UNS), (dict(H_q=34), UNS), (dict(max_len=4097), ARG),
              (dict(num_pages=63), ARG), (dict(max_blocks=40000, num_pages=40000), UNS), (dict(desc=0x4004), ARG)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_bad_four_bit_caches(kw, code):
    lib = sba.load()
    p = ctypes.byref(sba.select_params(16, 2))
    e = ctypes.byref(sba.evict_params(64))
    assert lib.sba_append_kv4(c4(**kw), 0x5000, 0x6000, 0x7000, 1, None) == code
    assert lib.sba_read_kv4(c4(**kw), 0x7000, 1, 0x5000, 0x6000, None) == code
    assert lib.sba_score_select_kv4(c4(**kw), 0x5000, 1, p, 0x6000, 0x7000, 16, 0x8000, 1 << 20, None) == code
    assert lib.sba_decode_kv4(c4(**kw), 0x5000, 1, None, None, 0, 0.1, 0x6000, 0, None, 0x8000, 1 << 30, None) == code
    assert lib.sba_accumulate_weights_kv4(c4(**kw), 0x5000, 1, None, None, 0, 0.1, 0x6000, 0x7000, 0x7000, None) == code
    assert lib.sba_evict_kv4(c4(**kw), 0x5000, e, c4(kv=0x9000), None, 0x6000, 0x7000, None) == code
    assert lib.sba_evict_kv4(c4(kv=0x9000), 0x5000, e, c4(**kw), None, 0x6000, 0x7000, None) == code
    assert lib.sba_decode_kv4_workspace_size(c4(**kw), 1, 0) == 0
    assert lib.sba_score_select_kv4_workspace_size(c4(**kw), p) == 0


def test_bad_append_and_read():
    lib = sba.load()
    ap, rd = lib.sba_append_kv4, lib.sba_read_kv4
    for k, v, pos, n in ((None, 0x6000, 0x7000, 1), (0x5000, None, 0x7000, 1), (0x5000, 0x6000, None, 1),
                         (0x5010, 0x6000, 0x7000, 1), (0x5000, 0x6010, 0x7000, 1), (0x5000, 0x6000, 0x7000, -1)):
        assert ap(c4(), k, v, pos, n, None) == ARG
        assert rd(c4(), pos, n, k, v, None) == ARG
    assert ap(c4(), 0x5000, 0x6000, 0x7000, 0, None) == sba.SBA_OK      # nothing to do
    assert rd(c4(), 0x7000, 0, 0x5000, 0x6000, None) == sba.SBA_OK
    assert ap(None, 0x5000, 0x6000, 0x7000, 1, None) == ARG


def test_bad_decode():
    lib = sba.load()

    def call(q=0x5000, M=1, idx=None, cnt=None, n=0, scale=0.1, out=0x6000, dt=0, ws=0x8000, size=1 << 30):
        return lib.sba_decode_kv4(c4(), q, M, idx, cnt, n, scale, out, dt, None, ws, size, None)

    assert call(q=None) == ARG and call(q=0x5008) == ARG and call(M=0) == ARG and call(M=1025) == ARG
    assert call(scale=0.0) == ARG and call(scale=float("nan")) == ARG and call(scale=float("inf")) == ARG
    assert call(out=None) == ARG and call(out=0x6004) == ARG and call(dt=2) == ARG
    assert call(idx=0x9000) == ARG and call(cnt=0x9000) == ARG and call(n=4) == ARG     # a selection is whole or absent
    assert call(idx=0x9000, cnt=0x9100, n=0) == ARG
    need = lib.sba_decode_kv4_workspace_size(c4(), 1, 0)
    assert need > 0 and call(ws=None) == WS and call(size=need - 1) == WS and call(ws=0x8008) == WS
    assert lib.sba_decode_kv4_workspace_size(c4(), 0, 0) == 0 and lib.sba_decode_kv4_workspace_size(c4(), 1, -1) == 0
    assert lib.sba_decode_kv4_workspace_size(c4(), 4, 0) > need                         # 16 rows instead of 8
    wide = dict(B=40000, H_q=508, H_kv=508, max_blocks=1, num_pages=60000, max_len=64, block_table=0x9000)
    assert lib.sba_decode_kv4(c4(**wide, b=64), 0x5000, 1024, None, None, 0, 0.1, 0x6000, 0, None, 0x8000, 1 << 40, None) == UNS
    gate = ctypes.byref(sba.select_params(16, 2, scorer=sba.SBA_SCORER_GATE))
    assert lib.sba_score_select_kv4(c4(), 0x5000, 1, gate, 0x6000, 0x7000, 16, 0x8000, 1 << 20, None) == UNS
    p = ctypes.byref(sba.select_params(16, 2))
    assert lib.sba_score_select_kv4(c4(desc=None), 0x5000, 1, p, 0x6000, 0x7000, 16, 0x8000, 1 << 20, None) == ARG
    assert lib.sba_score_select_kv4(c4(), 0x5000, 1, p, 0x6000, 0x7000, 15, 0x8000, 1 << 20, None) == ARG
    assert lib.sba_score_select_kv4(c4(), 0x5000, 1, p, 0x6000, 0x7000, 16, 0x8000, 16, None) == WS


def test_bad_weights():
    lib = sba.load()

    def call(q=0x5000, M=1, idx=None, cnt=None, bias=None, n=0, scale=0.1, lse=0x6000, a=0x7000, o=0x7000):
        return lib.sba_accumulate_weights(c16(), q, M, idx, cnt, bias, n, scale, lse, a, o, None)

    assert call(q=None) == ARG and call(M=0) == ARG and call(scale=-1.0) == ARG
    assert call(lse=None) == ARG and call(a=None) == ARG and call(o=None) == ARG and call(o=0x7002) == ARG
    assert call(bias=0x9000) == ARG                                                     # a bias belongs to selected blocks
    assert call(M=2, idx=0x9000, cnt=0x9100, n=4, bias=0x9200) == ARG
    assert call(idx=0x9000, n=4) == ARG
    assert lib.sba_accumulate_weights(c16(k=None), 0x5000, 1, None, None, None, 0, 0.1, 0x6000, 0x7000, 0x7000, None) == ARG


def test_bad_evict():
    lib = sba.load()

    def call(src=None, dst=None, acc=0x5000, p=(64, 0, 0), acc_dst=None, new=0x6000, kept=0x7000):
        return lib.sba_evict(src or c16(), acc, ctypes.byref(sba.evict_params(*p)),
                             dst or c16(k=0x100000, v=0x200000, desc=None), acc_dst, new, kept, None)

    assert call(acc=None) == ARG and call(acc=0x5008) == ARG and call(new=None) == ARG and call(kept=None) == ARG
    assert call(p=(0, 0, 0)) == ARG and call(p=(64, -1, 0)) == ARG and call(p=(64, 0, -1)) == ARG
    assert call(p=(64, 33, 32)) == ARG and call(p=(64, 2 ** 31 - 1, 2 ** 31 - 1)) == ARG
    assert call(p=(4097, 0, 0)) == ARG                                                  # dst has room for 4096
    other = dict(k=0x100000, v=0x200000, desc=None)
    assert call(dst=c16(**other, b=128)) == ARG and call(dst=c16(**other, H_kv=4, H_q=8)) == ARG
    assert call(dst=c16(**other, B=2, num_pages=128)) == ARG
    assert call(dst=c16(desc=None)) == ARG                                              # the same contiguous pages
    assert call(dst=c16(**{**other, "v": 0x2000})) == ARG
    assert call(new=0x3000) == ARG                                                      # src's own lengths
    assert call(acc_dst=0x5000) == ARG
    assert call(dst=c16(**{**other, "desc": 0x4000})) == ARG
    assert call(dst=c16(**other, d=64)) == UNS
    e = ctypes.byref(sba.evict_params(64))
    assert lib.sba_evict_kv4(c4(), 0x5000, e, c4(), None, 0x6000, 0x7000, None) == ARG
    assert lib.sba_evict(c16(), 0x5000, None, c16(**other), None, 0x6000, 0x7000, None) == ARG


def test_binding_takes_device_tensors_of_the_right_kind_only(monkeypatch):
    kv = torch.zeros((4, 2, 2, 4608), dtype=torch.uint8)
    lens = torch.zeros(1, dtype=torch.int32)
    good = dict(kv=kv, seq_lens=lens, H_q=4, max_blocks=4, max_len=256)
    rows = torch.zeros((1, 1, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        sba.sba_append_kv4(sba.Cache4(**good), rows, rows, lens)
    with pytest.raises(ValueError, match="kv must be"):
        sba.Cache4(**{**good, "kv": kv[..., :4600].contiguous()}).struct()
    # a cache's struct follows its fields
    c = sba.Cache4(**good)
    c.__dict__["_struct"] = "old"
    c.max_len = 128
    assert "_struct" not in c.__dict__ and c.max_len == 128 and c.B == 1
    # what each argument has to be (device -1 is the CPU's)
    for t, why in ((torch.zeros(4), "int32"), (torch.zeros(3, dtype=torch.int32), "at least 4"),
                   (torch.zeros((4, 2), dtype=torch.int32).t(), "not contiguous")):
        with pytest.raises(ValueError, match=why):
            sba._tensor(t, torch.int32, -1, 4, "x")
    with pytest.raises(ValueError, match="cuda:3"):
        sba._tensor(torch.zeros(4, dtype=torch.int32), torch.int32, 3, 4, "x")
    assert sba._tensor(None, torch.int32, 0, 4, "x") is None
    st = sba.sba_cache4(B=2, H_q=8, H_kv=2, d=128)
    assert sba._rows_of(st, -1, torch.zeros((2, 3, 8, 128), dtype=torch.bfloat16))[1] == 3
    assert sba._rows_of(st, -1, torch.zeros((2, 8, 128), dtype=torch.bfloat16))[1] == 1
    for shape in ((2, 8, 64), (1, 8, 128), (2, 3, 4, 128), (16, 128)):
        with pytest.raises(ValueError, match="q must be"):
            sba._rows_of(st, -1, torch.zeros(shape, dtype=torch.bfloat16))
    idx, cnt = torch.zeros((2, 2, 5), dtype=torch.int32), torch.zeros((2, 2), dtype=torch.int32)
    assert sba._selection(st, -1, idx, cnt)[2] == 5 and sba._selection(st, -1, None, None) == (None, None, 0)
    for i, c in ((idx, None), (None, cnt), (idx[0], cnt), (idx.long(), cnt), (idx, cnt[:1])):
        with pytest.raises(ValueError):
            sba._selection(st, -1, i, c)
    # kernels run on the current device: tensors of another one are refused
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        sba._current(0, None)


def test_a_replaced_tensor_is_seen_even_where_its_identity_comes_again(monkeypatch):
    # an object's identity may be a dead one's: the struct must not be looked up by it
    monkeypatch.setattr(sba, "_ptr", lambda t: None if t is None else ctypes.c_void_p(t.data_ptr()))
    k = torch.zeros((4, 2, 64, 128), dtype=torch.bfloat16)
    c = sba.Cache(k=k, v=torch.zeros_like(k), seq_lens=torch.zeros(1, dtype=torch.int32), H_q=4, max_blocks=4,
                  max_len=256)
    desc = torch.zeros(64, dtype=torch.bfloat16)
    c.desc = desc
    assert c.struct().desc == desc.data_ptr() and c.struct() is c.struct()
    monkeypatch.setattr(sba, "id", lambda t: 0, raising=False)
    c.struct()
    c.desc = torch.ones(64, dtype=torch.bfloat16)
    assert c.struct().desc == c.desc.data_ptr() != desc.data_ptr()
    c.desc = None
    assert c.struct().desc is None


def test_evict_refuses_new_lengths_that_overlap_the_old_ones():
    lib = sba.load()
    e = ctypes.byref(sba.evict_params(64))
    big = dict(B=4, num_pages=256, H_kv=2)
    for new in (0x3000, 0x3004, 0x300c, 0x2ffc, 0x2ff4):
        assert lib.sba_evict(c16(**big), 0x5000, e, c16(k=0x100000, v=0x200000, desc=None, **big), None, new, 0x7000, None) == ARG
