"""Thin Python binding of libsba.so (include/sba.h): argument marshalling only.

Every function here has the name of the C entry point it calls and forwards
torch tensors as raw device pointers plus the current CUDA stream.  All
computation happens in the CUDA kernels; there is no CPU path.  If the library
cannot be built or loaded, importing the package raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

from . import _build

SBA_OK = 0
SBA_ERR_INVALID_ARG = 1
SBA_ERR_UNSUPPORTED = 2
SBA_ERR_WORKSPACE = 3
SBA_ERR_CUDA = 4

SBA_DEV_BAD_PAGE = 1
SBA_DEV_BAD_POSITION = 2
SBA_DEV_BAD_SELECTION = 4
SBA_DEV_TIMEOUT = 8

SBA_SCORER_QUEST = 0
SBA_SCORER_GATE = 1
SBA_OUT_F32 = 0
SBA_OUT_BF16 = 1

SBA_LOG_GATE_OFF = 0
SBA_LOG_GATE_INNER = 1
SBA_LOG_GATE_OUTER = 2
SBA_GATE_SOFTMAX = 0
SBA_GATE_SIGMOID = 1
SBA_GATE_RAW = 2


class SbaError(RuntimeError):
    def __init__(self, code: int, where: str):
        msg = f"{where}: {sba_status_string(code)} (status {code})"
        if code == SBA_ERR_CUDA:
            msg += f": {load().sba_last_cuda_error().decode()}"
        super().__init__(msg)
        self.code = code


class sba_cache(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("B", ctypes.c_int32),
        ("H_q", ctypes.c_int32),
        ("H_kv", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("b", ctypes.c_int32),
        ("max_blocks", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_len", ctypes.c_int32),
        ("desc", ctypes.c_void_p),
        ("kg", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
    ]


class sba_gate(ctypes.Structure):
    _fields_ = [("Wq", ctypes.c_void_p), ("Wk", ctypes.c_void_p), ("dg", ctypes.c_int32)]


class sba_select_params(ctypes.Structure):
    _fields_ = [
        ("n_budget", ctypes.c_int32),
        ("n_local", ctypes.c_int32),
        ("n_min", ctypes.c_int32),
        ("keep_num", ctypes.c_int32),
        ("keep_den", ctypes.c_int32),
        ("scorer", ctypes.c_int32),
        ("log_gate", ctypes.c_int32),
        ("gate_act", ctypes.c_int32),
    ]


class sba_cache4(ctypes.Structure):
    _fields_ = [
        ("kv", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("B", ctypes.c_int32),
        ("H_q", ctypes.c_int32),
        ("H_kv", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("b", ctypes.c_int32),
        ("max_blocks", ctypes.c_int32),
        ("num_pages", ctypes.c_int32),
        ("max_len", ctypes.c_int32),
        ("desc", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
    ]


class sba_evict_params(ctypes.Structure):
    _fields_ = [("n_keep", ctypes.c_int32), ("n_sink", ctypes.c_int32), ("n_recent", ctypes.c_int32)]


_P = ctypes.c_void_p
_I = ctypes.c_int32
_C = ctypes.POINTER(sba_cache)
_C4 = ctypes.POINTER(sba_cache4)
_SEL = ctypes.POINTER(sba_select_params)
_EV = ctypes.POINTER(sba_evict_params)
_F = ctypes.c_float
_Z = ctypes.c_size_t
_SIGS = {
    "sba_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "sba_last_cuda_error": ([], ctypes.c_char_p),
    "sba_num_selected": ([_I, ctypes.POINTER(sba_select_params)], _I),
    "sba_budget_from_sparsity": ([_I, _I, _I], _I),
    "sba_default_num_splits": ([ctypes.POINTER(sba_cache), _I, _I], _I),
    "sba_workspace_size": ([ctypes.POINTER(sba_cache), ctypes.POINTER(sba_select_params)], ctypes.c_size_t),
    "sba_append_kv": ([ctypes.POINTER(sba_cache), _P, _P, _P, _I, _P], ctypes.c_int),
    "sba_update_descriptors": ([ctypes.POINTER(sba_cache), _P, _I, ctypes.POINTER(sba_gate), _P], ctypes.c_int),
    "sba_score_select": ([ctypes.POINTER(sba_cache), _P, ctypes.POINTER(sba_select_params), _P, _P, _P, _I, _P,
                          ctypes.c_size_t, _P], ctypes.c_int),
    "sba_sparse_decode": ([ctypes.POINTER(sba_cache), _P, _P, _P, _P, _I, ctypes.c_float, _I, _P, _P, _P],
                          ctypes.c_int),
    "sba_sparse_decode_outer": ([ctypes.POINTER(sba_cache), _P, _P, _P, _P, _I, ctypes.c_float, _I, _P, _P, _P],
                                ctypes.c_int),
    "sba_score_select_multi": ([ctypes.POINTER(sba_cache), _P, _I, ctypes.POINTER(sba_select_params), _P, _P, _I,
                                _P, ctypes.c_size_t, _P], ctypes.c_int),
    "sba_sparse_decode_multi": ([ctypes.POINTER(sba_cache), _P, _I, _P, _P, _I, ctypes.c_float, _I, _P, _P, _P],
                                ctypes.c_int),
    "sba_multi_row_groups": ([ctypes.POINTER(sba_cache), _I], _I),
    "sba_rectify": ([ctypes.POINTER(sba_cache), _P, _P, _P, _I, ctypes.c_float, _I, _P, _P, _P], ctypes.c_int),
    "sba_combine": ([_P, _P, _I, _I, _I, _I, _P, _I, _P, _P], ctypes.c_int),
    "sba_fold_gate": ([ctypes.POINTER(sba_gate), _P, _P], ctypes.c_int),
    "sba_static_scratch_bytes": ([], ctypes.c_size_t),
    "sba_selftest_wait_timeout": ([_P, ctypes.c_uint64, _P], ctypes.c_int),
    "sba_selftest_wait_vote": ([_P, _P, ctypes.c_uint64, _P], ctypes.c_int),
    "sba_score_select_static": ([ctypes.POINTER(sba_cache), _P, ctypes.POINTER(sba_select_params), _P, _P, _P, _I,
                                 _P], ctypes.c_int),
    "sba_decode_step_cluster": ([ctypes.POINTER(sba_cache), ctypes.POINTER(sba_select_params)], _I),
    "sba_decode_step": ([ctypes.POINTER(sba_cache), _P, _P, _P, _P, _I, _P, ctypes.POINTER(sba_select_params),
                         ctypes.c_float, _P, _I, _P, _P, _P, _P, _I, _P], ctypes.c_int),
    "sba_append_kv4": ([_C4, _P, _P, _P, _I, _P], ctypes.c_int),
    "sba_read_kv4": ([_C4, _P, _I, _P, _P, _P], ctypes.c_int),
    "sba_score_select_kv4_workspace_size": ([_C4, _SEL], _Z),
    "sba_score_select_kv4": ([_C4, _P, _I, _SEL, _P, _P, _I, _P, _Z, _P], ctypes.c_int),
    "sba_decode_kv4_workspace_size": ([_C4, _I, _I], _Z),
    "sba_decode_kv4": ([_C4, _P, _I, _P, _P, _I, _F, _P, _I, _P, _P, _Z, _P], ctypes.c_int),
    "sba_accumulate_weights": ([_C, _P, _I, _P, _P, _P, _I, _F, _P, _P, _P, _P], ctypes.c_int),
    "sba_accumulate_weights_kv4": ([_C4, _P, _I, _P, _P, _I, _F, _P, _P, _P, _P], ctypes.c_int),
    "sba_evict": ([_C, _P, _EV, _C, _P, _P, _P, _P], ctypes.c_int),
    "sba_evict_kv4": ([_C4, _P, _EV, _C4, _P, _P, _P, _P], ctypes.c_int),
}

_lib = None


def library_path() -> str:
    return _build.LIB


def load() -> ctypes.CDLL:
    """Build libsba.so if it is missing or older than its sources, then load it."""
    global _lib
    if _lib is None:
        path = _build.build()
        lib = ctypes.CDLL(path)
        for name, (args, res) in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libsba takes device tensors only")
    if not t.is_contiguous():
        raise ValueError("libsba takes contiguous tensors only")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _check(rc: int, where: str):
    if rc != SBA_OK:
        raise SbaError(rc, where)


@dataclass
class Cache:
    """Device tensors of one layer's KV cache and its descriptors (sba_cache).  Their addresses are kept from
    call to call: to use other memory, set the field to another tensor (a tensor's own storage stays)."""

    k: torch.Tensor                        # bf16 [num_pages][H_kv][b][d]
    v: torch.Tensor
    seq_lens: torch.Tensor                 # int32 [B]
    H_q: int
    max_blocks: int
    max_len: int
    block_table: Optional[torch.Tensor] = None   # int32 [B][max_blocks]
    desc: Optional[torch.Tensor] = None          # bf16 [num_pages][H_kv][2][d]
    kg: Optional[torch.Tensor] = None            # fp32 [num_pages][H_kv][d]
    status: Optional[torch.Tensor] = None        # int32 [1]

    @property
    def num_pages(self) -> int:
        return int(self.k.shape[0])

    @property
    def H_kv(self) -> int:
        return int(self.k.shape[1])

    @property
    def b(self) -> int:
        return int(self.k.shape[2])

    @property
    def d(self) -> int:
        return int(self.k.shape[3])

    @property
    def B(self) -> int:
        return int(self.seq_lens.shape[0])

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        self.__dict__.pop("_struct", None)  # a replaced tensor has another address; in-place updates keep it

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_struct"}  # (holds addresses: not copied)

    def struct(self) -> sba_cache:
        st = self.__dict__.get("_struct")
        if st is None:
            st = sba_cache(_ptr(self.k), _ptr(self.v), _ptr(self.block_table), _ptr(self.seq_lens),
                           self.B, self.H_q, self.H_kv, self.d, self.b, self.max_blocks, self.num_pages,
                           self.max_len, _ptr(self.desc), _ptr(self.kg), _ptr(self.status))
            self.__dict__["_struct"] = st
        return st


def select_params(n_budget=0, n_local=0, n_min=0, keep_num=0, keep_den=0, scorer=SBA_SCORER_QUEST,
                  log_gate=SBA_LOG_GATE_OFF, gate_act=SBA_GATE_SOFTMAX):
    return sba_select_params(n_budget, n_local, n_min, keep_num, keep_den, scorer, log_gate, gate_act)


def sba_status_string(code: int) -> str:
    return load().sba_status_string(code).decode()


def sba_num_selected(N: int, p: sba_select_params) -> int:
    return int(load().sba_num_selected(N, ctypes.byref(p)))


def sba_budget_from_sparsity(N: int, keep_num: int, keep_den: int) -> int:
    return int(load().sba_budget_from_sparsity(N, keep_num, keep_den))


def sba_default_num_splits(c: Cache, n_max: int, num_sms: Optional[int] = None) -> int:
    if num_sms is None:
        num_sms = torch.cuda.get_device_properties(c.k.device).multi_processor_count
    return int(load().sba_default_num_splits(ctypes.byref(c.struct()), n_max, num_sms))


def sba_workspace_size(c: Cache, p: sba_select_params) -> int:
    return int(load().sba_workspace_size(ctypes.byref(c.struct()), ctypes.byref(p)))


def sba_append_kv(c: Cache, k_new: torch.Tensor, v_new: torch.Tensor, pos_start: torch.Tensor, stream=None):
    n_new = int(k_new.shape[1])
    _check(load().sba_append_kv(ctypes.byref(c.struct()), _ptr(k_new), _ptr(v_new), _ptr(pos_start), n_new,
                                _stream(stream)), "sba_append_kv")


def sba_update_descriptors(c: Cache, pos_start: torch.Tensor, n_new: int, Wq: Optional[torch.Tensor] = None,
                           Wk: Optional[torch.Tensor] = None, stream=None):
    gate = None
    if Wq is not None:
        gate = ctypes.byref(sba_gate(_ptr(Wq), _ptr(Wk), int(Wq.shape[0])))
    _check(load().sba_update_descriptors(ctypes.byref(c.struct()), _ptr(pos_start), n_new, gate, _stream(stream)),
           "sba_update_descriptors")


def sba_score_select(c: Cache, q: torch.Tensor, p: sba_select_params, sel_idx: torch.Tensor, sel_cnt: torch.Tensor,
                     gate_bias: Optional[torch.Tensor], ws: torch.Tensor, stream=None):
    n_max = int(sel_idx.shape[-1])
    _check(load().sba_score_select(ctypes.byref(c.struct()), _ptr(q), ctypes.byref(p), _ptr(sel_idx),
                                   _ptr(sel_cnt), _ptr(gate_bias), n_max, _ptr(ws), ws.numel() * ws.element_size(),
                                   _stream(stream)), "sba_score_select")


def sba_static_scratch_bytes() -> int:
    return int(load().sba_static_scratch_bytes())


def sba_score_select_static(c: Cache, q: torch.Tensor, p: sba_select_params, sel_idx: torch.Tensor,
                            sel_cnt: torch.Tensor, gate_bias: Optional[torch.Tensor], stream=None):
    """sba_score_select without a workspace (for callers that cannot allocate):
    the library's static per-device scratch is used instead."""
    n_max = int(sel_idx.shape[-1])
    _check(load().sba_score_select_static(ctypes.byref(c.struct()), _ptr(q), ctypes.byref(p), _ptr(sel_idx),
                                          _ptr(sel_cnt), _ptr(gate_bias), n_max, _stream(stream)),
           "sba_score_select_static")


def sba_sparse_decode(c: Cache, q: torch.Tensor, sel_idx: torch.Tensor, sel_cnt: torch.Tensor,
                      gate_bias: Optional[torch.Tensor], softmax_scale: float, o_part: torch.Tensor,
                      lse_part: torch.Tensor, stream=None):
    n_max = int(sel_idx.shape[-1])
    num_splits = int(lse_part.shape[-1])
    _check(load().sba_sparse_decode(ctypes.byref(c.struct()), _ptr(q), _ptr(sel_idx), _ptr(sel_cnt),
                                    _ptr(gate_bias), n_max, float(softmax_scale), num_splits, _ptr(o_part),
                                    _ptr(lse_part), _stream(stream)), "sba_sparse_decode")


def sba_sparse_decode_outer(c: Cache, q: torch.Tensor, sel_idx: torch.Tensor, sel_cnt: torch.Tensor,
                            gate_bias: torch.Tensor, softmax_scale: float, o_part: torch.Tensor,
                            lse_part: torch.Tensor, stream=None):
    n_max = int(sel_idx.shape[-1])
    num_splits = int(lse_part.shape[-1])
    _check(load().sba_sparse_decode_outer(ctypes.byref(c.struct()), _ptr(q), _ptr(sel_idx), _ptr(sel_cnt),
                                          _ptr(gate_bias), n_max, float(softmax_scale), num_splits, _ptr(o_part),
                                          _ptr(lse_part), _stream(stream)), "sba_sparse_decode_outer")


def sba_score_select_multi(c: Cache, q: torch.Tensor, p: sba_select_params, sel_idx: torch.Tensor,
                           sel_cnt: torch.Tensor, ws: torch.Tensor, stream=None):
    """q: bf16 [B][M][H_q][d]; one Quest selection per (sequence, group) for all M tokens."""
    M = int(q.shape[1])
    n_max = int(sel_idx.shape[-1])
    _check(load().sba_score_select_multi(ctypes.byref(c.struct()), _ptr(q), M, ctypes.byref(p), _ptr(sel_idx),
                                         _ptr(sel_cnt), n_max, _ptr(ws), ws.numel() * ws.element_size(),
                                         _stream(stream)), "sba_score_select_multi")


def sba_multi_row_groups(c: Cache, M: int) -> int:
    return int(load().sba_multi_row_groups(ctypes.byref(c.struct()), M))


def sba_sparse_decode_multi(c: Cache, q: torch.Tensor, sel_idx: torch.Tensor, sel_cnt: torch.Tensor,
                            softmax_scale: float, o_part: torch.Tensor, lse_part: torch.Tensor, stream=None):
    """q: bf16 [B][M][H_q][d]; o_part fp32 [B][M][H_q][S][d], lse_part [B][M][H_q][S]."""
    M = int(q.shape[1])
    n_max = int(sel_idx.shape[-1])
    num_splits = int(lse_part.shape[-1])
    _check(load().sba_sparse_decode_multi(ctypes.byref(c.struct()), _ptr(q), M, _ptr(sel_idx), _ptr(sel_cnt), n_max,
                                          float(softmax_scale), num_splits, _ptr(o_part), _ptr(lse_part),
                                          _stream(stream)), "sba_sparse_decode_multi")


def sba_rectify(c: Cache, q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, softmax_scale: float,
                o_part: torch.Tensor, lse_part: torch.Tensor, stream=None):
    """q: bf16 [B][f][H_q][d]; k_new, v_new bf16 [B][f][H_kv][d] (the last f positions)."""
    f = int(q.shape[1])
    num_splits = int(lse_part.shape[-1])
    _check(load().sba_rectify(ctypes.byref(c.struct()), _ptr(q), _ptr(k_new), _ptr(v_new), f, float(softmax_scale),
                              num_splits, _ptr(o_part), _ptr(lse_part), _stream(stream)), "sba_rectify")


def sba_combine(o_part: torch.Tensor, lse_part: torch.Tensor, out: torch.Tensor,
                lse_out: Optional[torch.Tensor] = None, stream=None):
    if o_part.dim() == 5:  # multi-token partials [B][M][H_q][S][d]: merge M*H_q rows
        o_part = o_part.view(o_part.shape[0], -1, o_part.shape[3], o_part.shape[4])
    B, H_q, S, d = o_part.shape
    dt = SBA_OUT_BF16 if out.dtype == torch.bfloat16 else SBA_OUT_F32
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out must be fp32 or bf16")
    _check(load().sba_combine(_ptr(o_part), _ptr(lse_part), B, H_q, S, d, _ptr(out), dt, _ptr(lse_out),
                              _stream(stream)), "sba_combine")


def sba_fold_gate(Wq: torch.Tensor, Wk: torch.Tensor, A: torch.Tensor, stream=None):
    _check(load().sba_fold_gate(ctypes.byref(sba_gate(_ptr(Wq), _ptr(Wk), int(Wq.shape[0]))), _ptr(A),
                                _stream(stream)), "sba_fold_gate")


def sba_selftest_wait_timeout(status: torch.Tensor, limit_ns: int, stream=None):
    """Let one bounded wait run out on purpose (nothing arrives on its barrier): SBA_DEV_TIMEOUT
    is OR-ed into the int32 device `status`, the kernel returns."""
    _check(load().sba_selftest_wait_timeout(_ptr(status), int(limit_ns), _stream(stream)),
           "sba_selftest_wait_timeout")


def sba_selftest_wait_vote(status: torch.Tensor, verdicts: torch.Tensor, limit_ns: int, stream=None):
    """Let a wait of a whole warp run out for half of its lanes: int32 device `verdicts` [32] gets 0 for
    every lane, SBA_DEV_TIMEOUT is OR-ed into `status`."""
    dev = verdicts.get_device()
    _check(load().sba_selftest_wait_vote(_tensor(status, torch.int32, dev, 1, "status"),
                                         _tensor(verdicts, torch.int32, dev, 32, "verdicts"), int(limit_ns),
                                         _stream(stream)), "sba_selftest_wait_vote")


def sba_decode_step_cluster(c: Cache, p: sba_select_params) -> int:
    return int(load().sba_decode_step_cluster(ctypes.byref(c.struct()), ctypes.byref(p)))


def sba_decode_step(c: Cache, q: torch.Tensor, p: sba_select_params, softmax_scale: float, out: torch.Tensor,
                    lse_out: Optional[torch.Tensor] = None, k_new: Optional[torch.Tensor] = None,
                    v_new: Optional[torch.Tensor] = None, pos_start: Optional[torch.Tensor] = None,
                    gate_A: Optional[torch.Tensor] = None, sel_idx: Optional[torch.Tensor] = None,
                    sel_cnt: Optional[torch.Tensor] = None, gate_bias: Optional[torch.Tensor] = None,
                    stream=None):
    n_new = 0 if k_new is None else int(k_new.shape[1])
    n_max = int(sel_idx.shape[-1]) if sel_idx is not None else (int(gate_bias.shape[-1]) if gate_bias is not None
                                                               else 0)
    dt = SBA_OUT_BF16 if out.dtype == torch.bfloat16 else SBA_OUT_F32
    _check(load().sba_decode_step(ctypes.byref(c.struct()), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(pos_start),
                                  n_new, _ptr(gate_A), ctypes.byref(p), float(softmax_scale), _ptr(out), dt,
                                  _ptr(lse_out), _ptr(sel_idx), _ptr(sel_cnt), _ptr(gate_bias), n_max,
                                  _stream(stream)), "sba_decode_step")


# ---------------------------------------------------------------------------
# Four-bit caches, accumulated attention weights, eviction
# ---------------------------------------------------------------------------

STRIP_TOKENS = 32
STRIP_BYTES = 4608


@dataclass
class Cache4:
    """Device tensors of one layer's four-bit KV cache and its Quest descriptors (sba_cache4).  Their addresses
    are kept from call to call, as Cache's are."""

    kv: torch.Tensor                       # uint8 [num_pages][H_kv][b/32][4608]
    seq_lens: torch.Tensor                 # int32 [B]
    H_q: int
    max_blocks: int
    max_len: int
    block_table: Optional[torch.Tensor] = None   # int32 [B][max_blocks]
    desc: Optional[torch.Tensor] = None          # bf16 [num_pages][H_kv][2][d]
    status: Optional[torch.Tensor] = None        # int32 [1]

    @property
    def num_pages(self) -> int:
        return int(self.kv.shape[0])

    @property
    def H_kv(self) -> int:
        return int(self.kv.shape[1])

    @property
    def b(self) -> int:
        return int(self.kv.shape[2]) * STRIP_TOKENS

    @property
    def d(self) -> int:
        return 128

    @property
    def B(self) -> int:
        return int(self.seq_lens.shape[0])

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        self.__dict__.pop("_struct", None)  # a replaced tensor has another address; in-place updates keep it

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_struct"}  # (holds addresses: not copied)

    def struct(self) -> sba_cache4:
        st = self.__dict__.get("_struct")
        if st is None:
            if self.kv.dim() != 4 or self.kv.shape[3] != STRIP_BYTES:
                raise ValueError(f"kv must be uint8 [num_pages][H_kv][b/32][{STRIP_BYTES}]")
            if not self.kv.is_cuda:
                raise ValueError("libsba takes device tensors only")
            dev = self.kv.get_device()
            st = sba_cache4(_tensor(self.kv, torch.uint8, dev, 0, "kv"),
                            _tensor(self.block_table, torch.int32, dev, self.B * self.max_blocks, "block_table"),
                            _tensor(self.seq_lens, torch.int32, dev, self.B, "seq_lens"), self.B, self.H_q, self.H_kv,
                            self.d, self.b, self.max_blocks, self.num_pages, self.max_len,
                            _tensor(self.desc, torch.bfloat16, dev, self.num_pages * self.H_kv * 2 * self.d, "desc"),
                            _tensor(self.status, torch.int32, dev, 1, "status"))
            self.__dict__["_struct"] = st
        return st


def _tensor(t: Optional[torch.Tensor], dtype: torch.dtype, device: int, least: int, name: str):
    """Address of a contiguous tensor of `dtype` on CUDA device `device` with at least `least` elements
    (None stays None)."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == device and t.is_contiguous() and t.numel() >= least:
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor on cuda:{device} with at least {least} elements "
                     f"(got {t.dtype} on {t.device}, {t.numel()} elements"
                     f"{'' if t.is_contiguous() else ', not contiguous'})")


def _current(device: int, stream):
    """The stream to launch on; kernels run on the current device, so the tensors have to be there."""
    if device != torch.cuda.current_device():
        raise ValueError(f"tensors are on cuda:{device}, but the current device is cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def _opened(c):
    """A cache's struct (by reference), itself, and its device."""
    st = c.struct()
    t = c.kv if type(c) is Cache4 else c.k
    return ctypes.byref(st), st, t.get_device()


def _rows_of(st, device: int, q: torch.Tensor):
    """Address of q ([B][H_q][d], or [B][M][H_q][d]) and M."""
    shape = q.shape
    M = shape[1] if len(shape) == 4 else 1
    if shape != ((st.B, M, st.H_q, st.d) if len(shape) == 4 else (st.B, st.H_q, st.d)):
        raise ValueError(f"q must be [B][H_q][d] or [B][M][H_q][d] (got {tuple(shape)})")
    return _tensor(q, torch.bfloat16, device, 0, "q"), M


def _selection(st, device: int, sel_idx, sel_cnt):
    """Addresses of a selection and its row length (None, None, 0: every block)."""
    if sel_idx is None:
        if sel_cnt is not None:
            raise ValueError("sel_cnt without sel_idx")
        return None, None, 0
    shape = sel_idx.shape
    if sel_cnt is None or len(shape) != 3 or shape[0] != st.B or shape[1] != st.H_kv:
        raise ValueError("sel_idx must be int32 [B][H_kv][n_max], with sel_cnt [B][H_kv]")
    return (_tensor(sel_idx, torch.int32, device, 0, "sel_idx"),
            _tensor(sel_cnt, torch.int32, device, st.B * st.H_kv, "sel_cnt"), shape[2])


def _window(st, device: int, k: torch.Tensor, v: torch.Tensor, names):
    """Addresses of K and V rows [B][n][H_kv][d], and n."""
    at = k.shape
    n = at[1] if len(at) == 4 else -1
    want = (st.B, n, st.H_kv, 128)
    if at != want or v.shape != want:
        raise ValueError(f"{names[0]} and {names[1]} must be bf16 [B][n][H_kv][128] with the same n "
                         f"(got {tuple(at)} and {tuple(v.shape)})")
    return _tensor(k, torch.bfloat16, device, 0, names[0]), _tensor(v, torch.bfloat16, device, 0, names[1]), n


def evict_params(n_keep: int, n_sink: int = 0, n_recent: int = 0) -> sba_evict_params:
    return sba_evict_params(n_keep, n_sink, n_recent)


def sba_append_kv4(c: Cache4, k_new: torch.Tensor, v_new: torch.Tensor, pos_start: torch.Tensor, stream=None):
    """k_new, v_new: bf16 [B][n_new][H_kv][d] to positions pos_start[s] .. of a four-bit cache."""
    ref, st, dev = _opened(c)
    kp, vp, n_new = _window(st, dev, k_new, v_new, ("k_new", "v_new"))
    _check(load().sba_append_kv4(ref, kp, vp, _tensor(pos_start, torch.int32, dev, st.B, "pos_start"), n_new,
                                 _current(dev, stream)), "sba_append_kv4")


def sba_read_kv4(c: Cache4, pos_start: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor, stream=None):
    """Positions pos_start[s] .. as bf16 rows k_out, v_out [B][n][H_kv][d]."""
    ref, st, dev = _opened(c)
    kp, vp, n = _window(st, dev, k_out, v_out, ("k_out", "v_out"))
    _check(load().sba_read_kv4(ref, _tensor(pos_start, torch.int32, dev, st.B, "pos_start"), n, kp, vp,
                               _current(dev, stream)), "sba_read_kv4")


def sba_score_select_kv4_workspace_size(c: Cache4, p: sba_select_params) -> int:
    return int(load().sba_score_select_kv4_workspace_size(ctypes.byref(c.struct()), ctypes.byref(p)))


def sba_score_select_kv4(c: Cache4, q: torch.Tensor, p: sba_select_params, sel_idx: torch.Tensor,
                         sel_cnt: torch.Tensor, ws: torch.Tensor, stream=None):
    """q: bf16 [B][H_q][d] or [B][M][H_q][d]; one Quest selection per (sequence, group)."""
    ref, st, dev = _opened(c)
    qp, M = _rows_of(st, dev, q)
    si, sc, n_max = _selection(st, dev, sel_idx, sel_cnt)
    _check(load().sba_score_select_kv4(ref, qp, M, ctypes.byref(p), si, sc, n_max, _tensor(ws, torch.uint8, dev, 0, "ws"),
                                       ws.numel(), _current(dev, stream)), "sba_score_select_kv4")


def sba_decode_kv4_workspace_size(c: Cache4, M: int = 1, n_max: int = 0) -> int:
    return int(load().sba_decode_kv4_workspace_size(ctypes.byref(c.struct()), M, n_max))


def sba_decode_kv4(c: Cache4, q: torch.Tensor, softmax_scale: float, out: torch.Tensor, ws: torch.Tensor,
                   lse_out: Optional[torch.Tensor] = None, sel_idx: Optional[torch.Tensor] = None,
                   sel_cnt: Optional[torch.Tensor] = None, stream=None):
    """Attention over the selected blocks (or all) of a four-bit cache.  q, out: [B][H_q][d] or
    [B][M][H_q][d]; lse_out fp32 [B][M][H_q]; ws: uint8, zeroed once, of
    sba_decode_kv4_workspace_size(c, M, n_max) bytes."""
    ref, st, dev = _opened(c)
    qp, M = _rows_of(st, dev, q)
    si, sc, n_max = _selection(st, dev, sel_idx, sel_cnt)
    dt = out.dtype
    if dt is not torch.bfloat16 and dt is not torch.float32:
        raise ValueError("out must be fp32 or bf16")
    rows = st.B * M * st.H_q
    _check(load().sba_decode_kv4(ref, qp, M, si, sc, n_max, float(softmax_scale),
                                 _tensor(out, dt, dev, rows * st.d, "out"),
                                 SBA_OUT_BF16 if dt is torch.bfloat16 else SBA_OUT_F32,
                                 _tensor(lse_out, torch.float32, dev, rows, "lse_out"),
                                 _tensor(ws, torch.uint8, dev, 0, "ws"), ws.numel(), _current(dev, stream)),
           "sba_decode_kv4")


def _weights_args(st, dev, q, lse, acc_in, acc_out, sel_idx, sel_cnt):
    qp, M = _rows_of(st, dev, q)
    si, sc, n_max = _selection(st, dev, sel_idx, sel_cnt)
    cells = st.num_pages * st.H_kv * st.b
    return (qp, M, si, sc, n_max, _tensor(lse, torch.float32, dev, st.B * M * st.H_q, "lse"),
            _tensor(acc_in, torch.float32, dev, cells, "acc_in"), _tensor(acc_out, torch.float32, dev, cells, "acc_out"))


def sba_accumulate_weights(c: Cache, q: torch.Tensor, lse: torch.Tensor, softmax_scale: float, acc_in: torch.Tensor,
                           acc_out: torch.Tensor, sel_idx: Optional[torch.Tensor] = None,
                           sel_cnt: Optional[torch.Tensor] = None, gate_bias: Optional[torch.Tensor] = None,
                           stream=None):
    """acc_out[t] = acc_in[t] + the attention weight token t received from q's rows (fp32
    [num_pages][H_kv][b]; acc_out may be acc_in); lse as the step's attention returned it."""
    ref, st, dev = _opened(c)
    qp, M, si, sc, n_max, lp, ai, ao = _weights_args(st, dev, q, lse, acc_in, acc_out, sel_idx, sel_cnt)
    gb = _tensor(gate_bias, torch.float32, dev, st.B * st.H_q * n_max, "gate_bias")
    _check(load().sba_accumulate_weights(ref, qp, M, si, sc, gb, n_max, float(softmax_scale), lp, ai, ao,
                                         _current(dev, stream)), "sba_accumulate_weights")


def sba_accumulate_weights_kv4(c: Cache4, q: torch.Tensor, lse: torch.Tensor, softmax_scale: float,
                               acc_in: torch.Tensor, acc_out: torch.Tensor, sel_idx: Optional[torch.Tensor] = None,
                               sel_cnt: Optional[torch.Tensor] = None, stream=None):
    """sba_accumulate_weights on a four-bit cache."""
    ref, st, dev = _opened(c)
    qp, M, si, sc, n_max, lp, ai, ao = _weights_args(st, dev, q, lse, acc_in, acc_out, sel_idx, sel_cnt)
    _check(load().sba_accumulate_weights_kv4(ref, qp, M, si, sc, n_max, float(softmax_scale), lp, ai, ao,
                                             _current(dev, stream)), "sba_accumulate_weights_kv4")


def _evict(call, name, src, acc, p, dst, new_lens, kept, acc_dst, stream):
    (sref, ss, dev), (dref, ds, dst_dev) = _opened(src), _opened(dst)
    if dst_dev != dev:
        raise ValueError("source and destination caches are on different devices")
    _check(call(sref, _tensor(acc, torch.float32, dev, ss.num_pages * ss.H_kv * ss.b, "acc"), ctypes.byref(p), dref,
                _tensor(acc_dst, torch.float32, dev, ds.num_pages * ds.H_kv * ds.b, "acc_dst"),
                _tensor(new_lens, torch.int32, dev, ss.B, "new_lens"),
                _tensor(kept, torch.int32, dev, ss.B * ss.H_kv * p.n_keep, "kept"), _current(dev, stream)), name)


def sba_evict(src: Cache, acc: torch.Tensor, p: sba_evict_params, dst: Cache, new_lens: torch.Tensor,
              kept: torch.Tensor, acc_dst: Optional[torch.Tensor] = None, stream=None):
    """Keep p.n_keep tokens per (sequence, KV head) of src and move them, in order, to dst's pages.
    new_lens int32 [B] and kept int32 [B][H_kv][n_keep] are written."""
    _evict(load().sba_evict, "sba_evict", src, acc, p, dst, new_lens, kept, acc_dst, stream)


def sba_evict_kv4(src: Cache4, acc: torch.Tensor, p: sba_evict_params, dst: Cache4, new_lens: torch.Tensor,
                  kept: torch.Tensor, acc_dst: Optional[torch.Tensor] = None, stream=None):
    """sba_evict on four-bit caches."""
    _evict(load().sba_evict_kv4, "sba_evict_kv4", src, acc, p, dst, new_lens, kept, acc_dst, stream)


# ---------------------------------------------------------------------------
# Buffers of one decode step (allocation only; every step runs in the kernels)
# ---------------------------------------------------------------------------

@dataclass
class StepBuffers:
    sel_idx: torch.Tensor
    sel_cnt: torch.Tensor
    gate_bias: Optional[torch.Tensor]
    o_part: torch.Tensor
    lse_part: torch.Tensor
    out: torch.Tensor
    lse: torch.Tensor
    ws: torch.Tensor


def alloc_step(c: Cache, p: sba_select_params, num_splits: Optional[int] = None, n_max: Optional[int] = None,
               out_dtype=torch.float32) -> StepBuffers:
    dev = c.k.device
    N_max = (c.max_len + c.b - 1) // c.b
    if n_max is None:
        n_max = max(1, sba_num_selected(N_max, p))
    if num_splits is None:
        num_splits = sba_default_num_splits(c, n_max)
    ws_bytes = sba_workspace_size(c, p)
    return StepBuffers(
        sel_idx=torch.full((c.B, c.H_kv, n_max), -1, dtype=torch.int32, device=dev),
        sel_cnt=torch.zeros((c.B, c.H_kv), dtype=torch.int32, device=dev),
        gate_bias=(torch.zeros((c.B, c.H_q, n_max), dtype=torch.float32, device=dev)
                   if p.scorer == SBA_SCORER_GATE else None),
        o_part=torch.empty((c.B, c.H_q, num_splits, c.d), dtype=torch.float32, device=dev),
        lse_part=torch.empty((c.B, c.H_q, num_splits), dtype=torch.float32, device=dev),
        out=torch.empty((c.B, c.H_q, c.d), dtype=out_dtype, device=dev),
        lse=torch.empty((c.B, c.H_q), dtype=torch.float32, device=dev),
        ws=torch.zeros(((ws_bytes + 15) // 16 * 16,), dtype=torch.uint8, device=dev),
    )


def decode_step(c: Cache, q: torch.Tensor, p: sba_select_params, bufs: StepBuffers, softmax_scale: float,
                stream=None):
    """score_select -> sparse_decode -> combine for one layer (three library calls; the gate's
    position p.log_gate picks the decode call and whether it gets the log-gates)."""
    sba_score_select(c, q, p, bufs.sel_idx, bufs.sel_cnt, bufs.gate_bias, bufs.ws, stream)
    gate = p.scorer == SBA_SCORER_GATE
    if gate and p.log_gate == SBA_LOG_GATE_OUTER:
        sba_sparse_decode_outer(c, q, bufs.sel_idx, bufs.sel_cnt, bufs.gate_bias, softmax_scale, bufs.o_part,
                                bufs.lse_part, stream)
    else:
        bias = bufs.gate_bias if (gate and p.log_gate == SBA_LOG_GATE_INNER) else None
        sba_sparse_decode(c, q, bufs.sel_idx, bufs.sel_cnt, bias, softmax_scale, bufs.o_part, bufs.lse_part, stream)
    sba_combine(bufs.o_part, bufs.lse_part, bufs.out, bufs.lse, stream)
