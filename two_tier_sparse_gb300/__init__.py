"""Two-tier sparse attention (DeepSeek-V4.1) on one GB300: Python binding.

A thin ctypes layer over libdsa.so (include/dsa.h). It marshals torch tensors
(device pointers) and the current CUDA stream into the C calls and turns
status codes into exceptions; every step of the computation runs in the
library's CUDA kernels. There is no fallback: if libdsa.so is missing, every
call raises.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdsa.so")

FMT_BF16 = 0
FMT_MXFP8 = 1
FMT_MXFP4 = 2
_FMT = {"bf16": FMT_BF16, "mxfp8": FMT_MXFP8, "mxfp4": FMT_MXFP4}

STATUS = {
    0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_MISALIGNED", 3: "DSA_ERR_UNSUPPORTED",
    4: "DSA_ERR_WORKSPACE", 5: "DSA_ERR_CUDA", 6: "DSA_ERR_DEVICE_CHECK", 7: "DSA_ERR_TIMEOUT",
}

EXPORTS = ("dsa_default_config", "dsa_status_string", "dsa_workspace_size",
           "dsa_pool_index_keys", "dsa_index_blocks", "dsa_topk", "dsa_sparse_attn_decode",
           "dsa_decode_step", "dsa_sparse_attn_prefill", "dsa_read_device_status",
           "dsa_profile_events", "dsa_launch_counts", "dsa_topk_noalloc",
           "dsa_selftest_timeout", "dsa_sparse_attn_decode_paged", "dsa_decode_multi",
           "dsa_compress_append", "dsa_plan_step", "dsa_norm_rope", "dsa_kv_write",
           "dsa_kv_read", "dsa_full_attn_workspace_size", "dsa_full_attn_decode",
           "dsa_full_attn_multi", "dsa_plan_trim", "dsa_verify_drafts")

TOPK_NOALLOC_MAX_SCORES = 1 << 21

KERNEL_KINDS = ("pool", "scan", "select", "attn", "other")


class DsaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}")


class Config(ctypes.Structure):
    """dsa_config_t."""
    _fields_ = [("n_heads", ctypes.c_int), ("latent_dim", ctypes.c_int),
                ("n_idx_heads", ctypes.c_int), ("idx_dim", ctypes.c_int),
                ("block", ctypes.c_int), ("k_blocks", ctypes.c_int), ("k_tokens", ctypes.c_int),
                ("window", ctypes.c_int), ("ratio", ctypes.c_int), ("sm_scale", ctypes.c_float),
                ("kv_fmt", ctypes.c_int), ("kv_scale", ctypes.c_float)]


KV_BF16, KV_FP8_E4M3, KV_MXFP4 = 0, 1, 3
KV_MXFP4_ROW = 272  # bytes of a 4-bit row: 256 of codes, 16 scales


class _Pages(ctypes.Structure):
    """dsa_pages_t."""
    _fields_ = [("page_table", ctypes.c_void_p), ("page_rows", ctypes.c_int32),
                ("pages_per_seq", ctypes.c_int32), ("n_pages", ctypes.c_int64)]


class _Keys(ctypes.Structure):
    """dsa_keys_t / dsa_keys_out_t (same layout)."""
    _fields_ = [("fmt", ctypes.c_int), ("data", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("seq_stride_rows", ctypes.c_int64), ("pages", ctypes.POINTER(_Pages))]


class _PagePool(ctypes.Structure):
    """dsa_page_pool_t."""
    _fields_ = [("page_table", ctypes.c_void_p), ("page_rows", ctypes.c_int32),
                ("pages_per_seq", ctypes.c_int32), ("n_pages", ctypes.c_int64),
                ("free_ring", ctypes.c_void_p), ("ring_state", ctypes.c_void_p),
                ("ring_state_out", ctypes.c_void_p)]


class _StepPlan(ctypes.Structure):
    """dsa_step_plan_t."""
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("n_tokens", "n_latents", "swa_len", "cu_new", "token_seq", "positions",
                 "latent_slots", "window_slots")] + [("max_new", ctypes.c_int32)]


class _HeadsC(ctypes.Structure):
    """dsa_heads_t."""
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("dim", ctypes.c_int), ("x_token_stride", ctypes.c_int64),
                ("x_head_stride", ctypes.c_int64), ("out_token_stride", ctypes.c_int64),
                ("out_head_stride", ctypes.c_int64), ("weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("norm", ctypes.c_int), ("rope_start", ctypes.c_int)]


class _RopeC(ctypes.Structure):
    """dsa_rope_t."""
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rope_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("scale", ctypes.c_float)]


_lib = None


def load() -> ctypes.CDLL:
    """Loads libdsa.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m two_tier_sparse_gb300.build` (nvcc, sm_103a)")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        cp = ctypes.POINTER(Config)
        kp = ctypes.POINTER(_Keys)
        lib.dsa_default_config.argtypes = [cp]
        lib.dsa_default_config.restype = None
        lib.dsa_status_string.argtypes = [i32]
        lib.dsa_status_string.restype = ctypes.c_char_p
        lib.dsa_workspace_size.argtypes = [cp, i32, i64, ctypes.POINTER(sz)]
        lib.dsa_pool_index_keys.argtypes = [cp, kp, vp, i32, i64, i32, kp, vp, sz, vp]
        lib.dsa_index_blocks.argtypes = [cp, vp, vp, kp, vp, i32, i64, vp, vp, vp, sz, vp]
        lib.dsa_topk.argtypes = [cp, vp, vp, kp, vp, vp, i32, i64, vp, vp, vp, sz, vp]
        lib.dsa_sparse_attn_decode.argtypes = [cp, vp, vp, i64, vp, vp, vp, vp, i32, vp, vp, vp,
                                               sz, vp]
        lib.dsa_decode_step.argtypes = [cp, vp, vp, vp, kp, kp, i32, vp, i64, vp, i64, vp, vp, i32,
                                        vp, vp, vp, vp, vp, sz, vp]
        lib.dsa_sparse_attn_prefill.argtypes = [cp, i32, i64, vp, vp, vp, vp, kp, kp, vp, vp, vp,
                                                vp, vp, sz, vp]
        lib.dsa_read_device_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
        lib.dsa_profile_events.argtypes = [i32, ctypes.POINTER(vp), ctypes.POINTER(vp), i32]
        lib.dsa_launch_counts.argtypes = [ctypes.POINTER(ctypes.c_uint64), i32]
        lib.dsa_topk_noalloc.argtypes = [cp, vp, vp, kp, vp, vp, i32, i64, vp, vp]
        lib.dsa_selftest_timeout.argtypes = [vp, sz, vp]
        lib.dsa_sparse_attn_decode_paged.argtypes = [cp, vp, vp, ctypes.POINTER(_Pages), vp, vp,
                                                     vp, vp, i32, vp, vp, vp, sz, vp]
        lib.dsa_decode_multi.argtypes = [cp, i32, vp, vp, vp, vp, kp, kp, vp, i64, i64, vp, i32,
                                         vp, vp, vp, vp, sz, vp]
        lib.dsa_compress_append.argtypes = [cp, i32, vp, vp, vp, kp, vp, i64, kp, kp, i64, vp,
                                            sz, vp]
        lib.dsa_plan_step.argtypes = [cp, i32, vp, vp, ctypes.POINTER(_PagePool),
                                      ctypes.POINTER(_StepPlan), vp, sz, vp]
        lib.dsa_norm_rope.argtypes = [i32, vp, vp, i32, ctypes.POINTER(_HeadsC), i32,
                                      ctypes.POINTER(_RopeC), vp]
        lib.dsa_kv_write.argtypes = [cp, i32, vp, vp, i64, vp, vp, i64, vp, sz, vp]
        lib.dsa_kv_read.argtypes = [cp, i32, vp, vp, i64, vp, vp, i64, vp, sz, vp]
        pp = ctypes.POINTER(_Pages)
        lib.dsa_plan_trim.argtypes = lib.dsa_plan_step.argtypes
        lib.dsa_verify_drafts.argtypes = [i32, i32, i64, i32, vp, i64, vp, i64, vp, vp, vp, vp, vp,
                                          vp, vp, sz, vp]
        lib.dsa_full_attn_workspace_size.argtypes = [cp, i32, ctypes.POINTER(sz)]
        lib.dsa_full_attn_decode.argtypes = [cp, vp, vp, i64, pp, vp, i64, vp, vp, i32, vp, vp, vp,
                                             sz, vp]
        lib.dsa_full_attn_multi.argtypes = [cp, i32, vp, vp, vp, i64, pp, i64, vp, i32, vp, vp, vp,
                                            sz, vp]
        for f in EXPORTS:
            if f not in ("dsa_default_config", "dsa_status_string"):
                getattr(lib, f).restype = ctypes.c_int
        _lib = lib
    return _lib


_calls = None


class _NoCalls:
    """In the compiled part's place where it cannot be used: leaves every call to the binding."""

    @staticmethod
    def plan(*args):
        return None

    norm = rows = trim = full = verify = plan


def _load_calls():
    """The compiled part of the binding (csrc/calls.c), with the library's addresses. It only
    makes a plain call cheaper; without it the binding checks and passes every call itself."""
    global _calls
    lib = load()
    path = os.path.join(os.path.dirname(LIB_PATH),
                        "_calls" + importlib.machinery.EXTENSION_SUFFIXES[0])
    if _raw_stream is None or not os.path.exists(path):  # a torch without CUDA, or not built
        _calls = _NoCalls
        return _calls
    loader = importlib.machinery.ExtensionFileLoader("_calls", path)
    m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_calls", loader))
    loader.exec_module(m)
    m.init(tuple(ctypes.cast(f, ctypes.c_void_p).value for f in
                 (lib.dsa_plan_step, lib.dsa_norm_rope, lib.dsa_kv_write, lib.dsa_kv_read,
                  lib.dsa_plan_trim, lib.dsa_full_attn_decode, lib.dsa_full_attn_multi,
                  lib.dsa_verify_drafts)),
           (torch.int32, torch.bfloat16, torch.int16, torch.float16, torch.float32),
           torch._C._cuda_getDevice, _raw_stream)
    _calls = m
    return m


def _check(code: int, where: str) -> None:
    if code != 0:
        raise DsaError(code, where)


# Pointers and streams travel as plain integers (every argument is declared void*):
# building ctypes objects for them cost more than the call itself.
# (A torch without CUDA has no such function; no call gets as far as using it there.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = torch.cuda.current_device


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    return _raw_stream(_current_device()) if stream is None else stream.cuda_stream


def config(k_blocks=2048, k_tokens=512, window=128, ratio=1, sm_scale=0.0, kv_fmt=KV_BF16,
           kv_scale=1.0) -> Config:
    """kv_fmt: KV_BF16, KV_FP8_E4M3 (latents and window rows as E4M3 codes standing
    for code * kv_scale; decode attention and the decode step only) or KV_MXFP4
    (272-byte rows of e2m1 codes and their scales; the same calls and
    compress_append)."""
    c = Config()
    load().dsa_default_config(ctypes.byref(c))
    c.k_blocks, c.k_tokens, c.window, c.ratio = k_blocks, k_tokens, window, ratio
    c.sm_scale = sm_scale
    c.kv_fmt, c.kv_scale = kv_fmt, kv_scale
    return c


class Pages:
    """A page table (dsa_pages_t) over pools of n_pages pages of page_rows tokens:
    table is a device int32 tensor [B, pages_per_seq]."""

    def __init__(self, table: torch.Tensor, page_rows: int, n_pages: int):
        assert table.dtype == torch.int32 and table.dim() == 2
        self.table = table
        self.c = _Pages(table.data_ptr(), page_rows, table.shape[1], n_pages)
        self._key = (ctypes.addressof(self.c), table.shape[0] if table.is_contiguous() else -1,
                     table.get_device())


@dataclass
class Keys:
    """A key cache on the device: data [B, rows, 128] (bf16 as 16-bit words, or
    uint8 e4m3 codes) or [B, rows, 64] (uint8, two e2m1 codes a byte) and, for
    MXFP8 and MXFP4, scales uint8 [B, rows, 4]."""
    fmt: str
    data: torch.Tensor
    scales: Optional[torch.Tensor] = None
    pages: Optional[Pages] = None  # paged pool (data rows = n_pages x rows per page)

    def c(self) -> _Keys:
        stride = self.data.shape[-2] if self.data.dim() >= 3 else 0
        pages = ctypes.pointer(self.pages.c) if self.pages is not None else None
        return _Keys(_FMT[self.fmt], self.data.data_ptr(),
                     self.scales.data_ptr() if self.scales is not None else None, stride,
                     pages)


def workspace_size(cfg: Config, n_queries: int, max_latents: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().dsa_workspace_size(ctypes.byref(cfg), n_queries, max_latents, ctypes.byref(n)),
           "dsa_workspace_size")
    return int(n.value)


def workspace(cfg: Config, n_queries: int, max_latents: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace (the status word must start at zero)."""
    return torch.zeros(workspace_size(cfg, n_queries, max_latents), dtype=torch.uint8,
                       device=device)


def pool_index_keys(cfg, keys: Keys, n_latents, max_latents, pooled: Keys, ws, tail_only=False,
                    stream=None):
    B = n_latents.shape[0]
    _check(load().dsa_pool_index_keys(ctypes.byref(cfg), ctypes.byref(keys.c()), _p(n_latents), B,
                                      max_latents, int(tail_only), ctypes.byref(pooled.c()),
                                      _p(ws), ws.numel(), _stream(stream)), "dsa_pool_index_keys")


def index_blocks(cfg, q_idx, w, pooled: Keys, n_latents, max_latents, block_ids, ws,
                 block_scores=None, stream=None):
    B = q_idx.shape[0]
    _check(load().dsa_index_blocks(ctypes.byref(cfg), _p(q_idx), _p(w), ctypes.byref(pooled.c()),
                                   _p(n_latents), B, max_latents, _p(block_ids), _p(block_scores),
                                   _p(ws), ws.numel(), _stream(stream)), "dsa_index_blocks")


def topk(cfg, q_idx, w, keys: Keys, block_ids, n_latents, max_latents, token_ids, ws,
         token_scores=None, stream=None):
    B = q_idx.shape[0]
    _check(load().dsa_topk(ctypes.byref(cfg), _p(q_idx), _p(w), ctypes.byref(keys.c()),
                           _p(block_ids), _p(n_latents), B, max_latents, _p(token_ids),
                           _p(token_scores), _p(ws), ws.numel(), _stream(stream)), "dsa_topk")


def topk_noalloc(cfg, q_idx, w, keys: Keys, block_ids, n_latents, max_latents, token_ids,
                 stream=None):
    """dsa_topk without a workspace: for callers that cannot allocate device
    memory. Candidate scores go to a scratch array the library defines
    statically (at most TOPK_NOALLOC_MAX_SCORES values for the whole batch);
    calls that may overlap on the GPU share it and must be serialised."""
    B = q_idx.shape[0]
    _check(load().dsa_topk_noalloc(ctypes.byref(cfg), _p(q_idx), _p(w), ctypes.byref(keys.c()),
                                   _p(block_ids), _p(n_latents), B, max_latents, _p(token_ids),
                                   _stream(stream)), "dsa_topk_noalloc")


def sparse_attn_decode(cfg, q, latents, n_latents, token_ids, swa, swa_len, out, ws, lse=None,
                       stream=None):
    B = q.shape[0]
    _check(load().dsa_sparse_attn_decode(ctypes.byref(cfg), _p(q), _p(latents), latents.shape[1],
                                         _p(n_latents), _p(token_ids), _p(swa), _p(swa_len), B,
                                         _p(out), _p(lse), _p(ws), ws.numel(), _stream(stream)),
           "dsa_sparse_attn_decode")


def sparse_attn_decode_paged(cfg, q, latents, pages: Pages, n_latents, token_ids, swa, swa_len,
                             out, ws, lse=None, stream=None):
    """dsa_sparse_attn_decode over a paged latent pool (latents [n_pages * page_rows, 512])."""
    B = q.shape[0]
    _check(load().dsa_sparse_attn_decode_paged(ctypes.byref(cfg), _p(q), _p(latents),
                                               ctypes.byref(pages.c), _p(n_latents),
                                               _p(token_ids), _p(swa), _p(swa_len), B, _p(out),
                                               _p(lse), _p(ws), ws.numel(), _stream(stream)),
           "dsa_sparse_attn_decode_paged")


def decode_step(cfg, q, q_idx, w, keys: Keys, pooled: Keys, latents, n_latents, max_latents, swa,
                swa_len, out, ws, lse=None, block_ids=None, token_ids=None, update_pool=False,
                stream=None):
    B = q.shape[0]
    lat_stride = latents.shape[1] if keys.pages is None else 0
    _check(load().dsa_decode_step(ctypes.byref(cfg), _p(q), _p(q_idx), _p(w),
                                  ctypes.byref(keys.c()), ctypes.byref(pooled.c()),
                                  int(update_pool), _p(latents), lat_stride, _p(n_latents),
                                  max_latents, _p(swa), _p(swa_len), B, _p(block_ids),
                                  _p(token_ids), _p(out), _p(lse), _p(ws), ws.numel(),
                                  _stream(stream)), "dsa_decode_step")


def decode_multi(cfg, n_tokens, q, q_idx, w, keys: Keys, pooled: Keys, latents, max_latents, swa,
                 out, ws, lse=None, token_ids=None, stream=None):
    """Multi-query decode: q [B, n_q, 64, 512], each sequence's n_q queries at its
    last n_q positions (n_tokens [B] device int32)."""
    B, n_q = q.shape[0], q.shape[1]
    _check(load().dsa_decode_multi(ctypes.byref(cfg), n_q, _p(n_tokens), _p(q), _p(q_idx), _p(w),
                                   ctypes.byref(keys.c()), ctypes.byref(pooled.c()), _p(latents),
                                   latents.shape[1], max_latents, _p(swa), B, _p(out), _p(lse),
                                   _p(token_ids), _p(ws), ws.numel(), _stream(stream)),
           "dsa_decode_multi")


def compress_append(cfg, n_tokens, kv, gate, new_keys: Keys, latents, keys: Keys, pooled: Keys,
                    max_latents, ws, stream=None):
    """The cache append at the compression step: kv bf16 [B, ratio, 512], gate
    fp32 [B, ratio], new_keys one index-key row per sequence."""
    B = n_tokens.shape[0]
    lat_stride = latents.shape[1] if keys.pages is None else 0
    _check(load().dsa_compress_append(ctypes.byref(cfg), B, _p(n_tokens), _p(kv), _p(gate),
                                      ctypes.byref(new_keys.c()), _p(latents), lat_stride,
                                      ctypes.byref(keys.c()), ctypes.byref(pooled.c()),
                                      max_latents, _p(ws), ws.numel(), _stream(stream)),
           "dsa_compress_append")


def sparse_attn_prefill(cfg, ctx_len, q, q_idx, w, latents, keys: Keys, pooled: Keys, swa, out,
                        ws, lse=None, token_ids=None, stream=None):
    n_q = q.shape[0]
    _check(load().dsa_sparse_attn_prefill(ctypes.byref(cfg), n_q, ctx_len, _p(q), _p(q_idx),
                                          _p(w), _p(latents), ctypes.byref(keys.c()),
                                          ctypes.byref(pooled.c()), _p(swa), _p(out), _p(lse),
                                          _p(token_ids), _p(ws), ws.numel(), _stream(stream)),
           "dsa_sparse_attn_prefill")


def _launch_stream(t: torch.Tensor, stream):
    """The raw stream to launch on: the given one, or the current stream of t's
    device, which has to be the current device (the library launches there)."""
    dev = t.get_device()  # -1: on the host
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on {t.device}, which is not the current CUDA device")
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _one_device(*tensors):
    """Refuses tensors of different devices (None: not given)."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {tensors[0].device} and {t.device}")


def _i32(name, t, shape=None):
    if t.dtype != torch.int32 or not t.is_contiguous() or (shape is not None
                                                           and tuple(t.shape) != shape):
        raise ValueError(f"{name}: a contiguous int32 tensor"
                         + (f" of shape {list(shape)}" if shape is not None else "")
                         + f", not {t.dtype} {list(t.shape)}")


class PagePool:
    """A pool of pages and its free pages (dsa_page_pool_t): table int32
    [B, pages_per_seq], free_ring int32 [n_pages] with the free pages at positions
    head .. tail - 1 modulo n_pages, ring_state int64 {head, tail}. All are updated
    by plan_step; ring_state_out keeps ring_state as it is and takes its place."""

    def __init__(self, table: torch.Tensor, page_rows: int, free_ring: torch.Tensor,
                 ring_state: torch.Tensor, ring_state_out: Optional[torch.Tensor] = None):
        _i32("table", table)
        _i32("free_ring", free_ring)
        out = ring_state if ring_state_out is None else ring_state_out
        if table.dim() != 2 or free_ring.dim() != 1:
            raise ValueError("table has two dimensions and free_ring one")
        for r in (ring_state, out):
            if r.dtype != torch.int64 or r.numel() != 2 or not r.is_contiguous():
                raise ValueError("ring_state: two int64 values")
        _one_device(table, free_ring, ring_state, out)
        self.table, self.page_rows, self.free_ring = table, page_rows, free_ring
        self.ring_state, self.ring_state_out = ring_state, out
        self.B = table.shape[0]
        self.c = _PagePool(table.data_ptr(), page_rows, table.shape[1], free_ring.shape[0],
                           free_ring.data_ptr(), ring_state.data_ptr(), out.data_ptr())
        self._ref = ctypes.byref(self.c)
        self._key = ctypes.addressof(self.c), self.B, table.get_device()

    @classmethod
    def empty(cls, B: int, page_rows: int, pages_per_seq: int, n_pages: int, device="cuda"):
        """A pool with every page free and no request holding any."""
        return cls(torch.full((B, pages_per_seq), -1, dtype=torch.int32, device=device), page_rows,
                   torch.arange(n_pages, dtype=torch.int32, device=device),
                   torch.tensor([0, n_pages], dtype=torch.int64, device=device))

    def pages(self) -> Pages:
        """The pool's page table as the caches' calls take it."""
        return Pages(self.table, self.page_rows, self.free_ring.shape[0])


class StepPlan:
    """What plan_step writes (dsa_step_plan_t), int32 tensors: n_tokens, n_latents and
    swa_len [B], cu_new [B + 1], and per new token (max_new entries) token_seq,
    positions, latent_slots and window_slots. n_tokens may be the input lengths."""

    def __init__(self, n_tokens, n_latents, swa_len, cu_new, token_seq, positions, latent_slots,
                 window_slots):
        B, m = n_tokens.shape[0], token_seq.shape[0]
        for name, t, n in (("n_tokens", n_tokens, B), ("n_latents", n_latents, B),
                           ("swa_len", swa_len, B), ("cu_new", cu_new, B + 1),
                           ("token_seq", token_seq, m), ("positions", positions, m),
                           ("latent_slots", latent_slots, m), ("window_slots", window_slots, m)):
            _i32(name, t, (n,))
            setattr(self, name, t)
        _one_device(n_tokens, n_latents, swa_len, cu_new, token_seq, positions, latent_slots,
                    window_slots)
        self.B, self.max_new, self.shape = B, m, n_tokens.shape
        self.c = _StepPlan(n_tokens.data_ptr(), n_latents.data_ptr(), swa_len.data_ptr(),
                           cu_new.data_ptr(), token_seq.data_ptr(), positions.data_ptr(),
                           latent_slots.data_ptr(), window_slots.data_ptr(), m)
        self._ref = ctypes.byref(self.c)
        self._key = ctypes.addressof(self.c), B, n_tokens.get_device()

    @classmethod
    def empty(cls, B: int, max_new: int, device="cuda", n_tokens=None):
        """Tensors for B requests and up to max_new new tokens a step."""
        def new(n):
            return torch.zeros((n,), dtype=torch.int32, device=device)
        return cls(new(B) if n_tokens is None else n_tokens, new(B), new(B), new(B + 1),
                   new(max_new), new(max_new), new(max_new), new(max_new))

    @property
    def n_valid(self) -> torch.Tensor:
        """The step's number of new tokens, on the device (cu_new's last entry)."""
        return self.cu_new[-1:]


def plan_step(cfg, n_tokens, n_new, pool: PagePool, plan: StepPlan, ws, stream=None):
    """Block table and slot maps of a step (dsa_plan_step): n_tokens [B] lengths
    before the step, n_new [B] tokens added (negative: the request ends). ws: any workspace,
    workspace(cfg, 1, 0) will do."""
    if stream is None:  # the plain case (None: any other)
        code = (_calls or _load_calls()).plan(cfg, n_tokens, n_new, pool._key, plan._key, ws)
        if code is not None:
            return _check(code, "dsa_plan_step")
    B, i32 = plan.B, torch.int32
    if n_tokens.dtype is not i32 or n_new.dtype is not i32 or n_tokens.shape != plan.shape or \
            n_new.shape != plan.shape or pool.B != B or \
            not (n_tokens.is_contiguous() and n_new.is_contiguous()):
        raise ValueError(f"n_tokens and n_new: contiguous int32 tensors of the plan's {B} requests, "
                         f"the pool's table a row for each")
    dev = n_tokens.get_device()
    if n_new.get_device() != dev or pool.table.get_device() != dev or \
            plan.n_tokens.get_device() != dev or ws.get_device() != dev:
        _one_device(n_tokens, n_new, pool.table, plan.n_tokens, ws)
    code = load().dsa_plan_step(ctypes.byref(cfg), B, n_tokens.data_ptr(), n_new.data_ptr(),
                                pool._ref, plan._ref, ws.data_ptr(), ws.numel(),
                                _launch_stream(n_tokens, stream))
    if code:
        raise DsaError(code, "dsa_plan_step")


def plan_trim(cfg, n_tokens, n_drop, pool: PagePool, plan: StepPlan, ws, stream=None):
    """The requests' last n_drop [B] tokens taken off their n_tokens [B], the pages that held
    them back to the pool (dsa_plan_trim); writes plan's n_tokens (which may be the input
    lengths), n_latents and swa_len. ws: as for plan_step."""
    if stream is None:
        code = (_calls or _load_calls()).trim(cfg, n_tokens, n_drop, pool._key, plan._key, ws)
        if code is not None:
            return _check(code, "dsa_plan_trim")
    B = plan.B
    _i32("n_tokens", n_tokens, (B,))
    _i32("n_drop", n_drop, (B,))
    if pool.B != B:
        raise ValueError(f"a pool whose table has a row for each of the plan's {B} requests")
    _one_device(n_tokens, n_drop, pool.table, plan.n_tokens, ws)
    _check(load().dsa_plan_trim(ctypes.byref(cfg), B, n_tokens.data_ptr(), n_drop.data_ptr(),
                                pool._ref, plan._ref, ws.data_ptr(), ws.nbytes,
                                _launch_stream(n_tokens, stream)), "dsa_plan_trim")


_DT = {torch.bfloat16: 0, torch.int16: 0, torch.float16: 1, torch.float32: 2}


class Heads:
    """A group of heads for norm_rope (dsa_heads_t): x [n, heads, dim] or [n, dim]
    with contiguous elements and any token and head strides (a slice of a fused
    projection, say), out like x (x itself: in place). weight fp32 [dim] or None;
    norm=False rotates only; rope_start: first rotated element, None for no rotation."""

    def __init__(self, x: torch.Tensor, out: Optional[torch.Tensor] = None,
                 weight: Optional[torch.Tensor] = None, eps: float = 1e-6, norm: bool = True,
                 rope_start: Optional[int] = None):
        out = x if out is None else out
        if x.dtype not in _DT or out.dtype not in _DT or _DT[x.dtype] != _DT[out.dtype]:
            raise ValueError("x and out: bf16 (or its bits in int16), f16 or f32, both alike")
        if x.dim() not in (2, 3) or out.shape != x.shape or x.stride(-1) != 1 or \
                out.stride(-1) != 1:
            raise ValueError("x and out: [n, heads, dim] or [n, dim] with contiguous elements")
        if weight is not None and (weight.dtype != torch.float32 or not weight.is_contiguous()
                                   or weight.shape != x.shape[-1:]):
            raise ValueError("weight: contiguous fp32 [dim]")
        if any(t is not None and t.get_device() != x.get_device() for t in (out, weight)):
            raise ValueError("x, out and weight on one device")
        self.x, self.out, self.weight = x, out, weight
        self.n, self.dtype = x.shape[0], _DT[x.dtype]
        heads = x.shape[1] if x.dim() == 3 else 1

        def strides(t):
            return t.stride(0), t.stride(1) if t.dim() == 3 and heads > 1 else t.shape[-1]
        self.c = _HeadsC(x.data_ptr(), out.data_ptr(), heads, x.shape[-1], *strides(x),
                         *strides(out), weight.data_ptr() if weight is not None else None, eps,
                         int(norm), -1 if rope_start is None else rope_start)


class HeadSet:
    """The groups of heads of one norm_rope call, of one element type and token count."""

    def __init__(self, groups):
        groups = list(groups)
        if not groups or any(g.n != groups[0].n or g.dtype != groups[0].dtype or
                             g.x.get_device() != groups[0].x.get_device() for g in groups):
            raise ValueError("groups of one element type, token count and device")
        self.groups = groups
        self.n, self.dtype = groups[0].n, groups[0].dtype
        self.x, self.shape, self.count = groups[0].x, groups[0].x.shape[:1], len(groups)
        self._c = (_HeadsC * len(groups))(*[g.c for g in groups])
        self._key = (ctypes.addressof(self._c), self.count, self.n, self.dtype,
                     self.x.get_device())


class Rope:
    """A rotation (dsa_rope_t): inv_freq fp64 [rope_dim / 2] on the device, radians per
    position (finite; an infinity or NaN makes its pair NaN); interleaved pairs (2i, 2i + 1) or halves (i, i + rope_dim / 2); cosine
    and sine times scale."""

    def __init__(self, inv_freq: torch.Tensor, interleaved: bool = True, scale: float = 1.0):
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq: contiguous fp64 [rope_dim / 2]")
        self.inv_freq = inv_freq
        self.c = _RopeC(inv_freq.data_ptr(), 2 * inv_freq.shape[0], int(interleaved), scale)
        self._ref = ctypes.byref(self.c)
        self._key = ctypes.addressof(self.c), inv_freq.get_device()


def norm_rope(positions, heads: HeadSet, rope: Optional[Rope] = None, n_valid=None, stream=None):
    """Norms of heads and their rotation in one pass (dsa_norm_rope): positions int32
    [n]; n_valid: device int32 [1], tokens behind it are left as they were."""
    if stream is None:
        code = (_calls or _load_calls()).norm(positions, heads.x, heads._key,
                                              None if rope is None else rope._key, n_valid)
        if code is not None:
            return _check(code, "dsa_norm_rope")
    n = heads.n
    if rope is not None or positions is not None:
        if positions is None or positions.dtype is not torch.int32 or \
                positions.shape != heads.shape or not positions.is_contiguous():
            raise ValueError(f"positions: contiguous int32 [{n}]")
    if n_valid is not None:
        _i32("n_valid", n_valid, (1,))
    _one_device(heads.x, positions, n_valid, None if rope is None else rope.inv_freq)
    code = load().dsa_norm_rope(n, None if n_valid is None else n_valid.data_ptr(),
                                None if positions is None else positions.data_ptr(), heads.dtype,
                                heads._c, heads.count, None if rope is None else rope._ref,
                                _launch_stream(heads.x, stream))
    if code:
        raise DsaError(code, "dsa_norm_rope")


_KV_ROW = {KV_BF16: 1024, KV_FP8_E4M3: 512, KV_MXFP4: KV_MXFP4_ROW}


def _rows_call(name, cfg, rows, slots, cache, ws, n_valid, stream):
    """kv_write and kv_read: their checks and the call."""
    row = _KV_ROW.get(cfg.kv_fmt)
    if row is None:
        raise DsaError(1, "kv_fmt")
    shape = rows.shape
    if len(shape) != 2 or shape[1] != 512 or _DT.get(rows.dtype) != 0:
        raise ValueError("rows: bf16 (or its bits in int16) [n, 512] with contiguous elements")
    n, stride = shape[0], 512
    if not rows.is_contiguous():
        stride, unit = rows.stride()
        if unit != 1:
            raise ValueError("rows: contiguous elements")
    if slots.dtype is not torch.int32 or slots.numel() != n or slots.dim() != 1 or \
            not slots.is_contiguous():
        _i32("slots", slots, (n,))
    if n_valid is not None:
        _i32("n_valid", n_valid, (1,))
    if not cache.is_contiguous() or cache.shape[-1] * cache.element_size() != row:
        raise ValueError(f"cache: contiguous rows of {row} bytes")
    dev = rows.get_device()
    if slots.get_device() != dev or cache.get_device() != dev or ws.get_device() != dev or \
            (n_valid is not None and n_valid.get_device() != dev):
        _one_device(rows, slots, cache, ws, n_valid)
    s = _launch_stream(rows, stream)
    valid = None if n_valid is None else n_valid.data_ptr()
    n_rows, c = cache.nbytes // row, ctypes.byref(cfg)
    if name == "dsa_kv_write":
        code = load().dsa_kv_write(c, n, valid, rows.data_ptr(), stride, slots.data_ptr(),
                                   cache.data_ptr(), n_rows, ws.data_ptr(), ws.numel(), s)
    else:
        code = load().dsa_kv_read(c, n, valid, cache.data_ptr(), n_rows, slots.data_ptr(),
                                  rows.data_ptr(), stride, ws.data_ptr(), ws.numel(), s)
    if code:
        raise DsaError(code, name)


def kv_write(cfg, rows, slots, cache, ws, n_valid=None, stream=None):
    """bf16 rows [n, 512] into a cache of cfg.kv_fmt (dsa_kv_write): row r becomes cache
    row slots[r], negative slots skip; cache: [..., row] contiguous (a pool of pages, or
    the window rows). ws: any workspace, workspace(cfg, 1, 0) will do."""
    if stream is None:
        code = (_calls or _load_calls()).rows(True, cfg, rows, slots, cache, ws, n_valid)
        if code is not None:
            return _check(code, "dsa_kv_write")
    _rows_call("dsa_kv_write", cfg, rows, slots, cache, ws, n_valid, stream)


def kv_read(cfg, cache, slots, rows, ws, n_valid=None, stream=None):
    """Rows slots[r] of a cache back as bf16 rows [n, 512] (dsa_kv_read); rows with a
    negative slot are left as they were. ws: as for kv_write."""
    if stream is None:
        code = (_calls or _load_calls()).rows(False, cfg, rows, slots, cache, ws, n_valid)
        if code is not None:
            return _check(code, "dsa_kv_read")
    _rows_call("dsa_kv_read", cfg, rows, slots, cache, ws, n_valid, stream)


def full_attn_workspace(cfg: Config, n_queries: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace for full_attn_decode and full_attn_multi over n_queries queries (the
    calls that need no more than a status word take it too)."""
    n = ctypes.c_size_t(0)
    _check(load().dsa_full_attn_workspace_size(ctypes.byref(cfg), n_queries, ctypes.byref(n)),
           "dsa_full_attn_workspace_size")
    return torch.zeros(int(n.value), dtype=torch.uint8, device=device)


def _bf16(name, t, shape):
    if _DT.get(t.dtype) != 0 or not t.is_contiguous() or tuple(t.shape) != shape:
        raise ValueError(f"{name}: contiguous bf16 (or its bits in int16) {list(shape)}, "
                         f"not {t.dtype} {list(t.shape)}")


def _full_cache(cfg, latents, swa, pages: Optional[Pages], B, win_rows):
    """The caches' checks of the full attention: (stride, capacity) of the latents."""
    row = _KV_ROW.get(cfg.kv_fmt)
    if row is None:
        raise DsaError(1, "kv_fmt")
    for name, t in (("latents", latents), ("swa", swa)):
        if t is not None and (t.dim() == 0 or not t.is_contiguous() or t.shape[-1] * t.element_size() != row):
            raise ValueError(f"{name}: contiguous rows of {row} bytes")
    if swa is not None and tuple(swa.shape[:-1]) != (B, win_rows):
        raise ValueError(f"swa: [{B}, {win_rows}] rows, not {list(swa.shape[:-1])}")
    if pages is None:
        if latents.dim() != 3 or latents.shape[0] != B:
            raise ValueError(f"latents: [{B}, capacity] rows, not {list(latents.shape[:-1])}")
        return latents.shape[1], latents.shape[1]
    if pages.table.shape[0] != B or not pages.table.is_contiguous() or \
            latents.nbytes < pages.c.n_pages * pages.c.page_rows * row:
        raise ValueError(f"pages: a table of {B} rows, latents a row for every page row")
    return 0, pages.c.pages_per_seq * pages.c.page_rows


def full_attn_decode(cfg, q, latents, n_latents, out, ws, swa=None, swa_len=None,
                     pages: Optional[Pages] = None, lse=None, stream=None):
    """Attention over the whole cache and the window (dsa_full_attn_decode): q and out bf16
    [B, 64, 512], latents [B, capacity] rows of cfg.kv_fmt (pages: a pool's rows), n_latents
    int32 [B]; swa [B, window] rows with swa_len int32 [B], or neither. ws: full_attn_workspace."""
    if stream is None:
        code = (_calls or _load_calls()).full(False, cfg, n_latents, q, latents, out, ws, swa, swa_len,
                                              None if pages is None else pages._key, lse)
        if code is not None:
            return _check(code, "dsa_full_attn_decode")
    if q.dim() != 3:
        raise ValueError(f"q: [B, 64, 512], not {list(q.shape)}")
    B = q.shape[0]
    _bf16("q", q, (B, 64, 512))
    _bf16("out", out, (B, 64, 512))
    _i32("n_latents", n_latents, (B,))
    if (swa is None) != (swa_len is None):
        raise ValueError("swa and swa_len: both or neither")
    if swa_len is not None:
        _i32("swa_len", swa_len, (B,))
    stride, cap = _full_cache(cfg, latents, swa, pages, B, cfg.window)
    _check_lse(lse, (B, 64))
    _one_device(q, latents, n_latents, out, ws, swa, swa_len, lse,
                None if pages is None else pages.table)
    _check(load().dsa_full_attn_decode(ctypes.byref(cfg), q.data_ptr(), latents.data_ptr(), stride,
                                       None if pages is None else ctypes.byref(pages.c),
                                       n_latents.data_ptr(), cap, _p(swa), _p(swa_len), B,
                                       out.data_ptr(), _p(lse), ws.data_ptr(), ws.nbytes,
                                       _launch_stream(q, stream)), "dsa_full_attn_decode")


def _check_lse(lse, shape):
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous()
                            or tuple(lse.shape) != shape):
        raise ValueError(f"lse: contiguous fp32 {list(shape)}")


def full_attn_multi(cfg, n_tokens, q, latents, out, ws, swa=None, pages: Optional[Pages] = None,
                    lse=None, stream=None):
    """full_attn_decode for each sequence's last n_q positions (dsa_full_attn_multi): q and out
    bf16 [B, n_q, 64, 512], n_tokens int32 [B]; swa [B, window + n_q - 1] rows, by position as
    decode_multi takes them, or None."""
    if stream is None:
        code = (_calls or _load_calls()).full(True, cfg, n_tokens, q, latents, out, ws, swa, None,
                                              None if pages is None else pages._key, lse)
        if code is not None:
            return _check(code, "dsa_full_attn_multi")
    if q.dim() != 4:
        raise ValueError(f"q: [B, n_q, 64, 512], not {list(q.shape)}")
    B, n_q = q.shape[0], q.shape[1]
    _bf16("q", q, (B, n_q, 64, 512))
    _bf16("out", out, (B, n_q, 64, 512))
    _i32("n_tokens", n_tokens, (B,))
    stride, cap = _full_cache(cfg, latents, swa, pages, B, cfg.window + n_q - 1)
    _check_lse(lse, (B, n_q, 64))
    _one_device(q, latents, n_tokens, out, ws, swa, lse, None if pages is None else pages.table)
    _check(load().dsa_full_attn_multi(ctypes.byref(cfg), n_q, n_tokens.data_ptr(), q.data_ptr(),
                                      latents.data_ptr(), stride,
                                      None if pages is None else ctypes.byref(pages.c), cap,
                                      _p(swa), B, out.data_ptr(), _p(lse), ws.data_ptr(), ws.nbytes,
                                      _launch_stream(q, stream)), "dsa_full_attn_multi")


def _prob_rows(name, t, B, n):
    """The row stride of probabilities [B, n, vocab]: contiguous words, rows evenly spaced."""
    if t.dim() != 3 or t.shape[0] != B or t.shape[1] != n or t.dtype not in _PROBS or \
            (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name}: fp32, f16 or bf16 [{B}, {n}, vocab] with contiguous words")
    row = t.stride(1) if n > 1 else t.stride(0)
    if n > 1 and B > 1 and t.stride(0) != n * row:
        raise ValueError(f"{name}: rows evenly spaced")
    return row


_PROBS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def verify_drafts(target, draft_tokens, uniform, tokens, n_kept, ws, draft=None, n_drafts=None,
                  n_drop=None, stream=None):
    """Drafted tokens against the target's probabilities (dsa_verify_drafts): target
    [B, n_draft + 1, vocab] and draft [B, n_draft, vocab] (None: drafts of probability 1) fp32,
    f16 or bf16, both alike; draft_tokens int32 [B, n_draft]; n_drafts int32 [B] or None;
    uniform fp32 [B, n_draft + 1]. Writes tokens int32 [B, n_draft + 1] and, int32 [B], n_kept
    and n_drop (may be None). ws: any workspace, workspace(cfg, 1, 0) will do."""
    if stream is None:
        code = (_calls or _load_calls()).verify(target, draft, draft_tokens, n_drafts, uniform,
                                                tokens, n_kept, n_drop, ws)
        if code is not None:
            return _check(code, "dsa_verify_drafts")
    if uniform.dim() != 2 or uniform.shape[1] < 1 or uniform.dtype != torch.float32 or \
            not uniform.is_contiguous():
        raise ValueError("uniform: contiguous fp32 [B, n_draft + 1]")
    B, n = uniform.shape[0], uniform.shape[1] - 1
    p_stride = _prob_rows("target", target, B, n + 1)
    q_stride = 0
    if draft is not None:
        q_stride = _prob_rows("draft", draft, B, n)
        if draft.dtype != target.dtype or draft.shape[2] != target.shape[2]:
            raise ValueError("draft: of the target's type and vocabulary")
    _i32("draft_tokens", draft_tokens, (B, n))
    _i32("tokens", tokens, (B, n + 1))
    _i32("n_kept", n_kept, (B,))
    for name, t in (("n_drafts", n_drafts), ("n_drop", n_drop)):
        if t is not None:
            _i32(name, t, (B,))
    _one_device(target, draft_tokens, uniform, tokens, n_kept, ws, draft, n_drafts, n_drop)
    _check(load().dsa_verify_drafts(B, n, target.shape[2], _PROBS[target.dtype], target.data_ptr(),
                                    p_stride, _p(draft), q_stride, draft_tokens.data_ptr(),
                                    _p(n_drafts), uniform.data_ptr(), tokens.data_ptr(),
                                    n_kept.data_ptr(), _p(n_drop), ws.data_ptr(), ws.nbytes,
                                    _launch_stream(target, stream)), "dsa_verify_drafts")


def read_device_status(ws, stream=None):
    """(status code, info word); synchronises the stream and clears the status."""
    info = ctypes.c_uint32(0)
    code = load().dsa_read_device_status(_p(ws), _stream(stream), ctypes.byref(info))
    return int(code), int(info.value)


def selftest_timeout(ws, stream=None) -> None:
    """Launches the failure-report self-test: a wait that nothing satisfies
    runs out (about 1 ms) and records DSA_ERR_TIMEOUT in ws's status word (read
    it with read_device_status)."""
    _check(load().dsa_selftest_timeout(_p(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "dsa_selftest_timeout")


def profile_events(kind: str, starts, ends) -> None:
    """Brackets each later launch of kernel `kind` with the given torch.cuda.Events
    (recorded round-robin); pass empty lists to switch off."""
    n = len(starts)
    assert len(ends) == n
    for e in list(starts) + list(ends):
        if e.cuda_event == 0:
            e.record()  # torch creates its event lazily
    arr_s = (ctypes.c_void_p * max(n, 1))(*[ctypes.c_void_p(e.cuda_event) for e in starts])
    arr_e = (ctypes.c_void_p * max(n, 1))(*[ctypes.c_void_p(e.cuda_event) for e in ends])
    _profile_keepalive[kind] = (arr_s, arr_e, list(starts), list(ends))
    _check(load().dsa_profile_events(KERNEL_KINDS.index(kind), arr_s, arr_e, n),
           "dsa_profile_events")


_profile_keepalive: dict = {}


def launch_counts(reset: bool = False) -> dict:
    arr = (ctypes.c_uint64 * len(KERNEL_KINDS))()
    _check(load().dsa_launch_counts(arr, int(reset)), "dsa_launch_counts")
    return {k: int(arr[i]) for i, k in enumerate(KERNEL_KINDS)}


def default_tau() -> float:
    return 1.0 / math.sqrt(512.0)
