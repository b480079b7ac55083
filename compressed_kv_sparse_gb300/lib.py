"""Thin Python binding of libds4a.so (ctypes): argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; PyTorch only
provides device memory and streams. There is no CPU path: if the compiled
library is missing, ``load()`` raises.
"""
from __future__ import annotations

import copy
import ctypes
import math
import os
from typing import Dict, Optional

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libds4a.so")

DS4A_F32, DS4A_BF16 = 0, 1
CALL_APPEND, CALL_INDEX_TOPK, CALL_ATTN_DECODE, CALL_ATTN_PREFILL = 0, 1, 2, 3
STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported or inconsistent shape",
          -3: "capacity exceeded", -4: "position does not match the cache",
          -5: "unknown dtype", -6: "CUDA error", -7: "device wait timed out",
          -8: "workspace too small"}


class Ds4aError(RuntimeError):
    def __init__(self, status: int, call: str):
        msg = f"{call}: {STATUS.get(status, status)} ({status})"
        if status == -6 and _lib is not None:
            msg += ": " + _lib.ds4a_last_error().decode()
        super().__init__(msg)
        self.status = status


class ArgumentError(ValueError, AssertionError):
    """A tensor of another type, size, layout or device than the call reads."""


class LayerCacheC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in
                ("ratio", "head_dim", "n_rot", "index_dim", "index_rot", "batch", "cap_raw",
                 "comp_cap")] + [
        ("dtype", ctypes.c_int32), ("n_tokens", ctypes.c_uint32),
        ("raw_kv", ctypes.c_void_p), ("attn_comp_kv", ctypes.c_void_p),
        ("attn_state_kv", ctypes.c_void_p), ("attn_state_score", ctypes.c_void_p),
        ("index_comp_kv", ctypes.c_void_p), ("index_state_kv", ctypes.c_void_p),
        ("index_state_score", ctypes.c_void_p), ("index_norm", ctypes.c_void_p),
        ("index_norm_max", ctypes.c_void_p), ("rope_cos", ctypes.c_void_p),
        ("rope_sin", ctypes.c_void_p), ("index_rope_cos", ctypes.c_void_p),
        ("index_rope_sin", ctypes.c_void_p), ("rope_max_pos", ctypes.c_uint32),
        ("qat", ctypes.c_uint32), ("block_table", ctypes.c_void_p),
        ("max_blocks", ctypes.c_uint32), ("n_blocks", ctypes.c_uint32),
        ("seq_pos", ctypes.c_void_p)]

QAT_FP8_ATTN = 1    # DS4A_QAT_FP8_ATTN
QAT_FP4_INDEX = 2   # DS4A_QAT_FP4_INDEX
FP4_ROWS = 0x10000  # DS4A_FP4_ROWS: attn_comp_kv holds 4-bit rows
Q_ROTATED = 0x20000  # DS4A_Q_ROTATED: the attention's queries are rotated already
Q_READY = 0x80000   # DS4A_Q_READY: q and positions are written before the launch before it begins


class BlockPoolC(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_uint32), ("max_blocks", ctypes.c_uint32),
                ("n_blocks", ctypes.c_uint32), ("table", ctypes.c_void_p),
                ("held", ctypes.c_void_p), ("free_list", ctypes.c_void_p),
                ("state", ctypes.c_void_p)]


class StepTablesC(ctypes.Structure):
    _fields_ = [("max_tokens", ctypes.c_uint32)] + [
        (n, ctypes.c_void_p) for n in ("seq_pos", "cu_len", "tok_seq", "tok_pos", "raw_slot",
                                       "comp_slot4", "comp_slot128")]


EXPORTS = {
    "ds4a_cache_reset": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "ds4a_index_norms": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "ds4a_compress_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint32]
                             + [ctypes.c_void_p] * 11),
    "ds4a_compress_append_lanes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint32,
                                                  ctypes.c_uint32, ctypes.c_uint32]
                                   + [ctypes.c_void_p] * 11),
    "ds4a_index_topk": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint32,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint32,
                                       ctypes.c_uint32, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_size_t, ctypes.c_void_p]),
    "ds4a_sparse_attn_decode": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint32,
                                               ctypes.c_void_p, ctypes.c_uint32,
                                               ctypes.c_void_p, ctypes.c_uint32, ctypes.c_float,
                                               ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_size_t, ctypes.c_void_p]),
    "ds4a_sparse_attn_prefill_chunk": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint32,
                                                      ctypes.c_uint32, ctypes.c_void_p,
                                                      ctypes.c_uint32, ctypes.c_void_p,
                                                      ctypes.c_void_p, ctypes.c_uint32,
                                                      ctypes.c_float, ctypes.c_void_p,
                                                      ctypes.c_void_p, ctypes.c_size_t,
                                                      ctypes.c_void_p]),
    "ds4a_row_bytes": (ctypes.c_size_t, [ctypes.c_uint32, ctypes.c_uint32, ctypes.c_int]),
    "ds4a_pack_rows": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint32] + [ctypes.c_void_p] * 3),
    "ds4a_unpack_rows": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint32] + [ctypes.c_void_p] * 3),
    "ds4a_norm_rope": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_uint64, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_uint32, ctypes.c_void_p]),
    "ds4a_block_tables": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_uint32, ctypes.c_void_p, ctypes.c_void_p]),
    "ds4a_index_topk_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint32,
                                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint32,
                                               ctypes.c_uint32, ctypes.c_void_p, ctypes.c_void_p]),
    "ds4a_noalloc_status": (ctypes.c_int, [ctypes.c_void_p]),
    "ds4a_workspace_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "ds4a_workspace_clear_status": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t,
                                                   ctypes.c_void_p]),
    "ds4a_wait_selftest": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32,
                                          ctypes.c_void_p]),
    "ds4a_set_decode_cluster": (ctypes.c_int, [ctypes.c_uint32]),
    "ds4a_decode_cluster_size": (ctypes.c_uint32, [ctypes.c_void_p, ctypes.c_uint32,
                                                   ctypes.c_uint32]),
    "ds4a_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_void_p, ctypes.c_uint32,
                                               ctypes.c_uint32, ctypes.c_uint32]),
    "ds4a_rope_table": (ctypes.c_int, [ctypes.c_double, ctypes.c_uint32, ctypes.c_uint32,
                                       ctypes.c_void_p, ctypes.c_void_p]),
    "ds4a_cache_bytes": (ctypes.c_uint64, [ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32,
                                           ctypes.c_uint64, ctypes.c_uint32, ctypes.c_uint32]),
    "ds4a_layer_compress_ratio": (ctypes.c_uint32, [ctypes.c_int, ctypes.c_uint32]),
    "ds4a_prefill_chunk_cap": (ctypes.c_uint32, [ctypes.c_uint32]),
    "ds4a_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ds4a_launch_count": (ctypes.c_uint64, []),
    "ds4a_last_error": (ctypes.c_char_p, []),
}

_lib: Optional[ctypes.CDLL] = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libds4a.so and declare its signatures. Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m compressed_kv_sparse_gb300.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in EXPORTS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _refuse(t: torch.Tensor, dev: int):
    if not t.is_contiguous():
        raise ArgumentError("tensors passed to the library must be contiguous")
    raise ArgumentError(f"a tensor on {t.device}, where the call's are on "
                        + (f"cuda:{dev}" if dev >= 0 else "the CPU"))


def _ptr(t: Optional[torch.Tensor], dev: int) -> Optional[int]:
    """Address of a contiguous tensor on device `dev` (-1: the CPU)."""
    if t is None:
        return None
    if t.get_device() != dev or not t.is_contiguous():
        _refuse(t, dev)
    return t.data_ptr()


def _need(ok: bool, what: str):
    if not ok:
        raise ArgumentError(what)


def _stream(stream, dev: int) -> Optional[int]:
    """The stream of a call whose tensors are on device `dev`, the current one."""
    if dev < 0:
        raise ArgumentError("the call's tensors are not on a GPU")
    if torch._C._cuda_getDevice() != dev:
        raise ArgumentError(f"the call's tensors are on cuda:{dev}, which is not the current device")
    if stream is None:       # (the current stream without building its object)
        return torch._C._cuda_getCurrentRawStream(dev)
    if not hasattr(stream, "cuda_stream"):
        return stream
    if stream.device_index != dev:
        raise ArgumentError(f"a stream of cuda:{stream.device_index}, the call's tensors are on cuda:{dev}")
    return stream.cuda_stream


def _check(status: int, call: str):
    if status != 0:
        raise Ds4aError(status, call)


_tables: Dict[tuple, tuple] = {}


def rope_table(base: float, n_rot: int, n_pos: int, device) -> tuple:
    """Device cos / sin tables [n_pos][n_rot/2] built by ds4a_rope_table."""
    device = torch.empty(0, device=device).device   # (with its index)
    key = (float(base), int(n_rot), int(n_pos), str(device))
    if key not in _tables:
        lib = load()
        c = torch.empty((n_pos, n_rot // 2), dtype=torch.float32)
        s = torch.empty((n_pos, n_rot // 2), dtype=torch.float32)
        _check(lib.ds4a_rope_table(base, n_rot, n_pos, c.data_ptr(), s.data_ptr()),
               "ds4a_rope_table")
        _tables[key] = (c.to(device), s.to(device))
    return _tables[key]


class LayerCache:
    """Device memory of one layer's cache (torch tensors) and its C struct.

    block_table ([B][max_blocks] int32 on the device) makes the compressed rows
    paged: pools of n_blocks blocks of 256 token positions (256 / ratio rows);
    comp_cap is then max_blocks * 256 / ratio. ``logical(name)`` gathers a
    pool back into the contiguous [B][comp_cap][...] view."""

    def __init__(self, *, ratio: int, head_dim: int, n_rot: int, batch: int, comp_cap: int,
                 dtype: str, base: float, rope_max_pos: int, index_dim: int = 0,
                 index_rot: int = 0, cap_raw: int = 128, qat: int = 0, device="cuda",
                 block_table: Optional[torch.Tensor] = None, n_blocks: int = 0):
        td = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
        self.dtype, self.torch_dtype = dtype, td
        self.ratio, self.head_dim, self.n_rot = ratio, head_dim, n_rot
        self.index_dim, self.index_rot, self.batch = index_dim, index_rot, batch
        self.cap_raw, self.comp_cap, self.base = cap_raw, comp_cap, base
        W = {0: 0, 4: 8, 128: 128}[ratio]
        z = lambda *s, dt=td: torch.zeros(s, dtype=dt, device=device)
        self.block_table, self.n_blocks = block_table, n_blocks
        paged = block_table is not None
        if paged:
            _need(block_table.dtype == torch.int32 and block_table.shape[0] == batch,
                  "block_table: [batch][max_blocks] int32")
            _need(comp_cap == block_table.shape[1] * (256 // ratio),
                  "comp_cap: every row of max_blocks blocks")
        rpb = 256 // ratio if ratio else 0
        self.fp4_rows = bool(qat & FP4_ROWS)   # attn_comp_kv: 4-bit rows, as bytes
        # comp rows: [B][comp_cap][w] or a pool [n_blocks][rows per block][w]
        rows = (lambda w, r, dt=td: z(n_blocks, r, w, dt=dt)) if paged else \
               (lambda w, r, dt=td: z(batch, comp_cap, w, dt=dt))
        self.raw_kv = z(batch, cap_raw, head_dim)
        self.dev = dev = self.raw_kv.get_device()   # (-1: the CPU)
        self.attn_comp_kv = self.attn_state_kv = self.attn_state_score = None
        self.index_comp_kv = self.index_state_kv = self.index_state_score = None
        self.index_norm = self.index_norm_max = None
        if ratio:
            if self.fp4_rows:
                self.attn_comp_kv = rows(row_bytes(head_dim, n_rot, dtype), rpb, torch.uint8)
            else:
                self.attn_comp_kv = rows(head_dim, rpb)
            self.attn_state_kv = z(batch, W, head_dim, dt=torch.float32)
            self.attn_state_score = torch.full((batch, W, head_dim), float("-inf"),
                                               device=device)
        if ratio == 4:
            self.index_comp_kv = rows(index_dim, 64)
            self.index_state_kv = z(batch, 8, index_dim, dt=torch.float32)
            self.index_state_score = torch.full((batch, 8, index_dim), float("-inf"),
                                                device=device)
            self.index_norm = (z(n_blocks, 64, dt=torch.float32) if paged
                               else z(batch, comp_cap, dt=torch.float32))
            self.index_norm_max = z(batch, dt=torch.int32)
        self.rope_cos, self.rope_sin = rope_table(base, n_rot, rope_max_pos, device)
        self.index_rope_cos = self.index_rope_sin = None
        if ratio == 4:
            self.index_rope_cos, self.index_rope_sin = rope_table(base, index_rot,
                                                                  rope_max_pos, device)
        self.c = LayerCacheC(
            ratio=ratio, head_dim=head_dim, n_rot=n_rot, index_dim=index_dim,
            index_rot=index_rot, batch=batch, cap_raw=cap_raw, comp_cap=comp_cap,
            dtype=DS4A_BF16 if dtype == "bf16" else DS4A_F32, n_tokens=0,
            raw_kv=_ptr(self.raw_kv, dev), attn_comp_kv=_ptr(self.attn_comp_kv, dev),
            attn_state_kv=_ptr(self.attn_state_kv, dev), attn_state_score=_ptr(self.attn_state_score, dev),
            index_comp_kv=_ptr(self.index_comp_kv, dev), index_state_kv=_ptr(self.index_state_kv, dev),
            index_state_score=_ptr(self.index_state_score, dev), index_norm=_ptr(self.index_norm, dev),
            index_norm_max=_ptr(self.index_norm_max, dev), rope_cos=_ptr(self.rope_cos, dev),
            rope_sin=_ptr(self.rope_sin, dev), index_rope_cos=_ptr(self.index_rope_cos, dev),
            index_rope_sin=_ptr(self.index_rope_sin, dev), rope_max_pos=rope_max_pos, qat=qat,
            block_table=_ptr(block_table, dev), max_blocks=block_table.shape[1] if paged else 0,
            n_blocks=n_blocks if paged else 0)
        self._ref = ctypes.byref(self.c)

    def set_seq_pos(self, seq_pos: Optional[torch.Tensor]):
        """Ragged decode: [B] uint32/int32 device positions of this step's
        tokens (None: every sequence at the call's position). The tensor must
        stay alive while calls use it."""
        _need(seq_pos is None or (seq_pos.dtype in (torch.int32, torch.uint32)
                                  and seq_pos.numel() == self.batch), "seq_pos: [batch] int32 or uint32")
        self.c.seq_pos = _ptr(seq_pos, self.dev)
        self.seq_pos = seq_pos

    def rows(self, b0: int, b1: int) -> "LayerCache":
        """Sequences b0 .. b1 - 1 as a cache of their own on the same memory, with its own
        n_tokens: what runs together of a step whose sequences have different numbers of new
        tokens (positions are seq_pos's as it was set before)."""
        _need(0 <= b0 < b1 <= self.batch, f"sequences {b0} .. {b1 - 1} of {self.batch}")
        v = copy.copy(self)
        v.c, v.batch = LayerCacheC.from_buffer_copy(self.c), b1 - b0
        names = ["raw_kv", "attn_state_kv", "attn_state_score", "index_state_kv", "index_state_score",
                 "index_norm_max", "block_table", "seq_pos"]
        if self.block_table is None:
            names += ["attn_comp_kv", "index_comp_kv", "index_norm"]
        for n in names:
            t = getattr(self, n, None)
            if t is not None:
                setattr(v, n, t[b0:b1])
                setattr(v.c, n, _ptr(t[b0:b1], self.dev))
        v.c.batch, v._ref = v.batch, ctypes.byref(v.c)
        return v

    def logical(self, name: str) -> torch.Tensor:
        """[B][comp_cap][...] view of compressed rows / row norms (a gather
        through the block table when paged)."""
        t = getattr(self, name)
        if self.block_table is None or name not in ("attn_comp_kv", "index_comp_kv",
                                                     "index_norm"):
            return t
        tb = self.block_table.long()                       # [B][max_blocks]
        g = t[tb.clamp(0, self.n_blocks - 1)]              # [B][max_blocks][rpb](...)
        return g.reshape((self.batch, self.comp_cap) + tuple(t.shape[2:]))

    def slots(self, n: int) -> torch.Tensor:
        """[B][n] int32: the pool row of compressed rows 0 .. n - 1 of each sequence."""
        dev = self.raw_kv.device
        r = torch.arange(n, device=dev)
        if self.block_table is None:
            s = torch.arange(self.batch, device=dev)[:, None] * self.comp_cap + r
        else:
            rpb = 256 // self.ratio
            s = self.block_table.to(dev).long()[:, r // rpb] * rpb + r % rpb
        return s.int().contiguous()

    @property
    def n_tokens(self) -> int:
        return self.c.n_tokens

    @n_tokens.setter
    def n_tokens(self, v: int):
        self.c.n_tokens = v

    def ref(self):
        return self._ref

    def load_state(self, hist: Dict[str, torch.Tensor], n_tokens: int):
        """Copy a cache snapshot (same layout as the tensors here) in, set
        n_tokens and rebuild the indexer row norms (ds4a_index_norms). With 4-bit
        rows, attn_comp_kv may be given as values [B][n][D]: they are packed."""
        for name, t in hist.items():
            dst = getattr(self, name)
            if name == "attn_comp_kv" and self.fp4_rows and t.dtype != torch.uint8:
                ds4a_pack_rows(self, t.reshape(-1, self.head_dim).to(dst.device, self.torch_dtype),
                               self.slots(t.shape[1]).reshape(-1))
            elif self.block_table is not None and name in ("attn_comp_kv", "index_comp_kv"):
                rpb, nb = dst.shape[1], (t.shape[1] + dst.shape[1] - 1) // dst.shape[1]
                src = torch.zeros((self.batch, nb * rpb) + tuple(t.shape[2:]), dtype=t.dtype,
                                  device=t.device)
                src[:, :t.shape[1]] = t
                idx = self.block_table[:, :nb].reshape(-1).long().to(dst.device)
                dst[idx] = src.reshape((self.batch * nb, rpb) + tuple(t.shape[2:])).to(dst.device)
            elif name in ("attn_comp_kv", "index_comp_kv") and t.shape[1] < dst.shape[1]:
                dst[:, :t.shape[1]].copy_(t)
            else:
                dst.copy_(t)
        self.n_tokens = n_tokens
        if self.ratio == 4:
            ds4a_index_norms(self)

    def snapshot(self) -> Dict[str, torch.Tensor]:
        names = ["raw_kv", "attn_comp_kv", "attn_state_kv", "attn_state_score",
                 "index_comp_kv", "index_state_kv", "index_state_score"]
        return {n: getattr(self, n).clone() for n in names if getattr(self, n) is not None}

    def workspace_bytes(self, call: int, T: int, n_heads: int, top_k: int) -> int:
        return load().ds4a_workspace_bytes(call, self.ref(), T, n_heads, top_k)


def ds4a_cache_reset(cache: LayerCache, stream=None):
    _check(load().ds4a_cache_reset(cache.ref(), _stream(stream, cache.dev)), "ds4a_cache_reset")


def ds4a_index_norms(cache: LayerCache, stream=None):
    _check(load().ds4a_index_norms(cache.ref(), _stream(stream, cache.dev)), "ds4a_index_norms")


_APPEND = ("raw_kv_in", "attn_cand", "attn_score", "ape_attn", "gamma_attn", "idx_cand", "idx_score",
           "ape_idx", "gamma_idx")


def ds4a_compress_append(cache: LayerCache, pos0: int, T: int, inp: Dict[str, torch.Tensor],
                         raw_chunk_out: Optional[torch.Tensor] = None, stream=None):
    dev = cache.dev
    _check(load().ds4a_compress_append(
        cache.ref(), pos0, T, *[_ptr(inp.get(n), dev) for n in _APPEND], _ptr(raw_chunk_out, dev),
        _stream(stream, dev)), "ds4a_compress_append")


LANE_RAW, LANE_ATTN, LANE_INDEX = 1, 2, 4   # DS4A_LANE_*


def ds4a_compress_append_lanes(cache: LayerCache, pos0: int, T: int, lanes: int,
                               inp: Dict[str, torch.Tensor],
                               raw_chunk_out: Optional[torch.Tensor] = None, stream=None):
    """The parts `lanes` of an append; n_tokens is left for the caller to set."""
    dev = cache.dev
    _check(load().ds4a_compress_append_lanes(
        cache.ref(), pos0, T, lanes, *[_ptr(inp.get(n), dev) for n in _APPEND],
        _ptr(raw_chunk_out, dev), _stream(stream, dev)), "ds4a_compress_append_lanes")


def ds4a_index_topk(cache: LayerCache, pos0: int, T: int, q_idx: torch.Tensor, w: torch.Tensor,
                    n_heads: int, top_k: int, topk: torch.Tensor, ws: torch.Tensor, stream=None):
    dev = cache.dev
    _check(load().ds4a_index_topk(cache.ref(), pos0, T, _ptr(q_idx, dev), _ptr(w, dev), n_heads, top_k,
                                  _ptr(topk, dev), _ptr(ws, dev), _nbytes(ws), _stream(stream, dev)),
           "ds4a_index_topk")


def row_bytes(head_dim: int, n_rot: int, dtype: str) -> int:
    """Bytes of a compressed row held in 4 bits (ds4a_row_bytes)."""
    n = load().ds4a_row_bytes(head_dim, n_rot, DS4A_BF16 if dtype == "bf16" else DS4A_F32)
    if n == 0:
        raise Ds4aError(-2, "ds4a_row_bytes")
    return n


_I32 = torch.int32


def _rows_call(name: str, cache: LayerCache, rows: torch.Tensor, slots, stream):
    n, dev = rows.size(0), cache.dev
    if not (rows.dtype is cache.torch_dtype and rows.size(1) == cache.head_dim):
        raise ArgumentError("rows: [n][head_dim]")
    if not (slots is None or (slots.dtype is _I32 and slots.numel() == n)):
        raise ArgumentError("slots: [n] int32")
    _check(getattr(_lib or load(), name)(cache.ref(), n, _ptr(rows, dev), _ptr(slots, dev),
                                         _stream(stream, dev) if n else None), name)


def ds4a_pack_rows(cache: LayerCache, rows: torch.Tensor, slots: Optional[torch.Tensor] = None,
                   stream=None):
    """rows [n][D] into the 4-bit rows `slots` (None: 0 .. n - 1) of the cache's pool."""
    _rows_call("ds4a_pack_rows", cache, rows, slots, stream)


def ds4a_unpack_rows(cache: LayerCache, rows: torch.Tensor, slots: Optional[torch.Tensor] = None,
                     stream=None):
    """The values of 4-bit rows `slots` (None: 0 .. n - 1) into rows [n][D]."""
    _rows_call("ds4a_unpack_rows", cache, rows, slots, stream)


NORM_ROTATE_Q = 1   # DS4A_NORM_ROTATE_Q


def ds4a_norm_rope(cache: LayerCache, pos: torch.Tensor, *, q: Optional[torch.Tensor] = None,
                   gamma_q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                   kv: Optional[torch.Tensor] = None, gamma_kv: Optional[torch.Tensor] = None,
                   kv_out: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                   rot_q: bool = False, stream=None):
    """Norms of q [n][H][D] and kv [n][D] with the tail rotation. The tokens of q and kv
    may be strided (a slice of one projection's output); a token's own elements
    are contiguous. kv goes to kv_out [n][D] or, kv_out None, to rows `slots` of
    the raw window."""
    n, H, D, dt, q_stride, kv_stride = pos.numel(), 0, cache.head_dim, cache.torch_dtype, 0, 0
    dev = cache.dev
    # (the checks of this call and the next two in line: they are a good part of a small call)
    if not (pos.dtype is _I32 and (slots is None or (slots.dtype is _I32 and slots.numel() == n))):
        raise ArgumentError("pos and slots: [n] int32")
    if q is not None:
        (N, H, W), (q_stride, s1, s2) = q.shape, q.stride()
        if not (q.dtype is dt and N == n and W == D and s2 == 1 and (H == 1 or s1 == D)
                and q.get_device() == dev):
            raise ArgumentError("q: [n][heads][head_dim] with whole tokens, on the cache's device")
        if not ((q_out is None or (q_out.dtype is dt and q_out.numel() == n * H * D))
                and (gamma_q is None or (gamma_q.dtype is dt and gamma_q.numel() == D))):
            raise ArgumentError("q_out: like q; gamma_q: [head_dim]")
    if kv is not None:
        kv_stride, s1 = kv.stride()
        if not (kv.dtype is dt and kv.size(0) == n and kv.size(1) == D and s1 == 1
                and kv.get_device() == dev):
            raise ArgumentError("kv: [n][head_dim] with whole tokens, on the cache's device")
        if not ((kv_out is None or (kv_out.dtype is dt and kv_out.numel() == n * D))
                and (gamma_kv is None or (gamma_kv.dtype is dt and gamma_kv.numel() == D))):
            raise ArgumentError("kv_out: like kv; gamma_kv: [head_dim]")
    if n == 1:   # (one token: its stride is whatever the slice left)
        q_stride, kv_stride = H * D, D
    if n == 0:   # (empty tensors have no address)
        return
    _check((_lib or load()).ds4a_norm_rope(
        cache.ref(), n, _ptr(pos, dev), None if q is None else q.data_ptr(), q_stride, H,
        _ptr(gamma_q, dev), _ptr(q_out, dev), None if kv is None else kv.data_ptr(), kv_stride,
        _ptr(gamma_kv, dev), _ptr(kv_out, dev), _ptr(slots, dev), NORM_ROTATE_Q if rot_q else 0,
        _stream(stream, dev)), "ds4a_norm_rope")


class BlockPool:
    """Blocks of a paged cache and who holds them (ds4a_block_pool); all free at first."""

    def __init__(self, rows: int, max_blocks: int, n_blocks: int, device="cuda"):
        self.rows, self.max_blocks, self.n_blocks = rows, max_blocks, n_blocks
        i32 = dict(dtype=torch.int32, device=device)
        self.table = torch.full((rows, max_blocks), -1, **i32)
        self.held = torch.zeros(rows, **i32)
        self.free_list = torch.arange(n_blocks, **i32)
        self.state = torch.tensor([0, n_blocks, 0, 0], **i32)
        self.dev = dev = self.state.get_device()
        self.c = BlockPoolC(rows=rows, max_blocks=max_blocks, n_blocks=n_blocks,
                            table=_ptr(self.table, dev), held=_ptr(self.held, dev),
                            free_list=_ptr(self.free_list, dev), state=_ptr(self.state, dev))


class StepTables:
    """What ds4a_block_tables writes for a step (ds4a_step_tables)."""

    def __init__(self, rows: int, max_tokens: int, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.rows, self.max_tokens = rows, max_tokens
        self.seq_pos = torch.zeros(rows, **i32)
        self.cu_len = torch.zeros(rows + 1, **i32)
        tok = torch.full((5, max_tokens), -1, **i32)
        self.tok_seq, self.tok_pos, self.raw_slot, self.comp_slot4, self.comp_slot128 = tok
        self.dev = self.seq_pos.get_device()
        self.c = StepTablesC(max_tokens=max_tokens, **{
            n: _ptr(getattr(self, n), self.dev) for n in ("seq_pos", "cu_len", "tok_seq", "tok_pos",
                                                          "raw_slot", "comp_slot4", "comp_slot128")})


def ds4a_block_tables(pool: BlockPool, ctx_len: torch.Tensor, new_len: torch.Tensor, cap_raw: int,
                      step: StepTables, stream=None):
    """Blocks for rows of ctx_len [B] tokens (the last new_len [B] of them new), int32."""
    dev = pool.dev
    if not (ctx_len.dtype is _I32 and new_len.dtype is _I32
            and ctx_len.numel() == pool.rows == new_len.numel() == step.rows and step.dev == dev):
        raise ArgumentError("ctx_len, new_len: [rows] int32; a step of as many rows on the pool's device")
    _check((_lib or load()).ds4a_block_tables(
        ctypes.byref(pool.c), _ptr(ctx_len, dev), _ptr(new_len, dev), cap_raw, ctypes.byref(step.c),
        _stream(stream, dev)), "ds4a_block_tables")


STATIC_SCRATCH_BYTES = 8 << 20


def ds4a_index_topk_noalloc(cache: LayerCache, pos0: int, T: int, q_idx: torch.Tensor,
                            w: torch.Tensor, n_heads: int, top_k: int, topk: torch.Tensor,
                            stream=None):
    """ds4a_index_topk with the library's static scratch instead of a workspace."""
    dev = cache.dev
    _check(load().ds4a_index_topk_noalloc(cache.ref(), pos0, T, _ptr(q_idx, dev), _ptr(w, dev), n_heads,
                                          top_k, _ptr(topk, dev), _stream(stream, dev)),
           "ds4a_index_topk_noalloc")


def ds4a_sparse_attn_decode(cache: LayerCache, pos: int, q: torch.Tensor, n_heads: int,
                            topk: Optional[torch.Tensor], top_k: int, scale: float,
                            out: torch.Tensor, ws: Optional[torch.Tensor], stream=None):
    dev = cache.dev
    _check(load().ds4a_sparse_attn_decode(cache.ref(), pos, _ptr(q, dev), n_heads, _ptr(topk, dev), top_k,
                                          scale, _ptr(out, dev), _ptr(ws, dev), _nbytes(ws),
                                          _stream(stream, dev)),
           "ds4a_sparse_attn_decode")


def ds4a_sparse_attn_prefill_chunk(cache: LayerCache, pos0: int, T: int, q: torch.Tensor,
                                   n_heads: int, raw_chunk: torch.Tensor,
                                   topk: Optional[torch.Tensor], top_k: int, scale: float,
                                   out: torch.Tensor, ws: Optional[torch.Tensor], stream=None):
    dev = cache.dev
    _check(load().ds4a_sparse_attn_prefill_chunk(cache.ref(), pos0, T, _ptr(q, dev), n_heads,
                                                 _ptr(raw_chunk, dev), _ptr(topk, dev), top_k, scale,
                                                 _ptr(out, dev), _ptr(ws, dev), _nbytes(ws),
                                                 _stream(stream, dev)),
           "ds4a_sparse_attn_prefill_chunk")


def ds4a_cache_bytes(ratio, head_dim, index_dim, ctx, batch, elem_bytes) -> int:
    return load().ds4a_cache_bytes(ratio, head_dim, index_dim, ctx, batch, elem_bytes)


def ds4a_layer_compress_ratio(variant: int, il: int) -> int:
    return load().ds4a_layer_compress_ratio(variant, il)


def ds4a_prefill_chunk_cap(prompt_len: int) -> int:
    return load().ds4a_prefill_chunk_cap(prompt_len)


def ds4a_launch_count() -> int:
    return load().ds4a_launch_count()


def workspace(nbytes: int, device="cuda") -> Optional[torch.Tensor]:
    """A workspace buffer (uint8) of at least nbytes, 256-byte aligned by torch.
    Its first 256 bytes are zeroed, so its wait status starts clear."""
    if nbytes == 0:
        return None
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    ws[:min(nbytes, 256)].zero_()
    return ws


def _nbytes(ws: Optional[torch.Tensor]) -> int:
    return 0 if ws is None else ws.numel() * ws.element_size()


def ds4a_workspace_status(ws: torch.Tensor) -> int:
    """Timed-out device waits recorded in a workspace's error word (0: none).
    Synchronises nothing itself: call after the calls' stream is synchronised.
    Returns the count; the status (DS4A_OK / DS4A_ERR_TIMEOUT) follows from it."""
    n = ctypes.c_uint32(0)
    st = load().ds4a_workspace_status(_ptr(ws, ws.get_device()), _nbytes(ws), ctypes.byref(n))
    if st not in (0, -7):
        _check(st, "ds4a_workspace_status")
    assert (st == -7) == (n.value != 0)
    return n.value


def ds4a_workspace_clear_status(ws: torch.Tensor, stream=None):
    dev = ws.get_device()
    _check(load().ds4a_workspace_clear_status(_ptr(ws, dev), _nbytes(ws), _stream(stream, dev)),
           "ds4a_workspace_clear_status")


def ds4a_noalloc_status() -> int:
    """ds4a_workspace_status of the no-allocation variant's static scratch."""
    n = ctypes.c_uint32(0)
    st = load().ds4a_noalloc_status(ctypes.byref(n))
    if st not in (0, -7):
        _check(st, "ds4a_noalloc_status")
    return n.value


def ds4a_wait_selftest(ws: torch.Tensor, limit_us: int, stream=None):
    dev = ws.get_device()
    _check(load().ds4a_wait_selftest(_ptr(ws, dev), _nbytes(ws), limit_us, _stream(stream, dev)),
           "ds4a_wait_selftest")


def ds4a_set_decode_cluster(C: int):
    _check(load().ds4a_set_decode_cluster(C), "ds4a_set_decode_cluster")


def ds4a_decode_cluster_size(cache: "LayerCache", n_heads: int, top_k: int) -> int:
    return load().ds4a_decode_cluster_size(cache.ref(), n_heads, top_k)


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)
