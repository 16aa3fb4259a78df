"""Compressed sparse attention (c4a / c128a) for GB300: Python binding of libcsa.

A thin ctypes layer over the C ABI declared in include/csa.h.  It only
marshals arguments: torch tensors become device pointers, the current torch
stream becomes the launch stream.  Every step of the path runs in the CUDA
kernels of libcsa.so; there is no Python or CPU fallback, and every call
raises if the compiled library is missing.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa.so")

F32, BF16, E4M3, E2M1, E4M3R = 0, 1, 2, 3, 4
DTYPES = {"f32": F32, "bf16": BF16, "e4m3": E4M3, "e2m1": E2M1, "e4m3r": E4M3R}

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_DEVICE_BOUNDS, ERR_WORKSPACE, ERR_TIMEOUT = 0, -1, -2, -3, -4, -5, -6
ERR_NONFINITE = -7


class CsaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class Paged(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("rows_per_block", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("tail_bf16", ctypes.c_int32)]


class BlockTableC(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("num_seqs", ctypes.c_int32), ("stride", ctypes.c_int32)]


class QueryNormC(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_dtype", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("gamma", ctypes.c_void_p), ("q_out", ctypes.c_void_p), ("out_dtype", ctypes.c_int32)]


class Layer(ctypes.Structure):
    _fields_ = [("ratio", ctypes.c_int32), ("window", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("heads", ctypes.c_int32), ("swa", ctypes.c_int32),
                ("rope_theta", ctypes.c_float), ("rms_eps", ctypes.c_float), ("scale", ctypes.c_float)]


class Kv8C(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int32), ("rows_per_block", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("dim", ctypes.c_int32)]


class Kv8MaskC(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("slopes", ctypes.c_void_p), ("first", ctypes.c_void_p), ("prefix", ctypes.c_void_p)]


_lib = None

_VP, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_PP, _PB, _PL = ctypes.POINTER(Paged), ctypes.POINTER(BlockTableC), ctypes.POINTER(Layer)
_PQ = ctypes.POINTER(QueryNormC)
_PK, _PM = ctypes.POINTER(Kv8C), ctypes.POINTER(Kv8MaskC)

_SIGS = {
    "csa_compress_insert": (_I32, [_PL, _VP, _VP, _I32, _I32, _VP, _VP, _VP, _VP, _VP, _PP, _PB, _PP, _PB, _PP,
                                   _PB, _VP, _VP]),
    "csa_compress_insert_qnorm": (_I32, [_PL, _VP, _VP, _I32, _I32, _VP, _VP, _VP, _VP, _VP, _PP, _PB, _PP, _PB,
                                         _PP, _PB, _PQ, _VP, _VP]),
    "csa_cache_store": (_I32, [_VP, _I32, _VP, _VP, _PP, _PB, _VP, _VP]),
    "csa_indexer_topk": (_I32, [_VP, _I32, _VP, _I32, _I32, _I32, _VP, _VP, _I32, _I32, _PP, _PB, _I32, _I32, _VP,
                                _VP, _SZ, _VP, _VP]),
    "csa_indexer_topk_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "csa_sparse_attn_decode": (_I32, [_PL, _VP, _I32, _I32, _VP, _VP, _PP, _PB, _VP, _I32, _I32, _PP, _PB, _VP, _I32,
                                      _VP, _VP, _SZ, _VP, _VP]),
    "csa_sparse_attn_prefill": (_I32, [_PL, _VP, _I32, _I32, _VP, _VP, _PP, _PB, _VP, _I32, _I32, _PP, _PB, _VP,
                                       _I32, _VP, _VP, _SZ, _VP, _VP]),
    "csa_sparse_attn_workspace_size": (_SZ, [_PL, _I32, _I32]),
    "csa_indexer_topk_noalloc": (_I32, [_VP, _I32, _VP, _I32, _I32, _I32, _VP, _VP, _I32, _I32, _PP, _PB, _I32,
                                        _I32, _VP, _VP, _VP]),
    "csa_step_plan": (_I32, [_VP, _VP, _I32, _VP, _I32, _VP, _I32, _I32, _I32, _I32, _VP, _VP, _VP, _VP, _VP, _VP,
                             _VP]),
    "csa_kv8_store": (_I32, [_VP, _VP, _I32, _I64, _I64, _I32, _VP, _VP, _PK, _PB, _VP, _VP]),
    "csa_kv8_attn": (_I32, [_VP, _I32, _I64, _I32, _I32, _VP, _VP, _I32, _PK, _PB, _PM, _VP, _I32, _VP, _VP, _SZ,
                            _VP, _VP]),
    "csa_kv8_attn_workspace_size": (_SZ, [_I32, _I32, _I32, _PK, _I32]),
    "csa_read_status": (_I32, [_VP, _I32, _VP]),
    "csa_status_string": (ctypes.c_char_p, [_I32]),
    "csa_version": (_I32, []),
    "csa_launch_count": (ctypes.c_uint64, []),
}

EXPORTED = tuple(_SIGS)


def lib():
    """The loaded libcsa.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libcsa.so is not built ({LIB_PATH}); run "
                               "`python -m compressed_sparse_long_c128a_gb300.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().csa_status_string(int(status)).decode()


def version() -> int:
    return int(lib().csa_version())


def launch_count() -> int:
    """Kernel launches the library has enqueued in this process (host-side count)."""
    return int(lib().csa_launch_count())


def _check(status: int, what: str):
    if status != OK:
        raise CsaError(status, what)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on the CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _tdtype(t) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise ValueError(f"unsupported input dtype {t.dtype}")


@dataclass
class PagedCache:
    """A paged cache in device memory: `data` [num_blocks, rows_per_block, row] and,
    for quantised dtypes, `scales` (E4M3, E4M3R: float [num_blocks, rows_per_block];
    E2M1: uint8 [num_blocks, rows_per_block, dim/16]).  An E4M3R row is
    dim - tail_bf16 code bytes followed by tail_bf16 bf16 values."""

    data: torch.Tensor
    scales: torch.Tensor | None
    dtype: int
    rows_per_block: int
    dim: int
    tail_bf16: int = 0

    @staticmethod
    def empty(num_blocks: int, rows_per_block: int, dim: int, dtype: int, device="cuda",
              tail_bf16: int = 0) -> "PagedCache":
        shape = (num_blocks, rows_per_block)
        scales = None
        if dtype == F32:
            data = torch.zeros(*shape, dim, dtype=torch.float32, device=device)
        elif dtype == BF16:
            data = torch.zeros(*shape, dim, dtype=torch.bfloat16, device=device)
        elif dtype == E4M3:
            data = torch.zeros(*shape, dim, dtype=torch.uint8, device=device)
            scales = torch.zeros(*shape, dtype=torch.float32, device=device)
        elif dtype == E2M1:
            data = torch.zeros(*shape, dim // 2, dtype=torch.uint8, device=device)
            scales = torch.zeros(*shape, dim // 16, dtype=torch.uint8, device=device)
        elif dtype == E4M3R:
            data = torch.zeros(*shape, dim + tail_bf16, dtype=torch.uint8, device=device)
            scales = torch.zeros(*shape, dtype=torch.float32, device=device)
        else:
            raise ValueError(dtype)
        return PagedCache(data, scales, dtype, rows_per_block, dim, tail_bf16 if dtype == E4M3R else 0)

    @property
    def num_blocks(self) -> int:
        return self.data.shape[0]

    def c(self) -> Paged:
        return Paged(_ptr(self.data), _ptr(self.scales), self.dtype, self.num_blocks, self.rows_per_block, self.dim,
                     self.tail_bf16)


def block_table(t: torch.Tensor) -> BlockTableC:
    """C view of an int32 [num_seqs, stride] device block table."""
    if t.dtype != torch.int32 or t.dim() != 2:
        raise ValueError("block table must be int32 [num_seqs, stride]")
    return BlockTableC(_ptr(t), t.shape[0], t.shape[1])


def make_layer(ratio, window, dim, rope_dim, heads, swa=128, rope_theta=10000.0, rms_eps=1e-6, scale=None) -> Layer:
    return Layer(ratio, window, dim, rope_dim, heads, swa, rope_theta, rms_eps,
                 dim ** -0.5 if scale is None else scale)


# ------------------------------------------------------------------ entry points


def compress_insert(layer: Layer, kv, gate, seq_id, pos, bias, gamma_c, gamma_swa, state: PagedCache, state_bt,
                    swa: PagedCache | None, swa_bt, comp: PagedCache, comp_bt, err, stream=None):
    """swa=None (swa_bt and gamma_swa then ignored) writes no sliding-window rows:
    the indexer-key compressor, whose keys go to an indexer cache (comp may be E2M1)."""
    no_swa = swa is None
    st = lib().csa_compress_insert(ctypes.byref(layer), _ptr(kv), _ptr(gate), _tdtype(kv), kv.shape[0],
                                   _ptr(seq_id), _ptr(pos), _ptr(bias), _ptr(gamma_c),
                                   None if no_swa else _ptr(gamma_swa),
                                   ctypes.byref(state.c()), ctypes.byref(block_table(state_bt)),
                                   None if no_swa else ctypes.byref(swa.c()),
                                   None if no_swa else ctypes.byref(block_table(swa_bt)),
                                   ctypes.byref(comp.c()), ctypes.byref(block_table(comp_bt)), _ptr(err),
                                   _stream(stream))
    _check(st, "csa_compress_insert")


def compress_insert_qnorm(layer: Layer, kv, gate, seq_id, pos, bias, gamma_c, gamma_swa, state: PagedCache,
                          state_bt, swa: PagedCache | None, swa_bt, comp: PagedCache, comp_bt, q, gamma_q, q_out,
                          err, stream=None):
    """compress_insert plus q_out[j, h] := RMSNorm(q[j, h]; gamma_q) in the same launch.
    q, q_out: [n_tok, heads, D] (f32 or bf16; q_out may be q itself)."""
    if q.dim() != 3 or q_out.shape != q.shape or q.shape[0] != kv.shape[0]:
        raise ValueError("q and q_out must be [n_tok, heads, D] with n_tok rows of kv")
    qn = QueryNormC(_ptr(q), _tdtype(q), q.shape[1], _ptr(gamma_q), _ptr(q_out), _tdtype(q_out))
    no_swa = swa is None
    st = lib().csa_compress_insert_qnorm(ctypes.byref(layer), _ptr(kv), _ptr(gate), _tdtype(kv), kv.shape[0],
                                         _ptr(seq_id), _ptr(pos), _ptr(bias), _ptr(gamma_c),
                                         None if no_swa else _ptr(gamma_swa),
                                         ctypes.byref(state.c()), ctypes.byref(block_table(state_bt)),
                                         None if no_swa else ctypes.byref(swa.c()),
                                         None if no_swa else ctypes.byref(block_table(swa_bt)),
                                         ctypes.byref(comp.c()), ctypes.byref(block_table(comp_bt)),
                                         ctypes.byref(qn), _ptr(err), _stream(stream))
    _check(st, "csa_compress_insert_qnorm")


def cache_store(rows, seq_id, row_idx, cache: PagedCache, bt, err, stream=None):
    if rows.dtype != torch.float32:
        raise ValueError("rows must be float32")
    st = lib().csa_cache_store(_ptr(rows), rows.shape[0], _ptr(seq_id), _ptr(row_idx), ctypes.byref(cache.c()),
                               ctypes.byref(block_table(bt)), _ptr(err), _stream(stream))
    _check(st, "csa_cache_store")


def indexer_topk_workspace_size(n_rows: int, max_n: int, k: int) -> int:
    return int(lib().csa_indexer_topk_workspace_size(n_rows, max_n, k))


def indexer_topk(q_idx, w, seq_id, pos, ratio: int, window: int, idx_cache: PagedCache, bt, k: int, max_n: int,
                 out_idx, ws, err, stream=None):
    n_rows, heads, dim = q_idx.shape
    st = lib().csa_indexer_topk(_ptr(q_idx), _tdtype(q_idx), _ptr(w), n_rows, heads, dim, _ptr(seq_id), _ptr(pos),
                                ratio, window, ctypes.byref(idx_cache.c()), ctypes.byref(block_table(bt)), k, max_n,
                                _ptr(out_idx), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                _ptr(err), _stream(stream))
    _check(st, "csa_indexer_topk")


def indexer_topk_noalloc(q_idx, w, seq_id, pos, ratio: int, window: int, idx_cache: PagedCache, bt, k: int,
                         max_n: int, out_idx, err, stream=None):
    """indexer_topk without a workspace, for callers that cannot allocate device
    memory: its scratch is a fixed 16 MiB array inside the library, shared by
    every call (calls that may overlap on the GPU race; the first call on a
    device should come before any stream capture)."""
    n_rows, heads, dim = q_idx.shape
    st = lib().csa_indexer_topk_noalloc(_ptr(q_idx), _tdtype(q_idx), _ptr(w), n_rows, heads, dim, _ptr(seq_id),
                                        _ptr(pos), ratio, window, ctypes.byref(idx_cache.c()),
                                        ctypes.byref(block_table(bt)), k, max_n, _ptr(out_idx), _ptr(err),
                                        _stream(stream))
    _check(st, "csa_indexer_topk_noalloc")


def sparse_attn_workspace_size(layer: Layer, n_rows: int, k_or_max_n: int) -> int:
    return int(lib().csa_sparse_attn_workspace_size(ctypes.byref(layer), n_rows, k_or_max_n))


def _attn(name, layer, q, seq_id, pos, comp, comp_bt, topk, k, max_n, swa, swa_bt, out, out_dtype, out_scales, ws,
          err, stream):
    fn = getattr(lib(), name)
    st = fn(ctypes.byref(layer), _ptr(q), _tdtype(q), q.shape[0], _ptr(seq_id), _ptr(pos), ctypes.byref(comp.c()),
            ctypes.byref(block_table(comp_bt)), _ptr(topk), k, max_n, ctypes.byref(swa.c()),
            ctypes.byref(block_table(swa_bt)), _ptr(out), out_dtype, _ptr(out_scales), _ptr(ws),
            0 if ws is None else ws.numel() * ws.element_size(), _ptr(err), _stream(stream))
    _check(st, name)


def sparse_attn_decode(layer: Layer, q, seq_id, pos, comp: PagedCache, comp_bt, topk, k: int, max_n: int,
                       swa: PagedCache, swa_bt, out, out_dtype: int, out_scales, ws, err, stream=None):
    _attn("csa_sparse_attn_decode", layer, q, seq_id, pos, comp, comp_bt, topk, k, max_n, swa, swa_bt, out,
          out_dtype, out_scales, ws, err, stream)


def sparse_attn_prefill(layer: Layer, q, seq_id, pos, comp: PagedCache, comp_bt, topk, k: int, max_n: int,
                        swa: PagedCache, swa_bt, out, out_dtype: int, out_scales, ws, err, stream=None):
    _attn("csa_sparse_attn_prefill", layer, q, seq_id, pos, comp, comp_bt, topk, k, max_n, swa, swa_bt, out,
          out_dtype, out_scales, ws, err, stream)


# ------------------------------------------------------------------ step plan, 8-bit key / value cache


# These calls are short next to their launches, so the checks ask each tensor for little:
# raw device and stream numbers, one look at its shape and strides.


def _dev(t, dtype, what, device):
    """Device pointer of a dense tensor of the given type on `device`."""
    if t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor")
    if t.get_device() != device:
        raise ValueError(f"{what} must live on the current CUDA device")
    return t.data_ptr()


def _rows3(t, what, shape, device):
    """(pointer, elements between rows, type) of [rows, heads, dim] rows whose heads are dense."""
    st = t.stride()
    if len(st) != 3 or st[2] != 1 or (st[1] != shape[2] and shape[1] != 1):
        raise ValueError(f"{what} must be [rows, heads, dim] with dense heads")
    if t.get_device() != device:
        raise ValueError(f"{what} must live on the current CUDA device")
    return t.data_ptr(), st[0], _tdtype(t)


def _current(t):
    """The current device; t, the call's first tensor, must live there."""
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError("the tensors must live on the current CUDA device")
    return dev


def _raw_stream(stream, device):
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream


@dataclass
class Kv8Cache:
    """A paged key / value cache in 8 bits: e4m3 codes (uint8) [num_blocks, kv_heads, rows_per_block, dim]
    and one float scale for each block and head [num_blocks, kv_heads], for keys and for values."""

    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    def __post_init__(self):
        shape = tuple(self.k.shape)
        if len(shape) != 4 or tuple(self.v.shape) != shape:
            raise ValueError("k and v must be [num_blocks, kv_heads, rows_per_block, dim]")
        if tuple(self.k_scale.shape) != shape[:2] or tuple(self.v_scale.shape) != shape[:2]:
            raise ValueError("scales must be [num_blocks, kv_heads]")
        for t, dt in ((self.k, torch.uint8), (self.v, torch.uint8), (self.k_scale, torch.float32),
                      (self.v_scale, torch.float32)):
            if t.dtype is not dt:
                raise ValueError("codes are uint8 and scales float32")
            if t.device != self.k.device:
                raise ValueError("the cache's tensors must live on one device")
        self.num_blocks, self.kv_heads, self.rows_per_block, self.dim = shape
        self.device = self.k.get_device()
        self._c = Kv8C(_ptr(self.k), _ptr(self.v), _ptr(self.k_scale), _ptr(self.v_scale), shape[0], shape[2],
                       shape[1], shape[3])

    @staticmethod
    def empty(num_blocks: int, kv_heads: int, rows_per_block: int, dim: int, device="cuda") -> "Kv8Cache":
        codes = [torch.zeros(num_blocks, kv_heads, rows_per_block, dim, dtype=torch.uint8, device=device)
                 for _ in range(2)]
        scales = [torch.zeros(num_blocks, kv_heads, dtype=torch.float32, device=device) for _ in range(2)]
        return Kv8Cache(*codes, *scales)

    def c(self) -> Kv8C:
        return self._c


def step_plan(cached, n_new, free_blocks, bt, block_positions: int, num_blocks: int, row_start, seq_id, pos, slot,
              used, err, stream=None):
    """Row starts, sequence ids, positions, slots and the block table of a step from its requests' lengths
    (slot may be None).  bt [num_reqs, stride] is updated in place; rows past the step's become padding (-1)."""
    dev, i32 = _current(bt), torch.int32
    shape, n_rows = bt.shape, seq_id.numel()
    if len(shape) != 2 or cached.numel() != shape[0] or n_new.numel() != shape[0]:
        raise ValueError("cached and n_new must have one entry for each row of the block table")
    if row_start.numel() != shape[0] + 1 or pos.numel() != n_rows or used.numel() != 1:
        raise ValueError("row_start must be [num_reqs + 1], seq_id and pos of one length, used [1]")
    if slot is not None and slot.numel() != n_rows:
        raise ValueError("slot must have the length of seq_id")
    st = lib().csa_step_plan(_dev(cached, i32, "cached", dev), _dev(n_new, i32, "n_new", dev), shape[0],
                             _dev(free_blocks, i32, "free_blocks", dev), free_blocks.numel(),
                             _dev(bt, i32, "block table", dev), shape[1], block_positions, num_blocks, n_rows,
                             _dev(row_start, i32, "row_start", dev), _dev(seq_id, i32, "seq_id", dev),
                             _dev(pos, i32, "pos", dev),
                             None if slot is None else _dev(slot, torch.int64, "slot", dev),
                             _dev(used, i32, "used", dev), _dev(err, i32, "err", dev), _raw_stream(stream, dev))
    _check(st, "csa_step_plan")


def _kv8_lengths(row_start, cached, cache, bt, dev):
    """Pointers of row_start and cached, and the C block table, checked against each other."""
    if cache.device != dev:
        raise ValueError("the cache must live on the current CUDA device")
    shape = bt.shape
    if len(shape) != 2 or row_start.numel() != shape[0] + 1 or cached.numel() != shape[0]:
        raise ValueError("row_start must be [num_seqs + 1] and cached [num_seqs] for the block table's num_seqs")
    i32 = torch.int32
    return (_dev(row_start, i32, "row_start", dev), _dev(cached, i32, "cached", dev),
            BlockTableC(_dev(bt, i32, "block table", dev), shape[0], shape[1]))


def kv8_store(k, v, row_start, cached, cache: Kv8Cache, bt, err, stream=None):
    """Insert k, v [n_rows, kv_heads, dim] (f32 or bf16; rows may be strided) into the 8-bit cache: request b's
    rows row_start[b]..row_start[b+1] go to positions cached[b].. of row b of the block table."""
    dev, shape = _current(k), k.shape
    if shape != v.shape:
        raise ValueError("k and v must have one shape and type")
    kp, ks, dt = _rows3(k, "k", shape, dev)
    vp, vs, vt = _rows3(v, "v", shape, dev)
    if dt != vt:
        raise ValueError("k and v must have one shape and type")
    if shape[1] != cache.kv_heads or shape[2] != cache.dim:
        raise ValueError("k and v must have the cache's heads and dim")
    rs, ca, b = _kv8_lengths(row_start, cached, cache, bt, dev)
    st = lib().csa_kv8_store(kp, vp, dt, ks, vs, shape[0], rs, ca, cache.c(), b, _dev(err, torch.int32, "err", dev),
                             _raw_stream(stream, dev))
    _check(st, "csa_kv8_store")


def kv8_attn_workspace_size(n_rows: int, num_seqs: int, heads: int, cache: Kv8Cache, max_new: int) -> int:
    """Bytes of scratch of a kv8_attn call of these sizes; a call of fewer rows can need more."""
    return int(lib().csa_kv8_attn_workspace_size(n_rows, num_seqs, heads, cache.c(), max_new))


def kv8_attn(q, row_start, cached, cache: Kv8Cache, bt, max_new: int, out, ws, err, scale: float | None = None,
             softcap: float = 0.0, window: int = 0, slopes=None, first=None, prefix=None, lse=None, stream=None):
    """Attention of q [n_rows, heads, dim] (f32 or bf16; rows may be strided) over the 8-bit cache into out
    [n_rows, heads, dim] (f32 or bf16) and, if given, lse [n_rows, heads] (float).  Scores are capped by
    softcap * tanh(a / softcap), lowered by slopes[head] * distance, and masked by causality, `window`, `first`
    (int32 [n_rows], each row's first visible position) and `prefix` (int32 [num_seqs], tokens every row sees).
    The cache already holds the rows' own tokens; max_new is the most rows of a request."""
    dev, shape = _current(q), q.shape
    qp, qs, dt = _rows3(q, "q", shape, dev)
    n_rows, heads, dim = shape
    if dim != cache.dim or out.shape != shape:
        raise ValueError("q and out must be [n_rows, heads, dim] with the cache's dim")
    rs, ca, b = _kv8_lengths(row_start, cached, cache, bt, dev)
    i32, f32 = torch.int32, torch.float32
    m = Kv8MaskC(dim ** -0.5 if scale is None else scale, softcap, window)
    if slopes is not None:
        if slopes.numel() != heads:
            raise ValueError("slopes must be [heads]")
        m.slopes = _dev(slopes, f32, "slopes", dev)
    if first is not None:
        if first.numel() != n_rows:
            raise ValueError("first must be [n_rows]")
        m.first = _dev(first, i32, "first", dev)
    if prefix is not None:
        if prefix.numel() != b.num_seqs:
            raise ValueError("prefix must be [num_seqs]")
        m.prefix = _dev(prefix, i32, "prefix", dev)
    lp = wp = None
    nbytes = 0
    if lse is not None:
        if lse.numel() != n_rows * heads:
            raise ValueError("lse must be [n_rows, heads]")
        lp = _dev(lse, f32, "lse", dev)
    if ws is not None:
        wp, nbytes = _dev(ws, ws.dtype, "ws", dev), ws.numel() * ws.element_size()
    st = lib().csa_kv8_attn(qp, dt, qs, n_rows, heads, rs, ca, max_new, cache.c(), b, m,
                            _dev(out, out.dtype, "out", dev), _tdtype(out), lp, wp, nbytes,
                            _dev(err, i32, "err", dev), _raw_stream(stream, dev))
    _check(st, "csa_kv8_attn")


def read_status(err, reset: bool = True, stream=None) -> int:
    return int(lib().csa_read_status(_ptr(err), 1 if reset else 0, _stream(stream)))
