"""Python binding of libv4attn: DeepSeek-V4 hybrid compressed attention
(CSA / HCA) on B200.

Argument marshalling only: every function turns torch tensors into the
pointers and sizes of the C ABI (include/v4attn.h) and calls the library on
the current CUDA stream.  Every step of the hot path runs in the library's
CUDA kernels; there is no CPU or PyTorch fallback, and importing this module
raises when the library has not been built.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _abi
from ._abi import (BF16, CSA, E4M3_BF16ROPE, F16, F32, HCA, MXFP4, CompressArgs, DecodeArgs,
                   IndexArgs, KvDesc, LayerDesc, MqaArgs, ProjectArgs)

_lib = _abi.load()

__all__ = ["F32", "BF16", "F16", "E4M3_BF16ROPE", "MXFP4", "CSA", "HCA", "V4AttnError", "layer_desc",
           "workspace", "workspace_size", "workspace_init", "compress", "index_topk",
           "index_topk_noalloc", "noalloc_device_status", "debug_index_stall",
           "device_status_code", "tc_peak_probe",
           "sparse_mqa", "dense_mqa",
           "decode", "project", "device_status", "build_info", "row_bytes",
           "kv_desc", "kv_workspace", "kv_append", "paged_attention", "block_sparse_attention"]


class V4AttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = _lib.v4attn_status_string(status).decode()
        if status == _abi.ERR_CUDA:
            msg += ": " + _lib.v4attn_last_cuda_error().decode()
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


def _check(fn: str, status: int):
    if status != _abi.OK:
        raise V4AttnError(fn, status)


def _p(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on the GPU")
    return t.data_ptr()


def _stream(stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise ValueError(f"unsupported dtype {t.dtype}")


def row_bytes(fmt: int, c: int, d_rope: int = 64) -> int:
    if fmt == F32:
        return 4 * c
    if fmt == E4M3_BF16ROPE:
        return (c - d_rope) + 2 * d_rope
    if fmt == MXFP4:
        return c // 2
    raise ValueError(fmt)


def layer_desc(kind: int, m: int, H: int, d: int, d_rope: int, n_win: int = 128,
               rope_theta: float = 160000.0, softmax_scale: float = 0.0, H_I: int = 0,
               d_I: int = 0, top_k: int = 0, kv_dtype: int = E4M3_BF16ROPE,
               idx_dtype: int = MXFP4, rms_eps: float = 1e-6) -> LayerDesc:
    return LayerDesc(kind, m, n_win, H, d, d_rope, rope_theta, softmax_scale, H_I, d_I, top_k,
                     kv_dtype, idx_dtype, rms_eps)


def workspace_size(desc: LayerDesc, n_q: int, max_vis: int) -> int:
    n = _lib.v4attn_workspace_size(ctypes.byref(desc), n_q, max_vis)
    if n == 0:
        raise V4AttnError("v4attn_workspace_size", _abi.ERR_INVALID_ARG)
    return n


def workspace(desc: LayerDesc, n_q: int, max_vis: int, device="cuda") -> torch.Tensor:
    """A zero-status workspace for calls on this layer with <= n_q queries."""
    ws = torch.empty(workspace_size(desc, n_q, max_vis), dtype=torch.uint8, device=device)
    _check("v4attn_workspace_init", _lib.v4attn_workspace_init(_p(ws), ws.numel(), _stream()))
    return ws


def compress(desc: LayerDesc, *, m: int, overlap: bool, c: int, Ca, Za, Cb=None, Zb=None,
             in_rows: int, in_seq_stride: int, in_row_stride: int, bias=None, seq_len,
             entry_begin, n_entries: int, out_dtype: int, out, out_scale=None, out_rows: int,
             complete_only=False, apply_rmsnorm=True, apply_rope=True, ws=None, stream=None):
    a = CompressArgs(m, int(overlap), c, int(seq_len.numel()), _p(Ca), _p(Za), _p(Cb), _p(Zb),
                     _dt(Ca), in_seq_stride, in_row_stride, in_rows, _p(bias), _p(seq_len),
                     _p(entry_begin), n_entries, int(complete_only), int(apply_rmsnorm),
                     int(apply_rope), out_dtype, _p(out), _p(out_scale), out_rows)
    _check("v4attn_compress", _lib.v4attn_compress(ctypes.byref(desc), ctypes.byref(a), _p(ws),
                                                   0 if ws is None else ws.numel(),
                                                   _stream(stream)))


def _bt(block_table):
    """(pointer, blocks per sequence) of an int32 [B][blocks_per_seq] block table, or (None, 0)."""
    if block_table is None:
        return None, 0
    assert block_table.dim() == 2 and block_table.is_contiguous()
    return _p(block_table), int(block_table.shape[1])


def index_topk(desc: LayerDesc, *, qI, w, q_pos, keys, key_rows: int, max_vis: int, idx_out, ws,
               qI_sf=None, keys_sf=None, q_seq=None, B: Optional[int] = None, scores_out=None,
               score_dtype: int = F32, block_table=None, stream=None):
    """Indexer scores + top-k (see include/v4attn.h); with ``block_table``
    (int32 [B][blocks_per_seq]) the keys are a paged pool of ``key_rows`` rows."""
    n_q = int(q_pos.numel())
    bt, bps = _bt(block_table)
    a = IndexArgs(n_q, B if B is not None else n_q, _p(qI), _p(qI_sf), _p(w), _p(q_seq),
                  _p(q_pos), _p(keys), _p(keys_sf), key_rows, max_vis, _p(idx_out),
                  _p(scores_out), score_dtype, bt, bps)
    _check("v4attn_index_topk", _lib.v4attn_index_topk(ctypes.byref(desc), ctypes.byref(a),
                                                       _p(ws), ws.numel(), _stream(stream)))


def index_topk_noalloc(desc: LayerDesc, *, qI, w, q_pos, keys, key_rows: int, max_vis: int,
                       idx_out, qI_sf=None, keys_sf=None, q_seq=None, B: Optional[int] = None,
                       scores_out=None, stream=None):
    """index_topk with the library's built-in scratch instead of a workspace,
    for callers that cannot allocate device memory (see include/v4attn.h)."""
    n_q = int(q_pos.numel())
    a = IndexArgs(n_q, B if B is not None else n_q, _p(qI), _p(qI_sf), _p(w), _p(q_seq),
                  _p(q_pos), _p(keys), _p(keys_sf), key_rows, max_vis, _p(idx_out),
                  _p(scores_out), F32)
    _check("v4attn_index_topk_noalloc",
           _lib.v4attn_index_topk_noalloc(ctypes.byref(desc), ctypes.byref(a), _stream(stream)))


def noalloc_device_status(stream=None) -> int:
    """Raw status word of the last index_topk_noalloc call on this device
    (synchronises); raises on a device-side error."""
    bits = ctypes.c_uint32(0)
    st = _lib.v4attn_noalloc_device_status(_stream(stream), ctypes.byref(bits))
    _check("v4attn_noalloc_device_status", st)
    return bits.value


def debug_index_stall(desc: LayerDesc, *, qI, w, q_pos, keys, key_rows: int, max_vis: int, ws,
                      wait_ns: int, qI_sf=None, keys_sf=None, q_seq=None, B=None,
                      scores_out=None, idx_out=None, stream=None):
    """Failure-detection hook: index_topk with one wait of the tensor-core
    indexer made to run out after ``wait_ns`` (see include/v4attn.h)."""
    n_q = int(q_pos.numel())
    a = IndexArgs(n_q, B if B is not None else n_q, _p(qI), _p(qI_sf), _p(w), _p(q_seq),
                  _p(q_pos), _p(keys), _p(keys_sf), key_rows, max_vis, _p(idx_out),
                  _p(scores_out), F32)
    _check("v4attn_debug_index_stall",
           _lib.v4attn_debug_index_stall(ctypes.byref(desc), ctypes.byref(a), _p(ws), ws.numel(),
                                         int(wait_ns), _stream(stream)))


def tc_peak_probe(kind: int, n_iter: int, n_cols: int = 256, ws=None, stream=None):
    """Launch the tensor-core throughput probe (see include/v4attn.h);
    returns (dense FLOPs of the launch, CTAs)."""
    n = ctypes.c_int32(0)
    f = ctypes.c_double(0.0)
    _check("v4attn_tc_peak_probe",
           _lib.v4attn_tc_peak_probe(int(kind), int(n_cols), int(n_iter), ctypes.byref(n),
                                     ctypes.byref(f), _p(ws), _stream(stream)))
    return f.value, n.value


def device_status_code(ws, stream=None):
    """(status code, raw word) of a workspace, without raising."""
    bits = ctypes.c_uint32(0)
    st = _lib.v4attn_device_status(_p(ws), _stream(stream), ctypes.byref(bits))
    return st, bits.value


def workspace_init(ws, stream=None):
    _check("v4attn_workspace_init", _lib.v4attn_workspace_init(_p(ws), ws.numel(),
                                                                _stream(stream)))


def _mqa(fn, desc, Q, q_pos, kv, kv_rows, swa, swa_rows, out, ws, kv_scale, swa_scale, q_seq, B,
         idx, n_sel, max_vis, sink, lse, q_rmsnorm, stream, block_table=None):
    n_q = int(q_pos.numel())
    bt, bps = _bt(block_table)
    a = MqaArgs(n_q, B if B is not None else n_q, _p(Q), _dt(Q), int(q_rmsnorm), _p(q_seq),
                _p(q_pos), _p(kv), _p(kv_scale), kv_rows, _p(swa), _p(swa_scale), swa_rows,
                _p(idx), n_sel, max_vis, _p(sink), _p(out), _dt(out), _p(lse), bt, bps)
    _check(fn, getattr(_lib, fn)(ctypes.byref(desc), ctypes.byref(a), _p(ws), ws.numel(),
                                 _stream(stream)))


def sparse_mqa(desc: LayerDesc, *, Q, q_pos, kv, kv_rows: int, swa, swa_rows: int, idx, out, ws,
               kv_scale=None, swa_scale=None, q_seq=None, B=None, sink=None, lse=None,
               q_rmsnorm=False, block_table=None, stream=None):
    _mqa("v4attn_sparse_mqa", desc, Q, q_pos, kv, kv_rows, swa, swa_rows, out, ws, kv_scale,
         swa_scale, q_seq, B, idx, int(idx.shape[-1]), 0, sink, lse, q_rmsnorm, stream,
         block_table)


def dense_mqa(desc: LayerDesc, *, Q, q_pos, kv, kv_rows: int, swa, swa_rows: int, max_vis: int,
              out, ws, kv_scale=None, swa_scale=None, q_seq=None, B=None, sink=None, lse=None,
              q_rmsnorm=False, block_table=None, stream=None):
    _mqa("v4attn_dense_mqa", desc, Q, q_pos, kv, kv_rows, swa, swa_rows, out, ws, kv_scale,
         swa_scale, q_seq, B, None, 0, max_vis, sink, lse, q_rmsnorm, stream, block_table)


def decode(desc: LayerDesc, *, pos, x_main, tail, bias, kv, kv_rows: int, swa, swa_rows: int,
           Q, out, ws, max_vis: int, kv_scale=None, swa_scale=None, x_idx=None, itail=None,
           ibias=None, keys=None, keys_sf=None, key_rows: int = 0, qI=None, qI_sf=None, w=None,
           sink=None, lse=None, idx_out=None, block_table=None, stream=None):
    bt, bps = _bt(block_table)
    a = DecodeArgs(int(pos.numel()), _p(pos), _dt(x_main), _p(x_main), _p(tail), _p(bias),
                   _p(x_idx), _p(itail), _p(ibias), _p(kv), _p(kv_scale), kv_rows, _p(keys),
                   _p(keys_sf), key_rows, _p(swa), _p(swa_scale), swa_rows, _p(Q), _dt(Q),
                   _p(qI), _p(qI_sf), _p(w), _p(sink), _p(out), _dt(out), _p(lse), _p(idx_out),
                   max_vis, bt, bps)
    _check("v4attn_decode", _lib.v4attn_decode(ctypes.byref(desc), ctypes.byref(a), _p(ws),
                                               ws.numel(), _stream(stream)))


def project(X, W, Y, stream=None):
    """Y = X @ W for 2-D row-major views (leading-dimension strides allowed)."""
    M, K = X.shape
    K2, N = W.shape
    assert K == K2 and tuple(Y.shape) == (M, N)
    for t in (X, W, Y):
        assert t.stride(1) == 1
    a = ProjectArgs(M, N, K, _p(X), _dt(X), X.stride(0), _p(W), _dt(W), W.stride(0), _p(Y), _dt(Y),
                    Y.stride(0))
    _check("v4attn_project", _lib.v4attn_project(ctypes.byref(a), _stream(stream)))


# ---------------------------------------------------------------- 16-bit K/V layers
_KV_DTYPES = {torch.bfloat16: BF16, torch.float16: F16}
_KV_TORCH = {BF16: torch.bfloat16, F16: torch.float16}


def kv_desc(Hq: int, Hkv: int, d: int, *, dtype=torch.bfloat16, d_rope: Optional[int] = None,
            rope_theta: float = 160000.0, rope_halves: bool = False, softmax_scale: float = 0.0,
            n_win: int = 0) -> KvDesc:
    """An uncompressed layer: Hq query and Hkv K/V heads of d dims in ``dtype``
    (bfloat16 or float16), d_rope of them rotated (default: all); see "16-bit
    K/V layers" in include/v4attn.h."""
    if dtype not in _KV_DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    return KvDesc(Hq, Hkv, d, d if d_rope is None else d_rope, rope_theta, int(rope_halves),
                  softmax_scale, n_win, _KV_DTYPES[dtype])


def kv_workspace(desc: KvDesc, device="cuda") -> torch.Tensor:
    """A zero-status workspace for the calls on this layer, whatever their size."""
    n = _lib.v4attn_kv_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise V4AttnError("v4attn_kv_workspace_size", _abi.ERR_INVALID_ARG)
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    with torch.cuda.device(ws.device):
        _check("v4attn_workspace_init", _lib.v4attn_workspace_init(_p(ws), ws.numel(), _stream()))
    return ws


# A decode step's calls take a few microseconds on the GPU, so what checks and
# marshals their arguments asks each tensor for as little as it can.
def _kv_rows(name, t, shape, dtype, dev):
    """(pointer, token stride, head stride) of [T][H][d] rows; their last dim contiguous."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must be {shape} in {dtype} on cuda:{dev}, got "
                         f"{tuple(t.shape)} in {t.dtype} on {t.device}")
    tok, head, one = t.stride()
    T, H, d = shape
    if one != 1 and T:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    # a dimension of one element may have any stride: it is never taken
    return t.data_ptr(), tok if T > 1 else H * d, head if H > 1 else d


def _kv_small(name, t, shape, dtype, dev):
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on "
                         f"cuda:{dev}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


_I32, _I64, _F32 = torch.int32, torch.int64, torch.float32


def _kv_cache(d, Hkv, dtype, k_cache, v_cache, q_start, kv_len, block_table, ws):
    """Checked (device, B, pool and table fields) of a call on a 16-bit K/V layer."""
    dev = k_cache.get_device()
    pool, table = k_cache.shape, block_table.shape
    if len(pool) != 4 or len(table) != 2:
        raise ValueError("a cache is [n_blocks][Hkv][128][d], block_table [B][blocks_per_seq]")
    (n, H, rows, dims), (B, bps) = pool, table
    if (dev < 0 or v_cache.get_device() != dev or q_start.get_device() != dev
            or kv_len.get_device() != dev or block_table.get_device() != dev
            or ws.get_device() != dev):
        raise ValueError("k_cache, v_cache, q_start, kv_len, block_table and ws must live on one GPU")
    if not ws.is_contiguous():         # its bytes are counted from its shape
        raise ValueError("ws must be contiguous")
    if (H != Hkv or rows != 128 or dims != d or v_cache.shape != pool or k_cache.dtype is not dtype
            or v_cache.dtype is not dtype or not k_cache.is_contiguous()
            or not v_cache.is_contiguous()):
        raise ValueError(f"k_cache and v_cache must be contiguous [n_blocks][{Hkv}][128][{d}] in "
                         f"{dtype}, got {tuple(pool)} in {k_cache.dtype}, {tuple(v_cache.shape)} in "
                         f"{v_cache.dtype}")
    if (q_start.dtype is not _I32 or kv_len.dtype is not _I64 or block_table.dtype is not _I32
            or q_start.shape != (B + 1,) or kv_len.shape != (B,) or not q_start.is_contiguous()
            or not kv_len.is_contiguous() or not block_table.is_contiguous()):
        raise ValueError("q_start int32 [B + 1], kv_len int64 [B] and block_table int32 "
                         f"[B][blocks_per_seq] must be contiguous, got {tuple(q_start.shape)} in "
                         f"{q_start.dtype}, {tuple(kv_len.shape)} in {kv_len.dtype}, "
                         f"{tuple(table)} in {block_table.dtype}")
    return dev, B, (k_cache.data_ptr(), v_cache.data_ptr(), n, q_start.data_ptr(),
                    kv_len.data_ptr(), block_table.data_ptr(), bps)


_KV_CALLS = {fn: (_abi.packed_call(fn), fmt.pack) for fn, fmt in _abi.PACKED.items()}
# what torch.cuda asks, without its checks (1 us less a call); a torch without
# CUDA has neither, and imports this package all the same
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _kv_call(fn, desc, dev, ws, stream, *values):
    call, pack = _KV_CALLS[fn]
    if _current_device() != dev:       # on the tensors' device, whichever is current
        with torch.cuda.device(dev):
            return _kv_call(fn, desc, dev, ws, stream, *values)
    status = call(ctypes.addressof(desc), pack(*values), ws.data_ptr(), ws.nbytes,
                  _current_stream(dev) if stream is None else stream.cuda_stream)
    if status:
        raise V4AttnError(fn, status)


def kv_append(desc: KvDesc, *, k, v, k_cache, v_cache, q_start, kv_len, block_table, ws, q=None,
              q_out=None, stream=None):
    """Append new tokens to a paged K/V cache, K rotated to its position; with
    ``q`` also the queries, rotated into ``q_out`` (which may be ``q``).

    k, v [T][Hkv][d], q [T][Hq][d] (strided views allowed); k_cache, v_cache
    [n_blocks][Hkv][128][d]; q_start int32 [B + 1], kv_len int64 [B] (new tokens
    included), block_table int32 [B][blocks_per_seq]."""
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    d, Hkv, dtype, T = desc.d, desc.Hkv, _KV_TORCH.get(desc.dtype), k.shape[0]
    dev, B, cache = _kv_cache(d, Hkv, dtype, k_cache, v_cache, q_start, kv_len, block_table, ws)
    kv = (T, Hkv, d)
    if q is None:
        rows = (0, 0, 0, 0, 0, 0)
    else:
        qs = (T, desc.Hq, d)
        rows = (*_kv_rows("q", q, qs, dtype, dev), *_kv_rows("q_out", q_out, qs, dtype, dev))
    _kv_call("v4attn_kv_append", desc, dev, ws, stream, T, B, *_kv_rows("k", k, kv, dtype, dev),
             *_kv_rows("v", v, kv, dtype, dev), *rows, *cache)


def _kv_attention(fn, desc, q, k_cache, v_cache, q_start, kv_len, block_table, out, ws, lse, sink,
                  idx, n_local, stream):
    d, Hq, dtype, T = desc.d, desc.Hq, _KV_TORCH.get(desc.dtype), q.shape[0]
    dev, B, cache = _kv_cache(d, desc.Hkv, dtype, k_cache, v_cache, q_start, kv_len, block_table,
                              ws)
    rows = (T, Hq, d)
    n_lists, n_sel = 1, 0
    if idx is not None:
        if idx.dim() not in (2, 3):
            raise ValueError("idx must be [T][n_lists][n_sel] or [T][n_sel]")
        n_lists, n_sel = idx.shape[1] if idx.dim() == 3 else 1, idx.shape[-1]
        idx = _kv_small("idx", idx, (T, *idx.shape[1:]), _I32, dev)
    _kv_call(fn, desc, dev, ws, stream, T, B, *_kv_rows("q", q, rows, dtype, dev), *cache,
             idx or 0, n_lists, n_sel, n_local,
             0 if sink is None else _kv_small("sink", sink, (Hq,), _F32, dev),
             *_kv_rows("out", out, rows, dtype, dev),
             0 if lse is None else _kv_small("lse", lse, (T, Hq), _F32, dev))


def paged_attention(desc: KvDesc, *, q, k_cache, v_cache, q_start, kv_len, block_table, out, ws,
                    lse=None, sink=None, stream=None):
    """Attention of new tokens (decode steps, prefill chunks, or both in one
    batch) over a paged K/V cache; arguments as ``kv_append``, q and out
    [T][Hq][d], lse float32 [T][Hq], sink float32 [Hq]."""
    _kv_attention("v4attn_paged_attention", desc, q, k_cache, v_cache, q_start, kv_len,
                  block_table, out, ws, lse, sink, None, 0, stream)


def block_sparse_attention(desc: KvDesc, *, q, k_cache, v_cache, q_start, kv_len, block_table,
                           idx, n_local: int, out, ws, lse=None, sink=None, stream=None):
    """``paged_attention`` over the 128-token blocks selected for each query
    (idx int32 [T][n_lists][n_sel] or [T][n_sel]: ascending block ids, -1 behind
    them, e.g. from ``index_topk`` with m = 128; n_lists 1 or Hkv) and its last
    n_local blocks."""
    _kv_attention("v4attn_block_sparse_attention", desc, q, k_cache, v_cache, q_start, kv_len,
                  block_table, out, ws, lse, sink, idx, n_local, stream)


def device_status(ws, stream=None) -> int:
    """Synchronise and return the raw status word; raises on a device-side error."""
    bits = ctypes.c_uint32(0)
    st = _lib.v4attn_device_status(_p(ws), _stream(stream), ctypes.byref(bits))
    _check("v4attn_device_status", st)
    return bits.value


def build_info() -> str:
    return _lib.v4attn_build_info().decode()
