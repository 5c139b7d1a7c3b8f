"""Python binding of libstattn.so, the sm_100a spatial-temporal attention hot path.

Argument marshalling only: every step runs in the CUDA library.  Tensors are
torch CUDA tensors (PyTorch provides device memory and streams); the calls are
asynchronous on ``torch.cuda.current_stream()`` unless a stream is given.
Importing this module fails loudly when the library has not been built.

Entry points (same names as the C ABI in include/stattn.h):
    st_attn_spatial, st_attn_ring, st_attn_spatial_merge, st_attn_temporal, attn_chunk_merge, ulysses_relayout,
    ulysses_relayout_range, vmajor_mask_compact, vmajor_mask_compact_noalloc, vmajor_mask_compact_scatter,
    vmajor_scatter_rows, vmajor_workspace_bytes, vmajor_relayout_mask, vmajor_relayout_rows,
    st_rope_table, ulysses_relayout_rope,
    st_qk_norm_rope, st_attn_cross, st_attn_cross_workspace_bytes, st_attn_prefix, st_attn_prefix_workspace_bytes,
    st_check_device_status, st_status_string, st_set_sm_budget, st_get_sm_budget
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libstattn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m sequence_parallelism_st_b200.build` "
        "(there is no CPU fallback)")

lib = ctypes.CDLL(LIB_PATH)

# ---------------------------------------------------------------- C types
ST_OK, ST_ERR_NULL, ST_ERR_SHAPE, ST_ERR_DIVISIBILITY, ST_ERR_DTYPE = 0, -1, -2, -3, -4
ST_ERR_ALIGN, ST_ERR_UNSUPPORTED, ST_ERR_CUDA, ST_ERR_TIMEOUT = -5, -6, -7, -8
ST_F32, ST_BF16 = 0, 1
ST_S2T, ST_T2S, ST_SEQ2HEAD, ST_HEAD2SEQ = 0, 1, 2, 3
ST_ROPE_INTERLEAVED, ST_ROPE_HALVES = 0, 1
PAIRINGS = {"interleaved": ST_ROPE_INTERLEAVED, "halves": ST_ROPE_HALVES}
MODES = {"S2T": ST_S2T, "T2S": ST_T2S, "SEQ2HEAD": ST_SEQ2HEAD, "HEAD2SEQ": ST_HEAD2SEQ}

c_int, c_ll, c_float, c_void_p, c_size_t = (ctypes.c_int, ctypes.c_longlong, ctypes.c_float,
                                             ctypes.c_void_p, ctypes.c_size_t)


class st_attn_desc(ctypes.Structure):
    _fields_ = [("size", c_int), ("B", c_int), ("T", c_int), ("S", c_int), ("H", c_int), ("D", c_int),
                ("dtype", c_int), ("scale", c_float),
                ("stride_b", c_ll), ("stride_t", c_ll), ("stride_s", c_ll),
                ("t_block", c_int), ("stride_tb", c_ll), ("s_block", c_int), ("stride_sb", c_ll),
                ("n_slices", c_int), ("slice", c_int), ("kv_begin", c_int), ("kv_end", c_int),
                ("o_fp32", c_int)]


class st_qk_desc(ctypes.Structure):
    _fields_ = [("size", c_int), ("n_tokens", c_int), ("h_q", c_int), ("h_k", c_int), ("D", c_int),
                ("dtype", c_int), ("eps", c_float), ("pairing", c_int), ("pos_period", c_int),
                ("stride_q", c_ll), ("stride_k", c_ll), ("stride_q_out", c_ll), ("stride_k_out", c_ll)]


class st_kv_desc(ctypes.Structure):
    _fields_ = [("size", c_int), ("n_sets", c_int), ("L", c_int), ("H_kv", c_int), ("stride_set", c_ll),
                ("stride_l", c_ll), ("n_rows", c_ll), ("len", c_void_p), ("offsets", c_void_p), ("mask", c_void_p)]


def _proto(name, res, *args):
    f = getattr(lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_VP = c_void_p
_c = {
    "st_status_string": _proto("st_status_string", ctypes.c_char_p, c_int),
    "st_abi_version": _proto("st_abi_version", c_int),
    "st_attn_spatial": _proto("st_attn_spatial", c_int, ctypes.POINTER(st_attn_desc), _VP, _VP, _VP, _VP, _VP, _VP),
    "st_attn_temporal": _proto("st_attn_temporal", c_int, ctypes.POINTER(st_attn_desc), _VP, _VP, _VP, _VP, _VP, _VP),
    "st_attn_ring": _proto("st_attn_ring", c_int, ctypes.POINTER(st_attn_desc), _VP, _VP, _VP, _VP, _VP, c_int, _VP),
    "st_attn_spatial_merge": _proto("st_attn_spatial_merge", c_int, ctypes.POINTER(st_attn_desc), _VP, _VP, _VP,
                                    _VP, _VP, _VP, _VP, _VP),
    "attn_chunk_merge": _proto("attn_chunk_merge", c_int, c_int, ctypes.POINTER(_VP), ctypes.POINTER(_VP), c_ll,
                               c_int, c_int, c_int, _VP, c_int, _VP, _VP),
    "ulysses_relayout": _proto("ulysses_relayout", c_int, c_int, _VP, _VP, c_int, c_int, c_int, c_int, c_int,
                               c_int, c_int, c_int, c_int, c_int, c_int, c_int, _VP, c_int, c_float, _VP),
    "ulysses_relayout_range": _proto("ulysses_relayout_range", c_int, c_int, _VP, _VP, c_int, c_int, c_int, c_int,
                                     c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int, _VP,
                                     c_int, c_float, _VP),
    "vmajor_workspace_bytes": _proto("vmajor_workspace_bytes", c_size_t, c_ll),
    "vmajor_mask_compact": _proto("vmajor_mask_compact", c_int, _VP, _VP, c_ll, c_int, c_int, c_float, c_int,
                                  _VP, _VP, _VP, _VP, _VP, c_size_t, _VP),
    "vmajor_mask_compact_noalloc": _proto("vmajor_mask_compact_noalloc", c_int, _VP, _VP, c_ll, c_int, c_int,
                                          c_float, c_int, _VP, _VP, _VP, _VP, _VP),
    "vmajor_mask_compact_scatter": _proto("vmajor_mask_compact_scatter", c_int, _VP, _VP, c_ll, c_int, c_int,
                                          c_float, c_int, _VP, _VP, _VP, _VP, _VP, c_size_t,
                                          ctypes.POINTER(_VP), ctypes.POINTER(_VP), c_int, _VP),
    "vmajor_scatter_rows": _proto("vmajor_scatter_rows", c_int, _VP, _VP, c_ll, c_int, c_int,
                                  ctypes.POINTER(_VP), ctypes.POINTER(_VP), c_int, ctypes.POINTER(_VP), _VP),
    "st_check_device_status": _proto("st_check_device_status", c_int, _VP),
    "st_selftest_wait_timeout": _proto("st_selftest_wait_timeout", c_int, _VP),
    "st_selftest_ex2": _proto("st_selftest_ex2", c_int, _VP, _VP, _VP, c_int, _VP),
    "st_set_sm_budget": _proto("st_set_sm_budget", c_int, c_int),
    "vmajor_relayout_mask": _proto("vmajor_relayout_mask", c_int, _VP, _VP, _VP, c_int, c_int, c_int, c_int, c_int,
                                   c_int, c_int, c_int, c_float, c_int, _VP, _VP, _VP, _VP, _VP, c_size_t, _VP),
    "vmajor_relayout_rows": _proto("vmajor_relayout_rows", c_int, _VP, _VP, _VP, _VP, c_int, c_int, c_int, c_int,
                                   c_int, c_int, c_int, c_int, _VP, c_int, c_float, _VP, c_int, _VP),
    "st_rope_table": _proto("st_rope_table", c_int, c_int, c_int, c_float, _VP, _VP),
    "ulysses_relayout_rope": _proto("ulysses_relayout_rope", c_int, c_int, _VP, _VP, c_int, c_int, c_int, c_int,
                                    c_int, c_int, c_int, c_int, _VP, c_int, c_float, _VP, c_int, _VP),
    "st_get_sm_budget": _proto("st_get_sm_budget", c_int),
    "st_qk_norm_rope": _proto("st_qk_norm_rope", c_int, ctypes.POINTER(st_qk_desc), _VP, _VP, _VP, _VP, _VP, _VP, _VP,
                              c_int, _VP, _VP),
    "st_attn_cross": _proto("st_attn_cross", c_int, ctypes.POINTER(st_attn_desc), ctypes.POINTER(st_kv_desc), _VP, _VP,
                            _VP, _VP, _VP, _VP, c_size_t, _VP),
    "st_attn_cross_workspace_bytes": _proto("st_attn_cross_workspace_bytes", c_size_t, ctypes.POINTER(st_attn_desc),
                                            ctypes.POINTER(st_kv_desc)),
    "st_attn_prefix": _proto("st_attn_prefix", c_int, ctypes.POINTER(st_attn_desc), ctypes.POINTER(st_kv_desc),
                             ctypes.POINTER(st_kv_desc), _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, c_size_t, _VP),
    "st_attn_prefix_workspace_bytes": _proto("st_attn_prefix_workspace_bytes", c_size_t, ctypes.POINTER(st_attn_desc),
                                             ctypes.POINTER(st_kv_desc), ctypes.POINTER(st_kv_desc)),
}

EXPORTED = ["st_status_string", "st_abi_version", "st_attn_spatial", "st_attn_ring", "st_attn_spatial_merge",
            "st_attn_temporal",
            "attn_chunk_merge",
            "ulysses_relayout", "vmajor_workspace_bytes", "vmajor_mask_compact", "vmajor_mask_compact_noalloc",
            "vmajor_scatter_rows", "vmajor_mask_compact_scatter",
            "st_check_device_status", "st_selftest_wait_timeout", "ulysses_relayout_range", "st_set_sm_budget",
            "st_get_sm_budget", "vmajor_relayout_mask", "vmajor_relayout_rows", "st_rope_table",
            "ulysses_relayout_rope", "st_selftest_ex2", "st_qk_norm_rope", "st_attn_cross", "st_attn_cross_workspace_bytes",
            "st_attn_prefix", "st_attn_prefix_workspace_bytes"]


class StattnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {st_status_string(code)} ({code})")


def st_status_string(code: int) -> str:
    return _c["st_status_string"](int(code)).decode()


def _check(code: int, where: str) -> int:
    if code != ST_OK:
        raise StattnError(code, where)
    return code


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return ST_F32
    if t.dtype == torch.bfloat16:
        return ST_BF16
    raise StattnError(ST_ERR_DTYPE, f"dtype {t.dtype}")


def make_desc(B, T, S, H, D, dtype=ST_BF16, scale=0.0, stride_b=0, stride_t=0, stride_s=0, t_block=0,
              stride_tb=0, s_block=0, stride_sb=0, n_slices=1, slice=-1, kv_begin=0, kv_end=0,
              o_fp32=0) -> st_attn_desc:
    return st_attn_desc(ctypes.sizeof(st_attn_desc), B, T, S, H, D, dtype, scale, stride_b, stride_t,
                        stride_s, t_block, stride_tb, s_block, stride_sb, n_slices, slice, kv_begin, kv_end,
                        o_fp32)


# ---------------------------------------------------------------- attention
def st_attn_spatial(q, k, v, o, lse=None, *, desc: st_attn_desc | None = None, stream=None, raw=False, **kw):
    """Spatial attention per (b, t, head) over the S tokens of each frame.

    q, k, v, o: CUDA tensors; with no ``desc`` they are [B, T, S, H, D]
    contiguous and the descriptor is derived from their shape (keyword
    arguments override its fields).  Returns the status code when ``raw``.
    """
    if desc is None:
        B, T, S, H, D = q.shape
        desc = make_desc(B, T, S, H, D, _dtype_code(q), **kw)
    r = _c["st_attn_spatial"](ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _stream(stream))
    return r if raw else _check(r, "st_attn_spatial")


def st_attn_ring(q, k, v, o, lse=None, n_chunks=1, *, desc: st_attn_desc | None = None, stream=None, raw=False,
                 **kw):
    """Full attention over ``n_chunks`` KV ring chunks in one launch: each query
    block starts at the chunk holding its first row and carries its running
    statistics across the chunks (include/stattn.h)."""
    if desc is None:
        B, T, S, H, D = q.shape
        desc = make_desc(B, T, S, H, D, _dtype_code(q), **kw)
    r = _c["st_attn_ring"](ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), int(n_chunks),
                           _stream(stream))
    return r if raw else _check(r, "st_attn_ring")


def st_attn_spatial_merge(q, k, v, o_acc, lse_acc, o, lse=None, *, desc: st_attn_desc | None = None, stream=None,
                          raw=False, **kw):
    """Spatial attention over one KV chunk merged into the accumulated fp32
    partial ``o_acc`` and its LSE ``lse_acc``; ``o`` may be ``o_acc`` when the
    result is fp32 (``o_fp32=1``)."""
    if desc is None:
        B, T, S, H, D = q.shape
        desc = make_desc(B, T, S, H, D, _dtype_code(q), **kw)
    r = _c["st_attn_spatial_merge"](ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o_acc), _ptr(lse_acc),
                                    _ptr(o), _ptr(lse), _stream(stream))
    return r if raw else _check(r, "st_attn_spatial_merge")


def st_attn_temporal(q, k, v, o, lse=None, *, desc: st_attn_desc | None = None, stream=None, raw=False, **kw):
    """Temporal attention per (b, s, head) over the T frames of each token."""
    if desc is None:
        B, T, S, H, D = q.shape
        desc = make_desc(B, T, S, H, D, _dtype_code(q), **kw)
    r = _c["st_attn_temporal"](ctypes.byref(desc), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _stream(stream))
    return r if raw else _check(r, "st_attn_temporal")


def attn_chunk_merge(o_parts, lse_parts, n_units, S, H, D, o_out, lse_out=None, *, stream=None, raw=False):
    """Log-sum-exp merge of fp32 KV-chunk partials into o_out (bf16 or fp32)."""
    n = len(o_parts)
    op = (c_void_p * n)(*[t.data_ptr() for t in o_parts])
    lp = (c_void_p * n)(*[t.data_ptr() for t in lse_parts])
    r = _c["attn_chunk_merge"](n, op, lp, int(n_units), int(S), int(H), int(D), _ptr(o_out), _dtype_code(o_out),
                               _ptr(lse_out), _stream(stream))
    return r if raw else _check(r, "attn_chunk_merge")


# ---------------------------------------------------------------- relayout
def ulysses_relayout(mode, inp, out, P, B, T_or_N, S_or_H, C_or_D, n_t=1, n_s=1, blocks=None, rms_gamma=None,
                     rms_head_dim=0, rms_eps=1e-6, *, stream=None, raw=False):
    """All-to-all on a virtual partition of P shards (see include/stattn.h)."""
    m = MODES[mode] if isinstance(mode, str) else int(mode)
    i0, i1, j0, j1 = blocks if blocks is not None else (0, n_t, 0, n_s)
    r = _c["ulysses_relayout"](m, _ptr(inp), _ptr(out), inp.element_size(), P, B, T_or_N, S_or_H, C_or_D,
                               n_t, n_s, i0, i1, j0, j1, _ptr(rms_gamma), int(rms_head_dim), float(rms_eps),
                               _stream(stream))
    return r if raw else _check(r, "ulysses_relayout")


def ulysses_relayout_range(mode, inp, out, P, B, T_or_N, S_or_H, C_or_D, n_t=1, n_s=1, blocks=None, shards=None,
                           rms_gamma=None, rms_head_dim=0, rms_eps=1e-6, *, stream=None, raw=False):
    """ulysses_relayout restricted to the temporally sharded shards ``shards`` = (q0, q1)."""
    m = MODES[mode] if isinstance(mode, str) else int(mode)
    i0, i1, j0, j1 = blocks if blocks is not None else (0, n_t, 0, n_s)
    q0, q1 = shards if shards is not None else (0, P)
    r = _c["ulysses_relayout_range"](m, _ptr(inp), _ptr(out), inp.element_size(), P, B, T_or_N, S_or_H, C_or_D,
                                     n_t, n_s, i0, i1, j0, j1, q0, q1, _ptr(rms_gamma), int(rms_head_dim),
                                     float(rms_eps), _stream(stream))
    return r if raw else _check(r, "ulysses_relayout_range")


# ---------------------------------------------------------------- V-Major
def vmajor_workspace_bytes(n_tokens: int) -> int:
    return int(_c["vmajor_workspace_bytes"](int(n_tokens)))


def vmajor_mask_compact(v_cur, v_prev, tau, mask, idx, count, workspace, force_all=False, l1_out=None, *,
                        stream=None, raw=False):
    """Per-token L1 change mask and ascending compaction of active tokens."""
    n, C = v_cur.shape[0], v_cur[0].numel()
    r = _c["vmajor_mask_compact"](_ptr(v_cur), _ptr(v_prev), n, C, _dtype_code(v_cur), float(tau),
                                  1 if force_all else 0, _ptr(mask), _ptr(idx), _ptr(count), _ptr(l1_out),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    return r if raw else _check(r, "vmajor_mask_compact")


def vmajor_mask_compact_noalloc(v_cur, v_prev, tau, mask, idx, count, force_all=False, l1_out=None, *,
                                stream=None, raw=False):
    """vmajor_mask_compact with the library's own static scratch (no workspace, no allocation)."""
    n, C = v_cur.shape[0], v_cur[0].numel()
    r = _c["vmajor_mask_compact_noalloc"](_ptr(v_cur), _ptr(v_prev), n, C, _dtype_code(v_cur), float(tau),
                                          1 if force_all else 0, _ptr(mask), _ptr(idx), _ptr(count),
                                          _ptr(l1_out), _stream(stream))
    return r if raw else _check(r, "vmajor_mask_compact_noalloc")


def vmajor_mask_compact_scatter(v_cur, v_prev, tau, mask, idx, count, workspace, src, dst_cache, force_all=False,
                                l1_out=None, *, stream=None, raw=False):
    """vmajor_mask_compact and the cache update of the active tokens' rows in one call."""
    n, C = v_cur.shape[0], v_cur[0].numel()
    nt = len(src)
    sp = (c_void_p * nt)(*[t.data_ptr() for t in src])
    dp = (c_void_p * nt)(*[t.data_ptr() for t in dst_cache])
    r = _c["vmajor_mask_compact_scatter"](_ptr(v_cur), _ptr(v_prev), n, C, _dtype_code(v_cur), float(tau),
                                          1 if force_all else 0, _ptr(mask), _ptr(idx), _ptr(count), _ptr(l1_out),
                                          _ptr(workspace), workspace.numel() * workspace.element_size(), sp, dp, nt,
                                          _stream(stream))
    return r if raw else _check(r, "vmajor_mask_compact_scatter")


def vmajor_scatter_rows(idx, count, src, dst_cache, packed=None, *, stream=None, raw=False):
    """cache[idx[i]] <- src[idx[i]] for i < count (and the packed message)."""
    n = len(src)
    n_tok, C = src[0].shape[0], src[0][0].numel()
    sp = (c_void_p * n)(*[t.data_ptr() for t in src])
    dp = (c_void_p * n)(*[t.data_ptr() for t in dst_cache])
    pp = (c_void_p * n)(*[t.data_ptr() for t in packed]) if packed is not None else None
    r = _c["vmajor_scatter_rows"](_ptr(idx), _ptr(count), n_tok, C, src[0].element_size(), sp, dp, n, pp,
                                  _stream(stream))
    return r if raw else _check(r, "vmajor_scatter_rows")


def vmajor_relayout_mask(v_cur_x, v_prev_x, v_cache_y, P, B, T, S, C, n_t, n_s, tau, mask, idx, count, workspace,
                         force_all=False, l1_out=None, *, stream=None, raw=False):
    """Sender-side V-Major: mask of the L1 change of V on the x layout, rows of active
    tokens moved S->T into the V cache; mask/idx/count in y numbering."""
    r = _c["vmajor_relayout_mask"](_ptr(v_cur_x), _ptr(v_prev_x), _ptr(v_cache_y), P, B, T, S, C, n_t, n_s,
                                   _dtype_code(v_cur_x), float(tau), 1 if force_all else 0, _ptr(mask), _ptr(idx),
                                   _ptr(count), _ptr(l1_out), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream))
    return r if raw else _check(r, "vmajor_relayout_mask")


def vmajor_relayout_rows(in_x, out_y, idx, count, P, B, T, S, C, n_t, n_s, rms_gamma=None, rms_head_dim=0,
                         rms_eps=1e-6, rope_table=None, *, stream=None, raw=False):
    """S->T move of the destination rows idx[:count] (device), with the optional per-head RMSNorm
    and rotary embedding (rope_table from st_rope_table)."""
    n_pos = rope_table.shape[0] if rope_table is not None else 0
    r = _c["vmajor_relayout_rows"](_ptr(in_x), _ptr(out_y), _ptr(idx), _ptr(count), P, B, T, S, C, n_t, n_s,
                                   _dtype_code(in_x), _ptr(rms_gamma), int(rms_head_dim), float(rms_eps),
                                   _ptr(rope_table), n_pos, _stream(stream))
    return r if raw else _check(r, "vmajor_relayout_rows")


def st_rope_table(n_pos, head_dim, theta=10000.0, *, device="cuda", stream=None):
    """Rotary (cos, sin) table, fp32 [n_pos, head_dim // 2, 2], computed on the device."""
    import torch
    t = torch.empty((n_pos, head_dim // 2, 2), dtype=torch.float32, device=device)
    _check(_c["st_rope_table"](int(n_pos), int(head_dim), float(theta), _ptr(t), _stream(stream)), "st_rope_table")
    return t


def ulysses_relayout_rope(mode, inp, out, P, B, T_or_N, S_or_H, C_or_D, n_t=1, n_s=1, rms_gamma=None,
                          rms_head_dim=0, rms_eps=1e-6, rope_table=None, *, stream=None, raw=False):
    """ulysses_relayout (S2T / SEQ2HEAD) with the per-head RMSNorm and the rotary embedding."""
    m = MODES[mode] if isinstance(mode, str) else int(mode)
    n_pos = rope_table.shape[0] if rope_table is not None else 0
    r = _c["ulysses_relayout_rope"](m, _ptr(inp), _ptr(out), inp.element_size(), P, B, T_or_N, S_or_H, C_or_D, n_t,
                                    n_s, _ptr(rms_gamma), int(rms_head_dim), float(rms_eps), _ptr(rope_table), n_pos,
                                    _stream(stream))
    return r if raw else _check(r, "ulysses_relayout_rope")


# ---------------------------------------------------------------- conditioning
def _on_gpu(where, device):
    if device.type != "cuda":
        raise StattnError(ST_ERR_NULL, f"{where}: tensors must be on a CUDA device")


def _device_call(where, fn, device, stream, *args):
    """fn(*args, stream) with ``device`` current, on ``stream`` or the device's current stream."""
    import torch
    _on_gpu(where, device)
    # (the raw handle: a Stream object costs 3 us a call)
    s = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else _stream(stream)
    if device.index == torch.cuda.current_device():
        return fn(*args, s)
    with torch.cuda.device(device):
        return fn(*args, s)


def _addr(t):
    return None if t is None else t.data_ptr()


# The checks below run on every call and build their messages only when they fail.
def _same_device(where, index, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise StattnError(ST_ERR_SHAPE, f"{where}: tensors on different devices")


def _int32(where, t, n, index):
    """Pointer of an optional contiguous int32 tensor of n elements."""
    if t is None:
        return None
    import torch
    if t.dtype != torch.int32:
        raise StattnError(ST_ERR_DTYPE, f"{where}: lengths, offsets and positions are int32")
    if t.numel() != n or not t.is_contiguous() or t.get_device() != index:
        raise StattnError(ST_ERR_SHAPE, f"{where}: {n} contiguous int32 on the tensors' device expected")
    return t.data_ptr()


def _rows(where, t):
    """(tokens, H, D, elements between tokens) of a [..., H, D] tensor whose tokens have one stride."""
    size, stride = t.shape, t.stride()
    if len(size) < 3:
        raise StattnError(ST_ERR_SHAPE, f"{where}: [..., H, D] expected")
    H, D = size[-2], size[-1]
    if (D != 1 and stride[-1] != 1) or (H != 1 and stride[-2] != D):
        raise StattnError(ST_ERR_SHAPE, f"{where}: heads must be dense")
    n, step = 1, 0
    for i in range(len(size) - 3, -1, -1):
        if size[i] == 1:
            continue
        if n == 1:
            step = stride[i]
            if step <= 0:
                raise StattnError(ST_ERR_SHAPE, f"{where}: expanded tensors are not taken")
        elif stride[i] != n * step:
            raise StattnError(ST_ERR_SHAPE, f"{where}: tokens must have one stride")
        n *= size[i]
    return n, H, D, step


def st_qk_norm_rope(q, k=None, q_out=None, k_out=None, q_gamma=None, k_gamma=None, eps=1e-6, *, rope_table=None,
                    positions=None, pos_period=0, pairing="interleaved", stream=None, raw=False):
    """Per-head RMSNorm of Q and K and their rotary embedding in one pass (include/stattn.h).

    q, k: [..., H, D] with one stride between tokens (views of a fused projection
    included); either may be None.  Outputs default to in place."""
    import torch
    where = "st_qk_norm_rope"
    x = q if q is not None else k
    if x is None:
        raise StattnError(ST_ERR_NULL, f"{where}: q or k")
    d = st_qk_desc(size=ctypes.sizeof(st_qk_desc), dtype=_dtype_code(x), eps=float(eps), pos_period=int(pos_period),
                   pairing=PAIRINGS[pairing] if isinstance(pairing, str) else int(pairing))
    index, dtype = x.get_device(), x.dtype
    tokens = head_dim = None
    for name, t, out, gamma in (("q", q, q_out, q_gamma), ("k", k, k_out, k_gamma)):
        if t is None:
            if out is not None:
                raise StattnError(ST_ERR_NULL, f"{where}: {name}_out without {name}")
            continue
        n, H, D, step = _rows(where, t)
        if tokens is not None and (n != tokens or D != head_dim):
            raise StattnError(ST_ERR_SHAPE, f"{where}: q and k differ in tokens or D")
        tokens, head_dim, out_step = n, D, step
        if out is not None:
            if out.shape != t.shape:
                raise StattnError(ST_ERR_SHAPE, f"{where}: {name}_out has another shape")
            out_step = _rows(where, out)[3]
        if name == "q":
            d.h_q, d.stride_q, d.stride_q_out = H, step, out_step
        else:
            d.h_k, d.stride_k, d.stride_k_out = H, step, out_step
        _same_device(where, index, t, out, gamma)
        if t.dtype != dtype or (out is not None and out.dtype != dtype):
            raise StattnError(ST_ERR_DTYPE, f"{where}: one dtype for q, k and the outputs")
        if gamma is not None and (gamma.dtype != torch.float32 or gamma.numel() != D or not gamma.is_contiguous()):
            raise StattnError(ST_ERR_SHAPE, f"{where}: {name}_gamma is fp32 [D]")
    d.n_tokens, d.D = tokens, head_dim
    n_pos = 0
    if rope_table is not None:
        _same_device(where, index, rope_table)
        n_pos = rope_table.shape[0]
        if rope_table.dtype != torch.float32 or not rope_table.is_contiguous() or rope_table.numel() != n_pos * head_dim:
            raise StattnError(ST_ERR_SHAPE, f"{where}: rope_table is fp32 [n, D / 2, 2]")
    pos = _int32(where, positions, tokens, index)
    r = _device_call(where, _c["st_qk_norm_rope"], x.device, stream, ctypes.byref(d), _addr(q), _addr(k),
                     _addr(q if q_out is None else q_out), _addr(k if k_out is None else k_out), _addr(q_gamma),
                     _addr(k_gamma), _addr(rope_table), n_pos, pos)
    return r if raw else _check(r, where)


def _q_desc(where, q, o, kw):
    """Descriptor of Q and O [B, T, S, H, D], strides taken from the tensors."""
    size, st = q.shape, q.stride()
    if len(size) != 5:
        raise StattnError(ST_ERR_SHAPE, f"{where}: q is [B, T, S, H, D]")
    B, T, S, H, D = size
    if (D != 1 and st[4] != 1) or (H != 1 and st[3] != D) or (o is not None and o.shape != size):
        raise StattnError(ST_ERR_SHAPE, f"{where}: q and o are [B, T, S, H, D] with dense heads")
    so = st if o is None else o.stride()
    if so != st and ((D != 1 and so[4] != 1) or (H != 1 and so[3] != D)):
        raise StattnError(ST_ERR_SHAPE, f"{where}: q and o are [B, T, S, H, D] with dense heads")
    for i in range(3):
        if size[i] != 1 and (st[i] <= 0 or so[i] != st[i]):
            raise StattnError(ST_ERR_SHAPE, f"{where}: q and o need the same strides")
    sb, stt, ss = (st[i] if size[i] > 1 else 0 for i in range(3))
    if T > 1 and stt == S * (ss or H * D):
        stt = 0                                 # dense frames
    return make_desc(B, T, S, H, D, _dtype_code(q), stride_b=sb, stride_t=stt, stride_s=ss, **kw)


def _kv_desc(where, head_dim, q, k, v, length, offsets, mask, max_len):
    """st_kv_desc of K (and V) [n_sets, L, H_kv, D], or packed [rows, H_kv, D] with offsets."""
    packed = offsets is not None
    size, st = k.shape, k.stride()
    if len(size) != (3 if packed else 4):
        raise StattnError(ST_ERR_SHAPE, f"{where}: keys are [n_sets, L, H_kv, D], or [rows, H_kv, D] with offsets")
    L, H, D = size[-3:]
    if D != head_dim or (D != 1 and st[-1] != 1) or (H != 1 and st[-2] != D):
        raise StattnError(ST_ERR_SHAPE, f"{where}: keys need q's head dim and dense heads")
    if k.dtype != q.dtype or (v is not None and v.dtype != k.dtype):
        raise StattnError(ST_ERR_DTYPE, f"{where}: one dtype for q, k and v")
    if v is not None:
        sv = v.stride()
        if v.shape != size or (sv != st and any(n != 1 and a != b for n, a, b in zip(size, st, sv))):
            raise StattnError(ST_ERR_SHAPE, f"{where}: k and v need the same shape and strides")
    index = q.get_device()
    _same_device(where, index, k, v, length, offsets, mask)
    if L > 1 and st[-3] <= 0:
        raise StattnError(ST_ERR_SHAPE, f"{where}: expanded tensors are not taken")
    d = st_kv_desc(size=ctypes.sizeof(st_kv_desc), L=L, H_kv=H, stride_l=st[-3] if L > 1 else 0)
    if packed:
        if length is not None or mask is not None:
            raise StattnError(ST_ERR_SHAPE, f"{where}: offsets exclude lengths and mask")
        d.n_sets, d.n_rows = offsets.numel() - 1, L
        d.L = max(L, 1) if max_len is None else int(max_len)     # (no rows at all: sets without keys)
        d.offsets = _int32(where, offsets, d.n_sets + 1, index)
        return d
    n = size[0]
    d.n_sets = n
    if n > 1:
        if st[0] <= 0:
            raise StattnError(ST_ERR_SHAPE, f"{where}: expanded tensors are not taken")
        d.stride_set = st[0]
    if length is not None:
        d.len = _int32(where, length, n, index)
    if mask is not None:
        import torch
        if mask.dtype not in (torch.uint8, torch.bool):
            raise StattnError(ST_ERR_DTYPE, f"{where}: the mask is uint8 or bool")
        if mask.shape != size[:2] or not mask.is_contiguous():
            raise StattnError(ST_ERR_SHAPE, f"{where}: the mask is [n_sets, L]")
        d.mask = mask.data_ptr()
    return d


def _workspace(where, t, device):
    if t is None or t.numel() == 0:
        return None, 0
    if t.device != device or not t.is_contiguous():
        raise StattnError(ST_ERR_SHAPE, f"{where}: workspace")
    return _addr(t), t.numel() * t.element_size()


def _check_out(where, q, o, lse, o_fp32):
    import torch
    if o.dtype != (torch.float32 if o_fp32 else q.dtype):
        raise StattnError(ST_ERR_DTYPE, f"{where}: o's dtype")
    _same_device(where, q.get_device(), o, lse)
    if lse is not None:
        B, T, S, H, _ = q.shape
        if lse.dtype != torch.float32 or not lse.is_contiguous() or lse.numel() != B * T * H * S:
            raise StattnError(ST_ERR_SHAPE, f"{where}: lse is fp32 [B, T, H, S]")


def st_attn_cross(q, k, v, o, lse=None, *, kv_len=None, kv_offsets=None, kv_mask=None, max_len=None, workspace=None,
                  desc: st_attn_desc | None = None, stream=None, raw=False, **kw):
    """Cross attention of Q [B, T, S, H, D] to K, V [n_sets, L, H_kv, D] (include/stattn.h).

    With ``kv_offsets`` [n_sets + 1], K and V are packed [rows, H_kv, D], at most
    ``max_len`` rows of a set counted.  Strides come from the tensors (Q and O
    alike); ``desc`` overrides Q's.  ``workspace``: st_attn_cross_workspace_bytes
    bytes."""
    if desc is None:
        desc = _q_desc("st_attn_cross", q, o, kw)
        _check_out("st_attn_cross", q, o, lse, desc.o_fp32)
    kv = _kv_desc("st_attn_cross", desc.D, q, k, v, kv_len, kv_offsets, kv_mask, max_len)
    ws, n = _workspace("st_attn_cross", workspace, q.device)
    r = _device_call("st_attn_cross", _c["st_attn_cross"], q.device, stream, ctypes.byref(desc), ctypes.byref(kv),
                     _addr(q), _addr(k), _addr(v), _addr(o), _addr(lse), ws, n)
    return r if raw else _check(r, "st_attn_cross")


def st_attn_cross_workspace_bytes(q, k, *, kv_len=None, kv_offsets=None, kv_mask=None, max_len=None,
                                  desc: st_attn_desc | None = None, **kw) -> int:
    """Bytes of workspace st_attn_cross asks for with these arguments (0: none)."""
    desc = desc if desc is not None else _q_desc("st_attn_cross_workspace_bytes", q, None, kw)
    kv = _kv_desc("st_attn_cross_workspace_bytes", desc.D, q, k, None, kv_len, kv_offsets, kv_mask, max_len)
    _on_gpu("st_attn_cross_workspace_bytes", q.device)
    import torch
    with torch.cuda.device(q.device):
        return int(_c["st_attn_cross_workspace_bytes"](ctypes.byref(desc), ctypes.byref(kv)))


def st_attn_prefix(q, k_prefix, v_prefix, k, v, o, lse=None, *, prefix_len=None, prefix_offsets=None,
                   prefix_mask=None, prefix_max_len=None, kv_len=None, kv_offsets=None, kv_mask=None, max_len=None,
                   workspace=None, desc: st_attn_desc | None = None, stream=None, raw=False, **kw):
    """Attention of Q [B, T, S, H, D] over a prefix shared by several batches, then the batch's own keys
    (include/stattn.h).  Arguments as st_attn_cross, once for the prefix and once for the own keys."""
    if desc is None:
        desc = _q_desc("st_attn_prefix", q, o, kw)
        _check_out("st_attn_prefix", q, o, lse, desc.o_fp32)
    pre = _kv_desc("st_attn_prefix", desc.D, q, k_prefix, v_prefix, prefix_len, prefix_offsets, prefix_mask, prefix_max_len)
    kv = _kv_desc("st_attn_prefix", desc.D, q, k, v, kv_len, kv_offsets, kv_mask, max_len)
    ws, n = _workspace("st_attn_prefix", workspace, q.device)
    r = _device_call("st_attn_prefix", _c["st_attn_prefix"], q.device, stream, ctypes.byref(desc), ctypes.byref(pre),
                     ctypes.byref(kv), _addr(q), _addr(k_prefix), _addr(v_prefix), _addr(k), _addr(v), _addr(o), _addr(lse),
                     ws, n)
    return r if raw else _check(r, "st_attn_prefix")


def st_attn_prefix_workspace_bytes(q, k_prefix, k, *, prefix_len=None, prefix_offsets=None, prefix_mask=None,
                                   prefix_max_len=None, kv_len=None, kv_offsets=None, kv_mask=None, max_len=None,
                                   desc: st_attn_desc | None = None, **kw) -> int:
    """Bytes of workspace st_attn_prefix asks for with these arguments (0: none)."""
    where = "st_attn_prefix_workspace_bytes"
    desc = desc if desc is not None else _q_desc(where, q, None, kw)
    pre = _kv_desc(where, desc.D, q, k_prefix, None, prefix_len, prefix_offsets, prefix_mask, prefix_max_len)
    kv = _kv_desc(where, desc.D, q, k, None, kv_len, kv_offsets, kv_mask, max_len)
    _on_gpu(where, q.device)
    import torch
    with torch.cuda.device(q.device):
        return int(_c["st_attn_prefix_workspace_bytes"](ctypes.byref(desc), ctypes.byref(pre), ctypes.byref(kv)))


def st_check_device_status(stream=None) -> int:
    return int(_c["st_check_device_status"](_stream(stream)))


def st_set_sm_budget(sms: int) -> None:
    """Size the grids of this thread's later launches for at most ``sms`` SMs (0: all)."""
    _check(_c["st_set_sm_budget"](int(sms)), "st_set_sm_budget")


def st_get_sm_budget() -> int:
    return int(_c["st_get_sm_budget"]())


def st_selftest_wait_timeout(stream=None) -> int:
    return int(_c["st_selftest_wait_timeout"](_stream(stream)))


def st_selftest_ex2(x, y_poly, y_mufu, *, stream=None, raw=False):
    """The softmax's two exp2 implementations evaluated on the fp32 device tensor x."""
    r = _c["st_selftest_ex2"](_ptr(x), _ptr(y_poly), _ptr(y_mufu), int(x.numel()), _stream(stream))
    return r if raw else _check(r, "st_selftest_ex2")
