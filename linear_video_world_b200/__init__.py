"""Python binding of the B200 Hybrid Linear Temporal Attention library (libhlta.so).

Argument marshalling only: every function passes device pointers, sizes and the current
CUDA stream to the C ABI declared in include/hlta.h, and raises ``HltaError`` on a non-OK
status. Tensors are torch tensors on a CUDA device (torch provides memory and streams);
no computation happens here, and there is no fallback: if the compiled library is missing,
importing this package fails.

Function names match the C entry points (``hlta_swa_fwd`` ...). The convenience wrappers
at the end (``swa``, ``dswa``, ``gdn``, ``hybrid``, ``Stream``) allocate outputs and
workspaces with torch and then call those same entry points.
"""
from __future__ import annotations

import ctypes
import functools
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhlta.so")

HLTA_OK, HLTA_ERR_INVALID_ARG, HLTA_ERR_UNSUPPORTED, HLTA_ERR_CUDA, HLTA_ERR_TIMEOUT = range(5)
HLTA_BF16, HLTA_FP32 = 0, 1
HLTA_DEVERR_ATTN_WAIT, HLTA_DEVERR_GDN_WAIT, HLTA_DEVERR_SELFTEST = 0x1, 0x2, 0x4
HLTA_DEVERR_TABLE = 0x8
_STATUS = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "CUDA", 4: "TIMEOUT"}


class HltaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"HLTA_ERR_{_STATUS.get(status, status)}: {msg}")
        self.status = status


class hlta_rope_axes_t(ctypes.Structure):
    """The rotation of hlta_rope_axes and hlta_paged_append (include/hlta.h)."""
    _fields_ = [("pairs", ctypes.c_int * 3), ("layout", ctypes.c_int),
                ("shared_freq", ctypes.c_int), ("grid_h", ctypes.c_int),
                ("grid_w", ctypes.c_int), ("base", ctypes.c_float),
                ("pos", ctypes.c_void_p), ("t0", ctypes.c_void_p)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python linear_video_world_b200/build.py` (nvcc, sm_100a)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, L, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_float, ctypes.c_size_t
    sig = {
        "hlta_version": (I, []),
        "hlta_last_error": (ctypes.c_char_p, []),
        "hlta_swa_fwd": (I, [P, P, P, P, I, I, I, I, I, I, F, I, P]),
        "hlta_dswa_fwd": (I, [P, P, P, P, I, I, I, I, I, I, I, F, I, P]),
        "hlta_gdn_workspace_bytes": (Z, [I, I, L, I, I, I]),
        "hlta_gdn_chunk_fwd": (I, [P, P, P, P, P, P, P, P, I, I, L, I, I, P, Z, I, P]),
        "hlta_gdn_chunk_fwd_raw": (I, [P, P, P, P, P, F, P, P, P, I, I, L, I, I, P, Z, I, P]),
        "hlta_gdn_chunk_fwd_static": (I, [P, P, P, P, P, P, P, P, I, I, L, I, I, I, P]),
        "hlta_hybrid_workspace_bytes": (Z, [I, I, I, I, I, I, I]),
        "hlta_hybrid_fwd": (I, [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, I, F,
                                P, Z, I, P]),
        "hlta_hybrid_fwd_raw": (I, [P, P, P, P, P, F, P, P, P, I, I, I, I, I, I, I, I, I, I, I,
                                    F, P, Z, I, P]),
        "hlta_stream_create": (I, [ctypes.POINTER(P), I, I, I, I, I, I, I, I, I, I, F, I, P]),
        "hlta_stream_create_ex": (I, [ctypes.POINTER(P), I, I, I, I, I, I, I, I, I, I, F, I, I, P]),
        "hlta_stream_step": (I, [P, P, P, P, P, P, P, P]),
        "hlta_stream_step_frames": (I, [P, P, P, P, P, P, P, I, P]),
        "hlta_stream_state": (I, [P, ctypes.POINTER(P), ctypes.POINTER(I)]),
        "hlta_stream_destroy": (I, [P]),
        "hlta_stream_frame_counter": (I, [P, ctypes.POINTER(P)]),
        "hlta_stream_checkpoint_bytes": (Z, [P]),
        "hlta_stream_save": (I, [P, P, Z, P]),
        "hlta_stream_load": (I, [P, P, Z, P]),
        "hlta_rope": (I, [P, P, I, I, I, I, L, I, I, F, I, I, I, P]),
        "hlta_fp8_quantize_rows": (I, [P, P, I, I, L, I, L, I, P, P, P]),
        "hlta_fp8_quantize_channels": (I, [P, I, I, L, I, P, P, P]),
        "hlta_window_fp8_fwd": (I, [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P]),
        "hlta_window_fwd_lse": (I, [P, P, P, P, P, I, I, I, I, I, I, I, F, P]),
        "hlta_window_bwd_workspace_bytes": (Z, [I, I, I, I]),
        "hlta_window_bwd": (I, [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, P, Z, P]),
        "hlta_gdn_bwd_workspace_bytes": (Z, [I, I, L, I, I]),
        "hlta_gdn_chunk_bwd": (I, [P, P, P, P, P, P, P, P, P, P, P, P, P, P, I, I, L, I, I, P, Z, I,
                                   P]),
        "hlta_rope_axes": (I, [P, P, P, P, I, I, I, L, I, P, I, I, P]),
        "hlta_paged_append": (I, [P, P, P, P, P, P, P, I, I, L, I, L, I, I, P, I, P]),
        "hlta_paged_attn_workspace_bytes": (Z, [I, I, I, L, I, I, I, I, I]),
        "hlta_paged_attn_fwd": (I, [P] * 10 + [F, I, I, I, L, I, L, I, I, I, I, F, P, Z, I, P]),
        "hlta_paged_evict_workspace_bytes": (Z, [I, I, I]),
        "hlta_paged_evict": (I, [P] * 5 + [I, I, I, L, I, I, I, I, I, P, P, P, L, I, P, P, P, P, Z,
                                 I, P]),
        "hlta_gdn_step": (I, [P] * 10 + [I, I, L, I, L, I, P]),
        "hlta_gdn_step_raw": (I, [P] * 5 + [F] + [P] * 5 + [I, I, L, I, L, I, P]),
        "hlta_device_status": (I, [P, ctypes.POINTER(ctypes.c_uint)]),
        "hlta_kernel_launches": (ctypes.c_ulonglong, []),
        "hlta_wait_expiry_selftest": (I, [ctypes.c_ulonglong, P]),
        "hlta_set_profile_events": (I, [ctypes.POINTER(P)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()


def _check(status: int) -> None:
    if status != HLTA_OK:
        raise HltaError(status, (_lib.hlta_last_error() or b"").decode(errors="replace"))


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dt(t) -> int:
    torch = _th()
    if t.dtype == torch.bfloat16:
        return HLTA_BF16
    if t.dtype == torch.float32:
        return HLTA_FP32
    raise HltaError(HLTA_ERR_INVALID_ARG, f"unsupported dtype {t.dtype}")


def _need(t, name):
    if not t.is_cuda or not t.is_contiguous():
        raise HltaError(HLTA_ERR_INVALID_ARG, f"{name} must be a contiguous CUDA tensor")


# ---- entry points (same names as the C ABI) -----------------------------------------

def hlta_version() -> int:
    return int(_lib.hlta_version())


def hlta_swa_fwd(q, k, v, o, B, H, T, N, d, w, scale=0.0, stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _need(t, n)
    _check(_lib.hlta_swa_fwd(_p(q), _p(k), _p(v), _p(o), B, H, T, N, d, w, float(scale),
                             _dt(q), _stream(stream)))


def hlta_dswa_fwd(q, k, v, o, B, H, T, N, d, w, r, scale=0.0, stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _need(t, n)
    _check(_lib.hlta_dswa_fwd(_p(q), _p(k), _p(v), _p(o), B, H, T, N, d, w, r, float(scale),
                              _dt(q), _stream(stream)))


def hlta_gdn_workspace_bytes(B, H, L, d, chunk=64, dt=HLTA_BF16) -> int:
    return int(_lib.hlta_gdn_workspace_bytes(B, H, L, d, chunk, dt))


def hlta_gdn_chunk_fwd(q, k, v, a, b, o, S0, S_out, B, H, L, d, chunk, workspace,
                       stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (a, "a"), (b, "b"), (o, "o"), (workspace, "workspace")):
        _need(t, n)
    _check(_lib.hlta_gdn_chunk_fwd(_p(q), _p(k), _p(v), _p(a), _p(b), _p(o), _p(S0), _p(S_out),
                                   B, H, L, d, chunk, _p(workspace), workspace.numel() * workspace.element_size(),
                                   _dt(q), _stream(stream)))


def hlta_gdn_chunk_fwd_raw(q, k, v, x, y, c, o, S0, S_out, B, H, L, d, chunk, workspace,
                           stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (x, "x"), (y, "y"), (o, "o"), (workspace, "workspace")):
        _need(t, n)
    _check(_lib.hlta_gdn_chunk_fwd_raw(_p(q), _p(k), _p(v), _p(x), _p(y), float(c), _p(o), _p(S0),
                                       _p(S_out), B, H, L, d, chunk, _p(workspace),
                                       workspace.numel() * workspace.element_size(), _dt(q),
                                       _stream(stream)))


HLTA_STATIC_SCRATCH_BYTES = 32 * 1024 * 1024


def hlta_gdn_chunk_fwd_static(q, k, v, a, b, o, S0, S_out, B, H, L, d, chunk, stream=None):
    """hlta_gdn_chunk_fwd without a workspace argument: the library's built-in scratch is used
    (for callers that may not allocate device memory; see include/hlta.h)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (a, "a"), (b, "b"), (o, "o")):
        _need(t, n)
    _check(_lib.hlta_gdn_chunk_fwd_static(_p(q), _p(k), _p(v), _p(a), _p(b), _p(o), _p(S0),
                                          _p(S_out), B, H, L, d, chunk, _dt(q), _stream(stream)))


def hlta_hybrid_workspace_bytes(B, Hg, T, N, d, chunk=64, dt=HLTA_BF16) -> int:
    return int(_lib.hlta_hybrid_workspace_bytes(B, Hg, T, N, d, chunk, dt))


def hlta_hybrid_fwd(q, k, v, a, b, o, S0, S_out, B, Hs, Hd, Hg, T, N, d, w_swa, w_dswa, r,
                    chunk, scale, workspace, stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _need(t, n)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (_p(workspace), workspace.numel() * workspace.element_size())
    _check(_lib.hlta_hybrid_fwd(_p(q), _p(k), _p(v), _p(a), _p(b), _p(o), _p(S0), _p(S_out),
                                B, Hs, Hd, Hg, T, N, d, w_swa, w_dswa, r, chunk, float(scale),
                                ws_ptr, ws_bytes, _dt(q), _stream(stream)))


def hlta_hybrid_fwd_raw(q, k, v, x, y, c, o, S0, S_out, B, Hs, Hd, Hg, T, N, d, w_swa, w_dswa,
                        r, chunk, scale, workspace, stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o")):
        _need(t, n)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (_p(workspace), workspace.numel() * workspace.element_size())
    _check(_lib.hlta_hybrid_fwd_raw(_p(q), _p(k), _p(v), _p(x), _p(y), float(c), _p(o), _p(S0),
                                    _p(S_out), B, Hs, Hd, Hg, T, N, d, w_swa, w_dswa, r, chunk,
                                    float(scale), ws_ptr, ws_bytes, _dt(q), _stream(stream)))


def _need_types(x, x8, scales):
    import torch
    if x.dtype != torch.bfloat16 or x8.dtype != torch.uint8 or scales.dtype != torch.float32:
        raise HltaError(HLTA_ERR_INVALID_ARG, "FP8 quantisation takes bf16 x, uint8 codes and "
                        "float32 scales")


def hlta_fp8_quantize_rows(x, shift, B, H, L, d, frame_rows, block_rows, x8, scales,
                           stream=None):
    for t, n in ((x, "x"), (x8, "x8"), (scales, "scales")):
        _need(t, n)
    _need_types(x, x8, scales)
    if shift is not None:
        _need(shift, "shift")
    _check(_lib.hlta_fp8_quantize_rows(_p(x), _p(shift), B, H, L, d, frame_rows, block_rows,
                                       _p(x8), _p(scales), _stream(stream)))


def hlta_fp8_quantize_channels(x, B, H, L, d, x8, scales, stream=None):
    for t, n in ((x, "x"), (x8, "x8"), (scales, "scales")):
        _need(t, n)
    _need_types(x, x8, scales)
    _check(_lib.hlta_fp8_quantize_channels(_p(x), B, H, L, d, _p(x8), _p(scales),
                                           _stream(stream)))


def hlta_window_fp8_fwd(q8, qs, k8, ks, v8, vs, o, B, H, T, N, d, w, r, scale=0.0, stream=None):
    for t, n in ((q8, "q8"), (qs, "q_scales"), (k8, "k8"), (ks, "k_scales"), (v8, "v8"),
                 (vs, "v_scales"), (o, "o")):
        _need(t, n)
    _check(_lib.hlta_window_fp8_fwd(_p(q8), _p(qs), _p(k8), _p(ks), _p(v8), _p(vs), _p(o), B, H,
                                    T, N, d, w, r, float(scale), _stream(stream)))


def _need_bf16(*ts):
    import torch
    if any(t.dtype != torch.bfloat16 for t in ts):
        raise HltaError(HLTA_ERR_INVALID_ARG, "the attention training pair takes bf16 tensors")


def hlta_window_fwd_lse(q, k, v, o, lse, B, H, T, N, d, w, r, scale=0.0, stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (lse, "lse")):
        _need(t, n)
    _need_bf16(q, k, v, o)
    _check(_lib.hlta_window_fwd_lse(_p(q), _p(k), _p(v), _p(o), _p(lse), B, H, T, N, d, w, r,
                                    float(scale), _stream(stream)))


def hlta_window_bwd_workspace_bytes(B, H, T, N) -> int:
    return int(_lib.hlta_window_bwd_workspace_bytes(B, H, T, N))


def hlta_window_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, H, T, N, d, w, r, scale, workspace,
                    stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (lse, "lse"), (dO, "dO"), (dq, "dq"),
                 (dk, "dk"), (dv, "dv"), (workspace, "workspace")):
        _need(t, n)
    _need_bf16(q, k, v, o, dO, dq, dk, dv)
    _check(_lib.hlta_window_bwd(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(dO), _p(dq), _p(dk),
                                _p(dv), B, H, T, N, d, w, r, float(scale), _p(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream)))


def hlta_gdn_bwd_workspace_bytes(B, H, L, d=128, chunk=64) -> int:
    return int(_lib.hlta_gdn_bwd_workspace_bytes(B, H, L, d, chunk))


def hlta_rope(q, k, B, H, h0, Hr, L, N, d, base=10000.0, pos_mode=0, inverse=False,
              stream=None):
    for t, n in ((q, "q"), (k, "k")):
        if t is not None:
            _need(t, n)
    ref = q if q is not None else k
    _check(_lib.hlta_rope(_p(q), _p(k), B, H, h0, Hr, L, N, d, float(base), int(pos_mode),
                          1 if inverse else 0, _dt(ref), _stream(stream)))


def rope(q, k, N, heads=None, base=10000.0, pos_mode=0, inverse=False, stream=None):
    """Rotate q and k ([B, H, L, d]) in place; `heads` = (h0, Hr) or None for all heads."""
    ref = q if q is not None else k
    B, H, L, d = ref.shape
    h0, Hr = heads if heads is not None else (0, H)
    hlta_rope(q, k, B, H, h0, Hr, L, N, d, base, pos_mode, inverse, stream)
    return q, k


def hlta_gdn_chunk_bwd(q, k, v, a, b, S0, dO, dS_final, dq, dk, dv, da, db, dS0, B, H, L, d,
                       chunk, workspace, stream=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (a, "a"), (b, "b"), (dO, "dO"), (dq, "dq"),
                 (dk, "dk"), (dv, "dv"), (da, "da"), (db, "db"), (workspace, "workspace")):
        _need(t, n)
    for t, n in ((S0, "S0"), (dS_final, "dS_final"), (dS0, "dS0")):
        if t is not None:
            _need(t, n)
    _check(_lib.hlta_gdn_chunk_bwd(_p(q), _p(k), _p(v), _p(a), _p(b), _p(S0), _p(dO),
                                   _p(dS_final), _p(dq), _p(dk), _p(dv), _p(da), _p(db), _p(dS0),
                                   B, H, L, d, chunk, _p(workspace),
                                   workspace.numel() * workspace.element_size(), _dt(q),
                                   _stream(stream)))


# The serving calls (rotary axes, paged cache, recurrent gated delta rule) take a few microseconds
# on the GPU, so their checks are one pass over the tensors and torch is looked up once.
_torch = None


def _th():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _args(th, *wanted):
    """Addresses of (tensor, name, dtype, shape) tuples (None: a null pointer, any dtype or shape):
    each contiguous, on the current device (where the kernels are launched), as described."""
    out, dev = [], None
    for t, n, dtype, shape in wanted:
        if t is None:
            out.append(None)
            continue
        at = t.get_device()
        if dev is None and at >= 0:
            dev = th._C._cuda_getDevice()
        if (at != dev or not t.is_contiguous() or (dtype is not None and t.dtype is not dtype)
                or (shape is not None and t.shape != shape)):
            _misfit(t, n, dtype, shape, dev)
        out.append(t.data_ptr())
    return out


def _misfit(t, n, dtype, shape, dev):
    if dtype is not None and t.dtype != dtype:
        raise HltaError(HLTA_ERR_INVALID_ARG, f"{n} must be {dtype} (got {t.dtype})")
    if shape is not None and t.shape != shape:
        raise HltaError(HLTA_ERR_INVALID_ARG, f"{n} must be {list(shape)} (got {list(t.shape)})")
    if not t.is_cuda or not t.is_contiguous():
        raise HltaError(HLTA_ERR_INVALID_ARG, f"{n} must be a contiguous CUDA tensor")
    raise HltaError(HLTA_ERR_INVALID_ARG, f"{n} is on {t.device}, the current device is cuda:{dev}")


def _stream_address(th, stream):
    if stream is None:
        # the address alone: a Stream object costs as much as a launch
        return th._C._cuda_getCurrentRawStream(th._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_INT3 = ctypes.c_int * 3


def rope_axes_spec(pairs, grid=None, pos=None, t0=None, base=10000.0, halves=False,
                   shared_freq=False, B=None, L=None):
    """hlta_rope_axes_t from its parts: pairs = (time, height, width); grid = (height, width) of
    a frame, or pos [B, L, 3] int32; t0 [B] int32, the first frame's index of each rollout."""
    if (grid is None) == (pos is None):
        raise HltaError(HLTA_ERR_INVALID_ARG, "give either a grid or positions")
    if pos is not None and t0 is not None:
        raise HltaError(HLTA_ERR_INVALID_ARG, "t0 goes with a grid")
    gh, gw = (1, 1) if grid is None else grid
    at_pos = at_t0 = None
    if pos is not None or t0 is not None:
        th = _th()
        at_pos, at_t0 = _args(th, (pos, "pos", th.int32, None if B is None else (B, L, 3)),
                              (t0, "t0", th.int32, None if B is None else (B,)))
    return hlta_rope_axes_t(_INT3(*pairs), halves, shared_freq, gh, gw, base, at_pos,
                            at_t0)


def hlta_rope_axes(q, k, q_out, k_out, B, Hq, Hk, L, d, spec, inverse=False, stream=None):
    th, dt = _th(), (q if q is not None else k).dtype
    _check(_lib.hlta_rope_axes(
        *_args(th, (q, "q", dt, None), (k, "k", dt, None), (q_out, "q_out", dt, None),
               (k_out, "k_out", dt, None)),
        B, Hq, Hk, L, d, ctypes.byref(spec), 1 if inverse else 0, _dt(q if q is not None else k),
        _stream_address(th, stream)))


def hlta_paged_append(k, v, k_pages, v_pages, table, kv_lens, new_lens, B, Hkv, L, d, num_pages,
                      page, max_pages, spec=None, stream=None):
    th, dt = _th(), k.dtype
    i32 = th.int32
    _check(_lib.hlta_paged_append(
        *_args(th, (k, "k", dt, None), (v, "v", dt, None), (k_pages, "k_pages", dt, None),
               (v_pages, "v_pages", dt, None), (table, "table", i32, None),
               (kv_lens, "kv_lens", i32, None), (new_lens, "new_lens", i32, None)),
        B, Hkv, L, d, num_pages, page, max_pages, None if spec is None else ctypes.byref(spec),
        _dt(k), _stream_address(th, stream)))


def hlta_paged_attn_workspace_bytes(B, Hq, Hkv, L, d, page, max_pages, weights=False,
                                    dt=HLTA_BF16) -> int:
    return int(_lib.hlta_paged_attn_workspace_bytes(B, Hq, Hkv, L, d, page, max_pages,
                                                    1 if weights else 0, dt))


def hlta_paged_attn_fwd(q, k_pages, v_pages, table, kv_lens, new_lens, o, lse, w_in, w_out, decay,
                        B, Hq, Hkv, L, d, num_pages, page, max_pages, N, w, scale, workspace,
                        stream=None):
    th, dt = _th(), q.dtype
    i32, f32 = th.int32, th.float32
    *addr, ws = _args(th, (q, "q", dt, None), (k_pages, "k_pages", dt, None),
                      (v_pages, "v_pages", dt, None), (table, "table", i32, None),
                      (kv_lens, "kv_lens", i32, None), (new_lens, "new_lens", i32, None),
                      (o, "o", dt, None), (lse, "lse", f32, None), (w_in, "w_in", f32, None),
                      (w_out, "w_out", f32, None), (workspace, "workspace", None, None))
    _check(_lib.hlta_paged_attn_fwd(*addr, decay, B, Hq, Hkv, L, d, num_pages, page, max_pages, N,
                                    w, scale, ws, workspace.nbytes, _dt(q),
                                    _stream_address(th, stream)))


def hlta_paged_evict_workspace_bytes(B, Hkv, budget) -> int:
    return int(_lib.hlta_paged_evict_workspace_bytes(B, Hkv, budget))


def hlta_paged_evict(weights, k_pages, v_pages, table, kv_lens, B, Hkv, d, num_pages, page,
                     max_pages, budget, sink, recent, k_dst, v_dst, dst_table, num_dst, max_dst,
                     new_lens, kept, w_out, workspace, stream=None):
    th, dt = _th(), k_pages.dtype
    i32, f32 = th.int32, th.float32
    src = _args(th, (weights, "weights", f32, None), (k_pages, "k_pages", dt, None),
                (v_pages, "v_pages", dt, None), (table, "table", i32, None),
                (kv_lens, "kv_lens", i32, None))
    kd, vd, dst, nl, kp, wo, ws = _args(
        th, (k_dst, "k_dst", dt, None), (v_dst, "v_dst", dt, None),
        (dst_table, "dst_table", i32, None), (new_lens, "new_lens", i32, None),
        (kept, "kept", i32, None), (w_out, "w_out", f32, None), (workspace, "workspace", None, None))
    _check(_lib.hlta_paged_evict(*src, B, Hkv, d, num_pages, page, max_pages, budget, sink, recent,
                                 kd, vd, dst, num_dst, max_dst, nl, kp, wo, ws,
                                 0 if workspace is None else workspace.nbytes, _dt(k_pages),
                                 _stream_address(th, stream)))


def _gdn_step_args(th, q, k, v, a, b, o, S, S_out, slots, lens, qs=None, gs=None, ss=None, bs=None):
    dt, f32, i32 = q.dtype, th.float32, th.int32
    return _args(th, (q, "q", dt, qs), (k, "k", dt, qs), (v, "v", dt, qs), (a, "a", f32, gs),
                 (b, "b", f32, gs), (o, "o", dt, qs), (S, "S", f32, ss), (S_out, "S_out", f32, ss),
                 (slots, "slots", i32, bs), (lens, "lens", i32, bs))


def hlta_gdn_step(q, k, v, a, b, o, S, S_out, slots, lens, B, H, L, d, num_slots, stream=None):
    th = _th()
    _check(_lib.hlta_gdn_step(*_gdn_step_args(th, q, k, v, a, b, o, S, S_out, slots, lens), B, H, L,
                              d, num_slots, _dt(q), _stream_address(th, stream)))


def hlta_gdn_step_raw(q, k, v, x, y, c, o, S, S_out, slots, lens, B, H, L, d, num_slots,
                      stream=None):
    th = _th()
    args = _gdn_step_args(th, q, k, v, x, y, o, S, S_out, slots, lens)
    _check(_lib.hlta_gdn_step_raw(*args[:5], c, *args[5:], B, H, L, d, num_slots, _dt(q),
                                  _stream_address(th, stream)))


def hlta_device_status(stream=None) -> int:
    code = ctypes.c_uint(0)
    _check(_lib.hlta_device_status(_stream(stream), ctypes.byref(code)))
    return int(code.value)


def hlta_device_status_code(stream=None):
    """(status, raw device error word) without raising: hlta_device_status for callers that
    handle an expired wait themselves."""
    code = ctypes.c_uint(0)
    st = int(_lib.hlta_device_status(_stream(stream), ctypes.byref(code)))
    return st, int(code.value)


def hlta_kernel_launches() -> int:
    return int(_lib.hlta_kernel_launches())


def hlta_wait_expiry_selftest(cycles, stream=None):
    _check(_lib.hlta_wait_expiry_selftest(int(cycles), _stream(stream)))


def hlta_set_profile_events(events):
    """events: None, or 5 torch.cuda.Event objects (already created on the device)."""
    if events is None:
        _check(_lib.hlta_set_profile_events(None))
        return
    arr = (ctypes.c_void_p * 5)(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(_lib.hlta_set_profile_events(arr))


# ---- convenience wrappers (allocate with torch, then call the entry points) ----------

def _workspace(nbytes, device):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def swa(q, k, v, T, N, w, scale=0.0, out=None, stream=None):
    import torch
    B, H, _, d = q.shape
    o = torch.empty_like(q) if out is None else out
    hlta_swa_fwd(q, k, v, o, B, H, T, N, d, w, scale, stream)
    return o


def dswa(q, k, v, T, N, w, r, scale=0.0, out=None, stream=None):
    import torch
    B, H, _, d = q.shape
    o = torch.empty_like(q) if out is None else out
    hlta_dswa_fwd(q, k, v, o, B, H, T, N, d, w, r, scale, stream)
    return o


def fp8_quantize_rows(x, frame_rows, block_rows, shift=None, stream=None):
    """E4M3 codes (uint8, shape of x) and per-block scales [B, H, nframes, nblocks] of a bf16
    [B, H, L, d] tensor; blocks of block_rows rows inside frames of frame_rows rows."""
    import torch
    B, H, L, d = x.shape
    nf, nb = -(-L // frame_rows), -(-frame_rows // block_rows)
    x8 = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    sc = torch.empty((B, H, nf, nb), dtype=torch.float32, device=x.device)
    hlta_fp8_quantize_rows(x, shift, B, H, L, d, frame_rows, block_rows, x8, sc, stream)
    return x8, sc


def fp8_quantize_channels(x, stream=None):
    """E4M3 codes and per-channel scales [B, H, d] of a bf16 [B, H, L, d] tensor."""
    import torch
    B, H, L, d = x.shape
    x8 = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    sc = torch.empty((B, H, d), dtype=torch.float32, device=x.device)
    hlta_fp8_quantize_channels(x, B, H, L, d, x8, sc, stream)
    return x8, sc


def fp8_quantize_window_inputs(q, k, v, T, N, k_shift=None, stream=None):
    """The three quantisations the FP8 window attention takes: q in 128-row blocks of the
    head, k in 64-row runs of each frame (optionally minus a per-channel shift), v per channel.
    Returns (q8, qs, k8, ks, v8, vs)."""
    q8, qs = fp8_quantize_rows(q, T * N, 128, None, stream)
    k8, ks = fp8_quantize_rows(k, N, 64, k_shift, stream)
    v8, vs = fp8_quantize_channels(v, stream)
    return q8, qs, k8, ks, v8, vs


def window_fp8(q8, qs, k8, ks, v8, vs, T, N, w, r=1, scale=0.0, out=None, stream=None):
    """FP8 window attention (SWA for r = 1, DSWA otherwise); bf16 output [B, H, T*N, d]."""
    import torch
    B, H, L, d = q8.shape
    o = torch.empty((B, H, L, d), dtype=torch.bfloat16, device=q8.device) if out is None else out
    hlta_window_fp8_fwd(q8, qs, k8, ks, v8, vs, o, B, H, T, N, d, w, r, scale, stream)
    return o


def window_fwd_lse(q, k, v, T, N, w, r=1, scale=0.0, out=None, lse=None, stream=None):
    """Window attention forward that also returns the per-row log-sum-exp (for the backward)."""
    import torch
    B, H, L, d = q.shape
    o = torch.empty_like(q) if out is None else out
    ls = torch.empty((B, H, L), dtype=torch.float32, device=q.device) if lse is None else lse
    hlta_window_fwd_lse(q, k, v, o, ls, B, H, T, N, d, w, r, scale, stream)
    return o, ls


def window_bwd(q, k, v, o, lse, dO, T, N, w, r=1, scale=0.0, grads=None, workspace=None,
               stream=None):
    """Gradients (dq, dk, dv) of the window attention for the upstream gradient dO."""
    import torch
    B, H, L, d = q.shape
    dq, dk, dv = grads if grads is not None else (torch.empty_like(q) for _ in range(3))
    ws = workspace if workspace is not None else _workspace(
        hlta_window_bwd_workspace_bytes(B, H, T, N), q.device)
    hlta_window_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, H, T, N, d, w, r, scale, ws, stream)
    return dq, dk, dv


def gdn_bwd(q, k, v, a, b, dO, S0=None, dS_final=None, chunk=64, workspace=None, stream=None):
    """Gradients (dq, dk, dv, da, db, dS0) of the gated delta rule."""
    import torch
    B, H, L, d = q.shape
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    da, db = (torch.empty((B, H, L), dtype=torch.float32, device=q.device) for _ in range(2))
    dS0 = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    ws = workspace if workspace is not None else _workspace(
        hlta_gdn_bwd_workspace_bytes(B, H, L, d, chunk), q.device)
    hlta_gdn_chunk_bwd(q, k, v, a, b, S0, dO, dS_final, dq, dk, dv, da, db, dS0, B, H, L, d,
                       chunk, ws, stream)
    return dq, dk, dv, da, db, dS0


def gdn(q, k, v, a, b, S0=None, chunk=64, out=None, S_out=None, workspace=None, stream=None):
    import torch
    B, H, L, d = q.shape
    o = torch.empty_like(q) if out is None else out
    if S_out is None:
        S_out = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _workspace(hlta_gdn_workspace_bytes(B, H, L, d, chunk, _dt(q)), q.device)
    hlta_gdn_chunk_fwd(q, k, v, a, b, o, S0, S_out, B, H, L, d, chunk, workspace, stream)
    return o, S_out


def gdn_raw(q, k, v, x, y, c, S0=None, chunk=64, out=None, S_out=None, workspace=None,
            stream=None):
    """GDN heads from raw q, k and raw gate inputs x, y (see hlta_gdn_chunk_fwd_raw)."""
    import torch
    B, H, L, d = q.shape
    o = torch.empty_like(q) if out is None else out
    if S_out is None:
        S_out = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _workspace(hlta_gdn_workspace_bytes(B, H, L, d, chunk, _dt(q)), q.device)
    hlta_gdn_chunk_fwd_raw(q, k, v, x, y, c, o, S0, S_out, B, H, L, d, chunk, workspace, stream)
    return o, S_out


def hybrid_raw(q, k, v, x, y, c, Hs, Hd, Hg, T, N, w_swa, w_dswa, r, S0=None, chunk=64,
               scale=0.0, out=None, S_out=None, workspace=None, stream=None):
    """The hybrid operator with raw GDN inputs (see hlta_hybrid_fwd_raw)."""
    import torch
    B, H, L, d = q.shape
    o = torch.empty_like(q) if out is None else out
    if Hg and S_out is None:
        S_out = torch.empty((B, Hg, d, d), dtype=torch.float32, device=q.device)
    if Hg and workspace is None:
        workspace = _workspace(hlta_hybrid_workspace_bytes(B, Hg, T, N, d, chunk, _dt(q)), q.device)
    hlta_hybrid_fwd_raw(q, k, v, x, y, c, o, S0, S_out, B, Hs, Hd, Hg, T, N, d, w_swa, w_dswa,
                        r, chunk, scale, workspace, stream)
    return o, S_out


def hybrid(q, k, v, a, b, Hs, Hd, Hg, T, N, w_swa, w_dswa, r, S0=None, chunk=64, scale=0.0,
           out=None, S_out=None, workspace=None, stream=None):
    import torch
    B, H, L, d = q.shape
    o = torch.empty_like(q) if out is None else out
    if Hg and S_out is None:
        S_out = torch.empty((B, Hg, d, d), dtype=torch.float32, device=q.device)
    if Hg and workspace is None:
        workspace = _workspace(hlta_hybrid_workspace_bytes(B, Hg, T, N, d, chunk, _dt(q)), q.device)
    hlta_hybrid_fwd(q, k, v, a, b, o, S0, S_out, B, Hs, Hd, Hg, T, N, d, w_swa, w_dswa, r,
                    chunk, scale, workspace, stream)
    return o, S_out


def _made(stream, make, *args, **kw):
    """make(...): a tensor allocated, and filled, on the call's own stream (None: the current one), so
    that its memory is free there and a fill is ahead of the call."""
    if stream is None:
        return make(*args, **kw)
    th = _th()
    with th.cuda.stream(stream if hasattr(stream, "cuda_stream") else th.cuda.ExternalStream(int(stream))):
        return make(*args, **kw)


def rope_axes(q, k, pairs, grid=None, pos=None, t0=None, base=10000.0, halves=False,
              shared_freq=False, inverse=False, out=None, stream=None):
    """q and k ([B, H, L, d], either may be None) rotated by positions on three axes (see
    hlta_rope_axes); `out` = (q_out, k_out), which may be (q, k) for in place."""
    th, ref = _th(), q if q is not None else k
    if ref is None:
        raise HltaError(HLTA_ERR_INVALID_ARG, "neither q nor k is given")
    B, H, L, d = ref.shape
    Hk = k.shape[1] if k is not None else 0
    spec = rope_axes_spec(pairs, grid, pos, t0, base, halves, shared_freq, B, L)
    if out is None:
        out = (None if q is None else _made(stream, th.empty_like, q),
               None if k is None else _made(stream, th.empty_like, k))
    dt, qs, ks = ref.dtype, (B, H, L, d), (B, Hk, L, d)
    _check(_lib.hlta_rope_axes(
        *_args(th, (q, "q", dt, qs), (k, "k", dt, ks), (out[0], "q_out", dt, qs),
               (out[1], "k_out", dt, ks)),
        B, H, Hk, L, d, ctypes.byref(spec), 1 if inverse else 0, _dt(ref),
        _stream_address(th, stream)))
    return out


def paged_append(k, v, k_pages, v_pages, table, kv_lens, new_lens=None, rope=None, stream=None):
    """Append a chunk (k, v [B, Hkv, L, d]) to a paged cache (see hlta_paged_append); `rope`: the
    arguments of rope_axes_spec as a dict, for k to be rotated on the way."""
    th, dt = _th(), k.dtype
    i32, pages = th.int32, k_pages.shape
    num, H, page, d = pages
    B, width = table.shape
    L = k.shape[2]
    spec = None if rope is None else ctypes.byref(rope_axes_spec(**rope, B=B, L=L))
    cs, bs = (B, H, L, d), (B,)
    _check(_lib.hlta_paged_append(
        *_args(th, (k, "k", dt, cs), (v, "v", dt, cs), (k_pages, "k_pages", dt, pages),
               (v_pages, "v_pages", dt, pages), (table, "table", i32, None),
               (kv_lens, "kv_lens", i32, bs), (new_lens, "new_lens", i32, bs)),
        B, H, L, d, num, page, width, spec, _dt(k), _stream_address(th, stream)))


@functools.lru_cache(maxsize=1024)
def _attn_workspace(device, *shape):
    return _lib.hlta_paged_attn_workspace_bytes(*shape)


def paged_attn(q, k_pages, v_pages, table, kv_lens, new_lens=None, N=1, w=0, scale=0.0, out=None,
               lse=None, w_in=None, w_out=None, decay=1.0, workspace=None, stream=None):
    """Attention of a chunk (q [B, Hq, L, d]) over a paged cache it was appended to (see
    hlta_paged_attn_fwd). Rows behind a rollout's new tokens are left as they are in `out`
    (zeros when it is allocated here)."""
    th, dt = _th(), q.dtype
    i32, f32, pages, qs = th.int32, th.float32, k_pages.shape, q.shape
    num, H, page, d = pages
    B, width = table.shape
    Hq, L = qs[1], qs[2]
    if out is None:
        out = _made(stream, th.empty_like if new_lens is None else th.zeros_like, q)
    code = _dt(q)
    if workspace is None:
        need = _attn_workspace(q.get_device(), B, Hq, H, L, d, page, width,
                               0 if w_out is None else 1, code)
        workspace = _made(stream, q.new_empty, need, dtype=th.uint8)
    bs, ws_shape = (B,), (B, H, width * page)
    *addr, ws = _args(th, (q, "q", dt, (B, Hq, L, d)), (k_pages, "k_pages", dt, pages),
                      (v_pages, "v_pages", dt, pages), (table, "table", i32, None),
                      (kv_lens, "kv_lens", i32, bs), (new_lens, "new_lens", i32, bs),
                      (out, "out", dt, qs), (lse, "lse", f32, (B, Hq, L)),
                      (w_in, "w_in", f32, ws_shape), (w_out, "w_out", f32, ws_shape),
                      (workspace, "workspace", None, None))
    _check(_lib.hlta_paged_attn_fwd(*addr, decay, B, Hq, H, L, d, num, page, width, N, w, scale,
                                    ws, workspace.nbytes, code, _stream_address(th, stream)))
    return out


def paged_evict(weights, k_pages, v_pages, table, kv_lens, budget, sink, recent, k_dst, v_dst,
                dst_table, new_lens=None, kept=None, w_out=None, workspace=None, stream=None):
    """Copy the `budget` positions of largest accumulated weight (the first `sink` and the last
    `recent` always among them) of every rollout and key head to the destination's pages (see
    hlta_paged_evict). Returns the new lengths [B] int32."""
    th, dt = _th(), k_pages.dtype
    i32, f32, pages, to = th.int32, th.float32, k_pages.shape, k_dst.shape
    num, H, page, d = pages
    (B, width), (_, dwidth) = table.shape, dst_table.shape
    bs = (B,)
    if new_lens is None:
        new_lens = _made(stream, th.empty_like, kv_lens)
    if workspace is None and kept is None:
        need = _lib.hlta_paged_evict_workspace_bytes(B, H, budget)
        workspace = _made(stream, weights.new_empty, need, dtype=th.uint8)
    src = _args(th, (weights, "weights", f32, (B, H, width * page)),
                (k_pages, "k_pages", dt, pages), (v_pages, "v_pages", dt, pages),
                (table, "table", i32, None), (kv_lens, "kv_lens", i32, bs))
    kd, vd, dst, nl, kp, wo, ws = _args(
        th, (k_dst, "k_dst", dt, (to[0], H, page, d)), (v_dst, "v_dst", dt, to),
        (dst_table, "dst_table", i32, (B, dwidth)), (new_lens, "new_lens", i32, bs),
        (kept, "kept", i32, (B, H, budget)), (w_out, "w_out", f32, (B, H, dwidth * page)),
        (workspace, "workspace", None, None))
    _check(_lib.hlta_paged_evict(*src, B, H, d, num, page, width, budget, sink, recent, kd, vd, dst,
                                 to[0], dwidth, nl, kp, wo, ws,
                                 0 if workspace is None else workspace.nbytes, _dt(k_pages),
                                 _stream_address(th, stream)))
    return new_lens


def _gdn_step(raw, q, k, v, a, b, S, slots, lens, out, S_out, stream):
    th, qs = _th(), q.shape
    B, H, L, d = qs
    if out is None:
        out = _made(stream, th.empty_like if slots is None and lens is None else th.zeros_like, q)
    if S_out is None:
        S_out = S
    num = S.shape[0]
    args = _gdn_step_args(th, q, k, v, a, b, out, S, S_out, slots, lens, qs, (B, H, L),
                          (num, H, d, d), (B,))
    if raw is None:
        st = _lib.hlta_gdn_step(*args, B, H, L, d, num, _dt(q), _stream_address(th, stream))
    else:
        st = _lib.hlta_gdn_step_raw(*args[:5], raw, *args[5:], B, H, L, d, num, _dt(q),
                                    _stream_address(th, stream))
    _check(st)
    return out, S_out


def gdn_step(q, k, v, a, b, S, slots=None, lens=None, out=None, S_out=None, stream=None):
    """One step of one or a few tokens of the gated delta rule over a pool of states S
    [slots, H, d, d], updated in place unless S_out is given (see hlta_gdn_step). Returns
    (o, S_out). Outputs allocated here are zero where the call leaves rows as they are."""
    return _gdn_step(None, q, k, v, a, b, S, slots, lens, out, S_out, stream)


def gdn_step_raw(q, k, v, x, y, c, S, slots=None, lens=None, out=None, S_out=None, stream=None):
    """gdn_step from raw q, k and raw gate inputs (see hlta_gdn_step_raw)."""
    return _gdn_step(float(c), q, k, v, x, y, S, slots, lens, out, S_out, stream)


class PagedCache:
    """Paged key/value cache of B rollouts of different ages (paged_append / paged_attn /
    paged_evict): the page pool, and the tables that the host keeps and copies to the device when
    pages change hands. The pool's pages are handed out as rollouts grow, returned by `evict` and
    `release`. Everything runs on the current stream, which has to be the same one from call to call.
    `attend` may be captured into a CUDA graph and replayed for later chunks of as many rows (the cache's
    tensors stay the same ones); `append`, `evict` and `release` copy lengths and tables from the host,
    which blocks it, and cannot be captured.

    max_len: the longest a rollout may grow; num_pages: pages of the pool (an eviction needs free
    pages for what it keeps while it copies). weights: keep the attention weights that `attend`
    accumulates (times `decay` per call), which `evict` goes by; zero for positions of chunks that were
    never attended, and behind a rollout's end."""

    def __init__(self, B, Hkv, d, num_pages, max_len, page=64, dtype=None, weights=False, decay=1.0):
        th = _th()
        if B < 1 or Hkv < 1 or num_pages < 1 or max_len < 1 or page not in (16, 32, 64, 128):
            raise HltaError(HLTA_ERR_INVALID_ARG, f"bad cache: B={B} Hkv={Hkv} num_pages={num_pages} "
                            f"max_len={max_len} page={page}")
        self.B, self.page, self.max_len, self.decay = B, page, max_len, float(decay)
        self.width = -(-max_len // page)
        dt = th.bfloat16 if dtype is None else dtype
        self.k_pages, self.v_pages = (th.empty((num_pages, Hkv, page, d), dtype=dt, device="cuda")
                                      for _ in range(2))
        self.table = th.zeros((B, self.width), dtype=th.int32, device="cuda")
        self.kv_lens = th.zeros(B, dtype=th.int32, device="cuda")
        self.new_lens = th.zeros(B, dtype=th.int32, device="cuda")
        self.weights = th.zeros((B, Hkv, self.width * page), device="cuda") if weights else None
        self.lens = [0] * B                             # tokens cached, per rollout
        self._free = list(range(num_pages - 1, -1, -1))
        self._pages = [[] for _ in range(B)]

    def _grow(self, lens):
        """Pages for the given lengths, or an error that leaves everything as it was."""
        for b, n in enumerate(lens):
            if n > self.max_len:
                raise HltaError(HLTA_ERR_INVALID_ARG, f"rollout {b} would hold {n} tokens, at most {self.max_len}")
        want = [max(0, -(-n // self.page) - len(p)) for n, p in zip(lens, self._pages)]
        if sum(want) > len(self._free):
            raise HltaError(HLTA_ERR_INVALID_ARG, f"{sum(want)} pages wanted, {len(self._free)} free")
        for p, n in zip(self._pages, want):
            p.extend(self._free.pop() for _ in range(n))
        return sum(want) > 0

    def _tables(self, pages):
        if pages:
            self.table.copy_(_th().tensor([p + [0] * (self.width - len(p)) for p in self._pages],
                                          dtype=_th().int32))
        self.kv_lens.copy_(_th().tensor(self.lens, dtype=_th().int32))

    def append(self, k, v, new_lens=None, rope=None):
        """Append a chunk (k, v [B, Hkv, L, d]; new_lens: tokens that each rollout really has, a
        list, None for all L); `rope` as in paged_append."""
        L = k.shape[2]
        new = [L] * self.B if new_lens is None else [int(n) for n in new_lens]
        if len(new) != self.B or any(n < 0 or n > L for n in new):
            raise HltaError(HLTA_ERR_INVALID_ARG, f"new_lens must be {self.B} numbers in [0, {L}] (got {new})")
        before, held = self.lens, [len(p) for p in self._pages]
        lens = [a + n for a, n in zip(self.lens, new)]
        pages = self._grow(lens)
        self.lens = lens
        try:
            self._tables(pages)
            chunk = _th().tensor(new, dtype=_th().int32).to(self.new_lens.device)
            paged_append(k, v, self.k_pages, self.v_pages, self.table, self.kv_lens, chunk, rope)
        except Exception:
            # refused: the rollouts, their last chunk and the pool as they were
            self.lens = before
            for p, n in zip(self._pages, held):
                self._free.extend(reversed(p[n:]))
                del p[n:]
            self._tables(pages)
            raise
        self.new_lens.copy_(chunk)

    def attend(self, q, N=1, w=0, scale=0.0, out=None, lse=None):
        """Attention of the chunk appended last (q [B, Hq, L, d]; the rows of a rollout that was cut or
        released since are zero, or as they were in `out`); adds to the weights if kept."""
        return paged_attn(q, self.k_pages, self.v_pages, self.table, self.kv_lens, self.new_lens, N,
                          w, scale, out, lse, self.weights, self.weights, self.decay)

    def evict(self, budget, sink=0, recent=0):
        """Cut every rollout of more than `budget` tokens to that many (see hlta_paged_evict).
        Returns the rollouts that were cut."""
        th = _th()
        if self.weights is None:
            raise HltaError(HLTA_ERR_INVALID_ARG, "this cache keeps no weights")
        cut = [b for b, n in enumerate(self.lens) if n > budget]
        need = -(-budget // self.page)
        if need * len(cut) > len(self._free):
            raise HltaError(HLTA_ERR_INVALID_ARG, f"{need * len(cut)} pages wanted, {len(self._free)} free")
        if not cut:
            return cut
        # the copies go to free pages; rollouts that stay as they are take no part (length 0)
        to = {b: [self._free[-1 - i * need - j] for j in range(need)] for i, b in enumerate(cut)}
        dst = th.tensor([to.get(b, [0] * need) for b in range(self.B)], dtype=th.int32).cuda()
        lens = th.tensor([n if b in to else 0 for b, n in enumerate(self.lens)], dtype=th.int32).cuda()
        w_out = th.empty((self.B, self.weights.shape[1], need * self.page), device="cuda")
        paged_evict(self.weights, self.k_pages, self.v_pages, self.table, lens, budget, sink, recent,
                    self.k_pages, self.v_pages, dst, w_out=w_out)
        for b in cut:                                   # in place: a captured attend holds the tensor
            self.weights[b, :, :budget] = w_out[b, :, :budget]
            self.weights[b, :, budget:] = 0.0
        del self._free[len(self._free) - need * len(cut):]
        for b in cut:
            self._free.extend(self._pages[b])
            self._pages[b] = to[b]
            self.lens[b] = budget
            self.new_lens[b] = 0                        # its last chunk is no longer its last positions
        self._tables(True)
        return cut

    def release(self, b):
        """Empty rollout b: its pages go back to the pool."""
        self._free.extend(self._pages[b])
        self._pages[b] = []
        self.lens[b] = 0
        self.new_lens[b] = 0
        if self.weights is not None:
            self.weights[b] = 0.0
        self._tables(True)


class Stream:
    """Streaming cache (hlta_stream_create_ex / _step / _step_frames / _state /
    _frame_counter / _checkpoint_bytes / _save / _load / _destroy). A step may be captured into a CUDA graph and replayed for the
    following frames: the frame index lives in a device counter that every step advances."""

    def __init__(self, B, Hs, Hd, Hg, N, d, w_swa, w_dswa, r, chunk=64, scale=0.0,
                 dtype=None, S0=None, max_step_frames=1):
        import torch
        dt = HLTA_BF16 if dtype in (None, torch.bfloat16) else HLTA_FP32
        self._h = ctypes.c_void_p()
        _check(_lib.hlta_stream_create_ex(ctypes.byref(self._h), B, Hs, Hd, Hg, N, d, w_swa,
                                          w_dswa, r, chunk, float(scale), int(max_step_frames),
                                          dt, _p(S0)))
        self.B, self.H, self.Hg, self.N, self.d = B, Hs + Hd + Hg, Hg, N, d

    def step(self, q, k, v, a, b, out=None, stream=None):
        import torch
        o = torch.empty_like(q) if out is None else out
        _check(_lib.hlta_stream_step(self._h, _p(q), _p(k), _p(v), _p(a), _p(b), _p(o),
                                     _stream(stream)))
        return o

    def step_frames(self, q, k, v, a, b, frames, out=None, stream=None):
        """Append `frames` frames per rollout at once (inputs [B, H, frames*N, d])."""
        import torch
        o = torch.empty_like(q) if out is None else out
        _check(_lib.hlta_stream_step_frames(self._h, _p(q), _p(k), _p(v), _p(a), _p(b), _p(o),
                                            int(frames), _stream(stream)))
        return o

    def state(self):
        """(device address of the [B,Hg,d,d] fp32 state, frames appended so far)."""
        ptr, n = ctypes.c_void_p(), ctypes.c_int()
        _check(_lib.hlta_stream_state(self._h, ctypes.byref(ptr), ctypes.byref(n)))
        return ptr.value, n.value

    def frame_counter(self):
        """Device address of the cache's frame counter (an int advanced by every step, in
        stream order, replays of a captured step included)."""
        ptr = ctypes.c_void_p()
        _check(_lib.hlta_stream_frame_counter(self._h, ctypes.byref(ptr)))
        return ptr.value

    def checkpoint_bytes(self):
        return int(_lib.hlta_stream_checkpoint_bytes(self._h))

    def save(self, stream=None):
        """The cache's checkpoint image (hlta_stream_save) as a uint8 numpy array."""
        import numpy as np
        buf = np.empty(self.checkpoint_bytes(), dtype=np.uint8)
        _check(_lib.hlta_stream_save(self._h, buf.ctypes.data, buf.nbytes, _stream(stream)))
        return buf

    def load(self, image, stream=None):
        """Resume from a checkpoint image (hlta_stream_load)."""
        import numpy as np
        buf = np.ascontiguousarray(image, dtype=np.uint8)
        _check(_lib.hlta_stream_load(self._h, buf.ctypes.data, buf.nbytes, _stream(stream)))

    def state_tensor(self):
        """A torch copy of the carried state [B, Hg, d, d] fp32 (ordered on the current stream)."""
        import torch
        ptr, _ = self.state()

        class _View:   # exposes the cache's device buffer to torch without copying
            __cuda_array_interface__ = {"shape": (self.B, self.Hg, self.d, self.d),
                                        "typestr": "<f4", "data": (ptr, False), "version": 2}
        return torch.as_tensor(_View(), device="cuda").clone()

    def close(self):
        if self._h:
            _check(_lib.hlta_stream_destroy(self._h))
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
