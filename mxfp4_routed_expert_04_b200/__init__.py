"""Routed MXFP4 MoE FFN layer on B200 (sm_100a): Python binding of libmoe_mxfp4.so.

Thin ctypes marshalling over the C ABI in ``include/moe_mxfp4.h``: every
function here has the name of the C entry point it calls, takes torch tensors
(device memory) and passes their data pointers. All computation runs in the
library's CUDA kernels; there is no Python or CPU fallback. Importing the
package fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "MoeError", "MoeDims", "MoeLayerArgs", "ACT_BF16", "ACT_MXFP4", "library_path",
    "moe_status_string", "moe_workspace_size", "moe_x_op_size", "moe_workspace_init",
    "moe_device_status", "moe_route", "moe_route_biased", "moe_route_noalloc", "moe_permute", "moe_expert_ffn", "moe_combine",
    "moe_latent_down", "moe_layer", "moe_mxf4_layout_of", "moe_tile_scales",
    "moe_selftest_bounded_wait", "STATUS_BAD_EXPERT", "STATUS_REPEATED_EXPERT",
    "STATUS_WAIT_TIMEOUT", "SCORE_SOFTMAX", "SCORE_SIGMOID", "MoeLayer", "ExpertCache",
    "moe_expert_cache_bytes",
    "MoeLinearDims", "MoeFfnDims", "FfnSaved", "MoeFfn", "DTYPE_BF16", "DTYPE_F16", "FN_NONE", "FN_SILU",
    "FN_GELU", "FN_RELU", "SAVE_NONE", "SAVE_16", "SAVE_8", "moe_dense_workspace_init",
    "moe_linear_workspace_size", "moe_linear", "moe_linear_backward", "moe_ffn_workspace_size", "moe_ffn",
    "moe_ffn_backward", "moe_ckpt8_pack", "moe_ckpt8_unpack",
]

# bits of the device status word (moe_device_status)
STATUS_BAD_EXPERT, STATUS_REPEATED_EXPERT, STATUS_WAIT_TIMEOUT = 1, 2, 4

ACT_BF16 = 0
ACT_MXFP4 = 1

_PKG = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    return os.environ.get("MOE_MXFP4_LIB", os.path.join(_PKG, "libmoe_mxfp4.so"))


def _load():
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python mxfp4_routed_expert_04_b200/build.py` "
            "(there is no fallback implementation)")
    return ctypes.CDLL(path)


_lib = _load()


SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1


class MoeDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "I", "E", "k", "I_shared", "L", "act_mode",
                                              "score_fn", "n_group", "topk_group")] + \
               [("route_scale", ctypes.c_float)]

    @classmethod
    def of(cls, w, act_mode: int = ACT_BF16) -> "MoeDims":
        """Dims of a workload (anything with T, H, I, E, k, I_shared, L and,
        optionally, the router variant: score_fn, n_group, topk_group,
        route_scale)."""
        return cls(w.T, w.H, w.I, w.E, w.k, w.I_shared, w.L, act_mode,
                   getattr(w, "score_fn", 0), getattr(w, "n_group", 0),
                   getattr(w, "topk_group", 0), getattr(w, "route_scale", 1.0))


_P = ctypes.c_void_p


class MoeLayerArgs(ctypes.Structure):
    _fields_ = [(n, _P) for n in (
        "x", "w_router", "wg_q", "wg_s", "wu_q", "wu_s", "wd_q", "wd_s", "w_sgate",
        "ws_gate", "ws_up", "ws_down", "w_lat_down", "w_lat_up", "topk_idx", "topk_w",
        "counts", "offsets", "expert_list", "row_token", "row_slot", "slot_row", "x_lat", "x_op",
        "y_perm", "y", "e_bias")]


_lib.moe_status_string.restype = ctypes.c_char_p
_lib.moe_status_string.argtypes = [ctypes.c_int]
_lib.moe_last_error.restype = ctypes.c_char_p
_lib.moe_workspace_size.restype = ctypes.c_size_t
_lib.moe_workspace_size.argtypes = [ctypes.POINTER(MoeDims)]
_lib.moe_x_op_size.restype = ctypes.c_size_t
_lib.moe_x_op_size.argtypes = [ctypes.POINTER(MoeDims)]
_D = ctypes.POINTER(MoeDims)
_Z = ctypes.c_size_t
_sigs = {
    "moe_workspace_init": [_D, _P, _Z, _P],
    "moe_device_status": [_P, ctypes.POINTER(ctypes.c_int32), _P],
    "moe_route": [_D, _P, _P, _P, _P, _P, _P, _Z, _P],
    "moe_route_biased": [_D, _P, _P, _P, _P, _P, _P, _P, _Z, _P],
    "moe_route_noalloc": [_D, _P, _P, _P, _P, _P, _P],
    "moe_permute": [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _Z, _P],
    "moe_expert_ffn": [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _Z, _P],
    "moe_combine": [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _Z, _P],
    "moe_latent_down": [_D, _P, _P, _P, _P, _Z, _P],
    "moe_layer": [_D, ctypes.POINTER(MoeLayerArgs), _P, _Z, _P],
    "moe_mxf4_layout_of": [_D, ctypes.c_void_p],
    "moe_tile_scales": [_P, ctypes.c_int64, ctypes.c_int32, _P, _P],
    "moe_selftest_bounded_wait": [_P, _P, ctypes.c_int, ctypes.c_uint32, _P],
}
_sigs.update({
    "moe_expert_cache_create": [_D, ctypes.c_int32, _P, _Z, ctypes.POINTER(_P)],
    "moe_expert_cache_destroy": [_P],
    "moe_expert_cache_stats": [_P, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64),
                               ctypes.POINTER(ctypes.c_int64)],
    "moe_expert_ffn_streamed": [_P, _D, _P, ctypes.c_int32, _P, _P, _P, _P, _P, _P, _Z, _P],
})


class MoeLinearDims(ctypes.Structure):
    """Sizes of moe_linear / moe_linear_backward (pitches in elements, 0: packed rows)."""
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "N", "K", "fn", "dtype", "out_f32")] + \
               [(n, ctypes.c_int64) for n in ("ldx", "ldy", "ldr")]


class MoeFfnDims(ctypes.Structure):
    """Sizes of moe_ffn / moe_ffn_backward (pitches in elements, 0: packed rows)."""
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "I", "fn", "dtype", "save", "out_f32", "reserved")] + \
               [(n, ctypes.c_int64) for n in ("ldx", "ldy", "ldr")]


class _FfnSavedPtrs(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("g", "u", "g_s", "u_s", "x_q", "x_s")]


_DL = ctypes.POINTER(MoeLinearDims)
_DF = ctypes.POINTER(MoeFfnDims)
_DS = ctypes.POINTER(_FfnSavedPtrs)
_sigs.update({
    "moe_dense_workspace_init": [_P, _Z, _P],
    "moe_linear": [_DL] + [_P] * 7 + [_Z, _P],
    "moe_linear_backward": [_DL] + [_P] * 8 + [_Z, _P],
    "moe_ffn": [_DF] + [_P] * 6 + [_DS, _P, _Z, _P],
    "moe_ffn_backward": [_DF] + [_P] * 5 + [_DS] + [_P] * 5 + [_Z, _P],
    "moe_ckpt8_pack": [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, _P, ctypes.c_int64, _P, _P, _P],
    "moe_ckpt8_unpack": [ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, _P, _P, _P, ctypes.c_int64, _P],
})
for _n, _d in (("moe_linear_workspace_size", _DL), ("moe_ffn_workspace_size", _DF)):
    getattr(_lib, _n).restype = ctypes.c_size_t
    getattr(_lib, _n).argtypes = [_d]
for _n, _a in _sigs.items():
    getattr(_lib, _n).argtypes = _a
    getattr(_lib, _n).restype = ctypes.c_int
_lib.moe_expert_cache_bytes.restype = ctypes.c_size_t
_lib.moe_expert_cache_bytes.argtypes = [_D, ctypes.c_int32]


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{moe_status_string(status)} ({status}): {message}")
        self.status = status


def moe_status_string(status: int) -> str:
    return _lib.moe_status_string(status).decode()


def _check(status: int):
    if status != 0:
        raise MoeError(status, _lib.moe_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def moe_workspace_size(dims: MoeDims) -> int:
    return _lib.moe_workspace_size(ctypes.byref(dims))


def moe_x_op_size(dims: MoeDims) -> int:
    return _lib.moe_x_op_size(ctypes.byref(dims))


class MoeMxf4Layout(ctypes.Structure):
    _fields_ = [("x_codes", ctypes.c_size_t), ("x_scales", ctypes.c_size_t),
                ("tiles", ctypes.c_size_t), ("tile_base", ctypes.c_size_t),
                ("n_tiles", ctypes.c_size_t), ("h_codes", ctypes.c_size_t),
                ("h_scales", ctypes.c_size_t), ("max_tiles", ctypes.c_int32),
                ("tile_rows", ctypes.c_int32)]


def moe_mxf4_layout_of(dims) -> MoeMxf4Layout:
    """Byte offsets of the MOE_ACT_MXFP4 operands inside x_op and the workspace."""
    out = MoeMxf4Layout()
    _check(_lib.moe_mxf4_layout_of(ctypes.byref(dims), ctypes.addressof(out)))
    return out


def moe_tile_scales(src, rows: int, K: int, dst, stream=None):
    """Canonical E8M0 scales [rows, K/32] -> the tiled layout of the tensor-core path."""
    _check(_lib.moe_tile_scales(_ptr(src), int(rows), int(K), _ptr(dst), _stream(stream)))


def moe_selftest_bounded_wait(status, src, deliver: bool, limit: int, stream=None):
    """One CTA waits (bounded, ``limit`` tries) for a stage that a bulk copy
    from ``src`` fills (deliver) or that nothing fills; a timeout ORs
    STATUS_WAIT_TIMEOUT into the device int32 ``status``."""
    _check(_lib.moe_selftest_bounded_wait(_ptr(status), _ptr(src), 1 if deliver else 0,
                                          int(limit), _stream(stream)))


def moe_workspace_init(dims, ws, stream=None):
    _check(_lib.moe_workspace_init(ctypes.byref(dims), _ptr(ws), ws.numel() * ws.element_size(),
                                   _stream(stream)))


def moe_device_status(ws, stream=None) -> int:
    """Device status word (0 = no data error); raises nothing for a flagged word."""
    out = ctypes.c_int32(0)
    st = _lib.moe_device_status(_ptr(ws), ctypes.byref(out), _stream(stream))
    if st not in (0, 6):
        _check(st)
    return out.value


def _nbytes(t):
    return t.numel() * t.element_size()


def moe_route(dims, x, w_router, topk_idx, topk_w, logits, ws, stream=None):
    _check(_lib.moe_route(ctypes.byref(dims), _ptr(x), _ptr(w_router), _ptr(topk_idx),
                          _ptr(topk_w), _ptr(logits), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_route_biased(dims, x, w_router, e_bias, topk_idx, topk_w, logits, ws, stream=None):
    _check(_lib.moe_route_biased(ctypes.byref(dims), _ptr(x), _ptr(w_router), _ptr(e_bias),
                                 _ptr(topk_idx), _ptr(topk_w), _ptr(logits), _ptr(ws), _nbytes(ws),
                                 _stream(stream)))


def moe_route_noalloc(dims, x, w_router, topk_idx, topk_w, logits, stream=None):
    """moe_route without a workspace (partials in the library's static device array)."""
    _check(_lib.moe_route_noalloc(ctypes.byref(dims), _ptr(x), _ptr(w_router), _ptr(topk_idx),
                                  _ptr(topk_w), _ptr(logits), _stream(stream)))


def moe_permute(dims, topk_idx, x_in, counts, offsets, expert_list, row_token, row_slot, slot_row,
                x_op, ws, stream=None):
    _check(_lib.moe_permute(ctypes.byref(dims), _ptr(topk_idx), _ptr(x_in), _ptr(counts),
                            _ptr(offsets), _ptr(expert_list), _ptr(row_token), _ptr(row_slot),
                            _ptr(slot_row), _ptr(x_op), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_expert_ffn(dims, x_op, offsets, expert_list, row_token, wg_q, wg_s, wu_q, wu_s, wd_q, wd_s,
                   y_perm, ws, stream=None):
    _check(_lib.moe_expert_ffn(ctypes.byref(dims), _ptr(x_op), _ptr(offsets), _ptr(expert_list),
                               _ptr(row_token), _ptr(wg_q), _ptr(wg_s), _ptr(wu_q), _ptr(wu_s),
                               _ptr(wd_q), _ptr(wd_s), _ptr(y_perm), _ptr(ws), _nbytes(ws),
                               _stream(stream)))


def moe_combine(dims, y_perm, slot_row, topk_w, x, w_sgate, ws_gate, ws_up, ws_down, w_lat_up, y,
                ws, stream=None):
    _check(_lib.moe_combine(ctypes.byref(dims), _ptr(y_perm), _ptr(slot_row), _ptr(topk_w),
                            _ptr(x), _ptr(w_sgate), _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down),
                            _ptr(w_lat_up), _ptr(y), _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_latent_down(dims, x, w_lat_down, x_lat, ws, stream=None):
    _check(_lib.moe_latent_down(ctypes.byref(dims), _ptr(x), _ptr(w_lat_down), _ptr(x_lat),
                                _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_layer(dims, args: MoeLayerArgs, ws, stream=None):
    _check(_lib.moe_layer(ctypes.byref(dims), ctypes.byref(args), _ptr(ws), _nbytes(ws),
                          _stream(stream)))


def moe_expert_cache_bytes(dims, slots: int) -> int:
    return _lib.moe_expert_cache_bytes(ctypes.byref(dims), int(slots))


class ExpertCache:
    """An LRU cache of `slots` routed experts in device memory (one torch
    buffer) in front of experts kept in host memory (moe_expert_cache_*).

    host_experts: a sequence of E tuples (wg_q, wg_s, wu_q, wu_s, wd_q, wd_s)
    of host tensors (page-locked for asynchronous copies) in the canonical
    layout."""

    def __init__(self, dims: MoeDims, slots: int, host_experts, device="cuda"):
        self.dims = dims
        nbytes = moe_expert_cache_bytes(dims, slots)
        if nbytes == 0:
            raise MoeError(2, _lib.moe_last_error().decode())
        self.mem = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
        off = (-self.mem.data_ptr()) % 256
        self._host = list(host_experts)         # keeps the host tensors alive
        ptrs = (ctypes.c_void_p * (6 * dims.E))()
        for e, arrs in enumerate(self._host):
            for a, t in enumerate(arrs):
                ptrs[6 * e + a] = t.data_ptr()
        self._ptrs = ptrs
        h = ctypes.c_void_p()
        _check(_lib.moe_expert_cache_create(ctypes.byref(dims), int(slots), self.mem.data_ptr() + off,
                                            nbytes, ctypes.byref(h)))
        self._h = h

    def ffn(self, active, x_op, offsets, row_token, y_perm, ws, stream=None):
        """moe_expert_ffn_streamed for the experts in `active` (host ints)."""
        act = (ctypes.c_int32 * max(1, len(active)))(*[int(e) for e in active])
        _check(_lib.moe_expert_ffn_streamed(self._h, ctypes.byref(self.dims), act, len(active),
                                            _ptr(x_op), _ptr(offsets), _ptr(row_token), self._ptrs,
                                            _ptr(y_perm), _ptr(ws), _nbytes(ws), _stream(stream)))

    def stats(self):
        h, m, b = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
        _check(_lib.moe_expert_cache_stats(self._h, ctypes.byref(h), ctypes.byref(m), ctypes.byref(b)))
        return {"hits": h.value, "misses": m.value, "bytes_copied": b.value}

    def close(self):
        if self._h:
            _lib.moe_expert_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------------------
# dense operators
# ---------------------------------------------------------------------------

DTYPE_BF16, DTYPE_F16 = 0, 1
FN_NONE, FN_SILU, FN_GELU, FN_RELU = 0, 1, 2, 3
SAVE_NONE, SAVE_16, SAVE_8 = 0, 1, 2

_TORCH16 = (torch.bfloat16, torch.float16)


def _bad(message):
    return MoeError(1, message)


def _device():
    """The current CUDA device (-2, which no tensor is on, without one)."""
    try:
        return torch._C._cuda_getDevice()
    except (RuntimeError, AttributeError):
        return -2


def _tensor(t, name, dtype, shape, ld, dev):
    """Pointer of a tensor after its checks: type, shape, rows packed (or of
    pitch ld), on device dev. The library itself sees pointers only."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.get_device() == dev and \
            (t.is_contiguous() if not ld or ld == shape[-1] else _pitched(t, shape, ld)):
        return t.data_ptr()
    if t is None:
        raise _bad(f"{name} is None")
    if t.dtype is not dtype:
        raise _bad(f"{name} is {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise _bad(f"{name} has shape {tuple(t.shape)}, not {shape}")
    if t.get_device() != dev:
        raise _bad(f"{name} is on {t.device}, not on the current CUDA device")
    raise _bad(f"{name} has strides {t.stride()}, not rows of pitch {ld or shape[-1]}")


def _pitched(t, shape, ld):
    return (shape[1] == 1 or t.stride(1) == 1) and (shape[0] == 1 or t.stride(0) == ld)


def _opt(t, name, dtype, shape, ld, dev):
    return None if t is None else _tensor(t, name, dtype, shape, ld, dev)


def _ws_args(ws, dev):
    if ws.get_device() != dev or not ws.is_contiguous():
        raise _bad("the workspace is not a contiguous tensor on the current CUDA device")
    return ws.data_ptr(), ws.nbytes


def _raw_stream(stream, dev):
    """_stream() without building a Stream object for the current stream."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _types(dims):
    """(16-bit type, output type) of dims; dims out of range are left to the library."""
    t16 = _TORCH16[dims.dtype == DTYPE_F16]
    return t16, torch.float32 if dims.out_f32 else t16


def moe_dense_workspace_init(ws, stream=None):
    dev = _device()
    p, n = _ws_args(ws, dev)
    _check(_lib.moe_dense_workspace_init(p, n, _raw_stream(stream, dev)))


def _size(fn, dims):
    n = fn(ctypes.byref(dims))
    if n == 0:
        raise MoeError(2, _lib.moe_last_error().decode())
    return n


def moe_linear_workspace_size(dims: MoeLinearDims) -> int:
    """Bytes of workspace (raises for dims the library does not support)."""
    return _size(_lib.moe_linear_workspace_size, dims)


def moe_ffn_workspace_size(dims: MoeFfnDims) -> int:
    """Bytes of workspace (raises for dims the library does not support)."""
    return _size(_lib.moe_ffn_workspace_size, dims)


def moe_linear(dims, x, w, bias, residual, y, pre, ws, stream=None):
    """y = f(x W^T + bias) + residual; pre (or None) receives the argument of f."""
    t16, out = _types(dims)
    T, N, K, dev = dims.T, dims.N, dims.K, _device()
    wp, wn = _ws_args(ws, dev)
    _check(_lib.moe_linear(
        dims, _tensor(x, "x", t16, (T, K), dims.ldx, dev), _tensor(w, "w", t16, (N, K), 0, dev),
        _opt(bias, "bias", t16, (N,), 0, dev), _opt(residual, "residual", t16, (T, N), dims.ldr, dev),
        _tensor(y, "y", out, (T, N), dims.ldy, dev), _opt(pre, "pre", t16, (T, N), 0, dev), wp, wn,
        _raw_stream(stream, dev)))


def moe_linear_backward(dims, dy, x, w, pre, dx, dw, dbias, ws, stream=None):
    """Gradients of moe_linear; dx, dw and dbias may each be None (not wanted)."""
    t16, out = _types(dims)
    T, N, K, dev = dims.T, dims.N, dims.K, _device()
    wp, wn = _ws_args(ws, dev)
    _check(_lib.moe_linear_backward(
        dims, _tensor(dy, "dy", t16, (T, N), dims.ldy, dev), _opt(x, "x", t16, (T, K), dims.ldx, dev),
        _opt(w, "w", t16, (N, K), 0, dev), _opt(pre, "pre", t16, (T, N), 0, dev),
        _opt(dx, "dx", out, (T, K), dims.ldx, dev), _opt(dw, "dw", out, (N, K), 0, dev),
        _opt(dbias, "dbias", out, (N,), 0, dev), wp, wn, _raw_stream(stream, dev)))


class FfnSaved:
    """Saved activations of moe_ffn: g and u in 16 bits (SAVE_16), or g, u and
    x as 8-bit checkpoints (SAVE_8; keep_x=False when the caller keeps x
    itself). Buffers that are not given are allocated."""

    def __init__(self, dims: MoeFfnDims, g=None, u=None, keep_x=True, device="cuda"):
        T, H, I = dims.T, dims.H, dims.I
        self.g_s = self.u_s = self.x_q = self.x_s = None
        u8 = dict(dtype=torch.uint8, device=device)
        if dims.save == SAVE_16:
            t16 = _types(dims)[0]
            kind = dict(dtype=t16, device=device)
        elif dims.save == SAVE_8:
            kind = u8
            self.g_s = torch.empty(T, (I + 31) // 32, **u8)
            self.u_s = torch.empty(T, (I + 31) // 32, **u8)
            if keep_x:
                self.x_q = torch.empty(T, H, **u8)
                self.x_s = torch.empty(T, (H + 31) // 32, **u8)
        else:
            raise _bad("dims.save is SAVE_NONE: there is nothing to save")
        self.g = torch.empty(T, I, **kind) if g is None else g
        self.u = torch.empty(T, I, **kind) if u is None else u

    def _ptrs(self, dims, dev):
        T, H, I = dims.T, dims.H, dims.I
        t = torch.uint8 if dims.save == SAVE_8 else _types(dims)[0]
        ni, nh = (I + 31) // 32, (H + 31) // 32
        u8 = torch.uint8
        return _FfnSavedPtrs(
            _tensor(self.g, "saved.g", t, (T, I), 0, dev), _tensor(self.u, "saved.u", t, (T, I), 0, dev),
            _opt(self.g_s, "saved.g_s", u8, (T, ni), 0, dev), _opt(self.u_s, "saved.u_s", u8, (T, ni), 0, dev),
            _opt(self.x_q, "saved.x_q", u8, (T, H), 0, dev), _opt(self.x_s, "saved.x_s", u8, (T, nh), 0, dev))


def moe_ffn(dims, x, wg, wu, wd, residual, y, saved, ws, stream=None):
    """y = (f(x Wg^T) * (x Wu^T)) Wd^T + residual; saved: an FfnSaved, or None with SAVE_NONE."""
    t16, out = _types(dims)
    T, H, I, dev = dims.T, dims.H, dims.I, _device()
    wp, wn = _ws_args(ws, dev)
    _check(_lib.moe_ffn(
        dims, _tensor(x, "x", t16, (T, H), dims.ldx, dev), _tensor(wg, "wg", t16, (I, H), 0, dev),
        _tensor(wu, "wu", t16, (I, H), 0, dev), _tensor(wd, "wd", t16, (H, I), 0, dev),
        _opt(residual, "residual", t16, (T, H), dims.ldr, dev), _tensor(y, "y", out, (T, H), dims.ldy, dev),
        None if saved is None else saved._ptrs(dims, dev), wp, wn, _raw_stream(stream, dev)))


def moe_ffn_backward(dims, dy, x, wg, wu, wd, saved, dx, dwg, dwu, dwd, ws, stream=None):
    """Gradients of moe_ffn from `saved` (x None: from its 8-bit checkpoint);
    dx, dwd and the pair dwg, dwu may be None (not wanted)."""
    t16, out = _types(dims)
    T, H, I, dev = dims.T, dims.H, dims.I, _device()
    wp, wn = _ws_args(ws, dev)
    _check(_lib.moe_ffn_backward(
        dims, _tensor(dy, "dy", t16, (T, H), dims.ldy, dev), _opt(x, "x", t16, (T, H), dims.ldx, dev),
        _opt(wg, "wg", t16, (I, H), 0, dev), _opt(wu, "wu", t16, (I, H), 0, dev),
        _tensor(wd, "wd", t16, (H, I), 0, dev), None if saved is None else saved._ptrs(dims, dev),
        _opt(dx, "dx", out, (T, H), dims.ldx, dev), _opt(dwg, "dwg", out, (I, H), 0, dev),
        _opt(dwu, "dwu", out, (I, H), 0, dev), _opt(dwd, "dwd", out, (H, I), 0, dev), wp, wn,
        _raw_stream(stream, dev)))


def _rows16(t, name, dev):
    dtype = t.dtype
    if t.dim() != 2 or dtype not in _TORCH16:
        raise _bad(f"{name} is not a 2-D bf16 or f16 tensor")
    rows, cols = shape = t.shape
    ld = t.stride(0) if rows > 1 else cols
    return int(dtype is torch.float16), rows, cols, ld, _tensor(t, name, dtype, shape, ld, dev)


def moe_ckpt8_pack(src, q, s, stream=None):
    """src [rows, cols] (bf16 or f16, any row pitch) -> E4M3 codes q [rows, cols]
    and E8M0 scales s [rows, ceil(cols / 32)], both uint8."""
    dev = _device()
    dt, rows, cols, ld, p = _rows16(src, "src", dev)
    _check(_lib.moe_ckpt8_pack(dt, rows, cols, p, ld, _tensor(q, "q", torch.uint8, (rows, cols), 0, dev),
                               _tensor(s, "s", torch.uint8, (rows, (cols + 31) // 32), 0, dev),
                               _raw_stream(stream, dev)))


def moe_ckpt8_unpack(q, s, dst, stream=None):
    """The values an 8-bit checkpoint holds, into dst [rows, cols] (bf16 or f16)."""
    dev = _device()
    dt, rows, cols, ld, p = _rows16(dst, "dst", dev)
    _check(_lib.moe_ckpt8_unpack(dt, rows, cols, _tensor(q, "q", torch.uint8, (rows, cols), 0, dev),
                                 _tensor(s, "s", torch.uint8, (rows, (cols + 31) // 32), 0, dev), p, ld,
                                 _raw_stream(stream, dev)))


class MoeFfn:
    """Owns the device buffers of one gated feed-forward block (packed rows)
    and calls the C ABI on them. ``weights``: wg, wu [I, H] and wd [H, I]."""

    def __init__(self, dims: MoeFfnDims, weights: dict, device="cuda"):
        self.dims = dims
        self.w = {n: weights[n] for n in ("wg", "wu", "wd")}
        self.ws = torch.empty(moe_ffn_workspace_size(dims), dtype=torch.uint8, device=device)
        moe_dense_workspace_init(self.ws)
        t16, out = _types(dims)
        self.y = torch.empty(dims.T, dims.H, dtype=out, device=device)
        self.saved = None
        if dims.save != SAVE_NONE:
            self.saved = FfnSaved(dims, device=device)
            self.dx = torch.empty_like(self.y)
            self.dw = {n: torch.empty(w.shape, dtype=out, device=device) for n, w in self.w.items()}

    def __call__(self, x, residual=None, stream=None):
        w = self.w
        moe_ffn(self.dims, x, w["wg"], w["wu"], w["wd"], residual, self.y, self.saved, self.ws, stream)
        return self.y

    def backward(self, dy, x=None, stream=None):
        """(dx, {wg, wu, wd gradients}) of the last call; x is needed with SAVE_16."""
        w, dw = self.w, self.dw
        moe_ffn_backward(self.dims, dy, x, w["wg"], w["wu"], w["wd"], self.saved, self.dx, dw["wg"], dw["wu"],
                         dw["wd"], self.ws, stream)
        return self.dx, dw


# ---------------------------------------------------------------------------
# convenience: device buffers of one layer (allocation through torch only)
# ---------------------------------------------------------------------------

class MoeLayer:
    """Owns the device buffers of one layer shape and calls the C ABI on them.

    ``weights``: dict of device tensors (x excluded) named like the C ABI
    (w_router, wg_q, wg_s, wu_q, wu_s, wd_q, wd_s, w_sgate, ws_gate, ws_up,
    ws_down and, for latent layers, w_lat_down, w_lat_up; optionally e_bias,
    the router's fp32 selection bias [E]); bf16 tensors as
    int16/uint16 bit patterns or torch.bfloat16. Scales in the canonical
    layout; for ACT_MXFP4 the layer keeps tiled copies (moe_tile_scales) in
    ``self.w``, the weights every call uses.
    """

    def __init__(self, dims: MoeDims, weights: dict, device="cuda"):
        self.dims = dims
        d, T, k = dims, dims.T, dims.k
        W = d.L if d.L else d.H
        R = T * k
        self.w = dict(weights)
        if d.act_mode == ACT_MXFP4:
            for name, rows, K in (("wg_s", d.E * d.I, W), ("wu_s", d.E * d.I, W),
                                  ("wd_s", d.E * W, d.I)):
                tiled = torch.empty_like(weights[name])
                moe_tile_scales(weights[name], rows, K, tiled)
                self.w[name] = tiled
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        f32 = dict(dtype=torch.float32, device=dev)
        ws_bytes = moe_workspace_size(dims)
        if ws_bytes == 0:
            _check(1 if _lib.moe_last_error() else 2)
        self.ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        self.x_op = torch.empty(moe_x_op_size(dims), dtype=torch.uint8, device=dev)
        self.topk_idx = torch.empty(T, k, **i32)
        self.topk_w = torch.empty(T, k, **f32)
        self.logits = torch.empty(T, d.E, **f32)
        self.counts = torch.empty(d.E, **i32)
        self.offsets = torch.empty(d.E + 1, **i32)
        self.expert_list = torch.empty(d.E + 1, **i32)
        self.row_token = torch.empty(R, **i32)
        self.row_slot = torch.empty(R, **i32)
        self.slot_row = torch.empty(T, k, **i32)
        self.x_lat = torch.empty(T, d.L, dtype=torch.int16, device=dev) if d.L else None
        self.y_perm = torch.empty(R, W, **f32)
        self.y = torch.empty(T, d.H, **f32)
        moe_workspace_init(dims, self.ws)

    def layer_args(self, x) -> MoeLayerArgs:
        w = self.w
        g = lambda n: _ptr(w.get(n))
        return MoeLayerArgs(
            x=_ptr(x), w_router=g("w_router"), wg_q=g("wg_q"), wg_s=g("wg_s"), wu_q=g("wu_q"),
            wu_s=g("wu_s"), wd_q=g("wd_q"), wd_s=g("wd_s"), w_sgate=g("w_sgate"),
            ws_gate=g("ws_gate"), ws_up=g("ws_up"), ws_down=g("ws_down"),
            w_lat_down=g("w_lat_down"), w_lat_up=g("w_lat_up"), topk_idx=_ptr(self.topk_idx),
            topk_w=_ptr(self.topk_w), counts=_ptr(self.counts), offsets=_ptr(self.offsets),
            expert_list=_ptr(self.expert_list),
            row_token=_ptr(self.row_token), row_slot=_ptr(self.row_slot),
            slot_row=_ptr(self.slot_row), x_lat=_ptr(self.x_lat), x_op=_ptr(self.x_op),
            y_perm=_ptr(self.y_perm), y=_ptr(self.y), e_bias=g("e_bias"))

    def __call__(self, x, stream=None):
        """Whole layer (moe_layer); returns the fp32 output tensor [T, H]."""
        moe_layer(self.dims, self.layer_args(x), self.ws, stream)
        return self.y

    def stages(self, x, stream=None):
        """The same layer through the four step calls (route, [latent], permute,
        expert_ffn, combine); also fills self.logits."""
        d, w = self.dims, self.w
        moe_route_biased(d, x, w["w_router"], w.get("e_bias"), self.topk_idx, self.topk_w,
                         self.logits, self.ws, stream)
        xin = x
        if d.L:
            moe_latent_down(d, x, w["w_lat_down"], self.x_lat, self.ws, stream)
            xin = self.x_lat
        moe_permute(d, self.topk_idx, xin, self.counts, self.offsets, self.expert_list,
                    self.row_token, self.row_slot, self.slot_row, self.x_op, self.ws, stream)
        moe_expert_ffn(d, self.x_op, self.offsets, self.expert_list, self.row_token, w["wg_q"], w["wg_s"],
                       w["wu_q"], w["wu_s"], w["wd_q"], w["wd_s"], self.y_perm, self.ws, stream)
        moe_combine(d, self.y_perm, self.slot_row, self.topk_w, x, w["w_sgate"], w["ws_gate"],
                    w["ws_up"], w["ws_down"], w.get("w_lat_up"), self.y, self.ws, stream)
        return self.y
