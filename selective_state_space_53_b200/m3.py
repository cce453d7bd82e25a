"""ctypes binding of libm3.so (include/m3.h), argument marshalling only.

Every function takes torch tensors (device memory for tensor operands) and
passes raw pointers, sizes and the current CUDA stream to the C ABI.  All
arithmetic runs in the library's CUDA kernels; there is no other code path.
Loading fails loudly (``M3Error``) when the library is missing.
"""

from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libm3.so")

M3_F32, M3_BF16 = 0, 1
M3_FLAG_SEQUENTIAL = 1
M3_FLAG_ANGLE_DIRECT = 2
M3_FLAG_RAW_INPUTS = 4

_STATUS = {0: "M3_OK", -1: "M3_ERR_DIMS", -2: "M3_ERR_DTYPE", -3: "M3_ERR_ALIGN",
           -4: "M3_ERR_NULL", -5: "M3_ERR_WORKSPACE", -6: "M3_ERR_CUDA", -7: "M3_ERR_TIMEOUT",
           -8: "M3_ERR_UNSUPPORTED", -9: "M3_ERR_STATE"}


class M3Error(RuntimeError):
    def __init__(self, code, what=""):
        self.code = code
        name = _STATUS.get(code, str(code))
        super().__init__(f"{what}: {name}" if what else name)


class Dims(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("L", ctypes.c_int64), ("H", ctypes.c_int32),
                ("P", ctypes.c_int32), ("N", ctypes.c_int32), ("R", ctypes.c_int32),
                ("G", ctypes.c_int32), ("chunk", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


PAGES_MAX_BUF = 64


class PagesStruct(ctypes.Structure):
    """m3_pages: the buffers of a pool of states."""
    _fields_ = [("npages", ctypes.c_int32), ("nbuf", ctypes.c_int32), ("base", ctypes.c_void_p * PAGES_MAX_BUF),
                ("bytes", ctypes.c_int64 * PAGES_MAX_BUF)]


_lib = None

# Every symbol include/m3.h declares, with (restype, argtypes).
_VP, _SZ, _I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
_DP = ctypes.POINTER(Dims)
_PP = ctypes.POINTER(PagesStruct)
SIGNATURES = {
    "m3_state_bytes": (_I, [_DP, ctypes.POINTER(_SZ)]),
    "m3_state_alloc": (_I, [_DP, _VP, ctypes.POINTER(_VP)]),
    "m3_state_wrap": (_I, [_DP, _VP, _VP, _VP, ctypes.POINTER(_VP)]),
    "m3_state_free": (_I, [_VP]),
    "m3_state_tensors": (_I, [_VP, ctypes.POINTER(_VP), ctypes.POINTER(_VP), ctypes.POINTER(_VP)]),
    "m3_state_copy_to_host": (_I, [_VP, _VP, _SZ, _VP]),
    "m3_state_copy_from_host": (_I, [_VP, _VP, _SZ, _VP]),
    "m3_scan_workspace_size": (_I, [_DP, ctypes.POINTER(_SZ)]),
    "m3_scan_fwd": (_I, [_DP] + [_VP] * 14 + [_VP, _SZ, _VP]),
    "m3_scan_fwd_noalloc": (_I, [_DP] + [_VP] * 14 + [_VP]),
    "m3_decode_step": (_I, [_DP] + [_VP] * 15),
    "m3_output_norm": (_I, [_DP, _VP, _VP, _VP, ctypes.c_float, _VP, _VP]),
    "m3_frontend": (_I, [_DP] + [_VP] * 10 + [_VP]),
    "m3_scan_bwd_workspace_size": (_I, [_DP, ctypes.POINTER(_SZ)]),
    "m3_scan_bwd": (_I, [_DP] + [_VP] * 12 + [_VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "m3_scan_summary_workspace_size": (_I, [_DP, ctypes.POINTER(_SZ)]),
    "m3_scan_summary": (_I, [_DP] + [_VP] * 14 + [_VP, _SZ, _VP]),
    "m3_state_fold": (_I, [_DP, ctypes.c_int32] + [_VP] * 8 + [_VP, _VP]),
    "m3_linattn_workspace_size": (_I, [_DP, ctypes.POINTER(_SZ)]),
    "m3_linattn_fwd": (_I, [_DP] + [_VP] * 4 + [ctypes.c_float] + [_VP] * 3 + [ctypes.c_int64] + [_VP] * 3 + [_SZ, _VP]),
    "m3_linattn_step": (_I, [_DP] + [_VP] * 4 + [ctypes.c_float, _VP, ctypes.c_int64] + [_VP] * 3),
    "m3_linattn_bwd_workspace_size": (_I, [_DP, ctypes.POINTER(_SZ)]),
    "m3_linattn_bwd": (_I, [_DP] + [_VP] * 4 + [ctypes.c_float] + [_VP] * 9 + [_SZ, _VP]),
    "m3_pages_copy": (_I, [_PP, ctypes.c_int64] + [_VP] * 3),
    "m3_pages_fork": (_I, [_PP, _VP, ctypes.c_int64] + [_VP] * 3),
    "m3_pages_free": (_I, [_PP, _VP, ctypes.c_int64] + [_VP] * 2),
    "m3_pages_compact": (_I, [_PP] + [_VP] * 5),
    "m3_check": (_I, [_VP]),
    "m3_selftest_wait": (_I, [ctypes.c_uint64, _VP]),
    "m3_status_str": (ctypes.c_char_p, [_I]),
    "m3_version": (ctypes.c_char_p, []),
    "m3_last_error": (ctypes.c_char_p, []),
}


def lib():
    """Load libm3.so once; raise M3Error if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise M3Error(-6, f"{LIB_PATH} not built (python -m selective_state_space_53_b200.build)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(code, what):
    if code != 0:
        if code == -6:
            what = f"{what} ({lib().m3_last_error().decode()})"
        raise M3Error(code, what)


def make_dims(b, L, H, P, N, R, G=1, dtype="bf16", chunk=32, flags=0) -> Dims:
    dt = {"bf16": M3_BF16, "f32": M3_F32}[dtype] if isinstance(dtype, str) else int(dtype)
    return Dims(int(b), int(L), int(H), int(P), int(N), int(R), int(G), int(chunk), dt, int(flags))


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class State:
    """An m3_state handle.  ``State.wrap`` keeps torch tensors as the storage."""

    def __init__(self, handle, dims, keep=None):
        self.handle = handle
        self.dims = dims
        self._keep = keep

    @classmethod
    def alloc(cls, dims: Dims, stream=None):
        h = ctypes.c_void_p()
        _check(lib().m3_state_alloc(ctypes.byref(dims), _stream(stream), ctypes.byref(h)), "m3_state_alloc")
        return cls(h, dims)

    @classmethod
    def wrap(cls, dims: Dims, h, carry_B, carry_x):
        hd = ctypes.c_void_p()
        _check(lib().m3_state_wrap(ctypes.byref(dims), _ptr(h), _ptr(carry_B), _ptr(carry_x),
                                   ctypes.byref(hd)), "m3_state_wrap")
        return cls(hd, dims, keep=(h, carry_B, carry_x))

    def nbytes(self) -> int:
        n = ctypes.c_size_t()
        _check(lib().m3_state_bytes(ctypes.byref(self.dims), ctypes.byref(n)), "m3_state_bytes")
        return n.value

    def to_host(self, stream=None):
        import numpy as np
        buf = np.empty(self.nbytes() // 4, dtype=np.float32)
        _check(lib().m3_state_copy_to_host(self.handle, buf.ctypes.data_as(ctypes.c_void_p), buf.nbytes,
                                           _stream(stream)), "m3_state_copy_to_host")
        return buf

    def from_host(self, buf, stream=None):
        import numpy as np
        buf = np.ascontiguousarray(buf, dtype=np.float32)
        _check(lib().m3_state_copy_from_host(self.handle, buf.ctypes.data_as(ctypes.c_void_p), buf.nbytes,
                                             _stream(stream)), "m3_state_copy_from_host")

    def tensors(self):
        """(h, carry_B, carry_x) device pointers as ints."""
        a, b, c = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
        _check(lib().m3_state_tensors(self.handle, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)),
               "m3_state_tensors")
        return a.value, b.value, c.value

    def free(self):
        if self.handle is not None and self.handle.value:
            _check(lib().m3_state_free(self.handle), "m3_state_free")
        self.handle = None
        self._keep = None

    def __del__(self):
        try:
            if self.handle is not None and self.handle.value:
                lib().m3_state_free(self.handle)
        except Exception:
            pass


def m3_scan_workspace_size(dims: Dims) -> int:
    n = ctypes.c_size_t()
    _check(lib().m3_scan_workspace_size(ctypes.byref(dims), ctypes.byref(n)), "m3_scan_workspace_size")
    return n.value


def m3_scan_fwd(dims: Dims, x, dt, A, lam, B, C, theta, bias_B, bias_C, W_x, W_o, D, state: State, y,
                workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().m3_scan_fwd(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(lam), _ptr(B), _ptr(C),
                             _ptr(theta), _ptr(bias_B), _ptr(bias_C), _ptr(W_x), _ptr(W_o), _ptr(D),
                             state.handle, _ptr(y), _ptr(workspace), ws_bytes, _stream(stream)),
           "m3_scan_fwd")


def m3_scan_fwd_noalloc(dims: Dims, x, dt, A, lam, B, C, theta, bias_B, bias_C, W_x, W_o, D, state: State, y,
                        stream=None):
    """m3_scan_fwd without a workspace: the library's fixed 16 MiB device scratch is used
    (for callers that cannot allocate; calls overlapping on the GPU race on it)."""
    _check(lib().m3_scan_fwd_noalloc(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(lam), _ptr(B), _ptr(C),
                                     _ptr(theta), _ptr(bias_B), _ptr(bias_C), _ptr(W_x), _ptr(W_o), _ptr(D),
                                     state.handle, _ptr(y), _stream(stream)), "m3_scan_fwd_noalloc")


def m3_decode_step(dims: Dims, x_t, dt_t, A_t, lam_t, B_t, C_t, theta_t, bias_B, bias_C, W_x, W_o, D,
                   state: State, y_t, stream=None):
    _check(lib().m3_decode_step(ctypes.byref(dims), _ptr(x_t), _ptr(dt_t), _ptr(A_t), _ptr(lam_t), _ptr(B_t),
                                _ptr(C_t), _ptr(theta_t), _ptr(bias_B), _ptr(bias_C), _ptr(W_x), _ptr(W_o),
                                _ptr(D), state.handle, _ptr(y_t), _stream(stream)), "m3_decode_step")


def m3_scan_summary_workspace_size(dims: Dims) -> int:
    n = ctypes.c_size_t()
    _check(lib().m3_scan_summary_workspace_size(ctypes.byref(dims), ctypes.byref(n)),
           "m3_scan_summary_workspace_size")
    return n.value


def m3_scan_summary(dims: Dims, x, dt, A, lam, B, theta, bias_B, W_x, Z, logdec, angle, bp_first, carry_B,
                    carry_x, workspace, stream=None):
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib().m3_scan_summary(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(lam), _ptr(B), _ptr(theta),
                                 _ptr(bias_B), _ptr(W_x), _ptr(Z), _ptr(logdec), _ptr(angle), _ptr(bp_first),
                                 _ptr(carry_B), _ptr(carry_x), _ptr(workspace), ws_bytes, _stream(stream)),
           "m3_scan_summary")


def m3_state_fold(dims: Dims, nranges: int, Z, logdec, angle, bp_first, carry_B, carry_x, bias_B, W_x,
                  state: State, stream=None):
    _check(lib().m3_state_fold(ctypes.byref(dims), int(nranges), _ptr(Z), _ptr(logdec), _ptr(angle),
                               _ptr(bp_first), _ptr(carry_B), _ptr(carry_x), _ptr(bias_B), _ptr(W_x),
                               state.handle, _stream(stream)), "m3_state_fold")


def m3_frontend(dims: Dims, B_raw, C_raw, dt_raw, A_raw, lam_raw, B, C, dt, A, lam, stream=None):
    _check(lib().m3_frontend(ctypes.byref(dims), _ptr(B_raw), _ptr(C_raw), _ptr(dt_raw), _ptr(A_raw), _ptr(lam_raw),
                             _ptr(B), _ptr(C), _ptr(dt), _ptr(A), _ptr(lam), _stream(stream)), "m3_frontend")


def m3_output_norm(dims: Dims, y, z, weight, eps, out, stream=None):
    _check(lib().m3_output_norm(ctypes.byref(dims), _ptr(y), _ptr(z), _ptr(weight), float(eps), _ptr(out),
                                _stream(stream)), "m3_output_norm")


GRAD_KEYS = ("dx", "ddt", "dA", "dlam", "dB", "dC", "dtheta", "dbias_B", "dbias_C", "dW_x", "dW_o", "dD",
             "dh0", "dcarry_B", "dcarry_x")


class Grads(ctypes.Structure):
    """m3_grads: device pointers of the gradients (None where not wanted)."""
    _fields_ = [(k, ctypes.c_void_p) for k in GRAD_KEYS]


def m3_scan_bwd_workspace_size(dims: Dims) -> int:
    n = ctypes.c_size_t()
    _check(lib().m3_scan_bwd_workspace_size(ctypes.byref(dims), ctypes.byref(n)), "m3_scan_bwd_workspace_size")
    return n.value


def m3_scan_bwd(dims: Dims, x, dt, A, lam, B, C, theta, bias_B, bias_C, W_x, W_o, D, state0: State, dy,
                dh_final, grads: dict, workspace=None, stream=None):
    g = Grads(*[(None if grads.get(k) is None else grads[k].data_ptr()) for k in GRAD_KEYS])
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().m3_scan_bwd(ctypes.byref(dims), _ptr(x), _ptr(dt), _ptr(A), _ptr(lam), _ptr(B), _ptr(C),
                             _ptr(theta), _ptr(bias_B), _ptr(bias_C), _ptr(W_x), _ptr(W_o), _ptr(D), state0.handle,
                             _ptr(dy), _ptr(dh_final), ctypes.byref(g), _ptr(workspace), ws_bytes, _stream(stream)),
           "m3_scan_bwd")


def scan_backward(dims: Dims, dev: dict, state0: State, dy, dh_final=None, stream=None):
    """m3_scan_bwd on a dict from ``to_device``: allocates the gradients (every one of them) and
    the workspace; returns the gradients keyed by GRAD_KEYS."""
    import torch
    d = dev["x"].device
    b, L, H, P, N, R, G = dims.b, dims.L, dims.H, dims.P, dims.N, dims.R, dims.G
    f32 = dict(dtype=torch.float32, device=d)
    out = {"dx": torch.empty_like(dev["x"]), "ddt": torch.empty((b, L, H), **f32), "dA": torch.empty((b, L, H), **f32),
           "dlam": torch.empty((b, L, H), **f32), "dB": torch.empty_like(dev["B"]), "dC": torch.empty_like(dev["C"]),
           "dtheta": torch.empty((b, L, G, N // 2), **f32), "dbias_B": torch.empty((H, R, N), **f32),
           "dbias_C": torch.empty((H, R, N), **f32), "dW_x": torch.empty((H, R, P), **f32),
           "dW_o": torch.empty((H, R, P), **f32), "dD": torch.empty((H,), **f32),
           "dh0": torch.empty((b, H, N, P), **f32), "dcarry_B": torch.empty((b, H, R, N), **f32),
           "dcarry_x": torch.empty((b, H, P), **f32)}
    n = m3_scan_bwd_workspace_size(dims)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device=d)
    m3_scan_bwd(dims, *[dev[k] for k in _OPERANDS], state0, dy, dh_final, out, workspace=ws, stream=stream)
    return out


def _call_stream(index, stream):
    """Raw handle of the stream a call on tensors of CUDA device `index` runs on: `stream`, or the device's
    current one.  None when the call has to switch to that device or stream first (``_elsewhere``).  A stream
    of another device is refused: it could not order the work that the caller asks it to."""
    import torch
    if stream is not None and getattr(stream, "device_index", index) != index:
        raise M3Error(-1, f"stream is on cuda:{stream.device_index}, expected the tensors' device cuda:{index}")
    if stream is None and torch._C._cuda_getDevice() == index:
        return torch._C._cuda_getCurrentRawStream(index)
    return None


def _elsewhere(device, stream, *operands):
    """Context that makes the device current, and `stream` if given (allocations then belong to it too, and the
    operands' memory is not handed out again before it has run the call)."""
    import torch
    if stream is not None:
        for t in operands:
            if t is not None:
                t.record_stream(stream)
    return torch.cuda.device(device) if stream is None else torch.cuda.stream(stream)


def _expect(what, name, t, shape, dtype, device):
    if t.device != device or device.type != "cuda":
        raise M3Error(-1, f"{what}: {name} is on {t.device}, expected the CUDA device of the other tensors")
    if t.dtype != dtype:
        raise M3Error(-2, f"{what}: {name} is {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise M3Error(-1, f"{what}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise M3Error(-1, f"{what}: {name} is not contiguous")


def _la_dims(what, q, k, v, log_decay, token):
    """Dims of a linear attention call from its tensors, after their checks (token: no L axis)."""
    import torch
    sq, sv, dtype, dev = q.shape, v.shape, q.dtype, q.device
    if len(sq) != (3 if token else 4) or len(sv) != len(sq):
        raise M3Error(-1, f"{what}: q has {len(sq)} and v {len(sv)} dimensions, expected {3 if token else 4}")
    if dtype is torch.bfloat16:
        dt = M3_BF16
    elif dtype is torch.float32:
        dt = M3_F32
    else:
        raise M3Error(-2, f"{what}: q is {dtype}, expected bfloat16 or float32")
    b, G, N = sq[0], sq[-2], sq[-1]
    H, P = sv[-2], sv[-1]
    L = 1 if token else sq[1]
    if not (sv[0] == b and (token or sv[1] == L) and k.shape == sq and k.dtype is dtype and v.dtype is dtype
            and log_decay.dtype is torch.float32 and log_decay.shape == (H,) and dev.type == "cuda"
            and k.device == dev and v.device == dev and log_decay.device == dev and q.is_contiguous()
            and k.is_contiguous() and v.is_contiguous() and log_decay.is_contiguous()):
        _expect(what, "q", q, sq, dtype, dev)
        _expect(what, "k", k, sq, dtype, dev)
        _expect(what, "v", v, (b, H, P) if token else (b, L, H, P), dtype, dev)
        _expect(what, "log_decay", log_decay, (H,), torch.float32, dev)
    return Dims(b, L, H, P, N, 1, G, 0, dt, 0)


def _la_rows(what, dims, state, pages, device):
    """Rows of the state pool a call works on, after the checks of state and pages."""
    import torch
    rows = dims.b if pages is None else state.shape[0]
    shape = (rows, dims.H, dims.N, dims.P)
    if not (state.dtype is torch.float32 and state.shape == shape and state.device == device and state.is_contiguous()):
        _expect(what, "state", state, shape, torch.float32, device)
    if pages is not None and not (pages.dtype is torch.int32 and pages.shape == (dims.b,) and pages.device == device
                                  and pages.is_contiguous()):
        _expect(what, "pages", pages, (dims.b,), torch.int32, device)
    return rows


def _adr(t):
    return None if t is None else t.data_ptr()


def _raw(stream):
    """Raw handle of a stream, given as one already, as a torch stream or not at all (the current one)."""
    return stream if stream.__class__ is int else _stream(stream)


def m3_linattn_workspace_size(dims: Dims) -> int:
    n = ctypes.c_size_t()
    _check(lib().m3_linattn_workspace_size(ctypes.byref(dims), ctypes.byref(n)), "m3_linattn_workspace_size")
    return n.value


def m3_linattn_fwd(dims: Dims, q, k, v, log_decay, scale, lens, state_in, state_out, npages, pages, y,
                   workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().m3_linattn_fwd(ctypes.byref(dims), _adr(q), _adr(k), _adr(v), _adr(log_decay), scale, _adr(lens),
                                _adr(state_in), _adr(state_out), npages, _adr(pages), _adr(y), _adr(workspace),
                                ws_bytes, _raw(stream)), "m3_linattn_fwd")


def m3_linattn_step(dims: Dims, q_t, k_t, v_t, log_decay, scale, state, npages, pages, y_t, stream=None):
    _check(lib().m3_linattn_step(ctypes.byref(dims), _adr(q_t), _adr(k_t), _adr(v_t), _adr(log_decay), scale,
                                 _adr(state), npages, _adr(pages), _adr(y_t), _raw(stream)), "m3_linattn_step")


def m3_linattn_bwd_workspace_size(dims: Dims) -> int:
    n = ctypes.c_size_t()
    _check(lib().m3_linattn_bwd_workspace_size(ctypes.byref(dims), ctypes.byref(n)), "m3_linattn_bwd_workspace_size")
    return n.value


def m3_linattn_bwd(dims: Dims, q, k, v, log_decay, scale, lens, state_in, dy, dstate_out, dq, dk, dv, dstate_in,
                   workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().m3_linattn_bwd(ctypes.byref(dims), _adr(q), _adr(k), _adr(v), _adr(log_decay), scale, _adr(lens),
                                _adr(state_in), _adr(dy), _adr(dstate_out), _adr(dq), _adr(dk), _adr(dv),
                                _adr(dstate_in), _adr(workspace), ws_bytes, _raw(stream)), "m3_linattn_bwd")


def linattn(q, k, v, log_decay, scale=None, lens=None, state=None, pages=None, y=None, workspace=None, stream=None):
    """Linear attention with a decay per head over a batch of sequences (m3_linattn_fwd).

    q, k (b, L, G, N), v (b, L, H, P) in bf16 (products on the tensor cores where the sizes allow) or in fp32
    (fp32 arithmetic throughout), G dividing H; log_decay (H) fp32; scale: N ** -0.5 if not given; lens (b) int32: the lengths of a padded batch.  state (b, H, N, P) fp32, updated in
    place, or with pages (b) int32 the rows of a pool (npages, H, N, P); without it the sequences are
    fresh.  workspace: a contiguous tensor of m3_linattn_workspace_size bytes on the same device, else
    one is allocated.  Returns (y, state)."""
    import torch
    what = "linattn"
    dims = _la_dims(what, q, k, v, log_decay, False)
    dev = q.device
    if lens is not None:
        _expect(what, "lens", lens, (dims.b,), torch.int32, dev)
    if pages is not None and state is None:
        raise M3Error(-4, f"{what}: pages need a state pool")
    rows = dims.b if state is None else _la_rows(what, dims, state, pages, dev)
    if y is not None:
        _expect(what, "y", y, v.shape, v.dtype, dev)
    if workspace is not None:  # any type; its bytes are checked by the library
        _expect(what, "workspace", workspace, workspace.shape, workspace.dtype, dev)
    raw = _call_stream(dev.index, stream)
    if raw is None:
        with _elsewhere(dev, stream, q, k, v, log_decay, lens, state, pages, y, workspace):
            return linattn(q, k, v, log_decay, scale, lens, state, pages, y, workspace)
    out = state
    if out is None:
        out = torch.empty((dims.b, dims.H, dims.N, dims.P), dtype=torch.float32, device=dev)
    if y is None:
        y = torch.empty_like(v)
    if workspace is None:
        n = m3_linattn_workspace_size(dims)
        workspace = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    m3_linattn_fwd(dims, q, k, v, log_decay, dims.N ** -0.5 if scale is None else scale, lens, state, out, rows, pages,
                   y, workspace, raw)
    return y, out


def linattn_step(q, k, v, log_decay, state, scale=None, pages=None, y=None, stream=None):
    """One token of every sequence (m3_linattn_step): q, k (b, G, N), v (b, H, P); state and pages as
    for linattn, updated in place.  Returns y (b, H, P)."""
    import torch
    what = "linattn_step"
    dims = _la_dims(what, q, k, v, log_decay, True)
    dev = q.device
    rows = _la_rows(what, dims, state, pages, dev)
    if y is not None:
        _expect(what, "y", y, v.shape, v.dtype, dev)
    raw = _call_stream(dev.index, stream)
    if raw is None:
        with _elsewhere(dev, stream, q, k, v, log_decay, state, pages, y):
            return linattn_step(q, k, v, log_decay, state, scale, pages, y)
    if y is None:
        y = torch.empty_like(v)
    m3_linattn_step(dims, q, k, v, log_decay, dims.N ** -0.5 if scale is None else scale, state, rows, pages, y, raw)
    return y


def linattn_backward(q, k, v, log_decay, dy, scale=None, lens=None, state0=None, dstate=None, stream=None):
    """Gradients of linattn (m3_linattn_bwd): dy like v; state0 the states the sequences started from
    and dstate the gradient of the ones they ended in, (b, H, N, P) fp32 or None (zero).  Returns
    {"dq", "dk", "dv", "dstate0"}."""
    import torch
    what = "linattn_backward"
    dims = _la_dims(what, q, k, v, log_decay, False)
    dev = q.device
    _expect(what, "dy", dy, v.shape, v.dtype, dev)
    if lens is not None:
        _expect(what, "lens", lens, (dims.b,), torch.int32, dev)
    for name, t in (("state0", state0), ("dstate", dstate)):
        if t is not None:
            _expect(what, name, t, (dims.b, dims.H, dims.N, dims.P), torch.float32, dev)
    raw = _call_stream(dev.index, stream)
    if raw is None:
        with _elsewhere(dev, stream, q, k, v, log_decay, dy, lens, state0, dstate):
            return linattn_backward(q, k, v, log_decay, dy, scale, lens, state0, dstate)
    out = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
           "dstate0": torch.empty((dims.b, dims.H, dims.N, dims.P), dtype=torch.float32, device=dev)}
    n = m3_linattn_bwd_workspace_size(dims)
    ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    m3_linattn_bwd(dims, q, k, v, log_decay, dims.N ** -0.5 if scale is None else scale, lens, state0, dy, dstate,
                   *[out[g] for g in ("dq", "dk", "dv", "dstate0")], ws, raw)
    return out


class Pages:
    """A pool of recurrent states (m3_pages): `bufs` are the model's state buffers, contiguous tensors
    that share their leading axis; page i is row i of all of them.  `live` (npages) int32 marks the
    pages in use (all free if not given).  Page lists are int32 tensors on the pool's device; every
    call is asynchronous on the current stream (or `stream`)."""

    def __init__(self, bufs, live=None):
        import torch
        bufs = list(bufs)
        if not 1 <= len(bufs) <= PAGES_MAX_BUF:
            raise M3Error(-1, f"Pages: {len(bufs)} buffers, expected 1 to {PAGES_MAX_BUF}")
        self.device = bufs[0].device
        self.npages = bufs[0].shape[0] if bufs[0].dim() else 0
        if self.npages > 0x7fffffff:
            raise M3Error(-1, f"Pages: {self.npages} pages, expected fewer than 2^31")
        s = PagesStruct(self.npages, len(bufs))
        for j, t in enumerate(bufs):
            if t.dim() < 2:
                raise M3Error(-1, f"Pages: buffer {j} has no page axis")
            _expect("Pages", f"buffer {j}", t, (self.npages, *t.shape[1:]), t.dtype, self.device)
            s.base[j] = t.data_ptr()
            s.bytes[j] = t[0].numel() * t.element_size() if self.npages else 16
        if live is None:
            live = torch.zeros(self.npages, dtype=torch.int32, device=self.device)
        _expect("Pages", "live", live, (self.npages,), torch.int32, self.device)
        self.bufs, self.live, self.struct, self._ref = bufs, live, s, ctypes.byref(s)

    def _list(self, what, name, t):
        import torch
        shape = t.shape
        if len(shape) != 1:
            raise M3Error(-1, f"{what}: {name} has shape {tuple(shape)}, expected one axis")
        if not (t.dtype is torch.int32 and t.device == self.device and t.is_contiguous()):
            _expect(what, name, t, shape, torch.int32, self.device)
        return shape[0]

    def copy(self, src, dst, stream=None):
        """Page dst[i] becomes a copy of page src[i], in list order (m3_pages_copy)."""
        n = self._list("Pages.copy", "src", src)
        if self._list("Pages.copy", "dst", dst) != n:
            raise M3Error(-1, "Pages.copy: src and dst have different lengths")
        raw = _call_stream(self.device.index, stream)
        if raw is None:
            with _elsewhere(self.device, stream, src, dst, *self.bufs):
                return self.copy(src, dst)
        _check(lib().m3_pages_copy(self._ref, n, src.data_ptr(), dst.data_ptr(), raw), "m3_pages_copy")

    def fork(self, src, stream=None):
        """Take a free page for each entry and make it a copy of page src[i], or all zero where src[i]
        is negative (m3_pages_fork).  Returns the pages taken, (n) int32."""
        import torch
        n = self._list("Pages.fork", "src", src)
        raw = _call_stream(self.device.index, stream)
        if raw is None:
            with _elsewhere(self.device, stream, src, self.live, *self.bufs):
                return self.fork(src)
        dst = torch.empty_like(src)
        _check(lib().m3_pages_fork(self._ref, self.live.data_ptr(), n, src.data_ptr(), dst.data_ptr(), raw),
               "m3_pages_fork")
        return dst

    def free(self, idx, stream=None):
        """The pages idx become free (m3_pages_free)."""
        n = self._list("Pages.free", "idx", idx)
        raw = _call_stream(self.device.index, stream)
        if raw is None:
            with _elsewhere(self.device, stream, idx, self.live):
                return self.free(idx)
        _check(lib().m3_pages_free(self._ref, self.live.data_ptr(), n, idx.data_ptr(), raw), "m3_pages_free")

    def compact(self, stream=None):
        """Move the live pages to the front, in order (m3_pages_compact).  Returns (map, count): map
        (npages) int32 says where each page went (-1: it was free), count (1) int32 how many are live."""
        import torch
        raw = _call_stream(self.device.index, stream)
        if raw is None:
            with _elsewhere(self.device, stream, self.live, *self.bufs):
                return self.compact()
        n = self.npages
        out = torch.empty((2 * n + 2,), dtype=torch.int32, device=self.device)  # map, order, count
        at = out.data_ptr()
        _check(lib().m3_pages_compact(self._ref, self.live.data_ptr(), at, at + 4 * n, at + 8 * n, raw),
               "m3_pages_compact")
        return out[:n], out[2 * n:2 * n + 1]


def m3_check(stream=None) -> int:
    return int(lib().m3_check(_stream(stream)))


def m3_selftest_wait(limit_ns: int, stream=None):
    _check(lib().m3_selftest_wait(int(limit_ns), _stream(stream)), "m3_selftest_wait")


def m3_status_str(code: int) -> str:
    return lib().m3_status_str(int(code)).decode()


def m3_version() -> str:
    return lib().m3_version().decode()


# ---- marshalling helpers: seeded host draws -> device tensors

_OPERANDS = ("x", "dt", "A", "lam", "B", "C", "theta", "bias_B", "bias_C", "W_x", "W_o", "D")


def to_device(inp, device="cuda"):
    """Copy an ``inputs.Inputs`` draw to the device in its storage dtypes
    (x, B, C in the draw's dtype; everything else fp32).  Returns a dict."""
    import torch
    tdt = torch.bfloat16 if inp.dims["dtype"] == "bf16" else torch.float32
    out = {}
    for k in _OPERANDS:
        a = getattr(inp, k)
        if a is None:
            out[k] = None
            continue
        t = torch.from_numpy(a)
        if k in ("x", "B", "C"):
            t = t.to(tdt)
        out[k] = t.to(device).contiguous()
    return out


def dims_of(inp, L=None, flags=0, b=None) -> Dims:
    d = inp.dims
    return make_dims(d["b"] if b is None else b, d["L"] if L is None else L, d["H"], d["P"], d["N"], d["R"],
                     d["G"], d["dtype"], flags=flags)


def state_tensors(dims: Dims, device="cuda", h=None, carry_B=None, carry_x=None):
    """Torch-owned state buffers (zeros unless given) and their m3_state handle."""
    import torch
    b, H, N, P, R = dims.b, dims.H, dims.N, dims.P, dims.R
    th = torch.zeros((b, H, N, P), dtype=torch.float32, device=device) if h is None else \
        torch.as_tensor(h, dtype=torch.float32).to(device).contiguous()
    tb = torch.zeros((b, H, R, N), dtype=torch.float32, device=device) if carry_B is None else \
        torch.as_tensor(carry_B, dtype=torch.float32).to(device).contiguous()
    tx = torch.zeros((b, H, P), dtype=torch.float32, device=device) if carry_x is None else \
        torch.as_tensor(carry_x, dtype=torch.float32).to(device).contiguous()
    return State.wrap(dims, th, tb, tx), (th, tb, tx)


def scan(dims: Dims, dev: dict, state: State, y=None, workspace=None, stream=None):
    """m3_scan_fwd on a dict from ``to_device``; allocates y if not given."""
    import torch
    if y is None:
        y = torch.empty_like(dev["x"])
    if workspace is None:
        n = m3_scan_workspace_size(dims)
        workspace = torch.empty(n, dtype=torch.uint8, device=dev["x"].device) if n else None
    m3_scan_fwd(dims, *[dev[k] for k in _OPERANDS], state, y, workspace=workspace, stream=stream)
    return y


def decode(dims: Dims, tok: dict, state: State, y=None, stream=None):
    """m3_decode_step on one token's operands (dict with x (b,H,P), dt (b,H), ...)."""
    import torch
    if y is None:
        y = torch.empty_like(tok["x"])
    m3_decode_step(dims, *[tok[k] for k in _OPERANDS], state, y, stream=stream)
    return y
