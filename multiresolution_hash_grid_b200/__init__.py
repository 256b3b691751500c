"""Python binding of libhashgrid.so, the B200 (sm_100a) multiresolution hash-grid encoding.

Argument marshalling only: every step of the encoding runs in the library's CUDA kernels.
PyTorch supplies device memory and streams. The functions carry the C ABI's names
(``include/hashgrid.h`` documents semantics, layouts and errors) and take either torch
CUDA tensors or raw integer device pointers; ``stream`` defaults to torch's current
stream. A nonzero status raises ``HashGridError`` with the library's message.

The library must be built (``python multiresolution_hash_grid_b200/build.py``); importing
this package without it raises ImportError. There is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
# HASHGRID_CHECKED=1 loads the checked build (every global access of the kernels range-checked,
# violations returned as HASHGRID_ERR_DEVICE_CHECK; synchronous, for testing).
CHECKED = os.environ.get("HASHGRID_CHECKED", "0") not in ("", "0")
LIB_PATH = os.path.join(HERE, "libhashgrid_checked.so" if CHECKED else "libhashgrid.so")

HASHGRID_F32 = 0
HASHGRID_F16 = 1
HASHGRID_BF16 = 2
HASHGRID_E4M3 = 3

HASHGRID_ACT_NONE = 0
HASHGRID_ACT_RELU = 1
HASHGRID_ACT_GELU = 2
HASHGRID_ACT_SILU = 3
HASHGRID_ADAMW_BLOCK = 256

HASHGRID_OK = 0
HASHGRID_ERR_ARG = 1
HASHGRID_ERR_ALIGN = 2
HASHGRID_ERR_CUDA = 3
HASHGRID_ERR_OOM = 4
HASHGRID_ERR_DEVICE_CHECK = 5
HASHGRID_ERR_TIMEOUT = 6

MAX_LEVELS = 32

HASHGRID_OPT_FORWARD_GATHER = 0
HASHGRID_OPT_BACKWARD_MODE = 1
HASHGRID_OPT_SCHEDULE = 2
HASHGRID_SCHEDULE_AUTO = 0
HASHGRID_SCHEDULE_POINT_MAJOR = 1
HASHGRID_SCHEDULE_LEVEL_MAJOR = 2
HASHGRID_GATHER_AUTO = 0
HASHGRID_GATHER_CORNER = 1
HASHGRID_GATHER_SECTOR = 2
HASHGRID_GATHER_PAIR = 3
HASHGRID_GATHER_LANES = 4
HASHGRID_BACKWARD_AUTO = 0
HASHGRID_BACKWARD_ATOMIC = 1
HASHGRID_BACKWARD_WARP_DEDUP = 2
HASHGRID_BACKWARD_RUN_MERGE = 3
HASHGRID_BACKWARD_WARP_DEDUP_ADAPTIVE = 4
HASHGRID_BACKWARD_RUN_LANES = 5
HASHGRID_PROBE_GATHER = 0
HASHGRID_PROBE_RED = 1
HASHGRID_PROBE_RED_F16 = 2
HASHGRID_PROBE_RANDOM = 0
HASHGRID_PROBE_XPAIR = 1
HASHGRID_PROBE_SECTOR_PAIR = 2
HASHGRID_PROBE_LINE_PAIR = 3
HASHGRID_PROBE_STREAM = 4


class HashGridError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"hashgrid error {code}: {message}")
        self.code = code


class AdamwTensor(ctypes.Structure):
    """``struct hashgrid_adamw_tensor``."""
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("state_dtype", ctypes.c_int32), ("copy_dtype", ctypes.c_int32), ("lr_scale", ctypes.c_float),
                ("weight_decay", ctypes.c_float)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run `python multiresolution_hash_grid_b200/build.py"
                          f"{' --checked' if CHECKED else ''}`")
    lib = ctypes.CDLL(LIB_PATH)
    i32, i64, vp, sz = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    protos = {
        "hashgrid_create": (i32, [i32, i32, i32, i32, i32, i32, ctypes.POINTER(vp)]),
        "hashgrid_create_nd": (i32, [i32, i32, i32, i32, i32, i32, i32, ctypes.POINTER(vp)]),
        "hashgrid_dims": (i32, [vp]),
        "hashgrid_destroy": (i32, [vp]),
        "hashgrid_resolutions": (i32, [vp, ctypes.POINTER(i32)]),
        "hashgrid_table_elems": (sz, [vp]),
        "hashgrid_output_width": (i32, [vp]),
        "hashgrid_params": (i32, [vp] + [ctypes.POINTER(i32)] * 6),
        "hashgrid_set_option": (i32, [vp, i32, i32]),
        "hashgrid_get_option": (i32, [vp, i32, ctypes.POINTER(i32)]),
        "hashgrid_forward": (i32, [vp, vp, i64, vp, vp, vp]),
        "hashgrid_backward": (i32, [vp, vp, vp, i64, vp, vp]),
        "hashgrid_backward_input": (i32, [vp, vp, vp, i64, vp, vp, vp]),
        "hashgrid_backward_half": (i32, [vp, vp, vp, i64, vp, vp]),
        "hashgrid_adam_step": (i32, [vp, vp, vp, vp, vp, i64, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                     ctypes.c_float, i32, vp]),
        "hashgrid_mlp_forward": (i32, [vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
        "hashgrid_linear_create": (i32, [i32, i32, i32, i32, ctypes.POINTER(vp)]),
        "hashgrid_linear_destroy": (i32, [vp]),
        "hashgrid_linear_params": (i32, [vp] + [ctypes.POINTER(i32)] * 4),
        "hashgrid_linear_forward": (i32, [vp, vp, i64, i64, vp, vp, vp, i64, vp, i64, i32, vp, vp, sz, vp, vp]),
        "hashgrid_linear_forward_workspace": (sz, [vp, i64, i64]),
        "hashgrid_linear_backward_workspace": (sz, [vp, i64, i64, i64]),
        "hashgrid_linear_backward": (i32, [vp, vp, i64, vp, i64, i64, vp, vp, vp, i64, i32, vp, i32, vp, vp, sz, vp, vp]),
        "hashgrid_linear_status": (i32, []),
        "hashgrid_debug_wait_limit": (i32, [i64]),
        "hashgrid_adamw_create": (i32, [ctypes.POINTER(AdamwTensor), i32, ctypes.POINTER(vp)]),
        "hashgrid_adamw_destroy": (i32, [vp]),
        "hashgrid_adamw_step": (i32, [vp, i64, vp, ctypes.c_float, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                      ctypes.c_uint32, i32, vp]),
        "hashgrid_debug_indices": (i32, [vp, vp, i64, vp, vp]),
        "hashgrid_probe": (i32, [i32, i32, i32, vp, sz, i64, vp, ctypes.POINTER(i64), vp]),
        "hashgrid_last_error": (ctypes.c_char_p, []),
        "hashgrid_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in protos.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


lib = _load()


def _check(rc: int) -> None:
    if rc != HASHGRID_OK:
        raise HashGridError(rc, lib.hashgrid_last_error().decode())


def _ptr(a) -> int | None:
    if a is None or isinstance(a, int):
        return a
    return a.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _current_stream() -> int:
    """Torch's current stream on the current device."""
    global _current_stream
    import torch
    device, raw = torch.cuda.current_device, torch._C._cuda_getCurrentRawStream

    def _current_stream():
        return raw(device())
    return _current_stream()


def hashgrid_version() -> str:
    return lib.hashgrid_version().decode()


def hashgrid_last_error() -> str:
    return lib.hashgrid_last_error().decode()


def hashgrid_create(L: int, F: int, log2T: int, N_min: int, N_max: int, dtype: int = HASHGRID_F32) -> int:
    h = ctypes.c_void_p()
    _check(lib.hashgrid_create(L, F, log2T, N_min, N_max, dtype, ctypes.byref(h)))
    return h.value


def hashgrid_create_nd(D: int, L: int, F: int, log2T: int, N_min: int, N_max: int, dtype: int = HASHGRID_F32) -> int:
    h = ctypes.c_void_p()
    _check(lib.hashgrid_create_nd(D, L, F, log2T, N_min, N_max, dtype, ctypes.byref(h)))
    return h.value


def hashgrid_dims(h: int) -> int:
    return int(lib.hashgrid_dims(h))


def hashgrid_destroy(h: int) -> None:
    _check(lib.hashgrid_destroy(h))


def hashgrid_params(h: int) -> dict:
    vals = [ctypes.c_int() for _ in range(6)]
    _check(lib.hashgrid_params(h, *[ctypes.byref(v) for v in vals]))
    return dict(zip(("L", "F", "log2T", "N_min", "N_max", "dtype"), (v.value for v in vals)))


def hashgrid_resolutions(h: int) -> list[int]:
    arr = (ctypes.c_int * MAX_LEVELS)()
    _check(lib.hashgrid_resolutions(h, arr))
    return list(arr[: hashgrid_params(h)["L"]])


def hashgrid_set_option(h: int, option: int, value: int) -> None:
    _check(lib.hashgrid_set_option(h, option, value))


def hashgrid_get_option(h: int, option: int) -> int:
    v = ctypes.c_int()
    _check(lib.hashgrid_get_option(h, option, ctypes.byref(v)))
    return v.value


def hashgrid_table_elems(h: int) -> int:
    return int(lib.hashgrid_table_elems(h))


def hashgrid_output_width(h: int) -> int:
    return int(lib.hashgrid_output_width(h))


def hashgrid_forward(h: int, x, N: int, table, out, stream=None) -> None:
    _check(lib.hashgrid_forward(h, _ptr(x), N, _ptr(table), _ptr(out), _stream(stream)))


def hashgrid_backward(h: int, x, dL_dout, N: int, dL_dtable, stream=None) -> None:
    _check(lib.hashgrid_backward(h, _ptr(x), _ptr(dL_dout), N, _ptr(dL_dtable), _stream(stream)))


def hashgrid_backward_half(h: int, x, dL_dout, N: int, dL_dtable, stream=None) -> None:
    _check(lib.hashgrid_backward_half(h, _ptr(x), _ptr(dL_dout), N, _ptr(dL_dtable), _stream(stream)))


def hashgrid_backward_input(h: int, x, dL_dout, N: int, table, dL_dx, stream=None) -> None:
    _check(lib.hashgrid_backward_input(h, _ptr(x), _ptr(dL_dout), N, _ptr(table), _ptr(dL_dx), _stream(stream)))


def hashgrid_adam_step(h: int, table, adam_m, adam_v, dL_dtable, step: int, lr: float, beta1: float = 0.9,
                       beta2: float = 0.99, eps: float = 1e-15, zero_grad: bool = True, stream=None) -> None:
    _check(lib.hashgrid_adam_step(h, _ptr(table), _ptr(adam_m), _ptr(adam_v), _ptr(dL_dtable), step, lr, beta1,
                                  beta2, eps, 1 if zero_grad else 0, _stream(stream)))


def hashgrid_mlp_forward(h: int, x, N: int, table, w1, b1, w2, b2, w3, b3, y, device_status=None,
                         stream=None) -> None:
    _check(lib.hashgrid_mlp_forward(h, _ptr(x), N, _ptr(table), _ptr(w1), _ptr(b1), _ptr(w2), _ptr(b2), _ptr(w3),
                                    _ptr(b3), _ptr(y), _ptr(device_status), _stream(stream)))


def hashgrid_debug_indices(h: int, x, N: int, idx_out, stream=None) -> None:
    _check(lib.hashgrid_debug_indices(h, _ptr(x), N, _ptr(idx_out), _stream(stream)))


def hashgrid_linear_create(in_features: int, out_features: int, dtype: int = HASHGRID_BF16,
                           activation: int = HASHGRID_ACT_NONE) -> int:
    h = ctypes.c_void_p()
    _check(lib.hashgrid_linear_create(in_features, out_features, dtype, activation, ctypes.byref(h)))
    return h.value


def hashgrid_linear_destroy(layer: int) -> None:
    _check(lib.hashgrid_linear_destroy(layer))


def hashgrid_linear_params(layer: int) -> dict:
    vals = [ctypes.c_int() for _ in range(4)]
    _check(lib.hashgrid_linear_params(layer, *[ctypes.byref(v) for v in vals]))
    return dict(zip(("in", "out", "dtype", "activation"), (v.value for v in vals)))


def hashgrid_linear_forward(layer: int, x, ldx: int, N: int, w, b, residual, ldr: int, y, ldy: int, y_dtype: int, z=None,
                            workspace=None, workspace_bytes: int = 0, device_status=None, stream=None) -> None:
    _check(lib.hashgrid_linear_forward(layer, _ptr(x), ldx, N, _ptr(w), _ptr(b), _ptr(residual), ldr, _ptr(y), ldy,
                                       y_dtype, _ptr(z), _ptr(workspace), workspace_bytes, _ptr(device_status),
                                       _stream(stream)))


def hashgrid_linear_forward_workspace(layer: int, N: int, ldx: int) -> int:
    return int(lib.hashgrid_linear_forward_workspace(layer, N, ldx))


def hashgrid_linear_backward_workspace(layer: int, N: int, lddy: int, ldx: int) -> int:
    return int(lib.hashgrid_linear_backward_workspace(layer, N, lddy, ldx))


def hashgrid_linear_backward(layer: int, dL_dy, lddy: int, x, ldx: int, N: int, w, z, dL_dx, lddx: int, dx_dtype: int,
                             dL_dw, dw_dtype: int, dL_db, workspace, workspace_bytes: int, device_status=None,
                             stream=None) -> None:
    _check(lib.hashgrid_linear_backward(layer, _ptr(dL_dy), lddy, _ptr(x), ldx, N, _ptr(w), _ptr(z), _ptr(dL_dx), lddx,
                                        dx_dtype, _ptr(dL_dw), dw_dtype, _ptr(dL_db), _ptr(workspace), workspace_bytes,
                                        _ptr(device_status), _stream(stream)))


def hashgrid_linear_status() -> None:
    """Raises if an earlier layer call without a status word, its work done by now, left its outputs incomplete."""
    _check(lib.hashgrid_linear_status())


def hashgrid_debug_wait_limit(polls: int = -1) -> None:
    _check(lib.hashgrid_debug_wait_limit(polls))


def hashgrid_adamw_create(tensors) -> int:
    """``tensors``: AdamwTensor structs (device pointers)."""
    arr = (AdamwTensor * max(1, len(tensors)))(*tensors)
    h = ctypes.c_void_p()
    _check(lib.hashgrid_adamw_create(arr, len(tensors), ctypes.byref(h)))
    return h.value


def hashgrid_adamw_destroy(opt: int) -> None:
    _check(lib.hashgrid_adamw_destroy(opt))


def hashgrid_adamw_step(opt: int, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.99, eps: float = 1e-8,
                        seed: int = 0, zero_grad: bool = False, device_step=None, stream=None) -> None:
    if seed != 0 and seed & 0xFFFFFFFF == 0:
        raise HashGridError(HASHGRID_ERR_ARG, f"seed = {seed} is 0 in 32 bits, which would round to nearest")
    _check(lib.hashgrid_adamw_step(opt, step, _ptr(device_step), lr, beta1, beta2, eps, seed & 0xFFFFFFFF,
                                   1 if zero_grad else 0, _stream(stream)))


def hashgrid_probe(kind: int, width: int, pattern: int, buf, buf_bytes: int, ops: int, sink=None,
                   stream=None) -> int:
    """Runs one memory-system probe (include/hashgrid_probe.h); returns the number of lane
    operations the kernel performs."""
    done = ctypes.c_int64()
    _check(lib.hashgrid_probe(kind, width, pattern, _ptr(buf), buf_bytes, ops, _ptr(sink), ctypes.byref(done),
                              _stream(stream)))
    return done.value


class HashGrid:
    """Owns a handle and allocates outputs with torch; the encoding itself runs in the
    library. ``table`` arguments are CUDA tensors of shape [L, T, F] (float32 or float16,
    matching ``dtype``)."""

    def __init__(self, L: int = 16, F: int = 2, log2T: int = 19, N_min: int = 16, N_max: int = 512,
                 dtype: int = HASHGRID_F32, forward_gather: int = HASHGRID_GATHER_AUTO,
                 backward_mode: int = HASHGRID_BACKWARD_AUTO, schedule: int = HASHGRID_SCHEDULE_AUTO, D: int = 3):
        self.L, self.F, self.log2T, self.N_min, self.N_max, self.dtype, self.D = L, F, log2T, N_min, N_max, dtype, D
        self.T = 1 << log2T
        self.handle = hashgrid_create_nd(D, L, F, log2T, N_min, N_max, dtype)
        hashgrid_set_option(self.handle, HASHGRID_OPT_FORWARD_GATHER, forward_gather)
        hashgrid_set_option(self.handle, HASHGRID_OPT_BACKWARD_MODE, backward_mode)
        hashgrid_set_option(self.handle, HASHGRID_OPT_SCHEDULE, schedule)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and lib is not None:  # the module may already be torn down at interpreter exit
            lib.hashgrid_destroy(h)
            self.handle = None

    @property
    def resolutions(self) -> list[int]:
        return hashgrid_resolutions(self.handle)

    def forward(self, x, table, out=None, stream=None):
        import torch
        N = x.shape[0]
        if out is None:
            out = torch.empty((N, self.L * self.F), dtype=torch.float32, device=x.device)
        hashgrid_forward(self.handle, x, N, table, out, stream)
        return out

    def backward(self, x, dL_dout, dL_dtable=None, stream=None):
        import torch
        if dL_dtable is None:
            dL_dtable = torch.zeros((self.L, self.T, self.F), dtype=torch.float32, device=x.device)
        hashgrid_backward(self.handle, x, dL_dout, x.shape[0], dL_dtable, stream)
        return dL_dtable

    def backward_input(self, x, dL_dout, table, dL_dx=None, stream=None):
        import torch
        if dL_dx is None:
            dL_dx = torch.empty((x.shape[0], self.D), dtype=torch.float32, device=x.device)
        hashgrid_backward_input(self.handle, x, dL_dout, x.shape[0], table, dL_dx, stream)
        return dL_dx

    def indices(self, x, stream=None):
        import torch
        idx = torch.empty((x.shape[0], self.L, 1 << self.D), dtype=torch.int32, device=x.device)
        hashgrid_debug_indices(self.handle, x, x.shape[0], idx, stream)
        return idx


_CODES: dict = {}


def _dtype_code(t, name: str) -> int:
    """HASHGRID_* code of a torch tensor's type."""
    if not _CODES:
        import torch
        _CODES.update({torch.float32: HASHGRID_F32, torch.float16: HASHGRID_F16, torch.bfloat16: HASHGRID_BF16,
                       torch.float8_e4m3fn: HASHGRID_E4M3})
    code = _CODES.get(t.dtype)
    if code is None:
        raise HashGridError(HASHGRID_ERR_ARG, f"{name} has type {t.dtype}")
    return code


def _rows(t, n, width: int, dtypes, name: str) -> int:
    """Checks a [n, width] tensor with contiguous rows and returns its row stride."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[1] != width or (n is not None and shape[0] != n):
        raise HashGridError(HASHGRID_ERR_ARG, f"{name} has shape {tuple(shape)}, [{'N' if n is None else n}, {width}] is wanted")
    if t.dtype not in dtypes:
        raise HashGridError(HASHGRID_ERR_ARG, f"{name} has type {t.dtype}")
    if width > 1 and stride[1] != 1:
        raise HashGridError(HASHGRID_ERR_ARG, f"{name}: the elements of a row must be contiguous (strides {stride})")
    return stride[0] if shape[0] > 1 else width


def _flat(t, shape, dtypes, name: str) -> None:
    """Checks a contiguous tensor of the given shape."""
    if t.shape != shape or not t.is_contiguous():
        raise HashGridError(HASHGRID_ERR_ARG, f"{name} has shape {tuple(t.shape)}, strides {t.stride()}: contiguous {tuple(shape)} is wanted")
    if t.dtype not in dtypes:
        raise HashGridError(HASHGRID_ERR_ARG, f"{name} has type {t.dtype}")


class Linear:
    """A linear layer with its activation and residual, and its gradients (``hashgrid_linear_*``):
    ``z = x w^T + b``, ``y = act(z) + residual``. Holds a handle only; weights are arguments. Tensors
    are [N, features] with contiguous rows (any row stride), of the layer's 16-bit type where not
    said otherwise. A call that gave up a wait and left its outputs incomplete says so in ``device_status`` (an int32
    CUDA tensor of zeros), or, without one, through the next call's or ``hashgrid_linear_status()``'s error."""

    def __init__(self, in_features: int, out_features: int, dtype: int = HASHGRID_BF16,
                 activation: int = HASHGRID_ACT_NONE):
        self.in_features, self.out_features, self.dtype, self.activation = in_features, out_features, dtype, activation
        import torch
        own = torch.float16 if dtype == HASHGRID_F16 else torch.bfloat16
        self._shape, self._bias_shape = (out_features, in_features), (out_features,)
        self._own, self._either, self._f32 = (own,), (own, torch.float32), (torch.float32,)
        self.handle = hashgrid_linear_create(in_features, out_features, dtype, activation)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and lib is not None:
            lib.hashgrid_linear_destroy(h)
            self.handle = None

    def forward(self, x, w, b=None, residual=None, y=None, z=None, workspace=None, device_status=None, stream=None):
        """Returns y. ``w`` [out, in] contiguous; ``b`` [out] fp32; ``y`` (allocated if None, of ``residual``'s
        type or else the layer's) and ``residual`` of the layer's type or fp32; ``z``: a contiguous [N, out] tensor
        that receives the pre-activation, for ``backward``; ``workspace``: bytes from ``workspace()`` (allocated if
        None; only rows that do not begin on 16-byte boundaries need any)."""
        N, own = x.shape[0], self._own
        ldx = _rows(x, None, self.in_features, own, "x")
        _flat(w, self._shape, own, "w")
        if b is not None:
            _flat(b, self._bias_shape, self._f32, "b")
        if y is None:
            y = _empty((N, self.out_features), self._own[0] if residual is None else residual.dtype, x.device, stream)
        ldy = _rows(y, N, self.out_features, self._either, "y")
        y_dtype = self.dtype if y.dtype is own[0] else HASHGRID_F32
        ldr = 0 if residual is None else _rows(residual, N, self.out_features, (y.dtype,), "residual")
        if z is not None:
            _flat(z, (N, self.out_features), own, "z")
        size = 0
        if workspace is not None:
            size = workspace.numel() * workspace.element_size()
        elif ldx % 8 or self.in_features % 8:
            size = lib.hashgrid_linear_forward_workspace(self.handle, N, ldx)
            workspace = self._scratch(size, x.device, stream)
        _check(lib.hashgrid_linear_forward(self.handle, x.data_ptr(), ldx, N, w.data_ptr(), None if b is None else b.data_ptr(),
                                           None if residual is None else residual.data_ptr(), ldr, y.data_ptr(), ldy, y_dtype,
                                           _ptr(z), _ptr(workspace), size, _ptr(device_status), _stream(stream)))
        return y

    def workspace(self, N: int, device, lddy: int | None = None, ldx: int | None = None):
        """Workspace for ``forward`` and ``backward`` over up to N rows, of these row strides (any, if None)."""
        odd = lambda width, ld: 2 * width + 1 if ld is None else ld  # noqa: E731
        need = [hashgrid_linear_forward_workspace(self.handle, N, odd(self.in_features, ldx)),
                hashgrid_linear_backward_workspace(self.handle, N, odd(self.out_features, lddy), odd(self.in_features, ldx))]
        return self._scratch(max(need), device, None)

    def _scratch(self, size: int, device, stream):
        import torch
        return _empty((max(16, size),), torch.uint8, device, stream)

    def backward(self, dL_dy, x, w, z=None, dL_dx=True, dL_dw=True, dL_db=True, workspace=None, device_status=None,
                 stream=None):
        """Returns (dL_dx, dL_dw, dL_db). Each is a tensor to write (dL_dx and dL_dw of the layer's type or fp32, dL_db
        fp32), True to allocate it (the layer's type, fp32, fp32), or None to leave it out. ``z``: what ``forward``
        wrote (not needed without an activation)."""
        N, own, either = dL_dy.shape[0], self._own, self._either
        lddy = _rows(dL_dy, None, self.out_features, own, "dL_dy")
        ldx = _rows(x, N, self.in_features, own, "x")
        _flat(w, self._shape, own, "w")
        if z is not None:
            _flat(z, (N, self.out_features), own, "z")
        if dL_dx is True:
            dL_dx = _empty((N, self.in_features), own[0], x.device, stream)
        if dL_dw is True:
            dL_dw = _empty(self._shape, self._f32[0], x.device, stream)
        if dL_db is True:
            dL_db = _empty(self._bias_shape, self._f32[0], x.device, stream)
        lddx = 0 if dL_dx is None else _rows(dL_dx, N, self.in_features, either, "dL_dx")
        if dL_dw is not None:
            _flat(dL_dw, self._shape, either, "dL_dw")
        if dL_db is not None:
            _flat(dL_db, self._bias_shape, self._f32, "dL_db")
        if workspace is None:
            workspace = self._scratch(lib.hashgrid_linear_backward_workspace(self.handle, N, lddy, ldx), x.device, stream)
        _check(lib.hashgrid_linear_backward(
            self.handle, dL_dy.data_ptr(), lddy, x.data_ptr(), ldx, N, w.data_ptr(), _ptr(z), _ptr(dL_dx), lddx,
            self.dtype if dL_dx is not None and dL_dx.dtype is own[0] else HASHGRID_F32, _ptr(dL_dw),
            self.dtype if dL_dw is not None and dL_dw.dtype is own[0] else HASHGRID_F32, _ptr(dL_db), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _ptr(device_status), _stream(stream)))
        return dL_dx, dL_dw, dL_db


def _empty(shape, dtype, device, stream):
    """A tensor that is used on ``stream`` (None: the current one) first: its memory comes from that stream's pool, since
    what the current stream's pool hands out may still be in use there by what had it before."""
    import torch
    if stream is None or torch.device(device).type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)  # the caller goes on with it there
    return t


class AdamW:
    """One AdamW step over a list of tensors (``hashgrid_adamw_*``). Holds references to the tensors: they are
    updated in place, and the gradients are read from the same tensors at every step.

    params, grads: contiguous tensors, fp32, fp16 or bf16. m, v: the moments, allocated as zeros if None: fp32, or
    with ``bits=8`` e4m3 codes (torch.float8_e4m3fn or uint8) with ``block_scales = (m_scales, v_scales)``, one fp32
    tensor of ceil(n / 256) values per tensor each. copies: 16-bit tensors that receive the updated parameters.
    lr_scale, weight_decay: one number, or one per tensor."""

    def __init__(self, params, grads, m=None, v=None, bits: int = 32, block_scales=None, copies=None, lr_scale=1.0,
                 weight_decay=0.0):
        import torch
        params, grads = list(params), list(grads)
        count = len(params)
        if (m is None) != (v is None):
            raise HashGridError(HASHGRID_ERR_ARG, "m and v come together")
        if bits not in (8, 32):
            raise HashGridError(HASHGRID_ERR_ARG, f"bits = {bits} is neither 8 nor 32")
        if m is None:
            kind = torch.float32 if bits == 32 else torch.float8_e4m3fn
            m, v = ([torch.zeros(p.shape, dtype=torch.uint8 if bits == 8 else kind, device=p.device).view(kind)
                     for p in params] for _ in range(2))
        m, v = list(m), list(v)
        coded = [t.element_size() == 1 for t in m]
        if block_scales is None and any(coded):
            block_scales = tuple([torch.zeros(-(-p.numel() // HASHGRID_ADAMW_BLOCK), device=p.device) for p in params]
                                 for _ in range(2))
        ms, vs = (list(block_scales[0]), list(block_scales[1])) if block_scales is not None else ([None] * count,) * 2
        copies = list(copies) if copies is not None else [None] * count
        lr_scale = [float(lr_scale)] * count if isinstance(lr_scale, (int, float)) else [float(s) for s in lr_scale]
        weight_decay = ([float(weight_decay)] * count if isinstance(weight_decay, (int, float))
                        else [float(d) for d in weight_decay])
        for name, lst in (("grads", grads), ("m", m), ("v", v), ("block_scales", ms), ("block_scales", vs),
                          ("copies", copies), ("lr_scale", lr_scale), ("weight_decay", weight_decay)):
            if len(lst) != count:
                raise HashGridError(HASHGRID_ERR_ARG, f"{name}: {len(lst)} entries for {count} parameters")
        self.params, self.grads, self.m, self.v = params, grads, m, v
        self.m_scales, self.v_scales, self.copies = ms, vs, copies
        tensors = []
        for k, p in enumerate(params):
            n = p.numel()
            for name, t in (("param", p), ("grad", grads[k]), ("m", m[k]), ("v", v[k]), ("copy", copies[k])):
                if t is not None and (t.numel() != n or not t.is_contiguous()):
                    raise HashGridError(HASHGRID_ERR_ARG, f"tensor {k}: {name} has shape {tuple(t.shape)}, strides {t.stride()}: "
                                                          f"{n} contiguous elements are wanted")
            for t in (m[k], v[k]):
                kinds = (torch.float8_e4m3fn, torch.uint8) if coded[k] else (torch.float32,)
                if t.dtype not in kinds:
                    raise HashGridError(HASHGRID_ERR_ARG, f"tensor {k}: states of type {m[k].dtype} and {v[k].dtype}")
            blocks = -(-n // HASHGRID_ADAMW_BLOCK)
            for t in (ms[k], vs[k]):
                if coded[k] and (t is None or t.dtype != torch.float32 or t.numel() != blocks or not t.is_contiguous()):
                    raise HashGridError(HASHGRID_ERR_ARG, f"tensor {k}: {blocks} contiguous fp32 scales are wanted")
            tensors.append(AdamwTensor(
                _ptr(p), _ptr(grads[k]), _ptr(m[k]), _ptr(v[k]), _ptr(ms[k]) if coded[k] else None,
                _ptr(vs[k]) if coded[k] else None, _ptr(copies[k]), n, _dtype_code(p, "param"), _dtype_code(grads[k], "grad"),
                HASHGRID_E4M3 if coded[k] else HASHGRID_F32,
                HASHGRID_BF16 if copies[k] is None else _dtype_code(copies[k], "copy"), lr_scale[k], weight_decay[k]))
        self.handle = hashgrid_adamw_create(tensors)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and lib is not None:
            lib.hashgrid_adamw_destroy(h)
            self.handle = None

    def step(self, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.99, eps: float = 1e-8, seed: int = 0,
             zero_grad: bool = False, device_step=None, stream=None) -> None:
        """One step, t = ``step`` (from 1 on), or the int64 CUDA tensor ``device_step``'s value."""
        if device_step is not None and not isinstance(device_step, int) and (
                str(device_step.dtype) != "torch.int64" or device_step.numel() != 1):
            raise HashGridError(HASHGRID_ERR_ARG, "device_step is one int64")
        hashgrid_adamw_step(self.handle, step, lr, beta1, beta2, eps, seed, zero_grad, device_step, stream)
