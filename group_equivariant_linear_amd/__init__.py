"""Python binding of libeqlinear.so, the MI355X (gfx950) equivariant linear layers.

A thin ctypes layer over the C ABI in include/eqlinear.h: every function has the
C name, turns tensors into device pointers and the current torch stream into a
hipStream_t, checks shapes and dtypes, and raises EqlError on a non-OK status.
All arithmetic runs in the library's HIP kernels; there is no fallback path.
If the library has not been built, loading fails loudly.

Tensor arguments may be torch tensors on a ROCm device, or plain integers
(raw device addresses, for callers that manage memory themselves); where a call
takes strides, an address stands for contiguous rows, or comes with its strides
as an eqlinear_heads.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libeqlinear.so")

EQL_OK, EQL_ERR_INVALID, EQL_ERR_UNSUPPORTED, EQL_ERR_HIP, EQL_ERR_NOMEM = range(5)
EQL_F32, EQL_BF16, EQL_F16 = 0, 1, 2
EQL_KIND_CN, EQL_KIND_D8, EQL_KIND_ROTARY, EQL_KIND_MIXER, EQL_KIND_NORM, EQL_KIND_ATTENTION = range(6)
EQL_ACT_NONE, EQL_ACT_GELU, EQL_ACT_SILU = range(3)
EQL_ROTARY_HALF, EQL_ROTARY_INTERLEAVED = 0, 1
EQL_ROTARY_PLAIN, EQL_ROTARY_LINEAR, EQL_ROTARY_RAISED_BASE, EQL_ROTARY_BANDED = range(4)

# Every entry point of include/eqlinear.h.
ABI_FUNCTIONS = (
    "eqlinear_status_string", "eqlinear_plan", "eqlinear_d8_plan", "eqlinear_plan_destroy",
    "eqlinear_plan_info", "eqlinear_w_hat_elems", "eqlinear_weight_fft", "eqlinear_forward",
    "eqlinear_forward_tiled", "eqlinear_d8_forward", "eqlinear_expand_dense",
    "eqlinear_dense_forward", "eqlinear_w_hat_adjoint", "eqlinear_backward_data",
    "eqlinear_backward_weight_workspace", "eqlinear_backward_weight", "eqlinear_forward_bias_act",
    "eqlinear_d8_bias_act", "eqlinear_d8_to_fourier", "eqlinear_d8_to_regular", "eqlinear_dihedral_plan",
    "eqlinear_backward_weight_noalloc", "eqlinear_d8_regular_forward",
    "eqlinear_rotary_plan", "eqlinear_rotary", "eqlinear_mixer_plan", "eqlinear_linear_attention_workspace",
    "eqlinear_linear_attention", "eqlinear_linear_attention_backward", "eqlinear_linear_attention_step",
    "eqlinear_norm_plan", "eqlinear_group_norm_workspace", "eqlinear_group_norm", "eqlinear_group_norm_backward",
    "eqlinear_attention_plan", "eqlinear_attention_bucket", "eqlinear_attention_workspace", "eqlinear_attention",
    "eqlinear_attention_backward", "eqlinear_attention_step_workspace", "eqlinear_attention_step",
    "eqlinear_cache_tables_workspace", "eqlinear_cache_tables", "eqlinear_cache_store",
)

# Size of the library-held scratch array of eqlinear_backward_weight_noalloc.
EQL_NOALLOC_SCRATCH_BYTES = 32 << 20


class EqlError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {eqlinear_status_string(status)}")


class eqlinear_info(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32), ("dtype", ctypes.c_int32), ("N", ctypes.c_int32),
        ("C_in", ctypes.c_int32), ("C_out", ctypes.c_int32), ("bins", ctypes.c_int32),
        ("planes", ctypes.c_int32), ("has_nyquist", ctypes.c_int32),
        ("params", ctypes.c_int64), ("w_hat_elems", ctypes.c_int64),
        ("real_gemms", ctypes.c_int64), ("macs_per_token", ctypes.c_int64),
        ("dense_macs_per_token", ctypes.c_int64),
    ]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


class eqlinear_heads(ctypes.Structure):
    """A tensor [T][heads][d][N] with the last two axes contiguous; strides in elements."""

    _fields_ = [("ptr", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class eqlinear_pages(ctypes.Structure):
    """A cache [blocks][block_size][kv_heads][d][N] with the last two axes contiguous; strides in elements."""

    _fields_ = [("ptr", ctypes.c_void_p), ("block_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


_lib = None
_lock = threading.Lock()


def load_library(path: str | None = None):
    """Load libeqlinear.so (raises OSError if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise OSError(f"{p} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(p)
        vp, i32, i64, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int
        plan_p = ctypes.POINTER(ctypes.c_void_p)
        hp, f32, f64 = ctypes.POINTER(eqlinear_heads), ctypes.c_float, ctypes.c_double
        pp, size = ctypes.POINTER(eqlinear_pages), ctypes.c_size_t
        sig = {
            "eqlinear_status_string": ([st], ctypes.c_char_p),
            "eqlinear_plan": ([plan_p, i32, i32, i32, i32], st),
            "eqlinear_d8_plan": ([plan_p, i32, i32, i32], st),
            "eqlinear_plan_destroy": ([vp], st),
            "eqlinear_plan_info": ([vp, ctypes.POINTER(eqlinear_info)], st),
            "eqlinear_w_hat_elems": ([vp], ctypes.c_size_t),
            "eqlinear_weight_fft": ([vp, vp, vp], st),
            "eqlinear_forward": ([vp, vp, vp, vp, i64, vp], st),
            "eqlinear_forward_tiled": ([vp, vp, vp, vp, i64, vp, i32], st),
            "eqlinear_d8_forward": ([vp, vp, vp, vp, i64, vp], st),
            "eqlinear_expand_dense": ([vp, vp, vp, vp], st),
            "eqlinear_dense_forward": ([vp, vp, vp, vp, i64, vp], st),
            "eqlinear_w_hat_adjoint": ([vp, vp, vp, vp], st),
            "eqlinear_backward_data": ([vp, vp, vp, vp, i64, vp], st),
            "eqlinear_backward_weight_workspace": ([vp, i64], ctypes.c_size_t),
            "eqlinear_backward_weight": ([vp, vp, vp, vp, i64, vp, ctypes.c_size_t, vp], st),
            "eqlinear_backward_weight_noalloc": ([vp, vp, vp, vp, i64, vp], st),
            "eqlinear_forward_bias_act": ([vp, vp, vp, vp, i32, vp, i64, vp, i32], st),
            "eqlinear_d8_bias_act": ([vp, vp, vp, i32, vp, i64, vp], st),
            "eqlinear_dihedral_plan": ([ctypes.POINTER(ctypes.c_void_p), i32, i32, i32, i32], st),
            "eqlinear_d8_to_fourier": ([vp, vp, vp, i64, vp], st),
            "eqlinear_d8_regular_forward": ([vp, vp, vp, vp, i32, vp, i64, vp], st),
            "eqlinear_d8_to_regular": ([vp, vp, vp, i64, vp], st),
            "eqlinear_rotary_plan": ([plan_p] + [i32] * 6 + [f64, i32] + [f64] * 5 + [i32], st),
            "eqlinear_rotary": ([vp, hp, hp, vp, i32, hp, hp, i64, vp], st),
            "eqlinear_mixer_plan": ([plan_p] + [i32] * 6, st),
            "eqlinear_linear_attention_workspace": ([vp, i64, i64, i32], ctypes.c_size_t),
            "eqlinear_linear_attention": ([vp, hp, hp, hp, vp, f32, vp, i64, vp, vp, hp, i64, vp, ctypes.c_size_t, vp],
                                          st),
            "eqlinear_linear_attention_backward": ([vp, hp, hp, hp, hp, vp, f32, vp, i64, vp, vp, hp, hp, hp, vp, i64,
                                                    vp, ctypes.c_size_t, vp], st),
            "eqlinear_linear_attention_step": ([vp, hp, hp, hp, vp, f32, vp, hp, i64, vp], st),
            "eqlinear_norm_plan": ([plan_p] + [i32] * 4 + [f64, i32], st),
            "eqlinear_group_norm_workspace": ([vp, i64, i64, i32], ctypes.c_size_t),
            "eqlinear_group_norm": ([vp, vp, i64, vp, vp, vp, i64, vp, i64, vp, i64, vp, ctypes.c_size_t, vp], st),
            "eqlinear_group_norm_backward": ([vp, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, i64, vp, vp, i64, vp,
                                              ctypes.c_size_t, vp], st),
            "eqlinear_attention_plan": ([plan_p] + [i32] * 9, st),
            "eqlinear_attention_bucket": ([vp, i64], i32),
            "eqlinear_attention_workspace": ([vp, i64, i64, i64, i32], size),
            "eqlinear_attention": ([vp, hp, hp, hp, f32, vp, vp, vp, i64, hp, vp, i64, i64, vp, size, vp], st),
            "eqlinear_attention_backward": ([vp, hp, hp, hp, hp, hp, vp, f32, vp, vp, vp, i64, hp, hp, hp, vp, i64, i64,
                                             vp, size, vp], st),
            "eqlinear_attention_step_workspace": ([vp, i64], size),
            "eqlinear_attention_step": ([vp, hp, pp, pp, i64, i32, vp, i64, vp, f32, vp, hp, vp, i64, vp, size, vp], st),
            "eqlinear_cache_tables_workspace": ([i64], size),
            "eqlinear_cache_tables": ([vp, vp, vp, i64, vp, vp, i64, i32, vp, vp, vp, vp, vp, i64, i64, vp, size, vp], st),
            "eqlinear_cache_store": ([vp, hp, hp, vp, pp, pp, i64, i32, i64, vp], st),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, res
        if path is None:
            _lib = lib
        return lib


def eqlinear_status_string(status: int) -> str:
    return load_library().eqlinear_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != EQL_OK:
        raise EqlError(status, where)


class Plan:
    """Owns an eqlinear_plan_t; destroyed when garbage-collected."""

    def __init__(self, handle: int, lib):
        self.handle = ctypes.c_void_p(handle)
        self._lib = lib
        self.info = eqlinear_plan_info(self)
        self.kind, self.N, self.C = self.info["kind"], self.info["N"], self.info["C_in"]

    def __del__(self):
        # may run during interpreter shutdown, when module globals (ctypes among
        # them) are already gone: touch only what the instance holds
        h = getattr(self, "handle", None)
        lib = getattr(self, "_lib", None)
        if h is not None and lib is not None and h.value:
            lib.eqlinear_plan_destroy(h)
            h.value = None

    @property
    def dtype(self):
        return self.info["dtype"]

    @functools.cached_property
    def torch_dtype(self):
        return _torch_dtype(self)


def eqlinear_plan(N: int, C_in: int, C_out: int, dtype: int) -> Plan:
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.eqlinear_plan(ctypes.byref(h), N, C_in, C_out, int(dtype)), "eqlinear_plan")
    return Plan(h.value, lib)


def eqlinear_d8_plan(C_in: int, C_out: int, dtype: int) -> Plan:
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.eqlinear_d8_plan(ctypes.byref(h), C_in, C_out, int(dtype)), "eqlinear_d8_plan")
    return Plan(h.value, lib)


def eqlinear_dihedral_plan(n: int, C_in: int, C_out: int, dtype: int) -> Plan:
    """Plan of the D_n layer (dihedral group of the regular n-gon, order 2n; n = 4 is D8)."""
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.eqlinear_dihedral_plan(ctypes.byref(h), n, C_in, C_out, int(dtype)), "eqlinear_dihedral_plan")
    return Plan(h.value, lib)


def eqlinear_plan_destroy(plan: Plan):
    if plan.handle.value:
        _check(plan._lib.eqlinear_plan_destroy(plan.handle), "eqlinear_plan_destroy")
        plan.handle = ctypes.c_void_p(0)


def eqlinear_plan_info(plan: Plan) -> dict:
    inf = eqlinear_info()
    _check(plan._lib.eqlinear_plan_info(plan.handle, ctypes.byref(inf)), "eqlinear_plan_info")
    return inf.as_dict()


def eqlinear_w_hat_elems(plan: Plan) -> int:
    return int(plan._lib.eqlinear_w_hat_elems(plan.handle))


# --- tensor marshalling --------------------------------------------------------

def _torch_dtype(plan: Plan):
    import torch
    return {EQL_F32: torch.float32, EQL_BF16: torch.bfloat16, EQL_F16: torch.float16}[plan.dtype]


def _ptr(t, plan: Plan, numel: int | None, name: str):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor or a device address")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: tensor must live on the GPU, got {t.device}")
    if t.dtype != _torch_dtype(plan):
        raise ValueError(f"{name}: dtype {t.dtype} does not match the plan ({_torch_dtype(plan)})")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _widths(plan: Plan):
    inf = plan.info
    if inf["kind"] == EQL_KIND_CN:
        return inf["N"] * inf["C_in"], inf["N"] * inf["C_out"]
    return inf["C_in"], inf["C_out"]


def _tokens(x, T, K):
    if T is not None:
        return int(T)
    if isinstance(x, int):
        raise ValueError("T is required when x is a raw address")
    return x.numel() // K


def eqlinear_weight_fft(plan: Plan, w, w_hat):
    n = eqlinear_w_hat_elems(plan)
    _check(plan._lib.eqlinear_weight_fft(plan.handle, _ptr(w, plan, n, "w"),
                                         _ptr(w_hat, plan, n, "w_hat")), "eqlinear_weight_fft")


def eqlinear_forward(plan: Plan, x, w_hat, y, T: int | None = None, stream=None):
    K, M = _widths(plan)
    T = _tokens(x, T, K)
    n = eqlinear_w_hat_elems(plan)
    _check(plan._lib.eqlinear_forward(plan.handle, _ptr(x, plan, T * K, "x"),
                                      _ptr(w_hat, plan, n, "w_hat"), _ptr(y, plan, T * M, "y"),
                                      T, _stream(stream)), "eqlinear_forward")


def eqlinear_forward_tiled(plan: Plan, x, w_hat, y, tile: int, T: int | None = None, stream=None):
    K, M = _widths(plan)
    T = _tokens(x, T, K)
    n = eqlinear_w_hat_elems(plan)
    _check(plan._lib.eqlinear_forward_tiled(plan.handle, _ptr(x, plan, T * K, "x"),
                                            _ptr(w_hat, plan, n, "w_hat"),
                                            _ptr(y, plan, T * M, "y"), T, _stream(stream),
                                            int(tile)), "eqlinear_forward_tiled")


def eqlinear_forward_bias_act(plan: Plan, x, w_hat, bias, act: int, y, T: int | None = None, stream=None,
                              tile: int = -1):
    """y = act(layer(x) + bias[o]); bias may be None (no bias), act EQL_ACT_NONE or EQL_ACT_GELU."""
    K, M = _widths(plan)
    T = _tokens(x, T, K)
    n = eqlinear_w_hat_elems(plan)
    _check(plan._lib.eqlinear_forward_bias_act(plan.handle, _ptr(x, plan, T * K, "x"),
                                               _ptr(w_hat, plan, n, "w_hat"),
                                               _ptr(bias, plan, plan.info["C_out"], "bias"), int(act),
                                               _ptr(y, plan, T * M, "y"), T, _stream(stream), int(tile)),
           "eqlinear_forward_bias_act")


def eqlinear_d8_forward(plan: Plan, x, wb, y, T: int | None = None, stream=None):
    K, M = _widths(plan)
    T = _tokens(x, T, K)
    n = eqlinear_w_hat_elems(plan)
    _check(plan._lib.eqlinear_d8_forward(plan.handle, _ptr(x, plan, T * K, "x"),
                                         _ptr(wb, plan, n, "wb"), _ptr(y, plan, T * M, "y"),
                                         T, _stream(stream)), "eqlinear_d8_forward")


def eqlinear_d8_bias_act(plan: Plan, y_in, bias, act: int, y_out, T: int | None = None, stream=None):
    """y_out = F act(F^T y_in + bias[j]) per regular channel (y_out may be y_in); bias None or
    [C_out / group order]."""
    _, M = _widths(plan)
    T = _tokens(y_in, T, M)
    _check(plan._lib.eqlinear_d8_bias_act(plan.handle, _ptr(y_in, plan, T * M, "y_in"),
                                          _ptr(bias, plan, plan.info["C_out"] // plan.info["N"], "bias"), int(act),
                                          _ptr(y_out, plan, T * M, "y_out"), T, _stream(stream)),
           "eqlinear_d8_bias_act")


def eqlinear_d8_regular_forward(plan: Plan, x_reg, wb, bias, act: int, y_reg, T: int | None = None,
                                stream=None):
    """y_reg = act(to_regular(layer(to_fourier(x_reg))) + bias[j]) in one launch; bias None or
    [C_out / group order]."""
    K, M = _widths(plan)
    T = _tokens(x_reg, T, K)
    _check(plan._lib.eqlinear_d8_regular_forward(plan.handle, _ptr(x_reg, plan, T * K, "x_reg"),
                                                 _ptr(wb, plan, eqlinear_w_hat_elems(plan), "wb"),
                                                 _ptr(bias, plan, plan.info["C_out"] // plan.info["N"], "bias"),
                                                 int(act), _ptr(y_reg, plan, T * M, "y_reg"), T, _stream(stream)),
           "eqlinear_d8_regular_forward")


def eqlinear_d8_to_fourier(plan: Plan, x_reg, x_four, T: int | None = None, stream=None):
    K, _ = _widths(plan)
    T = _tokens(x_reg, T, K)
    _check(plan._lib.eqlinear_d8_to_fourier(plan.handle, _ptr(x_reg, plan, T * K, "x_reg"),
                                            _ptr(x_four, plan, T * K, "x_four"), T, _stream(stream)),
           "eqlinear_d8_to_fourier")


def eqlinear_d8_to_regular(plan: Plan, y_four, y_reg, T: int | None = None, stream=None):
    _, M = _widths(plan)
    T = _tokens(y_four, T, M)
    _check(plan._lib.eqlinear_d8_to_regular(plan.handle, _ptr(y_four, plan, T * M, "y_four"),
                                            _ptr(y_reg, plan, T * M, "y_reg"), T, _stream(stream)),
           "eqlinear_d8_to_regular")


def eqlinear_expand_dense(plan: Plan, w, w_dense, stream=None):
    K, M = _widths(plan)
    n = eqlinear_w_hat_elems(plan)
    _check(plan._lib.eqlinear_expand_dense(plan.handle, _ptr(w, plan, n, "w"),
                                           _ptr(w_dense, plan, K * M, "w_dense"),
                                           _stream(stream)), "eqlinear_expand_dense")


def eqlinear_dense_forward(plan: Plan, x, w_dense, y, T: int | None = None, stream=None):
    K, M = _widths(plan)
    T = _tokens(x, T, K)
    _check(plan._lib.eqlinear_dense_forward(plan.handle, _ptr(x, plan, T * K, "x"),
                                            _ptr(w_dense, plan, K * M, "w_dense"),
                                            _ptr(y, plan, T * M, "y"), T, _stream(stream)),
           "eqlinear_dense_forward")


def eqlinear_w_hat_adjoint(plan: Plan, w_hat, w_hat_adj, stream=None):
    n = eqlinear_w_hat_elems(plan)
    _check(plan._lib.eqlinear_w_hat_adjoint(plan.handle, _ptr(w_hat, plan, n, "w_hat"),
                                            _ptr(w_hat_adj, plan, n, "w_hat_adj"), _stream(stream)),
           "eqlinear_w_hat_adjoint")


def eqlinear_backward_data(plan: Plan, dy, w_hat_adj, dx, T: int | None = None, stream=None):
    K, M = _widths(plan)
    T = _tokens(dy, T, M)
    n = eqlinear_w_hat_elems(plan)
    _check(plan._lib.eqlinear_backward_data(plan.handle, _ptr(dy, plan, T * M, "dy"),
                                            _ptr(w_hat_adj, plan, n, "w_hat_adj"),
                                            _ptr(dx, plan, T * K, "dx"), T, _stream(stream)),
           "eqlinear_backward_data")


def eqlinear_backward_weight_workspace(plan: Plan, T: int) -> int:
    return int(plan._lib.eqlinear_backward_weight_workspace(plan.handle, int(T)))


def _raw_ptr(t, name: str, dtype=None, numel: int | None = None):
    """Device address of a tensor whose dtype does not follow the plan."""
    if isinstance(t, int):
        return t
    import torch
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name}: expected a GPU tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name}: expected {numel} elements, got {t.numel()}")
    return t.data_ptr()


def eqlinear_backward_weight(plan: Plan, x, dy, dw, workspace, T: int | None = None, stream=None):
    """dw (fp32, N*C_in*C_out elements) from x and dy; workspace: a GPU byte
    tensor of at least eqlinear_backward_weight_workspace(plan, T) bytes."""
    import torch
    K, M = _widths(plan)
    T = _tokens(x, T, K)
    n = eqlinear_w_hat_elems(plan)
    if isinstance(workspace, int):
        raise ValueError("workspace: pass a GPU tensor (its size is checked)")
    wbytes = workspace.numel() * workspace.element_size()
    _check(plan._lib.eqlinear_backward_weight(plan.handle, _ptr(x, plan, T * K, "x"), _ptr(dy, plan, T * M, "dy"),
                                              _raw_ptr(dw, "dw", torch.float32, n),
                                              T, _raw_ptr(workspace, "workspace"), wbytes, _stream(stream)),
           "eqlinear_backward_weight")


def eqlinear_backward_weight_noalloc(plan: Plan, x, dy, dw, T: int | None = None, stream=None):
    """dw (fp32, N*C_in*C_out elements) from x and dy, with the workspace in the
    library's own scratch array on the current GPU (no allocation anywhere)."""
    import torch
    K, M = _widths(plan)
    T = _tokens(x, T, K)
    n = eqlinear_w_hat_elems(plan)
    st = plan._lib.eqlinear_backward_weight_noalloc(plan.handle, _ptr(x, plan, T * K, "x"),
                                                    _ptr(dy, plan, T * M, "dy"),
                                                    _raw_ptr(dw, "dw", torch.float32, n), T, _stream(stream))
    if st == EQL_ERR_UNSUPPORTED:
        need = eqlinear_backward_weight_workspace(plan, T)
        raise EqlError(st, f"eqlinear_backward_weight_noalloc (workspace {need} bytes > the "
                           f"{EQL_NOALLOC_SCRATCH_BYTES}-byte library scratch, or past the 2 GiB plane limit)")
    _check(st, "eqlinear_backward_weight_noalloc")


# --- operators between the layers ---------------------------------------------------

def eqlinear_rotary_plan(N: int, heads: int, kv_heads: int, d: int, rot: int, layout: int, dtype: int,
                         base: float = 10000.0, scaling: int = EQL_ROTARY_PLAIN, factor: float = 1.0,
                         context: float = 0.0, turns_slow: float = 1.0, turns_fast: float = 32.0,
                         magnitude: float = 1.0) -> Plan:
    """Plan of rotary positions over the first rot of each head's d channels."""
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.eqlinear_rotary_plan(ctypes.byref(h), N, heads, kv_heads, d, rot, int(layout), base, int(scaling),
                                    factor, context, turns_slow, turns_fast, magnitude, int(dtype)),
           "eqlinear_rotary_plan")
    p = Plan(h.value, lib)
    p.heads, p.kv_heads, p.d = heads, kv_heads, d
    return p


def eqlinear_mixer_plan(N: int, heads: int, kv_heads: int, d_k: int, d_v: int, dtype: int) -> Plan:
    """Plan of linear attention: heads of d_k (queries, keys) and d_v (values) channels."""
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.eqlinear_mixer_plan(ctypes.byref(h), N, heads, kv_heads, d_k, d_v, int(dtype)), "eqlinear_mixer_plan")
    p = Plan(h.value, lib)
    p.heads, p.kv_heads, p.d_k, p.d_v = heads, kv_heads, d_k, d_v
    return p


def eqlinear_norm_plan(N: int, C: int, groups: int, act: int, dtype: int, eps: float = 1e-5) -> Plan:
    """Plan of a group norm with an activation over C channels."""
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.eqlinear_norm_plan(ctypes.byref(h), N, C, groups, int(act), eps, int(dtype)), "eqlinear_norm_plan")
    p = Plan(h.value, lib)
    p.groups = groups
    return p


@functools.lru_cache(maxsize=None)
def _torch():
    """The torch module: imported by the first call that has tensors."""
    import torch
    return torch


@functools.lru_cache(maxsize=None)
def _current_stream():
    """A function to the current device's current hipStream_t: torch's own short one where this torch has it (0.2 us;
    2.7 us through torch.cuda.current_stream(), of the 7 us that a call takes)."""
    torch = _torch()
    raw, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
    if raw is None or device is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw(device())


def _raw_stream(stream):
    """hipStream_t of a torch stream or an address; None: the current stream of the current device."""
    if stream is None:
        return _current_stream()()
    return stream if isinstance(stream, int) else stream.cuda_stream


def _heads(t, plan: Plan, T: int, heads: int, d: int, name: str):
    """A tensor [T, heads, d, N] (the last two axes contiguous), the address of a contiguous one, or an
    eqlinear_heads as it is."""
    if type(t) is eqlinear_heads:
        return t
    N = plan.N
    if type(t) is int:
        return eqlinear_heads(t, heads * d * N, d * N)
    _gpu(t, name, plan.torch_dtype)
    if t.shape != (T, heads, d, N):
        raise ValueError(f"{name}: expected shape {(T, heads, d, N)}, got {tuple(t.shape)}")
    ts, hs, sd, sn = t.stride()
    if (sn != 1 and N > 1) or (sd != N and d > 1):
        raise ValueError(f"{name}: the channel and group axes must be contiguous")
    return eqlinear_heads(t.data_ptr(), ts, hs)


def _gpu(t, name: str, dtype):
    try:
        fits = t.is_cuda and t.dtype is dtype
    except AttributeError:
        raise TypeError(f"{name}: expected a torch.Tensor") from None
    if not fits:
        if not t.is_cuda:
            raise ValueError(f"{name}: tensor must live on the GPU, got {t.device}")
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")


def _dense(t, name: str, dtype, shape):
    """Address of a contiguous GPU tensor of the given dtype and shape; None stays None, an address itself."""
    if t is None or type(t) is int:
        return t
    _gpu(t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")
    return t.data_ptr()


def _kind(plan: Plan, kind: int, where: str):
    if plan.kind != kind:
        raise EqlError(EQL_ERR_INVALID, where)


def _sequences(offsets, batch):
    """(address of the offsets or None, number of sequences)."""
    if offsets is None:
        return None, 1 if batch is None else int(batch)
    if isinstance(offsets, int):
        if batch is None:
            raise ValueError("batch is required when offsets is a raw address")
        return offsets, int(batch)
    n = offsets.numel() - 1
    if batch is not None and int(batch) != n:
        raise ValueError(f"offsets: expected batch + 1 = {int(batch) + 1} values, got {n + 1}")
    return _dense(offsets, "offsets", _torch().int64, (n + 1,)), n


def _workspace(workspace):
    """(address or None, bytes) of a workspace tensor."""
    if workspace is None:
        return None, 0
    if isinstance(workspace, int):
        raise ValueError("workspace: pass a GPU tensor (its size is checked)")
    return _raw_ptr(workspace, "workspace"), workspace.numel() * workspace.element_size()


def _count(t, T, name):
    if T is not None:
        return int(T)
    if isinstance(t, (int, eqlinear_heads)):
        raise ValueError(f"T is required when {name} is an address")
    return t.shape[0]


def eqlinear_rotary(plan: Plan, q, k, positions, q_out, k_out, inverse: bool = False, T: int | None = None,
                    stream=None):
    """Turn q [T, heads, d, N] and k [T, kv_heads, d, N] (k and k_out may be None) by positions
    (int32 [T]); q_out may be q and k_out k."""
    torch = _torch()
    _kind(plan, EQL_KIND_ROTARY, "eqlinear_rotary")
    T = _count(q, T, "q")
    H, K, d = plan.heads, plan.kv_heads, plan.d
    _check(plan._lib.eqlinear_rotary(
        plan.handle, _heads(q, plan, T, H, d, "q"), None if k is None else _heads(k, plan, T, K, d, "k"),
        _dense(positions, "positions", torch.int32, (T,)), int(bool(inverse)), _heads(q_out, plan, T, H, d, "q_out"),
        None if k_out is None else _heads(k_out, plan, T, K, d, "k_out"), T, _raw_stream(stream)), "eqlinear_rotary")


def eqlinear_linear_attention_workspace(plan: Plan, T: int, batch: int, backward: bool = False) -> int:
    return int(plan._lib.eqlinear_linear_attention_workspace(plan.handle, int(T), int(batch), int(bool(backward))))


def _state_shape(plan: Plan, batch: int):
    return (batch, plan.kv_heads, plan.d_k * plan.N, plan.d_v * plan.N)


def eqlinear_linear_attention(plan: Plan, q, k, v, log_decay, o, scale: float, offsets=None, batch: int | None = None,
                              state_in=None, state_out=None, workspace=None, T: int | None = None, stream=None):
    """Causal linear attention with a decay for each kv head: o [T, heads, d_v, N] and the fp32 state
    [batch, kv_heads, d_k N, d_v N] after the last token.  The sequences are offsets (int64 [batch + 1])
    or batch equal runs (default: one)."""
    torch = _torch()
    _kind(plan, EQL_KIND_MIXER, "eqlinear_linear_attention")
    T = _count(q, T, "q")
    H, K, dk, dv = plan.heads, plan.kv_heads, plan.d_k, plan.d_v
    off, B = _sequences(offsets, batch)
    ws, nb = _workspace(workspace)
    shape = _state_shape(plan, B)
    _check(plan._lib.eqlinear_linear_attention(
        plan.handle, _heads(q, plan, T, H, dk, "q"), _heads(k, plan, T, K, dk, "k"), _heads(v, plan, T, K, dv, "v"),
        _dense(log_decay, "log_decay", torch.float32, (K,)), scale, off, B,
        _dense(state_in, "state_in", torch.float32, shape), _dense(state_out, "state_out", torch.float32, shape),
        _heads(o, plan, T, H, dv, "o"), T, ws, nb, _raw_stream(stream)), "eqlinear_linear_attention")


def eqlinear_linear_attention_backward(plan: Plan, q, k, v, do, log_decay, dq, dk, dv, scale: float, offsets=None,
                                       batch: int | None = None, state_in=None, dstate_out=None, dstate_in=None,
                                       workspace=None, T: int | None = None, stream=None):
    """Gradients dq, dk, dv (and dstate_in) of eqlinear_linear_attention."""
    torch = _torch()
    _kind(plan, EQL_KIND_MIXER, "eqlinear_linear_attention_backward")
    T = _count(q, T, "q")
    H, K, ck, cv = plan.heads, plan.kv_heads, plan.d_k, plan.d_v
    off, B = _sequences(offsets, batch)
    ws, nb = _workspace(workspace)
    shape = _state_shape(plan, B)
    _check(plan._lib.eqlinear_linear_attention_backward(
        plan.handle, _heads(q, plan, T, H, ck, "q"), _heads(k, plan, T, K, ck, "k"), _heads(v, plan, T, K, cv, "v"),
        _heads(do, plan, T, H, cv, "do"), _dense(log_decay, "log_decay", torch.float32, (K,)), scale, off, B,
        _dense(state_in, "state_in", torch.float32, shape), _dense(dstate_out, "dstate_out", torch.float32, shape),
        _heads(dq, plan, T, H, ck, "dq"), _heads(dk, plan, T, K, ck, "dk"), _heads(dv, plan, T, K, cv, "dv"),
        _dense(dstate_in, "dstate_in", torch.float32, shape), T, ws, nb, _raw_stream(stream)),
        "eqlinear_linear_attention_backward")


def eqlinear_linear_attention_step(plan: Plan, q, k, v, log_decay, state, o, scale: float, batch: int | None = None,
                                   stream=None):
    """One token for each of batch sequences: state [batch, kv_heads, d_k N, d_v N] in place, o [batch, heads, d_v, N]."""
    torch = _torch()
    _kind(plan, EQL_KIND_MIXER, "eqlinear_linear_attention_step")
    B = _count(q, batch, "q")
    H, K, dk, dv = plan.heads, plan.kv_heads, plan.d_k, plan.d_v
    _check(plan._lib.eqlinear_linear_attention_step(
        plan.handle, _heads(q, plan, B, H, dk, "q"), _heads(k, plan, B, K, dk, "k"), _heads(v, plan, B, K, dv, "v"),
        _dense(log_decay, "log_decay", torch.float32, (K,)), scale,
        _dense(state, "state", torch.float32, _state_shape(plan, B)), _heads(o, plan, B, H, dv, "o"), B,
        _raw_stream(stream)), "eqlinear_linear_attention_step")


def eqlinear_group_norm_workspace(plan: Plan, T: int, batch: int, backward: bool = False) -> int:
    return int(plan._lib.eqlinear_group_norm_workspace(plan.handle, int(T), int(batch), int(bool(backward))))


def _tokens_of(t, plan: Plan, T: int, name: str):
    """(address, token stride) of a tensor [T, C, N] with the last two axes contiguous, of a contiguous one's
    address, or of an eqlinear_heads."""
    C, N = plan.C, plan.N
    if type(t) is int:
        return t, C * N
    if type(t) is eqlinear_heads:
        return t.ptr, t.token_stride
    _gpu(t, name, plan.torch_dtype)
    if t.shape != (T, C, N):
        raise ValueError(f"{name}: expected shape {(T, C, N)}, got {tuple(t.shape)}")
    ts, sc, sn = t.stride()
    if (sn != 1 and N > 1) or (sc != N and C > 1):
        raise ValueError(f"{name}: the channel and group axes must be contiguous")
    return t.data_ptr(), ts


def eqlinear_group_norm(plan: Plan, x, gamma, beta, y, stats=None, offsets=None, batch: int | None = None,
                        workspace=None, T: int | None = None, stream=None):
    """y = act(gamma (x - mean) / sqrt(var + eps) + beta), statistics over each sample's tokens, a group's
    channels and their group elements; x, y [T, C, N].  The samples are offsets (int64 [batch + 1]) or batch
    equal runs (default: one)."""
    torch = _torch()
    _kind(plan, EQL_KIND_NORM, "eqlinear_group_norm")
    T, C, dt = _count(x, T, "x"), plan.C, plan.torch_dtype
    off, B = _sequences(offsets, batch)
    ws, nb = _workspace(workspace)
    _check(plan._lib.eqlinear_group_norm(
        plan.handle, *_tokens_of(x, plan, T, "x"), _dense(gamma, "gamma", dt, (C,)), _dense(beta, "beta", dt, (C,)),
        off, B, *_tokens_of(y, plan, T, "y"), _dense(stats, "stats", torch.float32, (B, plan.groups, 2)), T, ws, nb,
        _raw_stream(stream)), "eqlinear_group_norm")


def eqlinear_group_norm_backward(plan: Plan, dy, x, gamma, beta, stats, dx, dgamma, dbeta, offsets=None,
                                 batch: int | None = None, workspace=None, T: int | None = None, stream=None):
    """Gradients of eqlinear_group_norm: dx [T, C, N] in the plan dtype, dgamma and dbeta fp32 [C] (or None)."""
    torch = _torch()
    _kind(plan, EQL_KIND_NORM, "eqlinear_group_norm_backward")
    T, C, dt = _count(x, T, "x"), plan.C, plan.torch_dtype
    off, B = _sequences(offsets, batch)
    ws, nb = _workspace(workspace)
    _check(plan._lib.eqlinear_group_norm_backward(
        plan.handle, *_tokens_of(dy, plan, T, "dy"), *_tokens_of(x, plan, T, "x"), _dense(gamma, "gamma", dt, (C,)),
        _dense(beta, "beta", dt, (C,)), _dense(stats, "stats", torch.float32, (B, plan.groups, 2)), off, B,
        *_tokens_of(dx, plan, T, "dx"), _dense(dgamma, "dgamma", torch.float32, (C,)),
        _dense(dbeta, "dbeta", torch.float32, (C,)), T, ws, nb, _raw_stream(stream)), "eqlinear_group_norm_backward")


# --- softmax attention and its paged cache -------------------------------------------

def eqlinear_attention_plan(N: int, heads: int, kv_heads: int, d_k: int, d_v: int, dtype: int, causal: bool = False,
                            buckets: int = 0, max_distance: int = 0) -> Plan:
    """Plan of softmax attention: heads of d_k (queries, keys) and d_v (values) channels; with buckets > 0 its calls
    may take a bias for every head and bucket of distances."""
    lib = load_library()
    h = ctypes.c_void_p()
    _check(lib.eqlinear_attention_plan(ctypes.byref(h), N, heads, kv_heads, d_k, d_v, int(bool(causal)), buckets,
                                       max_distance, int(dtype)), "eqlinear_attention_plan")
    p = Plan(h.value, lib)
    p.heads, p.kv_heads, p.d_k, p.d_v, p.buckets = heads, kv_heads, d_k, d_v, buckets
    return p


def eqlinear_attention_bucket(plan: Plan, distance: int) -> int:
    """Bucket of a distance (query's position less key's); -1: none."""
    return int(plan._lib.eqlinear_attention_bucket(plan.handle, int(distance)))


def eqlinear_attention_workspace(plan: Plan, T: int, T_kv: int, batch: int, backward: bool = False) -> int:
    return int(plan._lib.eqlinear_attention_workspace(plan.handle, int(T), int(T_kv), int(batch), int(bool(backward))))


def _two_sequences(offsets, kv_offsets, batch, T, T_kv):
    """(address of offsets, of kv_offsets, number of sequences); keys without offsets of their own share the queries'."""
    off, B = _sequences(offsets, batch)
    if kv_offsets is not None:
        kv, n = _sequences(kv_offsets, B if isinstance(kv_offsets, int) else None)
        if n != B and (offsets is not None or batch is not None):
            raise ValueError(f"kv_offsets: expected batch + 1 = {B + 1} values, got {n + 1}")
        return off, kv, n
    if off is not None and T != T_kv:
        raise ValueError("kv_offsets is required where k and v have other tokens than q")
    return off, off, B


def eqlinear_attention(plan: Plan, q, k, v, o, scale: float, bias=None, lse=None, offsets=None, kv_offsets=None,
                       batch: int | None = None, workspace=None, T: int | None = None, T_kv: int | None = None,
                       stream=None):
    """Softmax attention: o [T, heads, d_v, N] of q [T, heads, d_k, N] over k [T_kv, kv_heads, d_k, N] and
    v [T_kv, kv_heads, d_v, N]; bias [heads, buckets]; lse fp32 [heads, T] out (or None).  The sequences are offsets
    (int64 [batch + 1]; kv_offsets those of k and v, default: the same) or batch equal runs (default: one)."""
    torch = _torch()
    _kind(plan, EQL_KIND_ATTENTION, "eqlinear_attention")
    T, S = _count(q, T, "q"), _count(k, T_kv, "k")
    H, K, dk, dv = plan.heads, plan.kv_heads, plan.d_k, plan.d_v
    off, kv_off, B = _two_sequences(offsets, kv_offsets, batch, T, S)
    ws, nb = _workspace(workspace)
    _check(plan._lib.eqlinear_attention(
        plan.handle, _heads(q, plan, T, H, dk, "q"), _heads(k, plan, S, K, dk, "k"), _heads(v, plan, S, K, dv, "v"),
        scale, _dense(bias, "bias", plan.torch_dtype, (H, plan.buckets)), off, kv_off, B,
        _heads(o, plan, T, H, dv, "o"), _dense(lse, "lse", torch.float32, (H, T)), T, S, ws, nb, _raw_stream(stream)),
        "eqlinear_attention")


def eqlinear_attention_backward(plan: Plan, q, k, v, o, do, lse, dq, dk, dv, scale: float, bias=None, dbias=None,
                                offsets=None, kv_offsets=None, batch: int | None = None, workspace=None,
                                T: int | None = None, T_kv: int | None = None, stream=None):
    """Gradients dq, dk, dv (and dbias, fp32 [heads, buckets]) of eqlinear_attention from its o and lse."""
    torch = _torch()
    _kind(plan, EQL_KIND_ATTENTION, "eqlinear_attention_backward")
    T, S = _count(q, T, "q"), _count(k, T_kv, "k")
    H, K, ck, cv = plan.heads, plan.kv_heads, plan.d_k, plan.d_v
    off, kv_off, B = _two_sequences(offsets, kv_offsets, batch, T, S)
    ws, nb = _workspace(workspace)
    _check(plan._lib.eqlinear_attention_backward(
        plan.handle, _heads(q, plan, T, H, ck, "q"), _heads(k, plan, S, K, ck, "k"), _heads(v, plan, S, K, cv, "v"),
        _heads(o, plan, T, H, cv, "o"), _heads(do, plan, T, H, cv, "do"), _dense(lse, "lse", torch.float32, (H, T)),
        scale, _dense(bias, "bias", plan.torch_dtype, (H, plan.buckets)), off, kv_off, B,
        _heads(dq, plan, T, H, ck, "dq"), _heads(dk, plan, S, K, ck, "dk"), _heads(dv, plan, S, K, cv, "dv"),
        _dense(dbias, "dbias", torch.float32, (H, plan.buckets)), T, S, ws, nb, _raw_stream(stream)),
        "eqlinear_attention_backward")


def _pages(t, plan: Plan, d: int, blocks: int, block_size: int, name: str):
    """A cache [blocks, block_size, kv_heads, d, N] (the last two axes contiguous), the address of a contiguous one, or
    an eqlinear_pages as it is."""
    if type(t) is eqlinear_pages:
        return t
    K, N = plan.kv_heads, plan.N
    if type(t) is int:
        return eqlinear_pages(t, block_size * K * d * N, K * d * N, d * N)
    _gpu(t, name, plan.torch_dtype)
    if t.shape != (blocks, block_size, K, d, N):
        raise ValueError(f"{name}: expected shape {(blocks, block_size, K, d, N)}, got {tuple(t.shape)}")
    bs, ts, hs, sd, sn = t.stride()
    if (sn != 1 and N > 1) or (sd != N and d > 1):
        raise ValueError(f"{name}: the channel and group axes must be contiguous")
    return eqlinear_pages(t.data_ptr(), bs, ts, hs)


def _cache_shape(k_cache, blocks, block_size):
    """(blocks, block_size) of a cache: a tensor's own, or as given with an address."""
    if isinstance(k_cache, (int, eqlinear_pages)):
        if blocks is None or block_size is None:
            raise ValueError("blocks and block_size are required when k_cache is an address")
        return int(blocks), int(block_size)
    return k_cache.shape[0], k_cache.shape[1]


def eqlinear_attention_step_workspace(plan: Plan, batch: int) -> int:
    return int(plan._lib.eqlinear_attention_step_workspace(plan.handle, int(batch)))


def eqlinear_attention_step(plan: Plan, q, k_cache, v_cache, table, lengths, o, scale: float, bias=None, lse=None,
                            batch: int | None = None, blocks: int | None = None, block_size: int | None = None,
                            max_blocks: int | None = None, workspace=None, stream=None):
    """Attention of one new token for each of batch sequences: q [batch, heads, d_k, N] over the keys and values of
    k_cache [blocks, block_size, kv_heads, d_k, N] and v_cache that table (int32 [batch, max_blocks]) names, the first
    lengths[b] (int32) of them; o [batch, heads, d_v, N], lse fp32 [heads, batch] (or None)."""
    torch = _torch()
    _kind(plan, EQL_KIND_ATTENTION, "eqlinear_attention_step")
    B = _count(q, batch, "q")
    H, K, dk, dv = plan.heads, plan.kv_heads, plan.d_k, plan.d_v
    nb, bs = _cache_shape(k_cache, blocks, block_size)
    if max_blocks is None:
        if isinstance(table, int):
            raise ValueError("max_blocks is required when table is an address")
        max_blocks = table.shape[1]
    ws, n = _workspace(workspace)
    _check(plan._lib.eqlinear_attention_step(
        plan.handle, _heads(q, plan, B, H, dk, "q"), _pages(k_cache, plan, dk, nb, bs, "k_cache"),
        _pages(v_cache, plan, dv, nb, bs, "v_cache"), nb, bs, _dense(table, "table", torch.int32, (B, max_blocks)),
        max_blocks, _dense(lengths, "lengths", torch.int32, (B,)), scale,
        _dense(bias, "bias", plan.torch_dtype, (H, plan.buckets)), _heads(o, plan, B, H, dv, "o"),
        _dense(lse, "lse", torch.float32, (H, B)), B, ws, n, _raw_stream(stream)), "eqlinear_attention_step")


def eqlinear_cache_tables_workspace(batch: int) -> int:
    return int(load_library().eqlinear_cache_tables_workspace(int(batch)))


def eqlinear_cache_tables(lengths, added, free_blocks, cursor, table, block_size: int, lengths_out, cursor_out, slots,
                          positions, offsets, workspace, stream=None):
    """Tables of a paged cache for the next step: requests of lengths (int32 [batch]) tokens get added more, whose
    blocks come from free_blocks (int32) at cursor (int32 [1]) on; out: the new blocks in table (int32 [batch,
    max_blocks]), lengths_out, cursor_out, and for the packed new tokens slots (int64 [T]), positions (int32 [T]) and
    offsets (int64 [batch + 1]).  lengths_out may be lengths and cursor_out cursor."""
    torch = _torch()
    i32, i64 = torch.int32, torch.int64
    try:
        B, T, F, rows = lengths.numel(), slots.numel(), free_blocks.numel(), table.shape
    except AttributeError:
        raise TypeError("eqlinear_cache_tables: expected torch tensors (their sizes are checked)") from None
    if rows != (B, rows[-1]):
        raise ValueError(f"table: expected shape {(B, rows[-1])}, got {tuple(rows)}")
    ws, nb = _workspace(workspace)
    _check(load_library().eqlinear_cache_tables(
        _flat(lengths, "lengths", i32, B), _flat(added, "added", i32, B), _flat(free_blocks, "free_blocks", i32, F), F,
        _flat(cursor, "cursor", i32, 1), _flat(table, "table", i32, B * rows[1]), rows[1], block_size,
        _flat(lengths_out, "lengths_out", i32, B), _flat(cursor_out, "cursor_out", i32, 1), _flat(slots, "slots", i64, T),
        _flat(positions, "positions", i32, T), _flat(offsets, "offsets", i64, B + 1), B, T, ws, nb, _raw_stream(stream)),
        "eqlinear_cache_tables")


def _flat(t, name: str, dtype, numel: int):
    """Address of a contiguous GPU tensor of the given dtype and number of elements (whose shape is a single axis, or
    has been checked: half of _dense's cost)."""
    try:
        if t.is_cuda and t.dtype is dtype and t.numel() == numel and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _dense(t, name, dtype, (numel,))


def eqlinear_cache_store(plan: Plan, k, v, slots, k_cache, v_cache, T: int | None = None, blocks: int | None = None,
                         block_size: int | None = None, stream=None):
    """Rows of k [T, kv_heads, d_k, N] and v [T, kv_heads, d_v, N] to slots (int64 [T]) of k_cache [blocks, block_size,
    kv_heads, d_k, N] and v_cache; slots that the cache does not have are skipped."""
    torch = _torch()
    _kind(plan, EQL_KIND_ATTENTION, "eqlinear_cache_store")
    T = _count(k, T, "k")
    K, dk, dv = plan.kv_heads, plan.d_k, plan.d_v
    nb, bs = _cache_shape(k_cache, blocks, block_size)
    _check(plan._lib.eqlinear_cache_store(
        plan.handle, _heads(k, plan, T, K, dk, "k"), _heads(v, plan, T, K, dv, "v"),
        _dense(slots, "slots", torch.int64, (T,)), _pages(k_cache, plan, dk, nb, bs, "k_cache"),
        _pages(v_cache, plan, dv, nb, bs, "v_cache"), nb, bs, T, _raw_stream(stream)), "eqlinear_cache_store")


def built() -> bool:
    return os.path.exists(LIB_PATH)
