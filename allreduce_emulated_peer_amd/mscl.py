"""Thin ctypes binding over libmscl.so (C ABI in include/mscl.h).

Argument marshalling only: every step of the AllReduce, of the linear layer
and of layer norm runs in the HIP library.  Names mirror the C entry points without the ``mscl_`` prefix.
There is no fallback: if the library is missing, loading raises.

Pointers are plain integers (device addresses, e.g. ``tensor.data_ptr()``),
streams are ``hipStream_t`` values as integers (``torch.cuda.Stream.cuda_stream``;
0 = default stream).  ``allreduce_tensors`` and the operators' ``*_tensors``
are convenience wrappers that take torch tensors and the current torch stream.
"""

from __future__ import annotations

import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmscl.so")

FLOAT32, FLOAT16, BFLOAT16 = 0, 1, 2
ALGO_AUTO, ALGO_ONE_SHOT, ALGO_TWO_SHOT, ALGO_TWO_SHOT_FUSED, ALGO_TWO_SHOT_PORT = 0, 1, 2, 3, 4
ALGO_TWO_SHOT_FUSED_NOBARRIER = 5
ALGO_TWO_SHOT_PERTILE = 6
MAX_RANKS = 16

SUCCESS = 0
ERR_INVALID_ARGUMENT = 1
ERR_UNSUPPORTED = 2
ERR_MISALIGNED = 3
ERR_NOT_INITIALIZED = 4
ERR_OUT_OF_MEMORY = 5
ERR_HIP = 6
ERR_TIMEOUT = 7
ERR_PROTOCOL = 8

DTYPE_CODES = {"fp32": FLOAT32, "fp16": FLOAT16, "bf16": BFLOAT16}
ALGO_CODES = {"auto": ALGO_AUTO, "one_shot": ALGO_ONE_SHOT, "two_shot": ALGO_TWO_SHOT,
              "two_shot_fused": ALGO_TWO_SHOT_FUSED, "two_shot_port": ALGO_TWO_SHOT_PORT,
              "two_shot_fused_nobarrier": ALGO_TWO_SHOT_FUSED_NOBARRIER, "two_shot_pertile": ALGO_TWO_SHOT_PERTILE}

ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4
ACTIVATION_CODES = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH,
                    "silu": ACT_SILU}

# every function include/mscl.h declares
EXPORTS = (
    "mscl_version", "mscl_status_string", "mscl_last_error_string", "mscl_channel_create",
    "mscl_channel_destroy", "mscl_channel_check", "mscl_channel_reset", "mscl_allreduce",
    "mscl_select_algo", "mscl_channel_plan", "mscl_channel_set_fault_controls", "mscl_channel_set_checks",
    "mscl_reduce_scatter", "mscl_allgather", "mscl_channel_selftest", "mscl_allreduce_noalloc",
    "mscl_linear", "mscl_linear_workspace", "mscl_linear_backward", "mscl_linear_backward_workspace",
    "mscl_layer_norm", "mscl_layer_norm_backward", "mscl_layer_norm_backward_workspace",
)

# the argument records of include/mscl.h, field by field: pointers and sizes
# ("N": 8 bytes), then the codes ("i")
LINEAR = struct.Struct("14Nii")
LINEAR_BACKWARD = struct.Struct("16Nii")
LAYER_NORM = struct.Struct("10Ndii")
LAYER_NORM_BACKWARD = struct.Struct("13Nii")


class MsclError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: status {status} ({detail})")
        self.status = status


class Plan(ctypes.Structure):
    _fields_ = [
        ("algo", ctypes.c_int),
        ("nranks", ctypes.c_int),
        ("workgroups_per_rank", ctypes.c_int),
        ("threads_per_workgroup", ctypes.c_int),
        ("vectors_per_thread", ctypes.c_int),
        ("uses_barrier", ctypes.c_int),
        ("chunk_elems", ctypes.c_size_t),
        ("cached_puts", ctypes.c_int),
        ("held_tiles", ctypes.c_int),
        ("slices", ctypes.c_int),
        ("slice_elems", ctypes.c_size_t),
        ("tile_interleave", ctypes.c_int),
    ]


_lib = None


def load(path: str = LIB_PATH):
    """Open libmscl.so once; raises FileNotFoundError if it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is missing: build it with allreduce_emulated_peer_amd/build.py")
    lib = ctypes.CDLL(path)
    c_int, c_size, vp = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
    lib.mscl_version.restype = c_int
    lib.mscl_version.argtypes = []
    lib.mscl_status_string.restype = ctypes.c_char_p
    lib.mscl_status_string.argtypes = [c_int]
    lib.mscl_last_error_string.restype = ctypes.c_char_p
    lib.mscl_last_error_string.argtypes = []
    lib.mscl_channel_create.restype = c_int
    lib.mscl_channel_create.argtypes = [c_int, c_int, ctypes.POINTER(vp)]
    for name in ("mscl_channel_destroy", "mscl_channel_check", "mscl_channel_reset"):
        getattr(lib, name).restype = c_int
        getattr(lib, name).argtypes = [vp]
    for name in ("mscl_allreduce", "mscl_allreduce_noalloc"):
        getattr(lib, name).restype = c_int
        getattr(lib, name).argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), c_size, c_int, c_int, c_int, vp]
    for name in ("mscl_reduce_scatter", "mscl_allgather"):
        getattr(lib, name).restype = c_int
        getattr(lib, name).argtypes = [ctypes.POINTER(vp), ctypes.POINTER(vp), c_size, c_int, c_int, vp]
    lib.mscl_channel_selftest.restype = c_int
    lib.mscl_channel_selftest.argtypes = [vp, ctypes.c_uint32, ctypes.POINTER(ctypes.c_uint64)]
    lib.mscl_select_algo.restype = c_int
    lib.mscl_select_algo.argtypes = [c_size, c_int, c_int, ctypes.POINTER(c_int)]
    lib.mscl_channel_plan.restype = c_int
    lib.mscl_channel_plan.argtypes = [vp, c_size, c_int, c_int, c_int, ctypes.POINTER(Plan)]
    lib.mscl_channel_set_fault_controls.restype = c_int
    lib.mscl_channel_set_fault_controls.argtypes = [vp, ctypes.c_uint64, c_int]
    lib.mscl_channel_set_checks.restype = c_int
    lib.mscl_channel_set_checks.argtypes = [vp, c_int, c_int]
    for name in ("mscl_linear", "mscl_linear_backward", "mscl_layer_norm_backward"):
        getattr(lib, name).restype = c_int
        getattr(lib, name).argtypes = [ctypes.c_char_p, vp, c_size, vp]
        getattr(lib, name + "_workspace").restype = c_int
        getattr(lib, name + "_workspace").argtypes = [ctypes.c_char_p, ctypes.POINTER(c_size)]
    lib.mscl_layer_norm.restype = c_int
    lib.mscl_layer_norm.argtypes = [ctypes.c_char_p, vp]
    _lib = lib
    return lib


def _check(status: int, where: str) -> None:
    if status != SUCCESS:
        lib = load()
        detail = lib.mscl_last_error_string().decode() or lib.mscl_status_string(status).decode()
        raise MsclError(status, where, detail)


def version() -> int:
    return load().mscl_version()


def status_string(status: int) -> str:
    return load().mscl_status_string(status).decode()


def last_error_string() -> str:
    return load().mscl_last_error_string().decode()


def _ptr_array(ptrs):
    return (ctypes.c_void_p * len(ptrs))(*[ctypes.c_void_p(int(p)) if p else None for p in ptrs])


def raw_allreduce(inputs, outputs, count: int, dtype: int, nranks: int, algo: int, stream: int) -> int:
    """mscl_allreduce with no exception: returns the status code."""
    ins = _ptr_array(inputs) if inputs is not None else None
    outs = _ptr_array(outputs) if outputs is not None else None
    return load().mscl_allreduce(ins, outs, count, dtype, nranks, algo, ctypes.c_void_p(int(stream) or None))


def allreduce(inputs, outputs, count: int, dtype: int, nranks: int, algo: int = ALGO_AUTO, stream: int = 0) -> None:
    """mscl_allreduce: `inputs` / `outputs` are sequences of device addresses."""
    _check(raw_allreduce(inputs, outputs, count, dtype, nranks, algo, stream), "mscl_allreduce")


def raw_allreduce_noalloc(inputs, outputs, count: int, dtype: int, nranks: int, algo: int, stream: int) -> int:
    """mscl_allreduce_noalloc with no exception: returns the status code."""
    ins = _ptr_array(inputs) if inputs is not None else None
    outs = _ptr_array(outputs) if outputs is not None else None
    return load().mscl_allreduce_noalloc(ins, outs, count, dtype, nranks, algo, ctypes.c_void_p(int(stream) or None))


def allreduce_noalloc(inputs, outputs, count: int, dtype: int, nranks: int, algo: int = ALGO_AUTO,
                      stream: int = 0) -> None:
    """mscl_allreduce_noalloc: mscl_allreduce with no channel set and no allocation."""
    _check(raw_allreduce_noalloc(inputs, outputs, count, dtype, nranks, algo, stream), "mscl_allreduce_noalloc")


def raw_reduce_scatter(inputs, outputs, recvcount: int, dtype: int, nranks: int, stream: int) -> int:
    ins = _ptr_array(inputs) if inputs is not None else None
    outs = _ptr_array(outputs) if outputs is not None else None
    return load().mscl_reduce_scatter(ins, outs, recvcount, dtype, nranks, ctypes.c_void_p(int(stream) or None))


def reduce_scatter(inputs, outputs, recvcount: int, dtype: int, nranks: int, stream: int = 0) -> None:
    """mscl_reduce_scatter: inputs hold nranks*recvcount elements, outputs recvcount."""
    _check(raw_reduce_scatter(inputs, outputs, recvcount, dtype, nranks, stream), "mscl_reduce_scatter")


def raw_allgather(inputs, outputs, sendcount: int, dtype: int, nranks: int, stream: int) -> int:
    ins = _ptr_array(inputs) if inputs is not None else None
    outs = _ptr_array(outputs) if outputs is not None else None
    return load().mscl_allgather(ins, outs, sendcount, dtype, nranks, ctypes.c_void_p(int(stream) or None))


def allgather(inputs, outputs, sendcount: int, dtype: int, nranks: int, stream: int = 0) -> None:
    """mscl_allgather: inputs hold sendcount elements, outputs nranks*sendcount."""
    _check(raw_allgather(inputs, outputs, sendcount, dtype, nranks, stream), "mscl_allgather")


def channel_create(nranks: int, device: int) -> int:
    h = ctypes.c_void_p()
    _check(load().mscl_channel_create(nranks, device, ctypes.byref(h)), "mscl_channel_create")
    return h.value


def channel_destroy(handle: int) -> None:
    _check(load().mscl_channel_destroy(ctypes.c_void_p(handle)), "mscl_channel_destroy")


def channel_check(handle: int) -> int:
    """Status recorded on the device by earlier calls (SUCCESS, ERR_TIMEOUT, ERR_PROTOCOL, ...)."""
    return load().mscl_channel_check(ctypes.c_void_p(handle))


def channel_reset(handle: int) -> None:
    _check(load().mscl_channel_reset(ctypes.c_void_p(handle)), "mscl_channel_reset")


def channel_set_fault_controls(handle: int, wait_timeout_us: int = 0, drop_signal_rank: int = -1) -> None:
    _check(load().mscl_channel_set_fault_controls(ctypes.c_void_p(handle), wait_timeout_us, drop_signal_rank),
           "mscl_channel_set_fault_controls")


def channel_set_checks(handle: int, check_protocol: bool = True, double_signal_rank: int = -1) -> None:
    """mscl_channel_set_checks: protocol checks of every device-side wait, and
    the test control that makes one rank signal twice."""
    _check(load().mscl_channel_set_checks(ctypes.c_void_p(handle), int(bool(check_protocol)), double_signal_rank),
           "mscl_channel_set_checks")


def channel_selftest(handle: int, rounds: int) -> int:
    """mscl_channel_selftest: returns the number of mismatching words (expected 0)."""
    out = ctypes.c_uint64()
    _check(load().mscl_channel_selftest(ctypes.c_void_p(handle), rounds, ctypes.byref(out)), "mscl_channel_selftest")
    return out.value


def select_algo(count: int, dtype: int, nranks: int) -> int:
    out = ctypes.c_int()
    _check(load().mscl_select_algo(count, dtype, nranks, ctypes.byref(out)), "mscl_select_algo")
    return out.value


def channel_plan(handle: int, count: int, dtype: int, algo: int = ALGO_AUTO, in_place: bool = False) -> Plan:
    plan = Plan()
    _check(load().mscl_channel_plan(ctypes.c_void_p(handle), count, dtype, algo, int(in_place), ctypes.byref(plan)),
           "mscl_channel_plan")
    return plan


def allreduce_tensors(inputs, outputs, algo: int = ALGO_AUTO, stream=None) -> None:
    """AllReduce over lists of equal-shape contiguous CUDA(HIP) tensors.

    dtype comes from the tensors (float32 / float16 / bfloat16); the call
    runs with the tensors' device current (the channel set is looked up per
    device, so mscl_channel_create must have been called for that device and
    rank count); the stream defaults to torch's current stream there.
    """
    import torch

    codes = {torch.float32: FLOAT32, torch.float16: FLOAT16, torch.bfloat16: BFLOAT16}
    if len(inputs) != len(outputs) or not inputs:
        raise ValueError("need one output per input")
    t0 = inputs[0]
    if not t0.is_cuda:
        raise ValueError("tensors must be on a GPU")
    for t in list(inputs) + list(outputs):
        if t.dtype != t0.dtype or t.numel() != t0.numel() or not t.is_contiguous() or t.device != t0.device:
            raise ValueError("tensors must share dtype, size and device and be contiguous")
    if t0.dtype not in codes:
        raise ValueError(f"unsupported dtype {t0.dtype}")
    with torch.cuda.device(t0.device):
        if stream is None:
            stream = torch.cuda.current_stream(t0.device)
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        allreduce([t.data_ptr() for t in inputs], [t.data_ptr() for t in outputs], t0.numel(), codes[t0.dtype],
                  len(inputs), algo, handle)


# ---------------------------------------------------------------- linear layer and layer norm

# A call on small matrices takes as long on the host as on the GPU, so these
# functions look each thing up once and take the common case (a matrix, on the
# current device and stream) first.
_torch = None
_CODES = {}  # torch dtype -> element type code
_raw_stream = None
_outside_autograd = None


def _need_torch():
    global _torch, _raw_stream, _outside_autograd
    if _torch is None:
        import torch

        class OutsideAutograd(torch.autograd.Function):
            """call(), which autograd knows no gradient of: a backward pass through its results raises."""

            @staticmethod
            def forward(ctx, call, name, *inputs):
                ctx.name = name
                return call()

            @staticmethod
            def backward(ctx, *grads):
                raise RuntimeError(f"{ctx.name}_tensors is not part of autograd's graph: run {ctx.name}_backward_tensors, and "
                                   "call it under torch.no_grad() or detach what it takes or returns")

        _outside_autograd = OutsideAutograd.apply

        _CODES.update({torch.float32: FLOAT32, torch.float16: FLOAT16, torch.bfloat16: BFLOAT16})
        # the current stream's handle without a Stream object around it (2 us less), where torch has that
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _torch = torch
    return _torch


def _same_kind(like, name, t):
    """Checks shared by an operator's tensors: element type, device."""
    if t is not None:
        if t.device != like.device:
            raise ValueError(f"{name} must be on {like.device}")
        if t.dtype != like.dtype:
            raise ValueError(f"{name} must be of {like.dtype}")


def _matrix(name, t, cols):
    """`t` as rows of `cols` elements that lie next to each other: a view where strides allow one."""
    shape = t.shape
    if not shape or shape[-1] != cols:
        raise ValueError(f"{name} must have {cols} columns")
    if len(shape) != 2:
        t = t.reshape(-1, cols) if cols else t.reshape(shape[:-1].numel(), 0)
    if not t.is_contiguous():
        row, element = t.stride()
        if element != 1 and cols > 1:
            raise ValueError(f"the rows of {name} must be contiguous")
        if row < cols and t.shape[0] > 1:
            raise ValueError(f"the rows of {name} must not overlap")
    return t


def _vector(name, t, n):
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n}")


def _elsewhere(device, stream, tensors, call):
    """call() with `device` current and, if it is given, on `stream` (a torch stream or a handle)."""
    torch = _torch
    with torch.cuda.device(device):
        if stream is None:
            return call()
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        with torch.cuda.stream(stream):
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
            return call()


def _workspace(query, call, like):
    """The workspace that a call asks for, as (tensor or None, its bytes)."""
    need = ctypes.c_size_t()
    status = query(call, ctypes.byref(need))
    if status:
        _check(status, query.__name__)
    if need.value == 0:
        return None, 0
    return _torch.empty(need.value, dtype=_torch.uint8, device=like.device), need.value


def _address(t):
    return 0 if t is None else t.data_ptr()


def _row_stride(t):
    return 0 if t is None else t.stride(0)


def linear_tensors(x, weight, bias=None, residual=None, activation="none", return_preact=False, stream=None):
    """mscl_linear on torch tensors: activation(x @ weight.T + bias) + residual.

    x is (..., in), weight (out, in), bias (out), residual (..., out), all of
    one dtype (float32 / float16 / bfloat16) and device; rows may be strided,
    elements of a row must be contiguous.  activation is a name of
    ACTIVATION_CODES.  Returns y (..., out), or (y, preact) with return_preact:
    what linear_backward_tensors needs where there is an activation.  Autograd
    does not reach through it: where an input requires a gradient, so do the
    results, and a backward pass through them raises.
    """
    torch, lib = _torch or _need_torch(), _lib or load()
    dtype = _CODES.get(x.dtype)
    if dtype is None:
        raise ValueError(f"unsupported dtype {x.dtype}")
    if activation not in ACTIVATION_CODES:
        raise ValueError(f"unknown activation {activation!r}")
    if weight.dim() != 2:
        raise ValueError("weight must be a matrix")
    _same_kind(x, "weight", weight)
    _same_kind(x, "bias", bias)
    _same_kind(x, "residual", residual)
    if not x.is_cuda:
        raise ValueError("tensors must be on a GPU")
    n, k = weight.shape
    xm, wm = _matrix("x", x, k), _matrix("weight", weight, k)
    rows = xm.shape[0]
    if bias is not None:
        _vector("bias", bias, n)
    rm = None
    if residual is not None:
        if residual.shape != x.shape[:-1] + (n,):
            raise ValueError(f"residual must be {tuple(x.shape[:-1]) + (n,)}")
        rm = _matrix("residual", residual, n)

    index = x.device.index
    if stream is not None or index != torch.cuda.current_device():
        return _elsewhere(x.device, stream, (x, weight, bias, residual),
                          lambda: linear_tensors(x, weight, bias, residual, activation, return_preact))
    if torch.is_grad_enabled() and (x.requires_grad or weight.requires_grad or bias is not None and bias.requires_grad
                                    or residual is not None and residual.requires_grad):
        return _outside_autograd(lambda: linear_tensors(x, weight, bias, residual, activation, return_preact), "linear",
                                 x, weight, bias, residual)
    y = torch.empty((rows, n), dtype=x.dtype, device=x.device)
    z = torch.empty_like(y) if return_preact else None
    call = LINEAR.pack(xm.data_ptr(), xm.stride(0), wm.data_ptr(), wm.stride(0), _address(bias), _address(rm),
                       _row_stride(rm), y.data_ptr(), n, _address(z), n, rows, k, n, dtype,
                       ACTIVATION_CODES[activation])
    space, size = _workspace(lib.mscl_linear_workspace, call, x)
    status = lib.mscl_linear(call, _address(space), size, _raw_stream(index) or None)
    if status:
        _check(status, "mscl_linear")
    if x.dim() != 2:
        y = y.view(x.shape[:-1] + (n,))
        z = z.view(y.shape) if return_preact else None
    return (y, z) if return_preact else y


def linear_backward_tensors(dy, x, weight, preact=None, activation="none", need_dx=True, need_dw=True, need_db=True,
                            stream=None):
    """mscl_linear_backward on torch tensors: (dx, dw, db) of linear_tensors.

    dy is the gradient of y (..., out) (and of the residual), preact what
    linear_tensors returned with return_preact (needed unless activation is
    "none").  A gradient that is not needed is None.
    """
    torch, lib = _torch or _need_torch(), _lib or load()
    dtype = _CODES.get(dy.dtype)
    if dtype is None:
        raise ValueError(f"unsupported dtype {dy.dtype}")
    if activation not in ACTIVATION_CODES:
        raise ValueError(f"unknown activation {activation!r}")
    if weight.dim() != 2:
        raise ValueError("weight must be a matrix")
    if activation != "none" and preact is None:
        raise ValueError("an activation's gradient needs preact")
    if activation == "none":
        preact = None
    _same_kind(dy, "x", x)
    _same_kind(dy, "weight", weight)
    _same_kind(dy, "preact", preact)
    if not dy.is_cuda:
        raise ValueError("tensors must be on a GPU")
    n, k = weight.shape
    gm, xm, wm = _matrix("dy", dy, n), _matrix("x", x, k), _matrix("weight", weight, k)
    rows = gm.shape[0]
    if x.shape[:-1] != dy.shape[:-1]:
        raise ValueError("dy and x must have the same rows")
    zm = None
    if preact is not None:
        if preact.shape != dy.shape:
            raise ValueError("preact must have dy's shape")
        zm = _matrix("preact", preact, n)

    index = dy.device.index
    if stream is not None or index != torch.cuda.current_device():
        return _elsewhere(dy.device, stream, (dy, x, weight, preact),
                          lambda: linear_backward_tensors(dy, x, weight, preact, activation, need_dx, need_dw, need_db))
    dx = torch.empty((rows, k), dtype=dy.dtype, device=dy.device) if need_dx else None
    dw = torch.empty((n, k), dtype=dy.dtype, device=dy.device) if need_dw else None
    db = torch.empty((n,), dtype=dy.dtype, device=dy.device) if need_db else None
    call = LINEAR_BACKWARD.pack(gm.data_ptr(), gm.stride(0), xm.data_ptr(), xm.stride(0), wm.data_ptr(),
                                wm.stride(0), _address(zm), _row_stride(zm), _address(dx), k, _address(dw), k,
                                _address(db), rows, k, n, dtype, ACTIVATION_CODES[activation])
    space, size = _workspace(lib.mscl_linear_backward_workspace, call, dy)
    status = lib.mscl_linear_backward(call, _address(space), size, _raw_stream(index) or None)
    if status:
        _check(status, "mscl_linear_backward")
    if need_dx and x.dim() != 2:
        dx = dx.view(x.shape)
    return dx, dw, db


def _param_type(like, weight, bias, width):
    """The parameters' type: that of the rows, or float32; None says nothing."""
    if weight is None and bias is None:
        return like.dtype
    kind = bias.dtype if weight is None else weight.dtype
    if kind != like.dtype and kind != _torch.float32 or bias is not None and bias.dtype != kind:
        raise ValueError(f"parameters must all be of {like.dtype} or all of float32")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            if t.device != like.device:
                raise ValueError(f"{name} must be on {like.device}")
            _vector(name, t, width)
    return kind


def layer_norm_tensors(x, weight=None, bias=None, eps=1e-5, return_stats=False, stream=None):
    """mscl_layer_norm on torch tensors, over the last dimension of x.

    weight and bias have x's dtype or float32.  Returns y, or (y, mean, rstd)
    with return_stats: float32 of x's leading shape, what
    layer_norm_backward_tensors needs.  Autograd does not reach through it, as
    through linear_tensors.
    """
    torch, lib = _torch or _need_torch(), _lib or load()
    codes = _CODES
    if x.dtype not in codes:
        raise ValueError(f"unsupported dtype {x.dtype}")
    shape = x.shape
    if not shape or shape[-1] == 0:
        raise ValueError("x must have a last dimension of at least 1")
    if not eps >= 0:
        raise ValueError("eps must be at least 0")
    width = shape[-1]
    param = codes[_param_type(x, weight, bias, width)]
    if not x.is_cuda:
        raise ValueError("tensors must be on a GPU")
    xm = _matrix("x", x, width)
    rows = xm.shape[0]

    index = x.device.index
    if stream is not None or index != torch.cuda.current_device():
        return _elsewhere(x.device, stream, (x, weight, bias),
                          lambda: layer_norm_tensors(x, weight, bias, eps, return_stats))
    if torch.is_grad_enabled() and (x.requires_grad or weight is not None and weight.requires_grad
                                    or bias is not None and bias.requires_grad):
        return _outside_autograd(lambda: layer_norm_tensors(x, weight, bias, eps, return_stats), "layer_norm", x, weight,
                                 bias)
    y = torch.empty_like(xm) if xm.is_contiguous() else torch.empty((rows, width), dtype=x.dtype, device=x.device)
    mean = rstd = None
    if return_stats:
        mean = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    call = LAYER_NORM.pack(xm.data_ptr(), xm.stride(0), _address(weight), _address(bias), y.data_ptr(), width,
                           _address(mean), _address(rstd), rows, width, eps, codes[x.dtype], param)
    status = lib.mscl_layer_norm(call, _raw_stream(index) or None)
    if status:
        _check(status, "mscl_layer_norm")
    if xm is not x:
        y = y.view(shape)
    return (y, mean, rstd) if return_stats else y


def layer_norm_backward_tensors(dy, x, mean, rstd, weight=None, need_dx=True, need_dw=True, need_db=True, stream=None):
    """mscl_layer_norm_backward on torch tensors: (dx, dw, db) of layer_norm_tensors.

    mean and rstd are what it returned with return_stats.  dw and db have
    weight's dtype (dy's without a weight).  A gradient that is not needed is
    None.
    """
    torch, lib = _torch or _need_torch(), _lib or load()
    codes = _CODES
    if dy.dtype not in codes:
        raise ValueError(f"unsupported dtype {dy.dtype}")
    if dy.dim() == 0 or dy.shape[-1] == 0:
        raise ValueError("dy must have a last dimension of at least 1")
    if x.shape != dy.shape:
        raise ValueError("dy and x must have the same shape")
    _same_kind(dy, "x", x)
    width = dy.shape[-1]
    kind = _param_type(dy, weight, None, width)
    if not dy.is_cuda:
        raise ValueError("tensors must be on a GPU")
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or t.device != dy.device or t.shape != dy.shape[:-1] or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous, float32, on {dy.device} and {tuple(dy.shape[:-1])}")
    gm, xm = _matrix("dy", dy, width), _matrix("x", x, width)
    rows = gm.shape[0]

    index = dy.device.index
    if stream is not None or index != torch.cuda.current_device():
        return _elsewhere(dy.device, stream, (dy, x, mean, rstd, weight),
                          lambda: layer_norm_backward_tensors(dy, x, mean, rstd, weight, need_dx, need_dw, need_db))
    dx = torch.empty((rows, width), dtype=dy.dtype, device=dy.device) if need_dx else None
    dw = torch.empty((width,), dtype=kind, device=dy.device) if need_dw else None
    db = torch.empty((width,), dtype=kind, device=dy.device) if need_db else None
    call = LAYER_NORM_BACKWARD.pack(gm.data_ptr(), gm.stride(0), xm.data_ptr(), xm.stride(0), mean.data_ptr(),
                                    rstd.data_ptr(), _address(weight), _address(dx), width, _address(dw),
                                    _address(db), rows, width, codes[dy.dtype], codes[kind])
    space, size = _workspace(lib.mscl_layer_norm_backward_workspace, call, dy)
    status = lib.mscl_layer_norm_backward(call, _address(space), size, _raw_stream(index) or None)
    if status:
        _check(status, "mscl_layer_norm_backward")
    if need_dx and dy.dim() != 2:
        dx = dx.view(dy.shape)
    return dx, dw, db
