"""Python binding of liblq, the B200 LiftQuant decode library (argument marshalling only).

Every function here checks tensor placement and dtypes, then calls the extern "C"
entry point of the same name in liblq.so (declared in include/liblq.h). All
arithmetic runs in the library's CUDA kernels; torch only supplies device memory
and the current stream. There is no CPU fallback: if liblq.so has not been built,
the first call raises.
"""
import ctypes
import os

import torch

__all__ = [
    "LQError", "lib", "abi_version", "lifted_bits", "row_stride_bytes", "pack", "unpack",
    "whiten", "lift", "gemm_workspace_bytes", "gemm_launches", "gemm", "gemm_noalloc",
    "new_workspace",
    "device_status", "check_wait_timeout", "NOALLOC_SCRATCH_BYTES",
    "i8_row_bytes", "quant_i8", "Norm", "norm_residual", "norm_residual_i8", "gemm_i8",
    "gemm_i8_route", "gemm_i8_plan", "new_i8_workspace",
    "default_i8_workspace", "GEMM_I8_WORKSPACE_BYTES",
]

NOALLOC_SCRATCH_BYTES = 8 << 20   # LQ_NOALLOC_SCRATCH_BYTES

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblq.so")

LQ_OK, LQ_EINVAL, LQ_EUNSUPPORTED, LQ_ECUDA, LQ_ETIMEOUT, LQ_EDEVICE = range(6)
LQ_F32, LQ_F16, LQ_BF16 = 0, 1, 2
_DTYPES = {torch.float32: LQ_F32, torch.float16: LQ_F16, torch.bfloat16: LQ_BF16}

EXPORTS = ("lq_abi_version", "lq_lifted_bits", "lq_row_stride_bytes", "lq_pack", "lq_unpack", "lq_encode",
           "lq_whiten", "lq_lift", "lq_gemm_workspace_bytes", "lq_gemm_launches", "lq_gemm_route",
           "lq_gemm", "lq_gemm_on_route", "lq_gemm_route_workspace_bytes", "lq_gemv_staged_plan",
           "lq_codebook_workspace_bytes", "lq_codebook_round",
           "lq_i8_row_bytes", "lq_quant_i8", "lq_norm_residual", "lq_gemm_i8_route", "lq_gemm_i8_plan",
           "lq_gemm_i8",
           "lq_gemm_noalloc", "lq_check_wait_timeout",
           "lq_device_status", "lq_status_string", "lq_last_error")


class LQError(RuntimeError):
    def __init__(self, status, where, message):
        self.status = status
        super().__init__(f"{where}: status {status}: {message}")


class WhitenDesc(ctypes.Structure):
    _fields_ = [("sign", ctypes.c_void_p), ("chan_scale", ctypes.c_void_p),
                ("block", ctypes.c_int32)]


class NormDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("dtype", ctypes.c_int32)]


class GateDesc(ctypes.Structure):
    _fields_ = [("gate", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("tokens", ctypes.c_int32)]


_LIB = None


def _declare(L):
    i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    dp = ctypes.POINTER(WhitenDesc)
    sig = {
        "lq_abi_version": ([], i32),
        "lq_lifted_bits": ([i32, i32, i32], i64),
        "lq_row_stride_bytes": ([i32, i32, i32], i64),
        "lq_pack": ([vp, i32, i32, i32, i32, vp, vp], ctypes.c_int),
        "lq_encode": ([vp, i32, i32, vp, i32, i32, i32, vp, vp, vp], ctypes.c_int),
        "lq_unpack": ([vp, i32, i32, i32, i32, vp, vp], ctypes.c_int),
        "lq_whiten": ([vp, ctypes.c_int, i32, i32, dp, vp, vp], ctypes.c_int),
        "lq_lift": ([vp, ctypes.c_int, i32, i32, dp, vp, i32, i32, vp, vp], ctypes.c_int),
        "lq_gemm_workspace_bytes": ([i32, i32, i32, i32, i32], sz),
        "lq_gemm_launches": ([i32, i32, i32, i32, i32, i32], i32),
        "lq_gemm_route": ([i32, i32, i32, i32, i32, i32], i32),
        "lq_gemm": ([vp, ctypes.c_int, i32, dp, vp, vp, vp, ctypes.c_int, i32, i32, i32, i32, vp,
                     vp, sz, vp], ctypes.c_int),
        "lq_gemm_on_route": ([vp, ctypes.c_int, i32, dp, vp, vp, vp, ctypes.c_int, i32, i32, i32,
                              i32, vp, vp, sz, i32, vp], ctypes.c_int),
        "lq_gemm_route_workspace_bytes": ([i32, i32, i32, i32, i32, i32, i32], sz),
        "lq_gemv_staged_plan": ([i32, i32, i32, i32, i32, i32, ctypes.POINTER(i64)], ctypes.c_int),
        "lq_codebook_workspace_bytes": ([ctypes.c_int64, i32, i32], sz),
        "lq_codebook_round": ([vp, ctypes.c_int64, vp, i32, i32, i32, vp, vp, vp, sz, vp],
                              ctypes.c_int),
        "lq_gemm_noalloc": ([vp, ctypes.c_int, i32, dp, vp, vp, vp, ctypes.c_int, i32, i32, i32,
                             i32, vp, vp], ctypes.c_int),
        "lq_i8_row_bytes": ([i32], i64),
        "lq_quant_i8": ([vp, ctypes.c_int, i32, i32, i64, dp, vp, vp, vp, vp], ctypes.c_int),
        "lq_norm_residual": ([vp, ctypes.c_int, i64, vp, ctypes.c_int, i64, i32, i32,
                              ctypes.POINTER(NormDesc), ctypes.POINTER(GateDesc), ctypes.c_float,
                              ctypes.c_float, vp, ctypes.POINTER(NormDesc), vp, ctypes.c_int, dp,
                              vp, vp, vp], ctypes.c_int),
        "lq_gemm_i8_route": ([i32, i32, i32], i32),
        "lq_gemm_i8_plan": ([i32, i32, i32, i32, ctypes.POINTER(i64)], ctypes.c_int),
        "lq_gemm_i8": ([vp, vp, i32, vp, vp, vp, i32, i32, vp, ctypes.c_int, vp, sz, i32, vp],
                       ctypes.c_int),
        "lq_device_status": ([vp, ctypes.POINTER(i32), vp], ctypes.c_int),
        "lq_check_wait_timeout": ([vp, i32, vp], ctypes.c_int),
        "lq_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "lq_last_error": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    return L


def lib():
    """The loaded liblq.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m fractional_bit_weight_b200.build` (nvcc, sm_100a)")
        _LIB = _declare(ctypes.CDLL(LIB_PATH))
    return _LIB


def _check(rc, where):
    if rc != LQ_OK:
        msg = lib().lq_last_error().decode() or lib().lq_status_string(rc).decode()
        raise LQError(rc, where, msg)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dev(t, name, dtypes=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    return ctypes.c_void_p(t.data_ptr())


def _opt(t, name, dtypes):
    return None if t is None else _dev(t, name, dtypes)


def _whiten_desc(sign, chan_scale, block):
    if not block:
        return None
    sg = _opt(sign, "sign", (torch.int8,))
    cs = _opt(chan_scale, "chan_scale", (torch.float32,))
    return WhitenDesc(sg.value if sg is not None else None,
                      cs.value if cs is not None else None, int(block))


def _desc_ptr(desc):
    return None if desc is None else ctypes.byref(desc)


def abi_version():
    return int(lib().lq_abi_version())


def lifted_bits(K, d, D):
    return int(lib().lq_lifted_bits(K, d, D))


def row_stride_bytes(K, d, D):
    return int(lib().lq_row_stride_bytes(K, d, D))


def pack(b_pm1, K, d, D, out=None, stream=None):
    """int8 sign codes [N][ceil(K/d)*D] -> LQ_FORMAT_V1 rows as int32 [N][row_stride/4]."""
    N = b_pm1.shape[0]
    if out is None:
        out = torch.empty((N, row_stride_bytes(K, d, D) // 4), dtype=torch.int32,
                          device=b_pm1.device)
    _check(lib().lq_pack(_dev(b_pm1, "b_pm1", (torch.int8,)), N, K, d, D,
                         _dev(out, "packed", (torch.int32,)), _stream(stream)), "lq_pack")
    return out


LQ_ENCODE_EXACT, LQ_ENCODE_SEEDED = 0, 1


def encode(w, M, d, D, mode=LQ_ENCODE_SEEDED, with_err=True, stream=None):
    """Nearest-codeword codes of w [N][K] fp32 (see lq_encode): returns (b_pm1 int8
    [N][ceil(K/d)][D], err fp32 [N][ceil(K/d)] or None). Pack b_pm1.view(N, -1) with pack()."""
    N, K = w.shape
    G = -(-K // d)
    b = torch.empty((N, G, D), dtype=torch.int8, device=w.device)
    err = torch.empty((N, G), dtype=torch.float32, device=w.device) if with_err else None
    _check(lib().lq_encode(_dev(w, "w", (torch.float32,)), N, K, _dev(M, "M", (torch.float32,)),
                           d, D, int(mode), _dev(b, "b_pm1", (torch.int8,)),
                           _dev(err, "err", (torch.float32,)) if with_err else None,
                           _stream(stream)), "lq_encode")
    return b, err


def unpack(packed, K, d, D, out=None, stream=None):
    N = packed.shape[0]
    if out is None:
        out = torch.empty((N, lifted_bits(K, d, D)), dtype=torch.int8, device=packed.device)
    _check(lib().lq_unpack(_dev(packed, "packed", (torch.int32,)), N, K, d, D,
                           _dev(out, "b_pm1", (torch.int8,)), _stream(stream)), "lq_unpack")
    return out


def whiten(x, sign=None, chan_scale=None, block=0, out=None, stream=None):
    batch, K = x.shape
    if out is None:
        out = torch.empty((batch, K), dtype=torch.float32, device=x.device)
    desc = _whiten_desc(sign, chan_scale, block)
    _check(lib().lq_whiten(_dev(x, "x", _DTYPES), _DTYPES[x.dtype], batch, K, _desc_ptr(desc),
                           _dev(out, "xt", (torch.float32,)), _stream(stream)), "lq_whiten")
    return out


def lift(x, M, d, D, sign=None, chan_scale=None, block=0, out=None, stream=None):
    batch, K = x.shape
    if out is None:
        out = torch.empty((batch, lifted_bits(K, d, D)), dtype=torch.float32, device=x.device)
    desc = _whiten_desc(sign, chan_scale, block)
    _check(lib().lq_lift(_dev(x, "x", _DTYPES), _DTYPES[x.dtype], batch, K, _desc_ptr(desc),
                         _dev(M, "M", (torch.float32,)), d, D, _dev(out, "z", (torch.float32,)),
                         _stream(stream)), "lq_lift")
    return out


def gemm_workspace_bytes(batch, K, N, d, D):
    return int(lib().lq_gemm_workspace_bytes(batch, K, N, d, D))


STAGED_PLAN_FIELDS = ("ok", "S", "sc", "R", "rq", "rrem", "rows_per_stage", "wch", "NS", "nchunk",
                      "smem", "prep_smem")


def gemv_staged_plan(batch, K, N, d, D, block=0):
    """The TMA-staged GEMV's plan for a shape (host-only query), as a dict."""
    out = (ctypes.c_int64 * len(STAGED_PLAN_FIELDS))()
    _check(lib().lq_gemv_staged_plan(batch, K, N, d, D, block, out), "lq_gemv_staged_plan")
    return dict(zip(STAGED_PLAN_FIELDS, (int(v) for v in out)))


def gemm_launches(batch, K, N, d, D, block=0):
    """Kernels one lq_gemm call launches for this shape (host-only query)."""
    return int(lib().lq_gemm_launches(batch, K, N, d, D, block))


# lq_gemm_route codes (include/liblq.h)
ROUTE_GEMV_I8, ROUTE_NONE, ROUTE_GEMM_TC, ROUTE_GEMV_GROUPS, ROUTE_GEMV_BULK, ROUTE_GEMM_DQ = \
    0, 1, 2, 3, 4, 5


def gemm_route(batch, K, N, d, D, block=0):
    """Which kernels lq_gemm runs for this shape (host-only query; ROUTE_* codes)."""
    return int(lib().lq_gemm_route(batch, K, N, d, D, block))


def new_workspace(batch, K, N, d, D, device="cuda", block=0, route=None):
    """A zero-filled workspace tensor for lq_gemm (uint8, 256-byte aligned by torch); with a
    route, for lq_gemm_on_route on that route and Hadamard block."""
    if route is None:
        n = gemm_workspace_bytes(batch, K, N, d, D)
    else:
        n = int(lib().lq_gemm_route_workspace_bytes(batch, K, N, d, D, block, int(route)))
    if n == 0:
        raise ValueError("invalid sizes for lq_gemm")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def gemm(x, packed, M, s, d, D, sign=None, chan_scale=None, block=0, y=None, workspace=None,
         stream=None, route=None):
    """y[t][n] = s[n] * (W[n] . T(x[t])), float32 [batch][N].

    route=None lets the library pick the kernels (lq_gemm); a ROUTE_* code runs that route
    (lq_gemm_on_route), which must fit the shape."""
    batch, K = x.shape
    N = packed.shape[0]
    if y is None:
        y = torch.empty((batch, N), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = new_workspace(batch, K, N, d, D, device=x.device, block=block, route=route)
    desc = _whiten_desc(sign, chan_scale, block)
    args = (_dev(x, "x", _DTYPES), _DTYPES[x.dtype], batch, _desc_ptr(desc),
            _dev(packed, "packed", (torch.int32,)), _dev(M, "M", (torch.float32,)),
            _dev(s, "s", _DTYPES), _DTYPES[s.dtype], d, D, K, N,
            _dev(y, "y", (torch.float32,)), _dev(workspace, "workspace"),
            workspace.numel() * workspace.element_size())
    if route is None:
        _check(lib().lq_gemm(*args, _stream(stream)), "lq_gemm")
    else:
        _check(lib().lq_gemm_on_route(*args, int(route), _stream(stream)), "lq_gemm_on_route")
    return y


def gemm_noalloc(x, packed, M, s, d, D, sign=None, chan_scale=None, block=0, y=None,
                 stream=None):
    """lq_gemm without a workspace: the library's own fixed device scratch is used (batch 1..8).

    For callers that cannot allocate device memory. The first call on a device sets it up and
    should come before any stream capture; calls that overlap on the GPU share the scratch and
    must be serialised by the caller.
    """
    batch, K = x.shape
    N = packed.shape[0]
    if y is None:
        y = torch.empty((batch, N), dtype=torch.float32, device=x.device)
    desc = _whiten_desc(sign, chan_scale, block)
    _check(lib().lq_gemm_noalloc(_dev(x, "x", _DTYPES), _DTYPES[x.dtype], batch, _desc_ptr(desc),
                                 _dev(packed, "packed", (torch.int32,)),
                                 _dev(M, "M", (torch.float32,)), _dev(s, "s", _DTYPES),
                                 _DTYPES[s.dtype], d, D, K, N, _dev(y, "y", (torch.float32,)),
                                 _stream(stream)), "lq_gemm_noalloc")
    return y


def codebook_round(w, M, d, D, mode=0, b=None, mse=None, workspace=None, stream=None):
    """One round of the codebook fit on samples w [S][d] (fp32, device): nearest codewords
    under M, then the least-squares M. M (fp32 [d][D], device) is updated in place. Returns
    (M, codes int8 [S][D], mse fp64 tensor of one element) on the device."""
    S = w.shape[0]
    if b is None:
        b = torch.empty((S, D), dtype=torch.int8, device=w.device)
    if mse is None:
        mse = torch.empty(1, dtype=torch.float64, device=w.device)
    if workspace is None:
        n = int(lib().lq_codebook_workspace_bytes(S, d, D))
        if n == 0:
            raise ValueError("invalid sizes for lq_codebook_round")
        workspace = torch.empty(n, dtype=torch.uint8, device=w.device)
    _check(lib().lq_codebook_round(_dev(w, "w", (torch.float32,)), S,
                                   _dev(M, "M", (torch.float32,)), d, D, int(mode),
                                   _dev(b, "b", (torch.int8,)), _dev(mse, "mse", (torch.float64,)),
                                   _dev(workspace, "workspace"),
                                   workspace.numel() * workspace.element_size(), _stream(stream)),
           "lq_codebook_round")
    return M, b, mse


# ---- 8-bit linear layers and the block boundaries around them (include/liblq.h)

GEMM_I8_WORKSPACE_BYTES = 256   # LQ_GEMM_I8_WORKSPACE_BYTES
I8_ROUTE_GEMV, I8_ROUTE_TC, I8_ROUTE_PAIR, I8_ROUTE_SPLIT = 0, 1, 2, 3
_F32 = (torch.float32,)
_BYTES = (4, 2, 2)              # of LQ_F32, LQ_F16, LQ_BF16
_I8 = (torch.int8,)
_NORM_KINDS = {"rms": 1, "layer": 2}


def _arg(t, name, dtypes, device, shape=None):
    """The address of a dense tensor argument, after its checks."""
    try:
        if (t.get_device() == device and t.dtype in dtypes and t.is_contiguous() and
                (shape is None or t.shape == shape)):
            return t.data_ptr()
    except AttributeError:
        pass
    _device_of(t, name)
    _complain(t, name, dtypes, device, shape)
    raise ValueError(f"{name} must be contiguous")


def _complain(t, name, dtypes, device, shape):
    """Raises what is wrong with a CUDA tensor apart from its strides."""
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, expected cuda:{device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _rows(t, name, dtypes, device, shape=None):
    """(address, row stride) of a 2-D argument whose rows are dense and may lie apart."""
    try:
        if (t.get_device() == device and t.dtype in dtypes and t.is_contiguous() and t.dim() == 2 and
                (shape is None or t.shape == shape)):
            return t.data_ptr(), t.shape[1]
    except AttributeError:
        pass
    _device_of(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, not {t.dim()}")
    _complain(t, name, dtypes, device, shape)
    rows, K = t.shape
    step, unit = t.stride()
    if (unit != 1 and K > 1) or (step < K and rows > 1):
        raise ValueError(f"{name} must have dense rows (strides {t.stride()})")
    return t.data_ptr(), step if rows > 1 else K


# of a build of torch with CUDA; without it no call gets as far (its tensors are not CUDA tensors),
# but the host-only queries work
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)    # of a device, as an address


def _over_there(call, device, stream, inputs):
    """call() with `device` and `stream` (None: that device's current one) current, so that the
    outputs it allocates belong to the stream that writes them. The inputs' memory is kept until
    the stream has passed the call."""
    if stream is None:
        with torch.cuda.device(device):
            return call()
    if stream.device.index != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{device}")
    with torch.cuda.stream(stream):
        out = call()
        for t in inputs:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    return out


def _device_of(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


_INT32_MAX = 2 ** 31 - 1


def _int32(n, name):
    """n, which ctypes would cut down to its low 32 bits without a word."""
    if not -_INT32_MAX <= n <= _INT32_MAX:
        raise ValueError(f"{name} = {n} exceeds 32 bits")
    return n


def _whiten_arg(sign, chan_scale, block, K, device):
    if not block:
        if sign is not None or chan_scale is not None:
            raise ValueError("sign and chan_scale are parts of T, which block = 0 leaves out "
                             "(block = 1 applies them without mixing)")
        return None
    return ctypes.byref(WhitenDesc(
        None if sign is None else _arg(sign, "sign", _I8, device, (K,)),
        None if chan_scale is None else _arg(chan_scale, "chan_scale", _F32, device, (K,)),
        _int32(int(block), "block")))


def i8_row_bytes(K):
    """Bytes per row of int8 codes: K rounded up to a multiple of 16."""
    return int(lib().lq_i8_row_bytes(_int32(K, "K")))


def quant_i8(x, sign=None, chan_scale=None, block=0, values=False, stream=None):
    """Symmetric int8 rows of T(x) with a scale per row (see lq_quant_i8).

    x [rows][K] f32/f16/bf16; its rows may lie apart. block = 0 leaves T out, 1 applies sign and
    chan_scale alone. Returns (q int8 [rows][i8_row_bytes(K)],
    scale fp32 [rows]); with values=True also scale * q in x's type, [rows][K]."""
    device = _device_of(x, "x")
    if stream is not None or device != _current_device():
        return _over_there(lambda: quant_i8(x, sign, chan_scale, block, values), device, stream,
                           (x, sign, chan_scale))
    px, ldx = _rows(x, "x", _DTYPES, device)
    rows, K = x.shape
    if rows > _INT32_MAX or K > _INT32_MAX:
        raise ValueError(f"x of shape {tuple(x.shape)} exceeds 32 bits")
    q = x.new_empty((rows, (K + 15) // 16 * 16), dtype=torch.int8)
    scale = x.new_empty(rows, dtype=torch.float32)
    v = torch.empty_like(x, memory_format=torch.contiguous_format) if values else None
    _check(lib().lq_quant_i8(px, _DTYPES[x.dtype], rows, K, ldx,
                             _whiten_arg(sign, chan_scale, block, K, device), q.data_ptr(),
                             scale.data_ptr(), v.data_ptr() if values else None,
                             _raw_stream(device)), "lq_quant_i8")
    return (q, scale, v) if values else (q, scale)


class Norm:
    """A norm of lq_norm_residual: kind "rms" or "layer", weight and bias [K] (f32/f16/bf16, of
    one type) or None, eps. Holds its tensors; make it once per layer. Each call takes the tensors
    as they are then: they may have been given new storage or another type, or been replaced."""

    def __init__(self, kind, weight=None, bias=None, eps=1e-6):
        self.kind, self.weight, self.bias, self.eps = kind, weight, bias, float(eps)
        self._look()

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        if name in ("kind", "weight", "bias", "eps"):
            super().__setattr__("_held", None)

    def _look(self):
        """Makes the descriptor from what the tensors are now, after its checks."""
        self._held = None
        if self.kind not in _NORM_KINDS:
            raise ValueError(f"unknown norm kind {self.kind!r}, expected one of "
                             f"{sorted(_NORM_KINDS)}")
        device = size = None
        dtype = torch.float32
        held, address = [], {}
        for t, name in ((self.weight, "weight"), (self.bias, "bias")):
            if t is None:
                continue
            if device is not None and t.dtype != dtype:
                raise TypeError("weight and bias of a norm must have one dtype")
            address[name] = _arg(t, name, _DTYPES, _device_of(t, name) if device is None else device,
                                 (t.numel(),) if size is None else (size,))
            device, size, dtype = t.get_device(), t.numel(), t.dtype
            held.append((t, address[name]))
        # a new descriptor: another thread's call may be reading the last one
        self._ref = ctypes.byref(NormDesc(_NORM_KINDS[self.kind], self.eps, address.get("weight"),
                                          address.get("bias"), _DTYPES[dtype]))
        self.device, self.size, self._dtype, self._held = device, size, dtype, held

    def _arg(self, K, device):
        held = self._held
        if held is None:
            self._look()
        else:       # a tensor whose `.data` was replaced is the same tensor over other memory
            for t, address in held:
                if (t.data_ptr() != address or t.dtype is not self._dtype or
                        t.numel() != self.size or not t.is_contiguous()):
                    self._look()
                    break
        if self.size is not None and (self.size != K or self.device != device):
            raise ValueError(f"norm over {self.size} entries on cuda:{self.device}, rows of {K} "
                             f"on cuda:{device}")
        return self._ref

    def _tensors(self):
        return self.weight, self.bias


def _norm_arg(norm, K, device):
    if norm is None:
        return None
    if not isinstance(norm, Norm):
        raise TypeError("post and pre are Norm objects or None")
    return norm._arg(K, device)


def _clash(out, other, rows):
    """Whether `rows` rows at out overlap those at other, each (address, step, width) in bytes, other
    than by being the same. Rows of different steps count as overlapping where their extents do."""
    if out == other:
        return False
    first, last = sorted((out, other))
    if first[0] + (rows - 1) * first[1] + first[2] <= last[0]:
        return False
    shift = (last[0] - first[0]) % first[1]
    return first[1] != last[1] or first[2] > shift or shift + last[2] > first[1]


def _boundary(h, residual, post, pre, gate, gate_tokens, branch_scale, residual_scale,
              residual_out, dtype, codes, whiten):
    """The arguments' checks, outputs and call of lq_norm_residual on the current stream."""
    device = h.get_device()
    ph, ldh = _rows(h, "h", _DTYPES, device)
    rows, K = shape = h.shape
    if rows > _INT32_MAX or K > _INT32_MAX:
        raise ValueError(f"h of shape {tuple(shape)} exceeds 32 bits")
    hdt = _DTYPES[h.dtype]
    pr, ldr, rdt = None, 0, 0
    r_out = p_out = None
    if residual is not None:
        pr, ldr = _rows(residual, "residual", _DTYPES, device, shape)
        rdt = _DTYPES[residual.dtype]
        if residual_out is None:
            r_out = torch.empty_like(residual, memory_format=torch.contiguous_format)
            p_out = r_out.data_ptr()
        elif residual_out is residual:
            r_out, p_out = residual, pr
        else:
            r_out = residual_out
            p_out = _arg(r_out, "residual_out", (residual.dtype,), device, shape)
    elif residual_out is not None:
        r_out = residual_out
        p_out = _arg(r_out, "residual_out", _DTYPES, device, shape)
        rdt = _DTYPES[r_out.dtype]
    if residual_out is not None and rows:
        # each row of h and the residual is read before its row of residual_out is written, but
        # other rows may be read later
        ro, rh = _BYTES[rdt], _BYTES[hdt]
        out = (p_out, (ldr if r_out is residual else K) * ro, K * ro)
        if r_out is not residual and residual is not None and \
                _clash(out, (pr, ldr * ro, K * ro), rows):
            raise ValueError("residual_out overlaps residual")
        if _clash(out, (ph, ldh * rh, K * rh), rows):
            raise ValueError("residual_out overlaps h")
    g = None
    if gate is not None:
        pg = _arg(gate, "gate", _DTYPES, device)
        cols = gate.shape[-1] if gate.dim() == 2 else gate.numel()
        count = gate.numel() // cols if cols else 0
        tokens = int(gate_tokens) or (1 if count == rows else max(rows, 1))
        # no tokens: no row of the gate is read, be there none or one for all
        if tokens < 1 or count != -(-rows // tokens) and (rows or count != 1):
            raise ValueError(f"gate of shape {tuple(gate.shape)} does not give {rows} tokens a "
                             f"row each {tokens}")
        g = ctypes.byref(GateDesc(pg, _DTYPES[gate.dtype], _int32(cols, "gate's columns"),
                                  min(tokens, max(rows, 1))))
    n = q = scale = None
    if codes:
        q = h.new_empty((rows, (K + 15) // 16 * 16), dtype=torch.int8)
        scale = h.new_empty(rows, dtype=torch.float32)
    if dtype is not None:
        if dtype not in _DTYPES:
            raise TypeError(f"dtype {dtype}, expected one of {tuple(_DTYPES)}")
        n = torch.empty_like(h, dtype=dtype, memory_format=torch.contiguous_format)
    _check(lib().lq_norm_residual(
        ph, hdt, ldh, pr, rdt, ldr, rows, K, _norm_arg(post, K, device), g,
        branch_scale, residual_scale, p_out, _norm_arg(pre, K, device),
        None if n is None else n.data_ptr(), 0 if n is None else _DTYPES[dtype],
        _whiten_arg(*whiten, K, device) if codes else None,
        None if q is None else q.data_ptr(), None if scale is None else scale.data_ptr(),
        _raw_stream(device)), "lq_norm_residual")
    return r_out, n, q, scale


def _boundary_inputs(h, residual, post, pre, gate, *more):
    return (h, residual, gate, *(post._tensors() if isinstance(post, Norm) else ()),
            *(pre._tensors() if isinstance(pre, Norm) else ()), *more)


def norm_residual(h, residual=None, post=None, pre=None, gate=None, gate_tokens=0,
                  branch_scale=1.0, residual_scale=1.0, residual_out=None, dtype=None,
                  stream=None):
    """The boundary between two blocks of a residual model (see lq_norm_residual):

        c = residual_scale * residual + branch_scale * gate . post(h),   n = pre(c)

    h, residual [rows][K] f32/f16/bf16, rows may lie apart; post, pre Norm or None; gate [K] or
    [ceil(rows / gate_tokens)][K or 1], a row per gate_tokens tokens (0: one row for all, or one
    per token if there are that many). Returns (c in residual's type, n in `dtype`, h's if None).
    residual_out=residual updates it in place; without a residual c is only written if
    residual_out is given (else None is returned for it). A residual_out that overlaps h or the
    residual in any other way is refused."""
    device = _device_of(h, "h")
    if stream is not None or device != _current_device():
        return _over_there(
            lambda: norm_residual(h, residual, post, pre, gate, gate_tokens, branch_scale,
                                  residual_scale, residual_out, dtype),
            device, stream, _boundary_inputs(h, residual, post, pre, gate, residual_out))
    r, n, _, _ = _boundary(h, residual, post, pre, gate, gate_tokens, branch_scale,
                           residual_scale, residual_out, h.dtype if dtype is None else dtype,
                           False, None)
    return r, n


def norm_residual_i8(h, residual=None, post=None, pre=None, gate=None, gate_tokens=0,
                     branch_scale=1.0, residual_scale=1.0, residual_out=None, sign=None,
                     chan_scale=None, block=0, dtype=None, stream=None):
    """norm_residual with n leaving as int8 rows of T(n) and their scales, as quant_i8 makes them,
    for gemm_i8. Returns (c, q, scale); with a dtype also n in that type."""
    device = _device_of(h, "h")
    if stream is not None or device != _current_device():
        return _over_there(
            lambda: norm_residual_i8(h, residual, post, pre, gate, gate_tokens, branch_scale,
                                     residual_scale, residual_out, sign, chan_scale, block,
                                     dtype),
            device, stream,
            _boundary_inputs(h, residual, post, pre, gate, residual_out, sign, chan_scale))
    r, n, q, scale = _boundary(h, residual, post, pre, gate, gate_tokens, branch_scale,
                               residual_scale, residual_out, dtype, True,
                               (sign, chan_scale, block))
    return (r, q, scale) if dtype is None else (r, q, scale, n)


def _sizes(batch, K, N):
    return _int32(batch, "batch"), _int32(K, "K"), _int32(N, "N")


def gemm_i8_route(batch, K, N):
    """Which kernel lq_gemm_i8 runs for this shape on the current device, without one on a B200
    with 148 SMs (launches nothing; I8_ROUTE_* codes)."""
    return int(lib().lq_gemm_i8_route(*_sizes(batch, K, N)))


I8_PLAN_FIELDS = ("route", "cluster", "tiles", "rows", "tokens", "chunks", "stages", "smem")


def gemm_i8_plan(batch, K, N, route=None):
    """The tiles of lq_gemm_i8's tensor-core routes for a shape (launches nothing), as a dict."""
    out = (ctypes.c_int64 * len(I8_PLAN_FIELDS))()
    _check(lib().lq_gemm_i8_plan(*_sizes(batch, K, N),
                                 -1 if route is None else _int32(route, "route"), out),
           "lq_gemm_i8_plan")
    return dict(zip(I8_PLAN_FIELDS, (int(v) for v in out)))


def new_i8_workspace(device="cuda"):
    """A zero-filled workspace tensor for lq_gemm_i8 (its status word; see device_status)."""
    return torch.zeros(GEMM_I8_WORKSPACE_BYTES, dtype=torch.uint8, device=device)


_I8_WORKSPACES = {}     # by device index, for the calls that are given none


def default_i8_workspace(device="cuda"):
    """The workspace of a device's gemm_i8 calls that are given none: device_status reads there
    whether one of them failed on the device. Made by the first such call that is not captured (or
    here); a call captured before that gets one of its own, whose status is lost."""
    device = torch.device(device)
    index = torch.cuda.current_device() if device.index is None else device.index
    workspace = _I8_WORKSPACES.get(index)
    return _new_default(index, device) if workspace is None else workspace


def _new_default(index, device):
    workspace = new_i8_workspace(device)
    if torch.cuda.is_current_stream_capturing():
        return workspace        # the graph's own memory
    torch.cuda.current_stream(device).synchronize()     # zero before another stream's call
    return _I8_WORKSPACES.setdefault(index, workspace)


def gemm_i8(xq, xs, wq, ws, K=None, bias=None, dtype=torch.float32, y=None, workspace=None,
            stream=None, route=None):
    """y[t][n] = (xq[t] . wq[n]) * (xs[t] * ws[n]) + bias[n], [batch][N] of `dtype`.

    xq [batch][i8_row_bytes(K)] and wq [N][i8_row_bytes(K)] int8, xs [batch], ws [N] and bias [N]
    fp32. K None: the whole stored rows (quant_i8 pads them with zeros). route=None lets the
    library pick the kernel; an I8_ROUTE_* code runs that one. workspace None: the device's
    default_i8_workspace()."""
    device = _device_of(xq, "xq")
    if stream is not None or device != _current_device():
        return _over_there(lambda: gemm_i8(xq, xs, wq, ws, K, bias, dtype, y, workspace, None,
                                           route),
                           device, stream, (xq, xs, wq, ws, bias, y, workspace))
    if xq.dim() != 2 or wq.dim() != 2:
        raise ValueError("xq and wq must have two dimensions")
    batch, row = xq.shape
    N = wq.shape[0]
    if K is None:
        K = row
    if (K + 15) // 16 * 16 != row:
        raise ValueError(f"rows of {row} bytes, {(K + 15) // 16 * 16} expected for K = {K}")
    if batch > _INT32_MAX or K > _INT32_MAX or N > _INT32_MAX:
        raise ValueError(f"batch = {batch}, K = {K} or N = {N} exceeds 32 bits")
    pxq = _arg(xq, "xq", _I8, device)
    pwq = _arg(wq, "wq", _I8, device, (N, row))
    pxs = _arg(xs, "xs", _F32, device, (batch,))
    pws = _arg(ws, "ws", _F32, device, (N,))
    pb = None if bias is None else _arg(bias, "bias", _F32, device, (N,))
    if y is None:
        if dtype not in _DTYPES:
            raise TypeError(f"dtype {dtype}, expected one of {tuple(_DTYPES)}")
        y = xq.new_empty((batch, N), dtype=dtype)
    else:
        _arg(y, "y", _DTYPES, device, (batch, N))
    if workspace is None:
        workspace = _I8_WORKSPACES.get(device)
        if workspace is None:
            workspace = _new_default(device, xq.device)
    pw = _arg(workspace, "workspace", (torch.uint8,), device)
    _check(lib().lq_gemm_i8(pxq, pxs, batch, pwq, pws, pb, K, N, y.data_ptr(), _DTYPES[y.dtype],
                            pw, workspace.numel(), -1 if route is None else _int32(route, "route"),
                            _raw_stream(device)), "lq_gemm_i8")
    return y


def check_wait_timeout(workspace, limit_ms=20, stream=None):
    """Runs the device-side timeout check (see lq_check_wait_timeout); read the result with
    device_status(workspace)."""
    _check(lib().lq_check_wait_timeout(_dev(workspace, "workspace"), int(limit_ms),
                                       _stream(stream)), "lq_check_wait_timeout")


def device_status(workspace, stream=None):
    code = ctypes.c_int32(0)
    rc = lib().lq_device_status(_dev(workspace, "workspace"), ctypes.byref(code), _stream(stream))
    return int(rc), int(code.value)
