"""Thin Python binding of libadmmq.so (C ABI in include/admmq.h).

Argument marshalling only: torch provides device memory and streams, every
step of the solve runs in the library's CUDA kernels (and cuSOLVER for the
one-time eigendecomposition).  A missing library raises; there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

from .build import LIB

OK = 0
GRID_MINMAX, GRID_LSQ, GRID_FROZEN, GRID_MSE = 0, 1, 2, 3
GRID_MODES = {"minmax": GRID_MINMAX, "lsq": GRID_LSQ, "frozen": GRID_FROZEN, "mse": GRID_MSE}
SPLIT_MODES = {"auto": 0, "3xtf32": 1, "mixed": 2, "f16": 3}
SCHEDULES = {"fused": 0, "per_gemm": 1}
DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2
DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
MX_FORMATS = {"mxfp4": 0, "nvfp4": 1}
MX_BLOCK = {"mxfp4": 32, "nvfp4": 16}
_ACT_DTYPES = (torch.bfloat16, torch.float16)
BUFFERS = ["sigma", "rsig", "hdiag", "lambda", "V", "C0", "P_hi", "P_lo", "T_hi", "T_lo",
           "E_hi", "E_lo", "Ht", "status", "row_in", "row_out"]
ERR_INVALID_ARG, ERR_TIMEOUT, ERR_RANGE = -1, -6, -9


class AdmmqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class _Params(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int), ("group", ctypes.c_int), ("iters", ctypes.c_int),
                ("rho0", ctypes.c_float), ("gamma", ctypes.c_float),
                ("lambda_rel", ctypes.c_float), ("grid_mode", ctypes.c_int),
                ("split_mode", ctypes.c_int), ("no_scaling", ctypes.c_int),
                ("schedule", ctypes.c_int), ("rescale_dual", ctypes.c_int),
                ("fit_on_w", ctypes.c_int)]


@dataclass
class Params:
    bits: int = 3
    group: int = 128
    iters: int = 100
    rho0: float = 0.1
    gamma: float = 1.05
    lambda_rel: float = 0.01
    grid: str = "lsq"
    split: str = "auto"   # eigenbasis GEMM split precision: auto | 3xtf32 | mixed | f16
    scaling: bool = True  # False: Sigma = I (the unscaled ablation)
    schedule: str = "fused"  # fused: one launch per iterate call | per_gemm: two per iteration
    rescale_dual: bool = False  # V~ *= rho_t / rho_{t+1} after each iteration (a study variant)
    fit_on_w: bool = False  # refresh the grid from Sigma W~ instead of Sigma (W~ + V~) (a study variant)

    def c(self) -> _Params:
        return _Params(self.bits, self.group, self.iters, self.rho0, self.gamma, self.lambda_rel,
                       GRID_MODES[self.grid], SPLIT_MODES[self.split], int(not self.scaling),
                       SCHEDULES[self.schedule], int(self.rescale_dual), int(self.fit_on_w))


_lib = None
_vp, _i, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t


def _preload_solver_runtime():
    """Use the cuSOLVER build that matches torch's cuBLAS when torch ships one,
    so one process never mixes two cuBLAS versions."""
    try:
        import nvidia.cusolver  # type: ignore
        for base in nvidia.cusolver.__path__:
            p = os.path.join(base, "lib", "libcusolver.so.11")
            if os.path.exists(p):
                ctypes.CDLL(p, mode=ctypes.RTLD_GLOBAL)
                return
    except Exception:
        pass


def lib():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB):
        raise RuntimeError(f"{LIB} is missing: build it with "
                           "`python -m post_weight_quantization_10_b200.build`")
    torch.cuda.init() if torch.cuda.is_available() else None
    _preload_solver_runtime()
    L = ctypes.CDLL(LIB)
    sig = {
        "admmq_status_string": (ctypes.c_char_p, [_i]),
        "admmq_version": (_i, []),
        "admmq_launch_count": (ctypes.c_int64, []),
        "admmq_gram_workspace_bytes": (_sz, [_i64, _i]),
        "admmq_build_hessian": (_i, [_vp, _i64, _i, _vp, _i, _vp, _sz, _vp]),
        "admmq_workspace_bytes": (_sz, [_i, _i, ctypes.POINTER(_Params)]),
        "admmq_create": (_i, [ctypes.POINTER(_vp), _i, _i, ctypes.POINTER(_Params), _vp, _sz]),
        "admmq_destroy": (None, [_vp]),
        "admmq_prepare": (_i, [_vp, _vp, _vp, _i, _vp]),
        "admmq_eigh": (_i, [_vp, _vp]),
        "admmq_setup": (_i, [ctypes.POINTER(_vp), _vp, _vp, _i, _i, _i, ctypes.POINTER(_Params),
                             _vp, _sz, _vp]),
        "admmq_init": (_i, [_vp, _vp, _vp, _vp, _vp]),
        "admmq_iterate": (_i, [_vp, _i, _i, _vp, _vp, _vp, _vp]),
        "admmq_finish": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp]),
        "admmq_solve": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp]),
        "admmq_pack": (_i, [_vp, _i, _i, _i, _vp, _vp]),
        "admmq_get_buffer": (_i, [_vp, _i, ctypes.POINTER(_vp), ctypes.POINTER(_sz)]),
        "admmq_debug_dump_wtilde": (_i, [_vp, _vp]),
        "admmq_set_timing": (_i, [_vp, _i]),
        "admmq_get_timing": (_i, [_vp, ctypes.POINTER(ctypes.c_double),
                                  ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]),
        "admmq_project": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp,
                               _vp, _vp, _vp, _vp, _vp, ctypes.c_float, _i, _vp]),
        "admmq_split_mode": (_i, [_vp]),
        "admmq_set_split": (_i, [_vp, _i, _vp]),
        "admmq_check": (_i, [_vp, _vp]),
        "admmq_debug_skew_ready": (_i, [_vp, _i]),
        "admmq_debug_rint_div": (_i, [_vp, _vp, _i64, _vp, _vp]),
        "admmq_gptq_workspace_bytes": (_sz, [_i, _i, _i]),
        "admmq_gptq": (_i, [_vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float, _i, _vp, _vp, _vp, _vp,
                            _sz, _vp]),
        "admmq_packed_matmul": (_i, [_vp, _i, _i64, _i64, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _i,
                                     _vp]),
        "admmq_operators_check": (_i, [_vp]),
        "admmq_debug_give_up": (_i, [_i, _vp]),
        "admmq_debug_packed_plan": (_i, [_i64, _i, _i, _i, _i, _i, _vp]),
        "admmq_mx_scale_bytes": (_sz, [_i64, _i, _i]),
        "admmq_mx_quantize": (_i, [_vp, _i, _i64, _i, _i64, _i, _vp, _vp, _vp, _vp]),
        "admmq_mx_dequantize": (_i, [_vp, _vp, _i64, _i, _i, _vp, _vp, _i, _i64, _vp]),
        "admmq_mx_linear_workspace_bytes": (_sz, [_i64, _i, _i, _i]),
        "admmq_mx_linear": (_i, [_vp, _i, _i64, _i64, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _i, _vp,
                                 _sz, _vp]),
        "admmq_mx_matmul": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i, _i, _i, _vp, _i, _vp]),
    }
    for name, (res, args) in sig.items():
        if name.startswith("admmq_debug_") and not hasattr(L, name):
            continue  # test hooks of another build; calling one raises
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def launch_count() -> int:
    """Kernels launched by libadmmq.so in this process."""
    return int(lib().admmq_launch_count())


def status_string(s: int) -> str:
    return lib().admmq_status_string(s).decode()


def _check(rc: int, where: str):
    if rc != OK:
        raise AdmmqError(rc, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# ------------------------------------------------------------------ Hessian


def gram_workspace_bytes(n: int, d_in: int) -> int:
    return int(lib().admmq_gram_workspace_bytes(n, d_in))


def build_hessian(X: torch.Tensor, H: torch.Tensor | None = None, accumulate: bool = False,
                  workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """H = X^T X (fp32, both triangles) from bf16 activations X [n][d_in]."""
    assert X.is_cuda and X.dtype == torch.bfloat16 and X.dim() == 2 and X.is_contiguous()
    n, d = X.shape
    if H is None:
        H = torch.empty((d, d), dtype=torch.float32, device=X.device)
    need = gram_workspace_bytes(n, d)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    _check(lib().admmq_build_hessian(_ptr(X), n, d, _ptr(H), int(accumulate), _ptr(workspace),
                                     workspace.numel(), _stream(stream)), "admmq_build_hessian")
    return H


# ------------------------------------------------------------------- solver


class Solver:
    """One layer solve: owns the workspace tensor and the C context."""

    def __init__(self, d_in: int, d_out: int, params: Params, device="cuda"):
        self.d_in, self.d_out, self.params = d_in, d_out, params
        self._cp = params.c()
        need = int(lib().admmq_workspace_bytes(d_in, d_out, ctypes.byref(self._cp)))
        if need == 0:
            raise AdmmqError(-1, "admmq_workspace_bytes")
        self.workspace = torch.empty(need, dtype=torch.uint8, device=device)
        self._ctx = ctypes.c_void_p()
        _check(lib().admmq_create(ctypes.byref(self._ctx), d_in, d_out, ctypes.byref(self._cp),
                                  _ptr(self.workspace), need), "admmq_create")
        self._W_hat = None
        ng = d_in // params.group
        self.codes = torch.empty((d_out, d_in), dtype=torch.uint8, device=device)
        self.scale = torch.empty((d_out, ng), dtype=torch.float32, device=device)
        self.zero = torch.empty((d_out, ng), dtype=torch.float32, device=device)
        self.resid = torch.zeros((max(params.iters, 1), 2), dtype=torch.float64, device=device)
        self.objective = torch.zeros(1, dtype=torch.float64, device=device)

    def close(self):
        if self._ctx:
            lib().admmq_destroy(self._ctx)
            self._ctx = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def prepare(self, G: torch.Tensor, W_hat: torch.Tensor, stream=None):
        assert G.dtype == torch.float32 and G.shape == (self.d_in, self.d_in) and G.is_contiguous()
        assert W_hat.shape == (self.d_out, self.d_in) and W_hat.is_contiguous()
        dt = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}[W_hat.dtype]
        self._W_hat = W_hat  # the library reads it again in finish()
        _check(lib().admmq_prepare(self._ctx, _ptr(G), _ptr(W_hat), dt, _stream(stream)),
               "admmq_prepare")

    def eigh(self, stream=None):
        _check(lib().admmq_eigh(self._ctx, _stream(stream)), "admmq_eigh")

    def init(self, stream=None):
        _check(lib().admmq_init(self._ctx, _ptr(self.codes), _ptr(self.scale), _ptr(self.zero),
                                _stream(stream)), "admmq_init")

    def iterate(self, t0: int, count: int, stream=None):
        _check(lib().admmq_iterate(self._ctx, t0, count, _ptr(self.codes), _ptr(self.scale),
                                   _ptr(self.zero), _stream(stream)), "admmq_iterate")

    def finish(self, resid=True, objective=True, stream=None):
        _check(lib().admmq_finish(self._ctx, _ptr(self.codes), _ptr(self.scale), _ptr(self.zero),
                                  _ptr(self.resid) if resid else None,
                                  _ptr(self.objective) if objective else None, _stream(stream)),
               "admmq_finish")

    def objective_of(self, codes, scale, zero, stream=None) -> float:
        """1/2 Tr((D - W_hat)^T H (D - W_hat)) of any codes on any grid of this
        layer (e.g. a GPTQ result), through the same eigenbasis GEMM."""
        out = torch.zeros(1, dtype=torch.float64, device=codes.device)
        _check(lib().admmq_finish(self._ctx, _ptr(codes), _ptr(scale), _ptr(zero), None,
                                  _ptr(out), _stream(stream)), "admmq_finish")
        return float(out.cpu())

    def solve(self, stream=None):
        _check(lib().admmq_solve(self._ctx, _ptr(self.codes), _ptr(self.scale), _ptr(self.zero),
                                 _ptr(self.resid), _ptr(self.objective), _stream(stream)),
               "admmq_solve")

    def kernel_status(self) -> int:
        """The kernels' status word (0 = ok, 1 = a bounded wait gave up);
        synchronises with the device."""
        return int(self.buffer("status")[0].item())

    def check(self, stream=None):
        """Synchronise and raise AdmmqError if a kernel's bounded wait gave up
        (ERR_TIMEOUT) or an fp16-split operand left fp16's range (ERR_RANGE)."""
        _check(lib().admmq_check(self._ctx, _stream(stream)), "admmq_check")

    def debug_skew_ready(self, iterations: int):
        """Failure-path test hook (see include/admmq.h)."""
        _check(lib().admmq_debug_skew_ready(self._ctx, iterations), "admmq_debug_skew_ready")

    def buffer(self, name: str) -> torch.Tensor:
        """A torch view of a workspace buffer (see include/admmq.h for layouts)."""
        which = BUFFERS.index(name)
        p, nb = ctypes.c_void_p(), ctypes.c_size_t()
        _check(lib().admmq_get_buffer(self._ctx, which, ctypes.byref(p), ctypes.byref(nb)),
               "admmq_get_buffer")
        off = p.value - self.workspace.data_ptr()
        raw = self.workspace[off:off + nb.value]
        d, m = self.d_in, self.d_out
        if name in ("sigma", "rsig", "hdiag", "lambda", "row_in", "row_out"):
            return raw.view(torch.float32)
        if name in ("V", "C0"):
            return raw.view(torch.float32).view(m, d)
        mixed = self.split == "mixed"
        if self.split == "f16" and name in ("P_hi", "P_lo", "T_hi", "T_lo"):   # fp16 bit patterns
            return raw[:2 * m * d].view(torch.int16).view(m, d)
        if self.split == "f16" and name in ("E_hi", "E_lo"):
            return raw[:2 * d * d].view(torch.int16).view(d, d)
        if name in ("P_hi", "T_hi") or (name in ("P_lo", "T_lo") and not mixed):
            return raw.view(torch.float32).view(m, d)
        if name in ("P_lo", "T_lo"):   # bf16 correction rows (bit patterns)
            return raw.view(torch.int16).view(m, 2 * d)
        if name == "E_hi" or (name == "E_lo" and not mixed):
            return raw.view(torch.float32).view(d, d)
        if name == "E_lo":
            return raw.view(torch.int16).view(d, 2 * d)
        if name == "Ht":
            return raw.view(torch.float64).view(d, d)
        return raw.view(torch.int32)

    @property
    def split(self) -> str:
        """The eigenbasis GEMMs' split precision: "3xtf32", "mixed" or "f16"."""
        mode = int(lib().admmq_split_mode(self._ctx))
        return {1: "3xtf32", 2: "mixed", 3: "f16"}[mode]

    def set_split(self, split: str, stream=None):
        """Switch to another split precision after eigh(); init() or solve()
        must come next (see admmq_set_split in include/admmq.h)."""
        _check(lib().admmq_set_split(self._ctx, SPLIT_MODES[split], _stream(stream)),
               "admmq_set_split")

    def dump_wtilde(self, out: torch.Tensor | None):
        _check(lib().admmq_debug_dump_wtilde(self._ctx, _ptr(out)), "admmq_debug_dump_wtilde")

    def set_timing(self, enable: bool):
        _check(lib().admmq_set_timing(self._ctx, int(enable)), "admmq_set_timing")

    def get_timing(self):
        """([ms GEMM 1, ms GEMM 2], [launches, launches], iterations timed); with
        the fused schedule index 0 is the fused launches and index 1 is zero."""
        ms = (ctypes.c_double * 2)()
        n = (ctypes.c_int * 2)()
        iters = ctypes.c_int(0)
        _check(lib().admmq_get_timing(self._ctx, ms, n, ctypes.byref(iters)), "admmq_get_timing")
        return [ms[0], ms[1]], [n[0], n[1]], iters.value


# --------------------------------------------------------------- pack etc.


def pack(codes: torch.Tensor, bits: int, out: torch.Tensor | None = None, stream=None):
    m, d = codes.shape
    if out is None:
        out = torch.empty((m, d * bits // 32), dtype=torch.int32, device=codes.device)
    _check(lib().admmq_pack(_ptr(codes), d, m, bits, _ptr(out), _stream(stream)), "admmq_pack")
    return out


def _invalid(what: str):
    raise AdmmqError(ERR_INVALID_ARG, what)


def _is_matrix(x: torch.Tensor, dtypes) -> bool:
    """A matrix on the GPU with unit column stride (rows may lie apart)."""
    return x.is_cuda and x.dim() == 2 and x.dtype in dtypes and (x.stride(1) == 1 or x.shape[1] == 1)


def _row_stride(x: torch.Tensor) -> int:
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


# The raw handle of a device's current stream: on the decode path a call's host
# time counts, and a Stream object costs more than the launch.
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else lambda i: torch.cuda.current_stream(i).cuda_stream


def _launch(name: str, device: torch.device, stream, *args):
    """Call entry point `name` with `device` current, on `stream` (None: the
    device's current stream)."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(name, device, stream, *args)
    _call(name, device, stream, *args)


def _call(name: str, device: torch.device, stream, *args):
    """_launch where `device` is current already."""
    rc = getattr(_lib or lib(), name)(
        *args, _raw_stream(device.index) if stream is None else stream.cuda_stream)
    if rc != OK:
        raise AdmmqError(rc, name)


def _empty(shape, dtype, device, stream):
    """A new contiguous tensor of one or two dimensions that belongs to the
    stream its kernel runs on.  (With strides given, torch takes half the time.)"""
    strides = (1,) if len(shape) == 1 else (max(shape[1], 1), 1)
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, strides, dtype=dtype, device=device)


def _output(out, shape, dtype, x: torch.Tensor, stream, where: str):
    """`out` after a check of its shape, type, device and layout, or a new tensor."""
    if out is None:
        return _empty(shape, dtype, x.device, stream)
    if not (out.shape == shape and out.dtype == dtype and out.device == x.device
            and out.is_contiguous()):
        _invalid(f"{where}: out")
    return out


def packed_matmul(x: torch.Tensor, packed: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor,
                  bits: int, dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """x [m][d_in] (bf16 or fp16) times the layer whose codes `pack` packed:
    sum over groups of scale * (code - zero) . x, [m][d_out] in `dtype`
    (x's by default).  The group size is d_in / scale.shape[1]."""
    if not _is_matrix(x, _ACT_DTYPES):
        _invalid("packed_matmul: x")
    m, d = x.shape
    device = x.device
    if not (packed.dim() == 2 and packed.dtype == torch.int32 and packed.is_contiguous()
            and packed.shape[1] * 32 == d * bits and packed.device == device):
        _invalid("packed_matmul: packed")
    n = packed.shape[0]
    if not (scale.dtype == torch.float32 and zero.dtype == torch.float32 and scale.dim() == 2
            and scale.shape == zero.shape and scale.shape[0] == n and scale.is_contiguous()
            and zero.is_contiguous() and scale.device == device and zero.device == device):
        _invalid("packed_matmul: scale and zero")
    groups = scale.shape[1]
    if groups < 1 or d % groups:
        _invalid("packed_matmul: groups")
    dtype = dtype or x.dtype
    if dtype not in DTYPES:
        _invalid("packed_matmul: dtype")
    out = _output(out, (m, n), dtype, x, stream, "packed_matmul")
    _launch("admmq_packed_matmul", device, stream, x.data_ptr(), DTYPES[x.dtype], m,
            _row_stride(x), packed.data_ptr(), scale.data_ptr(), zero.data_ptr(), d, n, bits,
            d // groups, out.data_ptr(), DTYPES[dtype])
    return out


def debug_packed_plan(m: int, d_in: int, d_out: int, bits: int, group: int, sms: int = 0) -> dict:
    """How packed_matmul lays out a call (test hook, see include/admmq.h)."""
    plan = (ctypes.c_int * 10)()
    _check(lib().admmq_debug_packed_plan(m, d_in, d_out, bits, group, sms, plan),
           "admmq_debug_packed_plan")
    return dict(zip(("tokens", "rows", "tiles", "at_once", "ranks", "range", "stage", "groups",
                     "staged", "vec_scales"), plan))


# ------------------------------------------- microscaled 4-bit floating point


@dataclass(frozen=True)
class MxTensor:
    """A matrix [rows][k] of 4-bit elements with a scale per block of a row
    (layouts in include/admmq.h): `codes` u8 [rows][k / 2], `scale` u8 in tiles
    of 128 rows x 4 blocks, `fmt` "mxfp4" or "nvfp4", `tensor_scale` fp32 [1]
    on the device (nvfp4; None means 1)."""
    codes: torch.Tensor
    scale: torch.Tensor
    fmt: str = "mxfp4"
    tensor_scale: torch.Tensor | None = None

    def __post_init__(self):
        c, s = self.codes, self.scale
        if self.fmt not in MX_FORMATS:
            _invalid("MxTensor: fmt")
        if not (c.is_cuda and c.dtype == torch.uint8 and c.dim() == 2 and c.is_contiguous()
                and c.shape[1] > 0 and c.shape[1] % 16 == 0):
            _invalid("MxTensor: codes")
        if not (s.dtype == torch.uint8 and s.device == c.device and s.is_contiguous()
                and s.numel() == _mx_scale_numel(c.shape[0], 2 * c.shape[1], self.fmt)):
            _invalid("MxTensor: scale")
        _check_tensor_scale(self.tensor_scale, self.fmt, c.device, "MxTensor")

    @classmethod
    def _of(cls, codes, scale, fmt, tensor_scale):
        """One that the library made itself."""
        q = cls.__new__(cls)
        q.__dict__.update(codes=codes, scale=scale, fmt=fmt, tensor_scale=tensor_scale)
        return q

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def k(self) -> int:
        return 2 * self.codes.shape[1]

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def _ptrs(self):
        g = self.tensor_scale
        return self.codes.data_ptr(), self.scale.data_ptr(), None if g is None else g.data_ptr()


def _mx_scale_numel(rows: int, k: int, fmt: str) -> int:
    return -(-rows // 128) * -(-k // (4 * MX_BLOCK[fmt])) * 512


def _check_tensor_scale(g, fmt: str, device, where: str):
    if g is not None and not (fmt == "nvfp4" and g.dtype == torch.float32 and g.numel() == 1
                              and g.device == device):
        _invalid(f"{where}: tensor_scale")


def _check_mx_input(x: torch.Tensor, fmt: str, tensor_scale, where: str):
    if not _is_matrix(x, DTYPES):
        _invalid(f"{where}: x")
    if fmt not in MX_FORMATS:
        _invalid(f"{where}: fmt")
    _check_tensor_scale(tensor_scale, fmt, x.device, where)
    if x.shape[1] == 0 or x.shape[1] % 32:
        _invalid(f"{where}: k is a positive multiple of 32")


def _ptr_or_null(t):
    return None if t is None else t.data_ptr()


def mx_quantize(x: torch.Tensor, fmt: str = "mxfp4", tensor_scale: torch.Tensor | None = None,
                stream=None) -> MxTensor:
    """Round x [rows][k] (fp32, bf16 or fp16; k a multiple of 32) to a
    microscaled 4-bit format: "mxfp4" (blocks of 32, power-of-two scales) or
    "nvfp4" (blocks of 16, e4m3 scales on top of `tensor_scale`, usually
    amax(x) / (448 * 6), fp32 [1] on the device)."""
    _check_mx_input(x, fmt, tensor_scale, "mx_quantize")
    rows, k = x.shape
    device = x.device
    codes = _empty((rows, k // 2), torch.uint8, device, stream)
    scale = _empty((_mx_scale_numel(rows, k, fmt),), torch.uint8, device, stream)
    _launch("admmq_mx_quantize", device, stream, x.data_ptr(), DTYPES[x.dtype], rows, k,
            _row_stride(x), MX_FORMATS[fmt], _ptr_or_null(tensor_scale), codes.data_ptr(),
            scale.data_ptr())
    return MxTensor._of(codes, scale, fmt, tensor_scale)


def mx_dequantize(q: MxTensor, dtype: torch.dtype = torch.bfloat16,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of q, [rows][k] in `dtype` (fp32, bf16 or fp16)."""
    if dtype not in DTYPES:
        _invalid("mx_dequantize: dtype")
    codes = q.codes
    rows, half = codes.shape
    out = _output(out, (rows, 2 * half), dtype, codes, stream, "mx_dequantize")
    _launch("admmq_mx_dequantize", codes.device, stream, codes.data_ptr(), q.scale.data_ptr(), rows,
            2 * half, MX_FORMATS[q.fmt], _ptr_or_null(q.tensor_scale), out.data_ptr(),
            DTYPES[dtype], 2 * half)
    return out


def _check_mx_weights(w: MxTensor, fmt: str, k: int, device, dtype, where: str):
    if not (w.fmt == fmt and w.k == k and w.device == device):
        _invalid(f"{where}: operands differ in format, k or device")
    if w.rows == 0 or dtype not in DTYPES:
        _invalid(f"{where}: no weights, or dtype")


def mx_matmul(a: MxTensor, b: MxTensor, dtype: torch.dtype = torch.bfloat16,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """a [m][k] times b [n][k] transposed (activations and nn.Linear weights,
    both in one microscaled format), [m][n] in `dtype` (fp32, bf16 or fp16)."""
    _check_mx_weights(b, a.fmt, a.k, a.device, dtype, "mx_matmul")
    out = _output(out, (a.rows, b.rows), dtype, a.codes, stream, "mx_matmul")
    _launch("admmq_mx_matmul", a.device, stream, *a._ptrs(), *b._ptrs(), a.rows, b.rows, a.k,
            MX_FORMATS[a.fmt], out.data_ptr(), DTYPES[dtype])
    return out


def mx_linear(x: torch.Tensor, w: MxTensor, dtype: torch.dtype | None = None,
              tensor_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """mx_matmul(mx_quantize(x, w.fmt, tensor_scale), w): a linear layer with
    4-bit weights whose activations are quantised on the way in."""
    fmt = w.fmt
    _check_mx_input(x, fmt, tensor_scale, "mx_linear")
    m, k = x.shape
    device = x.device
    if device.index != torch.cuda.current_device():  # the workspace's size depends on the device
        with torch.cuda.device(device):
            return mx_linear(x, w, dtype, tensor_scale, out, stream)
    dtype = dtype or x.dtype
    _check_mx_weights(w, fmt, k, device, dtype, "mx_linear")
    n = w.codes.shape[0]
    out = _output(out, (m, n), dtype, x, stream, "mx_linear")
    f = MX_FORMATS[fmt]
    need = (_lib or lib()).admmq_mx_linear_workspace_bytes(m, n, k, f)
    ws = _empty((need,), torch.uint8, device, stream) if need else None
    _call("admmq_mx_linear", device, stream, x.data_ptr(), DTYPES[x.dtype], m, _row_stride(x),
          _ptr_or_null(tensor_scale), *w._ptrs(), n, k, f, out.data_ptr(), DTYPES[dtype],
          _ptr_or_null(ws), need)
    return out


def operators_check(device=None, stream=None):
    """Wait for the stream and raise AdmmqError (ERR_TIMEOUT) if a kernel of the
    packed or mx operators gave up a bounded wait on `device` since the last
    check: the outputs that it could not compute are NaN."""
    index = None if device is None else torch.device(device).index
    if index is None:
        index = torch.cuda.current_device()
    _launch("admmq_operators_check", torch.device("cuda", index), stream)


def debug_give_up(unit: int, stream=None):
    """Failure-path test hook (see include/admmq.h)."""
    _check(lib().admmq_debug_give_up(unit, _stream(stream)), "admmq_debug_give_up")


def project(wtilde, V, sigma, rsig, hdiag, bits, group, grid, codes, scale, zero, P_hi, P_lo,
            resid=None, split="mixed", row_scale=None, range_flag=None, dual_scale=1.0,
            fit_on_w=False, stream=None):
    """Stand-alone projection; P planes in the encoding of `split`: "3xtf32"
    fp32 [m][d] x2, "mixed" fp32 [m][d] + int16 (bf16 bit patterns) [m][2d],
    "f16" int16 (fp16 bit patterns) [m][d] x2 with the rows' scales
    `row_scale` (fp32 [m]; None = 1) and an optional int32 range flag;
    `dual_scale` multiplies the new V~ (the dual rescaling); `fit_on_w`
    refreshes the grid from sigma W~ alone."""
    m, d = wtilde.shape
    if resid is None:
        resid = torch.zeros(2, dtype=torch.float64, device=wtilde.device)
    _check(lib().admmq_project(_ptr(wtilde), _ptr(V), _ptr(sigma), _ptr(rsig), _ptr(hdiag), d, m,
                               bits, group, GRID_MODES[grid], SPLIT_MODES[split], _ptr(codes),
                               _ptr(scale), _ptr(zero), _ptr(P_hi), _ptr(P_lo), _ptr(row_scale),
                               _ptr(range_flag), _ptr(resid), ctypes.c_float(dual_scale),
                               int(fit_on_w), _stream(stream)),
           "admmq_project")
    return resid


def debug_rint_div(y: torch.Tensor, s: torch.Tensor, stream=None) -> torch.Tensor:
    """rint(y / s[i // 8]) as the projection computes it (tests)."""
    out = torch.empty_like(y)
    _check(lib().admmq_debug_rint_div(_ptr(y), _ptr(s), y.numel(), _ptr(out), _stream(stream)),
           "admmq_debug_rint_div")
    return out


def gptq(G: torch.Tensor, W_hat: torch.Tensor, bits: int, group: int, lambda_rel: float = 0.01,
         block: int = 128, stream=None):
    """GPTQ on the fixed min/max grid of W_hat: returns (codes, scale, zero)."""
    m, d = W_hat.shape
    assert G.dtype == torch.float32 and G.shape == (d, d) and G.is_contiguous()
    assert W_hat.is_contiguous()
    dt = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}[W_hat.dtype]
    need = int(lib().admmq_gptq_workspace_bytes(d, m, block))
    if need == 0:
        raise AdmmqError(-1, "admmq_gptq_workspace_bytes")
    ws = torch.empty(need, dtype=torch.uint8, device=W_hat.device)
    codes = torch.empty((m, d), dtype=torch.uint8, device=W_hat.device)
    scale = torch.empty((m, d // group), dtype=torch.float32, device=W_hat.device)
    zero = torch.empty_like(scale)
    _check(lib().admmq_gptq(_ptr(G), _ptr(W_hat), dt, d, m, bits, group, lambda_rel, block,
                            _ptr(codes), _ptr(scale), _ptr(zero), _ptr(ws), need, _stream(stream)),
           "admmq_gptq")
    return codes, scale, zero


def solve_layer(X: torch.Tensor, W_hat: torch.Tensor, params: Params, stream=None) -> Solver:
    """Gram -> setup -> solve for one layer; the Solver holds codes/scale/zero,
    the residual history and the objective.  Synchronises once at the end to
    read the status words: when the fp16 split's range word is set, the layer
    is solved again with the mixed split (admmq_set_split); any other error
    raises AdmmqError."""
    H = build_hessian(X, stream=stream)
    s = Solver(X.shape[1], W_hat.shape[0], params, device=X.device)
    s.prepare(H, W_hat, stream)
    s.eigh(stream)
    s.solve(stream)
    try:
        s.check(stream)
    except AdmmqError as e:
        if e.status != ERR_RANGE:
            raise
        s.set_split("mixed", stream)
        s.solve(stream)
        s.check(stream)
    return s
