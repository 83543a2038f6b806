"""Thin Python binding over libck.so (include/ck.h): argument marshalling only.

Each function takes CUDA torch tensors, passes their device pointers, sizes and
strides to the C entry point of the same name, and raises CkError on a non-OK
status.  Every step of the computation runs in the library's CUDA kernels; there is
no CPU path.  Loading fails loudly if libck.so has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import os
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libck.so")

CK_OK, CK_ERR_INVALID_ARG, CK_ERR_UNSUPPORTED, CK_ERR_OVERFLOW = 0, 1, 2, 3
CK_ERR_WORKSPACE, CK_ERR_CUDA, CK_ERR_TIMEOUT = 4, 5, 6
CK_F32, CK_F16, CK_BF16, CK_I8, CK_FP4 = 0, 1, 2, 3, 4
CK_MXFP4, CK_NVFP4 = 0, 1
FP4_BLOCK = {CK_MXFP4: 32, CK_NVFP4: 16}

DTYPE_CODE = {torch.float32: CK_F32, torch.float16: CK_F16, torch.bfloat16: CK_BF16,
              torch.int8: CK_I8}
CODE_DTYPE = {v: k for k, v in DTYPE_CODE.items()}

# every entry point include/ck.h declares, with its ctypes signature
_P, _I64, _I, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
SIGNATURES = {
    "ck_rotate_quant": ([_P, _I, _I64, _I64, _I64, _I64, _P, _I, _P, _P, _I64, _P, _P, _P], _I),
    "ck_w4a4_linear": ([_P, _I, _I64, _I64, _I64, _I64, _P, _I, _P, _P, _I64, _I64, _P, _I, _P,
                        _P, _I, _I64, _P, _SZ, _P, _P], _I),
    "ck_w4a4_linear_workspace_bytes": ([_I64, _I64, _I64, _I64], _SZ),
    "ck_workspace_codes_pitch": ([_I64], _I64),
    "ck_workspace_scales_offset": ([_I64, _I64], _SZ),
    "ck_w4a4_linear_noalloc": ([_P, _I, _I64, _I64, _I64, _I64, _P, _I, _P, _P, _I64, _I64, _P,
                                _I, _P, _P, _I, _I64, _P, _P], _I),
    "ck_w4a4_grouped_linear": ([_P, _I, _I64, _I64, _I64, _I64, _P, _I, _P, _P, _I64, _P, _I, _P,
                                _I, _P, _P, _P, _I, _P, _SZ, _P, _P], _I),
    "ck_unpack_w4": ([_P, _I64, _I64, _I64, _P, _I64, _P], _I),
    "ck_rotate_quant_int8": ([_P, _I, _I64, _I64, _I64, _I64, _P, _I, _P, _P, _I64, _P, _P, _P],
                             _I),
    "ck_w8a8_linear": ([_P, _I, _I64, _I64, _I64, _I64, _P, _I, _P, _P, _I64, _I64, _P, _I, _P,
                        _P, _I, _I64, _P, _SZ, _P, _P], _I),
    "ck_w8a8_linear_workspace_bytes": ([_I64, _I64, _I64, _I64], _SZ),
    "ck_rotate_quant_packed": ([_P, _I, _I64, _I64, _I64, _I64, _P, _I, _P, _I, ctypes.c_uint64,
                                ctypes.c_uint64, _P, _I64, _P, _P], _I),
    "ck_fp4_scales_bytes": ([_I64, _I64, _I, _I], _SZ),
    "ck_fp4_linear_workspace_bytes": ([_I64, _I64, _I, _I], _SZ),
    "ck_quant_fp4": ([_P, _I, _I64, _I64, _I64, _I64, _I, _P, _P, _I, _P, _I64, _P, _P], _I),
    "ck_dequant_fp4": ([_P, _I64, _P, _I64, _I64, _I, _P, _P, _I, _P, _I, _I64, _P], _I),
    "ck_fp4_linear": ([_P, _I, _I64, _I64, _I64, _I64, _I, _P, _P, _P, _I64, _I64, _P, _P, _P, _I,
                       _P, _I, _I64, _P, _SZ, _P, _P], _I),
    "ck_fp4_expert_linear": ([_P, _I, _I64, _I64, _I64, _I64, _I, _P, _P, _P, _I, _P, _I64, _I64,
                              _I64, _P, _P, _P, _I, _P, _I, _I64, _P, _SZ, _P, _P], _I),
    "ck_status_string": ([_I], ctypes.c_char_p),
}


class CkError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_lib = None
_bind = None      # the native host side of the fp4 calls, once libck.so is loaded


def load_library(path: str) -> ctypes.CDLL:
    """Load a build of the library at `path` with every entry point's ctypes signature set."""
    if not os.path.exists(path):
        raise ImportError(f"{os.path.basename(path)} not found at {path}; run "
                          "`python -m rotated_w4a4_quantized_group_b200.build`")
    L = ctypes.CDLL(path)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    return L


def lib() -> ctypes.CDLL:
    """Load libck.so (raises if it is missing: build it with the package's build module)."""
    global _lib, _bind
    if _lib is None:
        _lib = load_library(LIB_PATH)
        try:
            from . import _ck_bind
        except ImportError:     # not built: the fp4 calls take Python's way, with the same results
            pass
        else:
            built_for = getattr(_ck_bind, "torch_version", None)
            if built_for == str(torch.__version__):
                _ck_bind.load(LIB_PATH)
                _bind = _ck_bind
            else:               # its view of a tensor may be another's
                warnings.warn(f"_ck_bind was built against torch {built_for}, this is "
                              f"{torch.__version__}: the fp4 calls do without it until the package is built again")
    return _lib


def status_string(status: int) -> str:
    return lib().ck_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != CK_OK:
        raise CkError(status, where)


def _stream(stream) -> int | None:
    """The caller's stream, or torch's current stream of the current device (every entry
    point makes its tensors' device current before asking)."""
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t) -> int | None:
    """Device address of a tensor argument (None stays NULL, an int is taken as an address).
    A tensor outside GPU memory is refused here: the library would hand its host address to
    the device."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError(f"ck: tensor arguments must live on a CUDA device, got one on {t.device}")
    return t.data_ptr()


def workspace_bytes(M: int, N: int, K: int, w_ld: int) -> int:
    return int(lib().ck_w4a4_linear_workspace_bytes(M, N, K, w_ld))


def workspace_codes_pitch(K: int) -> int:
    return int(lib().ck_workspace_codes_pitch(K))


def workspace_scales_offset(M: int, K: int) -> int:
    return int(lib().ck_workspace_scales_offset(M, K))


def _check_rotation(x: torch.Tensor, R: torch.Tensor, g: int):
    # the C ABI reads R as g*g row-major elements of x's dtype
    if tuple(R.shape) != (g, g) or R.dtype != x.dtype or not R.is_contiguous():
        raise ValueError(f"R must be a contiguous ({g}, {g}) tensor of {x.dtype}; got "
                         f"{tuple(R.shape)} {R.dtype} strides {R.stride()}")


def ck_rotate_quant(x: torch.Tensor, R: torch.Tensor, g: int, scale_in: torch.Tensor | None = None,
                    codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                    dev_status: torch.Tensor | None = None, stream=None):
    """Stage 1 on a 2-D (M, K) CUDA view; returns (codes int8 (M, K), scales fp32 (M,))."""
    M, K = x.shape
    _check_rotation(x, R, g)
    _same_device(x, R, scale_in, codes, scales, dev_status)
    if codes is None:
        codes = torch.empty(M, K, dtype=torch.int8, device=x.device)
    if scales is None:
        scales = torch.empty(M, dtype=torch.float32, device=x.device)
    if codes.dtype != torch.int8 or tuple(codes.shape) != (M, K) or codes.stride(1) != 1:
        raise ValueError(f"codes must be an int8 ({M}, {K}) view with unit inner stride")
    if scales.dtype != torch.float32 or scales.numel() < M or not scales.is_contiguous():
        raise ValueError(f"scales must be a contiguous fp32 tensor of at least {M} values")
    with torch.cuda.device(x.device):
        st = lib().ck_rotate_quant(_ptr(x), DTYPE_CODE[x.dtype], M, K, x.stride(0), x.stride(1),
                                   _ptr(R), g, _ptr(scale_in), _ptr(codes), codes.stride(0),
                                   _ptr(scales), _ptr(dev_status), _stream(stream))
    _check(st, "ck_rotate_quant")
    return codes, scales


def _check_weights(w_packed: torch.Tensor, N: int, K: int):
    # the library reads N rows of K/2 bytes through the row pitch w_packed.stride(0)
    if w_packed.dtype != torch.int8 or w_packed.dim() != 2 or w_packed.stride(1) != 1 or \
            tuple(w_packed.shape) != (N, K // 2):
        raise ValueError(f"w_packed must be an int8 (N, K/2) = ({N}, {K // 2}) view with unit inner "
                         f"stride; got {tuple(w_packed.shape)} {w_packed.dtype} strides "
                         f"{w_packed.stride()}")


def _check_out(out: torch.Tensor, M: int, N: int, x: torch.Tensor):
    # the library writes M rows of N values through the row pitch out.stride(0)
    if tuple(out.shape) != (M, N) or out.stride(1) != 1 or out.device != x.device:
        raise ValueError(f"out must be an (M, N) = ({M}, {N}) view with unit inner stride on "
                         f"{x.device}; got {tuple(out.shape)} strides {out.stride()} on {out.device}")


def _same_device(x: torch.Tensor, *ts):
    """Every tensor argument on x's CUDA device (a host tensor's address would be read by the
    device; a tensor on another GPU would be read through the wrong device's memory)."""
    _ptr(x)
    for t in ts:
        if t is not None and not isinstance(t, int) and t.device != x.device:
            raise ValueError(f"every tensor must be on {x.device}; got one on {t.device}")


def ck_w4a4_linear(x: torch.Tensor, R: torch.Tensor | None, g: int, w_packed: torch.Tensor,
                   w_scale: torch.Tensor, bias: torch.Tensor | None = None, *,
                   a_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   out_dtype: torch.dtype | None = None, workspace: torch.Tensor | None = None,
                   dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The whole W4A4 linear.  x is (M, K) activations (fp32/fp16/bf16) or int8 codes (with
    a_scale); w_packed is (N, K/2) int8.  Returns out (M, N)."""
    M, K = x.shape
    N = w_packed.shape[0]
    if x.dtype != torch.int8:
        _check_rotation(x, R, g)
    _check_weights(w_packed, N, K)
    _same_device(x, R, w_packed, w_scale, bias, a_scale, workspace, dev_status)
    if out is None:
        odt = out_dtype or (x.dtype if x.dtype != torch.int8 else w_scale.dtype)
        out = torch.empty(M, N, dtype=odt, device=x.device)
    _check_out(out, M, N, x)
    with torch.cuda.device(x.device):
        if workspace is None:
            nbytes = workspace_bytes(M, N, K, w_packed.stride(0))
            workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
        st = lib().ck_w4a4_linear(
            _ptr(x), DTYPE_CODE[x.dtype], M, K, x.stride(0), x.stride(1), _ptr(R), int(g),
            _ptr(a_scale), _ptr(w_packed), N, w_packed.stride(0), _ptr(w_scale),
            DTYPE_CODE[w_scale.dtype], _ptr(bias), _ptr(out), DTYPE_CODE[out.dtype],
            out.stride(0), _ptr(workspace), workspace.numel(), _ptr(dev_status), _stream(stream))
    _check(st, "ck_w4a4_linear")
    return out


def ck_w4a4_linear_noalloc(x: torch.Tensor, R: torch.Tensor | None, g: int,
                           w_packed: torch.Tensor, w_scale: torch.Tensor,
                           bias: torch.Tensor | None = None, *, out: torch.Tensor,
                           a_scale: torch.Tensor | None = None,
                           dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """ck_w4a4_linear with the library's built-in 32 MiB scratch instead of a workspace, for
    callers that cannot allocate device memory; `out` must be given (nothing is allocated)."""
    M, K = x.shape
    N = w_packed.shape[0]
    if x.dtype != torch.int8:
        _check_rotation(x, R, g)
    _check_weights(w_packed, N, K)
    _same_device(x, R, w_packed, w_scale, bias, a_scale, dev_status)
    _check_out(out, M, N, x)
    with torch.cuda.device(x.device):
        st = lib().ck_w4a4_linear_noalloc(
            _ptr(x), DTYPE_CODE[x.dtype], M, K, x.stride(0), x.stride(1), _ptr(R), int(g),
            _ptr(a_scale), _ptr(w_packed), N, w_packed.stride(0), _ptr(w_scale),
            DTYPE_CODE[w_scale.dtype], _ptr(bias), _ptr(out), DTYPE_CODE[out.dtype],
            out.stride(0), _ptr(dev_status), _stream(stream))
    _check(st, "ck_w4a4_linear_noalloc")
    return out


def fuse_linear_weights(parts):
    """Stack the packed weights, weight scales and biases of several linears that share one
    input along N (one-time weight preparation, done on the device by torch): parts is a list
    of (w_packed (N_i, K/2) int8, w_scale (N_i,), bias (N_i,) or None).  Returns
    (w_packed (N, K/2), w_scale (N,), bias (N,) or None, [N_i]); biases that are None become
    zeros when another part has one."""
    if not parts:
        raise ValueError("fuse_linear_weights needs at least one linear")
    ws = torch.cat([p[0] for p in parts], 0).contiguous()
    sc = torch.cat([p[1] for p in parts], 0).contiguous()
    if all(p[2] is None for p in parts):
        bias = None
    else:
        bias = torch.cat([p[2] if p[2] is not None else torch.zeros_like(p[1]) for p in parts],
                         0).contiguous()
    return ws, sc, bias, [int(p[0].shape[0]) for p in parts]


def ck_w4a4_grouped_linear(x: torch.Tensor, R: torch.Tensor | None, g: int,
                           w_packed: torch.Tensor, w_scale: torch.Tensor,
                           bias: torch.Tensor | None, group_n, *, outs=None,
                           a_scale: torch.Tensor | None = None,
                           out_dtype: torch.dtype | None = None,
                           workspace: torch.Tensor | None = None,
                           dev_status: torch.Tensor | None = None, stream=None):
    """Several linears sharing x as one call: w_packed/w_scale/bias are the groups' weights
    stacked along N (fuse_linear_weights), group_n the channels of each group.  Returns the
    list of per-group outputs (M, N_i)."""
    M, K = x.shape
    N = int(sum(group_n))
    if x.dtype != torch.int8:
        _check_rotation(x, R, g)
    _check_weights(w_packed, N, K)
    _same_device(x, R, w_packed, w_scale, bias, a_scale, workspace, dev_status)
    odt = out_dtype or (x.dtype if x.dtype != torch.int8 else w_scale.dtype)
    if outs is None:
        outs = [torch.empty(M, int(n), dtype=odt, device=x.device) for n in group_n]
    if len(outs) != len(group_n):
        raise ValueError("one output per group")
    for o, n in zip(outs, group_n):
        _check_out(o, M, int(n), x)
        if o.dtype != outs[0].dtype:
            raise ValueError("every group's output has the same dtype")
    G = len(group_n)
    gn = (ctypes.c_int64 * G)(*[int(n) for n in group_n])
    ptrs = (ctypes.c_void_p * G)(*[o.data_ptr() for o in outs])
    ldos = (ctypes.c_int64 * G)(*[o.stride(0) for o in outs])
    with torch.cuda.device(x.device):
        if workspace is None:
            nbytes = workspace_bytes(M, N, K, w_packed.stride(0))
            workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
        st = lib().ck_w4a4_grouped_linear(
            _ptr(x), DTYPE_CODE[x.dtype], M, K, x.stride(0), x.stride(1), _ptr(R), int(g),
            _ptr(a_scale), _ptr(w_packed), w_packed.stride(0), _ptr(w_scale),
            DTYPE_CODE[w_scale.dtype], _ptr(bias), G, gn, ptrs, ldos, DTYPE_CODE[outs[0].dtype],
            _ptr(workspace), workspace.numel(), _ptr(dev_status), _stream(stream))
    _check(st, "ck_w4a4_grouped_linear")
    return outs


def ck_rotate_quant_int8(x: torch.Tensor, R: torch.Tensor, g: int,
                         scale_in: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                         scales: torch.Tensor | None = None,
                         dev_status: torch.Tensor | None = None, stream=None):
    """The W8A8 variant's stage 1: INT8 codes (qmax 127) and fp32 row scales of a 2-D view."""
    M, K = x.shape
    _check_rotation(x, R, g)
    _same_device(x, R, scale_in, codes, scales, dev_status)
    if codes is None:
        codes = torch.empty(M, K, dtype=torch.int8, device=x.device)
    if scales is None:
        scales = torch.empty(M, dtype=torch.float32, device=x.device)
    if codes.dtype != torch.int8 or tuple(codes.shape) != (M, K) or codes.stride(1) != 1:
        raise ValueError(f"codes must be an int8 ({M}, {K}) view with unit inner stride")
    if scales.dtype != torch.float32 or scales.numel() < M or not scales.is_contiguous():
        raise ValueError(f"scales must be a contiguous fp32 tensor of at least {M} values")
    with torch.cuda.device(x.device):
        st = lib().ck_rotate_quant_int8(_ptr(x), DTYPE_CODE[x.dtype], M, K, x.stride(0),
                                        x.stride(1), _ptr(R), g, _ptr(scale_in), _ptr(codes),
                                        codes.stride(0), _ptr(scales), _ptr(dev_status),
                                        _stream(stream))
    _check(st, "ck_rotate_quant_int8")
    return codes, scales


def ck_w8a8_linear(x: torch.Tensor, R: torch.Tensor | None, g: int, w: torch.Tensor,
                   w_scale: torch.Tensor, bias: torch.Tensor | None = None, *,
                   a_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   out_dtype: torch.dtype | None = None, workspace: torch.Tensor | None = None,
                   dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The W8A8 linear: x (M, K) activations (or INT8 codes with a_scale), w (N, K) int8."""
    M, K = x.shape
    N = w.shape[0]
    if x.dtype != torch.int8:
        _check_rotation(x, R, g)
    if w.dtype != torch.int8 or w.dim() != 2 or w.stride(1) != 1 or tuple(w.shape) != (N, K):
        raise ValueError(f"w must be an int8 (N, K) = ({N}, {K}) view with unit inner stride")
    _same_device(x, R, w, w_scale, bias, a_scale, workspace, dev_status)
    if out is None:
        odt = out_dtype or (x.dtype if x.dtype != torch.int8 else w_scale.dtype)
        out = torch.empty(M, N, dtype=odt, device=x.device)
    _check_out(out, M, N, x)
    with torch.cuda.device(x.device):
        if workspace is None:
            nbytes = int(lib().ck_w8a8_linear_workspace_bytes(M, N, K, w.stride(0)))
            workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
        st = lib().ck_w8a8_linear(
            _ptr(x), DTYPE_CODE[x.dtype], M, K, x.stride(0), x.stride(1), _ptr(R), int(g),
            _ptr(a_scale), _ptr(w), N, w.stride(0), _ptr(w_scale), DTYPE_CODE[w_scale.dtype],
            _ptr(bias), _ptr(out), DTYPE_CODE[out.dtype], out.stride(0), _ptr(workspace),
            workspace.numel(), _ptr(dev_status), _stream(stream))
    _check(st, "ck_w8a8_linear")
    return out


def ck_rotate_quant_packed(x: torch.Tensor, R: torch.Tensor, g: int, *, stochastic: bool = False,
                           seed: int = 0, offset: int = 0, scale_in: torch.Tensor | None = None,
                           packed: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                           stream=None):
    """The public packed quantizer: (packed uint8 (M, K/2), scales fp32 (M,)); stochastic
    rounding draws from Philox4x32-10 keyed by seed at counter (element index, offset)."""
    M, K = x.shape
    _check_rotation(x, R, g)
    _same_device(x, R, scale_in, packed, scales)
    if packed is None:
        packed = torch.empty(M, K // 2, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(M, dtype=torch.float32, device=x.device)
    if packed.dtype != torch.uint8 or tuple(packed.shape) != (M, K // 2) or packed.stride(1) != 1:
        raise ValueError(f"packed must be a uint8 ({M}, {K // 2}) view with unit inner stride")
    with torch.cuda.device(x.device):
        st = lib().ck_rotate_quant_packed(_ptr(x), DTYPE_CODE[x.dtype], M, K, x.stride(0),
                                          x.stride(1), _ptr(R), g, _ptr(scale_in),
                                          1 if stochastic else 0, seed & (2 ** 64 - 1),
                                          offset & (2 ** 64 - 1), _ptr(packed), packed.stride(0),
                                          _ptr(scales), _stream(stream))
    _check(st, "ck_rotate_quant_packed")
    return packed, scales


def ck_unpack_w4(packed: torch.Tensor, K: int, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """(N, K/2) packed int8 -> (N, K) int8 codes."""
    N = packed.shape[0]
    if out is None:
        out = torch.empty(N, K, dtype=torch.int8, device=packed.device)
    if packed.dim() != 2 or packed.stride(1) != 1 or packed.shape[1] < K // 2 or \
            out.dim() != 2 or out.stride(1) != 1 or tuple(out.shape) != (N, K):
        raise ValueError("ck_unpack_w4: packed must be (N, >= K/2) and out (N, K), unit inner strides")
    _same_device(packed, out)
    with torch.cuda.device(packed.device):
        st = lib().ck_unpack_w4(_ptr(packed), N, K, packed.stride(0), _ptr(out), out.stride(0),
                                _stream(stream))
    _check(st, "ck_unpack_w4")
    return out


# ------------------------------------------------------------------ microscaled fp4
#
# A small call's time is mostly the host's.  Usual calls go through _ck_bind, which does what the code
# here does in a fifth of the time and declines (None) whatever it has any objection to; the code here
# then says what is wrong, or handles it.  It checks each tensor once and with the cheapest accessors
# (get_device() is -1 for a host tensor), and enters a device context only when another device is
# current.

@functools.lru_cache(maxsize=4096)
def fp4_scales_bytes(M: int, K: int, fmt: int, n_experts: int = 0) -> int:
    return int(lib().ck_fp4_scales_bytes(M, K, fmt, n_experts))


@functools.lru_cache(maxsize=4096)
def fp4_workspace_bytes(M: int, K: int, fmt: int, n_experts: int = 0) -> int:
    return int(lib().ck_fp4_linear_workspace_bytes(M, K, fmt, n_experts))


_FLOAT_CODE = {torch.float32: CK_F32, torch.float16: CK_F16, torch.bfloat16: CK_BF16}


def _on_device(x: torch.Tensor, *ts) -> int:
    """x's CUDA device index; every other tensor must be there too."""
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"ck: tensor arguments must live on a CUDA device, got one on {x.device}")
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"every tensor must be on {x.device}; got one on {t.device}")
    return dev


def _on_stream(stream, like: torch.Tensor, fn, *args, **kw):
    """fn(*args, **kw) with a caller's stream (a torch stream or a handle) current, so that what the
    call allocates is allocated there too: memory freed on another stream may still be in use by it."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _launch(name: str, dev: int, args):
    """The library's `name` on torch's current stream of `dev`, with `dev` current."""
    fn = getattr(lib(), name)
    if dev == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st != CK_OK:
        raise CkError(st, name)


def _bound(r, name: str):
    """The result of a _ck_bind call: a status of the library is raised."""
    if r.__class__ is int:
        raise CkError(r, name)
    return r


def _check_fp4(fmt: int, K: int):
    if fmt not in FP4_BLOCK:
        raise ValueError(f"fmt must be CK_MXFP4 or CK_NVFP4, got {fmt!r}")
    if K <= 0 or K % FP4_BLOCK[fmt]:
        raise ValueError(f"K = {K} must be a positive multiple of the block, {FP4_BLOCK[fmt]}")


def _check_codes(t: torch.Tensor, what: str, shape: tuple):
    if t.dtype != torch.uint8 or t.shape != shape or (t.stride(-1) != 1 and shape[-1] != 1):
        raise ValueError(f"{what} must be a uint8 {shape} view with unit inner stride; got "
                         f"{tuple(t.shape)} {t.dtype} strides {t.stride()}")


def _pitch(t: torch.Tensor, what: str) -> int:
    """Distance of a (rows, width) view's rows, which the library walks: at least a row (broadcast and
    overlapping rows are refused).  A single row's is never used and may be anything."""
    rows, width = t.shape[-2:]
    ld = t.stride(-2)
    if ld < width:
        if rows > 1:
            raise ValueError(f"{what}'s rows must not overlap: {rows} rows of {width} at a pitch of {ld}")
        ld = width
    return ld


def _check_scales(t: torch.Tensor, what: str, nbytes: int):
    if t.dtype != torch.uint8 or t.numel() < nbytes or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous uint8 tensor of at least {nbytes} bytes; got "
                         f"{t.numel()} of {t.dtype}")


def _check_memory(t: torch.Tensor, what: str):
    if t.is_neg():
        raise ValueError(f"{what} is a negated view, whose memory does not hold its values: pass "
                         f"{what}.resolve_neg()")


def _check_tensor_scale(t: torch.Tensor, what: str, n: int, fmt: int):
    if fmt == CK_MXFP4:
        raise ValueError(f"{what}: CK_MXFP4 has no tensor scale")
    _check_memory(t, what)
    if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous fp32 tensor of {n} values; got {t.numel()} of "
                         f"{t.dtype}")


def _check_offsets(offsets: torch.Tensor) -> int:
    """Number of experts."""
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous() or \
            offsets.numel() < 2:
        raise ValueError("offsets must be a contiguous 1-D int32 tensor of one more value than "
                         f"experts; got {tuple(offsets.shape)} {offsets.dtype}")
    return offsets.numel() - 1


def _float_code(t: torch.Tensor, what: str) -> int:
    code = _FLOAT_CODE.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be fp32, fp16 or bf16; got {t.dtype}")
    _check_memory(t, what)
    return code


def ck_quant_fp4(x: torch.Tensor, fmt: int, *, tensor_scale: torch.Tensor | None = None,
                 offsets: torch.Tensor | None = None, codes: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None, stream=None):
    """A 2-D (M, K) view to microscaled fp4 (fmt CK_MXFP4 or CK_NVFP4); returns (codes uint8
    (M, K/2) with rows at a pitch of 16 bytes, scales uint8 in tiles).  offsets (n_experts + 1 int32
    on the device): rows sorted by expert, each expert's scales in tiles of its own."""
    if _bind is not None and stream is None:
        r = _bind.quant(x, fmt, tensor_scale, offsets, codes, scales)
        if r is not None:
            return _bound(r, "ck_quant_fp4")
    if stream is not None:
        return _on_stream(stream, x, ck_quant_fp4, x, fmt, tensor_scale=tensor_scale, offsets=offsets,
                          codes=codes, scales=scales)
    M, K = x.shape
    _check_fp4(fmt, K)
    dt = _float_code(x, "x")
    dev = _on_device(x, tensor_scale, offsets, codes, scales)
    if tensor_scale is not None:
        _check_tensor_scale(tensor_scale, "tensor_scale", 1, fmt)
    E = 0 if offsets is None else _check_offsets(offsets)
    nbytes = fp4_scales_bytes(M, K, fmt, E)
    half = K // 2
    if codes is None:
        codes = torch.empty(M, (half + 15) // 16 * 16, dtype=torch.uint8, device=x.device)
        if half % 16:
            codes = codes[:, :half]
    else:
        _check_codes(codes, "codes", (M, half))
    if scales is None:
        scales = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    else:
        _check_scales(scales, "scales", nbytes)
    sm, sk = x.stride()
    _launch("ck_quant_fp4", dev, (
        x.data_ptr(), dt, M, K, sm, sk, fmt, None if tensor_scale is None else tensor_scale.data_ptr(),
        None if offsets is None else offsets.data_ptr(), E, codes.data_ptr(),
        _pitch(codes, "codes"), scales.data_ptr()))
    return codes, scales


def ck_dequant_fp4(codes: torch.Tensor, scales: torch.Tensor, fmt: int, *,
                   tensor_scale: torch.Tensor | None = None, offsets: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.bfloat16,
                   stream=None) -> torch.Tensor:
    """The values that codes (M, K/2) and their scale tiles stand for, (M, K)."""
    if _bind is not None and stream is None and out is None:
        r = _bind.dequant(codes, scales, fmt, tensor_scale, offsets, out_dtype)
        if r is not None:
            return _bound(r, "ck_dequant_fp4")
    if stream is not None:
        return _on_stream(stream, codes, ck_dequant_fp4, codes, scales, fmt, tensor_scale=tensor_scale,
                          offsets=offsets, out=out, out_dtype=out_dtype)
    M, half = codes.shape
    K = 2 * half
    _check_fp4(fmt, K)
    dev = _on_device(codes, scales, tensor_scale, offsets)
    _check_codes(codes, "codes", (M, half))
    if tensor_scale is not None:
        _check_tensor_scale(tensor_scale, "tensor_scale", 1, fmt)
    E = 0 if offsets is None else _check_offsets(offsets)
    _check_scales(scales, "scales", fp4_scales_bytes(M, K, fmt, E))
    if out is None:
        out = torch.empty(M, K, dtype=out_dtype, device=codes.device)
    else:
        _check_out(out, M, K, codes)
    odt = _float_code(out, "out")
    _launch("ck_dequant_fp4", dev, (
        codes.data_ptr(), _pitch(codes, "codes"), scales.data_ptr(), M, K, fmt,
        None if tensor_scale is None else tensor_scale.data_ptr(),
        None if offsets is None else offsets.data_ptr(), E, out.data_ptr(), odt, _pitch(out, "out")))
    return out


def _fp4_product(x, offsets, w, E, N, w_scales, fmt, bias, x_scales, x_tensor_scale, w_tensor_scale,
                 out, out_dtype, workspace, dev_status, stream):
    """Both products: E weight matrices w of N channels; offsets None for the plain linear."""
    if stream is not None:
        return _on_stream(stream, x, _fp4_product, x, offsets, w, E, N, w_scales, fmt, bias, x_scales,
                          x_tensor_scale, w_tensor_scale, out, out_dtype, workspace, dev_status, None)
    M, K = x.shape
    dt = _FLOAT_CODE.get(x.dtype)
    if dt is None:
        if x.dtype != torch.uint8:
            raise ValueError(f"x must be fp32, fp16 or bf16, or uint8 codes; got {x.dtype}")
        dt, K = CK_FP4, 2 * K
    _check_memory(x, "x")
    _check_fp4(fmt, K)
    dev = _on_device(x, w, w_scales, bias, x_tensor_scale, w_tensor_scale, offsets, out, x_scales,
                     workspace, dev_status)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous; got strides {workspace.stride()}")
    if dev_status is not None and (dev_status.dtype != torch.int32 or dev_status.numel() < 1):
        raise ValueError(f"dev_status must be an int32 tensor; got {dev_status.numel()} of {dev_status.dtype}")
    half = K // 2
    nE = 0 if offsets is None else E
    w_strides = w.stride()
    if w.shape[-1] != half or w.dtype != torch.uint8 or w_strides[-1] != 1:
        raise ValueError(f"w_codes must be uint8 of {half} bytes a row with unit inner stride; got "
                         f"{tuple(w.shape)} {w.dtype} strides {w.stride()}")
    per = fp4_scales_bytes(N, K, fmt)
    _check_scales(w_scales, "w_scales", E * per)
    if nE:
        if w_scales.shape != (E, per):
            raise ValueError(f"w_scales must be (n_experts, {per}); got {tuple(w_scales.shape)}")
        if _check_offsets(offsets) != E:
            raise ValueError(f"offsets must hold {E + 1} values for {E} experts; got {offsets.numel()}")
    if x_tensor_scale is not None:
        _check_tensor_scale(x_tensor_scale, "x_tensor_scale", 1, fmt)
    if w_tensor_scale is not None:
        _check_tensor_scale(w_tensor_scale, "w_tensor_scale", E, fmt)
    bdt = CK_F32
    if bias is not None:
        bdt = _float_code(bias, "bias")
        if bias.numel() != E * N or not bias.is_contiguous():
            raise ValueError(f"bias must hold {E} x {N} contiguous values; got {tuple(bias.shape)}")
    sm, sk = x.stride()
    wsb, ws = 0, None
    if dt == CK_FP4:
        _check_codes(x, "x", (M, half))
        if x_scales is None:
            raise ValueError("x holds fp4 codes: x_scales must be given")
        _check_scales(x_scales, "x_scales", fp4_scales_bytes(M, K, fmt, nE))
        # one row's pitch is never used, and need not be one that TMA could
        sm, sk = (_pitch(x, "x") if M > 1 else (half + 15) // 16 * 16), 1
    else:
        x_scales = None
        if workspace is None:
            wsb = fp4_workspace_bytes(M, K, fmt, nE)
            if wsb:
                workspace = torch.empty(wsb, dtype=torch.uint8, device=x.device)
                ws = workspace.data_ptr()
        else:
            wsb = workspace.numel() * workspace.element_size()
            ws = workspace.data_ptr()
    if out is None:
        if out_dtype is None:
            out_dtype = x.dtype if dt != CK_FP4 else torch.bfloat16 if bias is None else bias.dtype
        out = torch.empty(M, N, dtype=out_dtype, device=x.device)
        ldo = N
    else:
        _check_out(out, M, N, x)
        ldo = _pitch(out, "out")
    odt = _float_code(out, "out")
    head = (x.data_ptr(), dt, M, K, sm, sk, fmt, None if x_scales is None else x_scales.data_ptr(),
            None if x_tensor_scale is None else x_tensor_scale.data_ptr())
    tail = (w_scales.data_ptr(), None if w_tensor_scale is None else w_tensor_scale.data_ptr(),
            None if bias is None else bias.data_ptr(), bdt, out.data_ptr(), odt, ldo,
            ws, wsb, None if dev_status is None else dev_status.data_ptr())
    w_ld = _pitch(w, "w_codes") if N > 1 else (half + 15) // 16 * 16
    if nE:
        _launch("ck_fp4_expert_linear", dev, (
            *head, offsets.data_ptr(), E, w.data_ptr(), N, w_ld, w_strides[0], *tail))
    else:
        _launch("ck_fp4_linear", dev, (*head, w.data_ptr(), N, w_ld, *tail))
    return out


def ck_fp4_linear(x: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor, fmt: int,
                  bias: torch.Tensor | None = None, *, x_scales: torch.Tensor | None = None,
                  x_tensor_scale: torch.Tensor | None = None,
                  w_tensor_scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  out_dtype: torch.dtype | None = None, workspace: torch.Tensor | None = None,
                  dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The linear on microscaled fp4: x (M, K) activations (quantized on the way), or uint8 codes
    (M, K/2) with x_scales; w_codes (N, K/2) and w_scales as ck_quant_fp4 returns them.  Returns
    out (M, N)."""
    if _bind is not None and stream is None:
        r = _bind.product(x, None, w_codes, w_scales, fmt, bias, x_scales, x_tensor_scale, w_tensor_scale,
                          out, out_dtype, workspace, dev_status)
        if r is not None:
            return _bound(r, "ck_fp4_linear")
    if w_codes.dim() != 2:
        raise ValueError(f"w_codes must be (N, K/2); got {tuple(w_codes.shape)}")
    return _fp4_product(x, None, w_codes, 1, w_codes.shape[0], w_scales, fmt, bias, x_scales,
                        x_tensor_scale, w_tensor_scale, out, out_dtype, workspace, dev_status, stream)


def ck_fp4_expert_linear(x: torch.Tensor, offsets: torch.Tensor, w_codes: torch.Tensor,
                         w_scales: torch.Tensor, fmt: int, bias: torch.Tensor | None = None, *,
                         x_scales: torch.Tensor | None = None,
                         x_tensor_scale: torch.Tensor | None = None,
                         w_tensor_scale: torch.Tensor | None = None,
                         out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                         workspace: torch.Tensor | None = None,
                         dev_status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """ck_fp4_linear with rows sorted by expert: rows [offsets[e], offsets[e+1]) of x times
    w_codes[e] (n_experts, N, K/2) with w_scales[e] (n_experts, bytes), w_tensor_scale[e] and
    bias[e].  offsets stays on the device; rows of no expert keep what `out` held."""
    if _bind is not None and stream is None and offsets is not None:
        r = _bind.product(x, offsets, w_codes, w_scales, fmt, bias, x_scales, x_tensor_scale,
                          w_tensor_scale, out, out_dtype, workspace, dev_status)
        if r is not None:
            return _bound(r, "ck_fp4_expert_linear")
    if offsets is None or w_codes.dim() != 3:
        raise ValueError("offsets must be given, and w_codes be (n_experts, N, K/2); got "
                         f"{tuple(w_codes.shape)}")
    return _fp4_product(x, offsets, w_codes, w_codes.shape[0], w_codes.shape[1], w_scales, fmt, bias,
                        x_scales, x_tensor_scale, w_tensor_scale, out, out_dtype, workspace, dev_status,
                        stream)
