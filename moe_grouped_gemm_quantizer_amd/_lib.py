"""ctypes binding of libfp8gemm.so (argument marshalling only).

Each function has the name of the C entry point it calls, takes torch tensors
that already live on the current GPU, passes their device pointers, sizes and
the current torch stream, and raises on a non-zero status. No arithmetic of the
method happens here, and there is no fallback: if the library cannot be
loaded, every call raises.
"""

import array
import bisect
import ctypes
import itertools
import operator
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libfp8gemm.so")

ENTRY_POINTS = ("fp8_quantize", "fp8_quantize_bf16", "fp8_quantize_tensor", "gemm_fp8_blockscaled",
                "gemm_fp8_pertensor", "gemm_fp8_pertensor_fmt", "fp8_quantize_delayed",
                "gemm_fp8_blockscaled_quant",
                "grouped_gemm_fp8_contiguous", "grouped_gemm_fp8_contiguous_workspace_size",
                "grouped_gemm_fp8_contiguous_ws", "grouped_gemm_fp8_contiguous_noalloc",
                "grouped_gemm_fp8_masked", "fp8g_clock_probe", "fp8g_warmup",
                "fp8g_set_shape_specialisation", "fp8g_gemm_kernel_name",
                "moe_route", "moe_route_workspace_size", "moe_route_backward",
                "fp8_quantize_transpose", "grouped_gemm_fp8_wgrad", "grad_norm_sq",
                "grad_norm_sq_workspace_size", "grad_clip",
                "moe_route_scored", "moe_route_scored_backward",
                "adamw_step", "adamw_table", "adamw_table_size", "int8_quantize", "gemm_int8", "grouped_gemm_int8_contiguous",
                "grouped_gemm_int8_masked",
                "fp8g_status_string", "fp8g_abi_version")

_c_i64 = ctypes.c_int64
_c_int = ctypes.c_int
_c_vp = ctypes.c_void_p
_c_sz = ctypes.c_size_t
_c_f = ctypes.c_float
_c_d = ctypes.c_double

_SIGS = {
    "fp8_quantize": [_c_vp, _c_i64, _c_i64, _c_i64, _c_int, _c_vp, _c_i64, _c_vp, _c_i64, _c_i64, _c_vp],
    "fp8_quantize_bf16": [_c_vp, _c_i64, _c_i64, _c_i64, _c_int, _c_vp, _c_i64, _c_vp, _c_i64, _c_i64,
                          _c_vp],
    "fp8_quantize_tensor": [_c_vp, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp, _c_vp],
    "gemm_fp8_blockscaled": [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_vp],
    "gemm_fp8_pertensor": [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_vp],
    "gemm_fp8_pertensor_fmt": [_c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_i64, _c_i64,
                               _c_i64, _c_vp],
    "fp8_quantize_delayed": [_c_vp, _c_i64, _c_i64, _c_i64, _c_int, _c_vp, _c_int, _c_int, _c_vp,
                             _c_i64, _c_vp, _c_vp],
    "gemm_fp8_blockscaled_quant": [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64,
                                   _c_i64, _c_vp],
    "grouped_gemm_fp8_contiguous": [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_i64,
                                    _c_i64, _c_i64, _c_vp],
    "grouped_gemm_fp8_contiguous_workspace_size": [_c_int, _c_i64, _c_i64, _c_i64,
                                                   ctypes.POINTER(_c_sz)],
    "grouped_gemm_fp8_contiguous_ws": [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_i64,
                                       _c_i64, _c_i64, _c_vp, _c_sz, _c_vp],
    "grouped_gemm_fp8_contiguous_noalloc": [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int,
                                            _c_i64, _c_i64, _c_i64, _c_vp],
    "grouped_gemm_fp8_masked": [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_i64,
                                _c_i64, _c_i64, _c_int, _c_vp],
    "fp8g_clock_probe": [_c_vp, _c_int, _c_vp],
    "fp8g_warmup": [],
    "fp8g_set_shape_specialisation": [_c_int],
    "fp8g_gemm_kernel_name": [_c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int,
                              ctypes.c_char_p, _c_sz],
    "moe_route": [_c_vp, _c_int, _c_i64, _c_int, _c_i64, _c_vp, _c_int, _c_int, _c_f, _c_int, _c_i64,
                  _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp],
    "moe_route_workspace_size": [_c_i64, _c_int, ctypes.POINTER(_c_sz)],
    "moe_route_backward": [_c_vp, _c_int, _c_i64, _c_int, _c_i64, _c_vp, _c_int, _c_int, _c_f, _c_vp,
                           _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp],
    "fp8_quantize_transpose": [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_vp, _c_i64, _c_vp,
                               _c_vp],
    "grouped_gemm_fp8_wgrad": [_c_vp, _c_int, _c_i64, _c_vp, _c_vp, _c_int, _c_i64, _c_vp, _c_vp,
                               _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp],
    "grad_norm_sq": [_c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_sz, _c_vp],
    "grad_norm_sq_workspace_size": [_c_vp, _c_int, ctypes.POINTER(_c_sz)],
    "grad_clip": [_c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_f, _c_vp, _c_vp],
    "moe_route_scored": [_c_vp, _c_int, _c_i64, _c_int, _c_i64, _c_vp, _c_int, _c_int, _c_int, _c_int, _c_vp,
                         _c_int, _c_int, _c_f, _c_f, _c_int, _c_i64, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp,
                         _c_vp, _c_vp, _c_vp, _c_vp, _c_sz, _c_vp],
    "moe_route_scored_backward": [_c_vp, _c_int, _c_i64, _c_int, _c_i64, _c_int, _c_vp, _c_int, _c_int, _c_f,
                                  _c_f, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp],
    "adamw_step": [_c_vp] * 11 + [_c_int, _c_vp, _c_i64, _c_vp, _c_d, _c_d, _c_d, _c_d, _c_d, _c_vp, _c_f,
                                  _c_vp, ctypes.c_uint32, _c_vp, _c_vp],
    "adamw_table": [_c_vp] * 11 + [_c_int, _c_vp],
    "adamw_table_size": [_c_int, ctypes.POINTER(ctypes.c_size_t)],
    "int8_quantize": [_c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_vp, _c_i64, _c_vp, _c_vp],
    "gemm_int8": [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_i64, _c_vp],
    "grouped_gemm_int8_contiguous": [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_i64, _c_i64,
                                     _c_i64, _c_vp],
    "grouped_gemm_int8_masked": [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_i64, _c_i64,
                                 _c_i64, _c_int, _c_vp],
}

LAYOUTS = {"dense": 0, "contiguous": 1, "masked": 2, "pertensor": 3}
FORMATS = {"e4m3": 0, "e5m2": 1}
SCORES = {"sigmoid": 0, "softmax": 1}

_lib = None


class Fp8GemmError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: status {status} ({status_string(status)})")


def load(path=LIB_PATH):
    """Load the shared library (once) and declare every entry point."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m moe_grouped_gemm_quantizer_amd.build`")
    lib = ctypes.CDLL(path)
    for name, args in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.fp8g_status_string.argtypes = [ctypes.c_int]
    lib.fp8g_status_string.restype = ctypes.c_char_p
    lib.fp8g_abi_version.argtypes = []
    lib.fp8g_abi_version.restype = ctypes.c_int
    _lib = lib
    return lib


def status_string(status):
    return load().fp8g_status_string(int(status)).decode()


def fp8g_abi_version():
    return load().fp8g_abi_version()


_raw_stream = None


def _current_stream():
    """The current device's current stream, as its handle. (torch's own
    integer form takes 0.1 us, the Stream object 2.9.)"""
    global _raw_stream
    if _raw_stream is None:
        import torch
        torch.cuda.current_stream()                 # (initialises the device)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_stream = ((lambda: raw(torch._C._cuda_getDevice())) if raw is not None
                       else (lambda: torch.cuda.current_stream().cuda_stream))
    return _raw_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _torchs_stream(stream, handle):
    """The Stream object that `stream` (as _stream takes it) means, or None where
    it is not one of torch's own: a handle made elsewhere may be destroyed while
    torch's allocator still wants to record an event on it."""
    torch = _torch()
    if stream is None or isinstance(stream, int):
        # (not ExternalStream(handle): that of 0 is no default stream but another, new one)
        s = torch.cuda.current_stream()
        if s.cuda_stream != handle:
            s = torch.cuda.default_stream()
    else:
        s = stream
    if not isinstance(s, torch.cuda.Stream) or s.cuda_stream != handle or (handle != 0 and s.stream_id == handle):
        return None                          # (a foreign stream's id is its handle)
    return s


def _ptr(t):
    return None if t is None else t.data_ptr()


def _nb(n):
    """128-wide blocks covering n (the last may be partial)."""
    return -(-int(n) // 128)


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _check(status, what):
    if status != 0:
        raise Fp8GemmError(status, what)


def _dev(*ts):
    for t in ts:
        _need(t.is_cuda, "tensors must live on the GPU")
        _need(t.is_contiguous(), "tensors must be contiguous")


def _gemm_dtypes(a, sa, b, sb, d, meta=None):
    """The C calls read raw bytes: a wrong element type would be misread, not
    converted, so it is refused here."""
    import torch
    codes = (torch.uint8, torch.float8_e4m3fn)
    _need(a.dtype in codes and b.dtype in codes, "a and b must be e4m3 codes (uint8 or float8_e4m3fn)")
    _need(sa.dtype == torch.float32 and sb.dtype == torch.float32, "sa and sb must be float32")
    _need(d.dtype in (torch.int16, torch.bfloat16, torch.uint16),
          "d must hold bf16 values (bfloat16, or int16/uint16 bit patterns)")
    if meta is not None:
        _need(meta.dtype == torch.int32, "group metadata must be int32")


def fp8_quantize(x, block_rows, q, scales, s_stride_row, s_stride_col, stream=None):
    """x float32 [rows][cols] -> q uint8 [rows][cols], scales float32 (strided).

    block_rows 1: A operand, call with s_stride_row=1, s_stride_col=rows.
    block_rows 128: B operand, s_stride_row=cols//128, s_stride_col=1.
    """
    import torch
    _need(x.dim() == 2 and q.dim() == 2 and x.shape == q.shape, "x and q must be same-shape 2-D")
    _need(x.dtype == torch.float32 and q.dtype == torch.uint8 and scales.dtype == torch.float32,
          "x float32, q uint8, scales float32")
    _dev(x, q, scales)
    rows, cols = x.shape
    nrb = -(-rows // block_rows)
    ncb = -(-cols // 128)
    if rows and cols:
        need = (nrb - 1) * s_stride_row + (ncb - 1) * s_stride_col + 1
        _need(scales.numel() >= need, "scales tensor too small for the blocking")
    st = load().fp8_quantize(_ptr(x), rows, cols, cols, int(block_rows), _ptr(q), cols,
                             _ptr(scales), int(s_stride_row), int(s_stride_col), _stream(stream))
    _check(st, "fp8_quantize")


def fp8_quantize_bf16(x, block_rows, q, scales, s_stride_row, s_stride_col, stream=None):
    """x bfloat16 (or int16 bit patterns) [rows][cols] -> q uint8, scales float32;
    arguments and result as for fp8_quantize on x's exact float32 values."""
    import torch
    _need(x.dim() == 2 and q.dim() == 2 and x.shape == q.shape, "x and q must be same-shape 2-D")
    _need(x.dtype in (torch.bfloat16, torch.int16) and q.dtype == torch.uint8
          and scales.dtype == torch.float32, "x bfloat16, q uint8, scales float32")
    _dev(x, q, scales)
    rows, cols = x.shape
    nrb = -(-rows // block_rows)
    ncb = -(-cols // 128)
    if rows and cols:
        need = (nrb - 1) * s_stride_row + (ncb - 1) * s_stride_col + 1
        _need(scales.numel() >= need, "scales tensor too small for the blocking")
    st = load().fp8_quantize_bf16(_ptr(x), rows, cols, cols, int(block_rows), _ptr(q), cols,
                                  _ptr(scales), int(s_stride_row), int(s_stride_col),
                                  _stream(stream))
    _check(st, "fp8_quantize_bf16")


def gemm_fp8_blockscaled_quant(a, sa, b, sb, d, qd, sd, stream=None):
    """gemm_fp8_blockscaled with the result also quantised 1x128 for the next
    GEMM: qd uint8 [M][N] codes, sd float32 [N/128][M] scales; d bf16 [M][N]
    or None."""
    import torch
    M, K = a.shape
    N = b.shape[0]
    _need(b.shape[1] == K, "a and b disagree on K")
    _need(tuple(sa.shape) == (_nb(K), M), "sa must be [ceil(K/128)][M] (1x128 per-token scales)")
    _need(tuple(sb.shape) == (_nb(N), _nb(K)), "sb must be [ceil(N/128)][ceil(K/128)] (128x128 block scales)")
    _need(tuple(qd.shape) == (M, N) and qd.dtype == torch.uint8, "qd must be uint8 [M][N]")
    _need(tuple(sd.shape) == (_nb(N), M) and sd.dtype == torch.float32, "sd must be float32 [ceil(N/128)][M]")
    dd = d if d is not None else torch.empty(0, dtype=torch.int16)
    _gemm_dtypes(a, sa, b, sb, dd)
    if d is not None:
        _need(tuple(d.shape) == (M, N), "d must be [M][N]")
        _dev(d)
    _dev(a, sa, b, sb, qd, sd)
    st = load().gemm_fp8_blockscaled_quant(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(d), _ptr(qd),
                                           _ptr(sd), M, N, K, _stream(stream))
    _check(st, "gemm_fp8_blockscaled_quant")


def fp8_quantize_tensor(x, q, scale, stream=None):
    """x float32 [rows][cols] -> q uint8 [rows][cols] with one scale: scale
    is a float32 device tensor of one element (receives amax / 448)."""
    import torch
    _need(x.dim() == 2 and q.dim() == 2 and x.shape == q.shape, "x and q must be same-shape 2-D")
    _need(x.dtype == torch.float32 and q.dtype == torch.uint8 and scale.dtype == torch.float32
          and scale.numel() == 1, "x float32, q uint8, scale float32 [1]")
    _dev(x, q, scale)
    rows, cols = x.shape
    st = load().fp8_quantize_tensor(_ptr(x), rows, cols, cols, _ptr(q), cols, _ptr(scale),
                                    _stream(stream))
    _check(st, "fp8_quantize_tensor")


def gemm_fp8_pertensor(a, scale_a, b, scale_b, d, stream=None):
    """a uint8 [M][K], scale_a float32 [1], b uint8 [N][K], scale_b float32 [1],
    d bf16 (int16/bfloat16) [M][N]."""
    import torch
    M, K = a.shape
    N = b.shape[0]
    _need(b.shape[1] == K, "a and b disagree on K")
    _need(scale_a.numel() == 1 and scale_b.numel() == 1, "per-tensor scales are one float each")
    _need(tuple(d.shape) == (M, N), "d must be [M][N]")
    _gemm_dtypes(a, scale_a, b, scale_b, d)
    _dev(a, scale_a, b, scale_b, d)
    st = load().gemm_fp8_pertensor(_ptr(a), _ptr(scale_a), _ptr(b), _ptr(scale_b), _ptr(d), M, N,
                                   K, _stream(stream))
    _check(st, "gemm_fp8_pertensor")


def _fmt(name):
    if name not in FORMATS:
        raise ValueError(f"format must be one of {sorted(FORMATS)}")
    return FORMATS[name]


def _codes_dtype_ok(t, fmt):
    import torch
    ok = (torch.uint8, torch.float8_e4m3fn) if fmt == "e4m3" else (torch.uint8, torch.float8_e5m2)
    return t.dtype in ok


def gemm_fp8_pertensor_fmt(a, fmt_a, scale_a, b, fmt_b, scale_b, d, stream=None):
    """gemm_fp8_pertensor with each operand's format: fmt_a, fmt_b 'e4m3' or
    'e5m2' (codes as uint8, or torch's float8 dtype of that format)."""
    import torch
    fa, fb = _fmt(fmt_a), _fmt(fmt_b)
    M, K = a.shape
    N = b.shape[0]
    _need(b.shape[1] == K, "a and b disagree on K")
    _need(scale_a.numel() == 1 and scale_b.numel() == 1, "per-tensor scales are one float each")
    _need(tuple(d.shape) == (M, N), "d must be [M][N]")
    _need(_codes_dtype_ok(a, fmt_a) and _codes_dtype_ok(b, fmt_b),
          "a and b must be codes of their formats (uint8 or the matching float8 dtype)")
    _need(scale_a.dtype == torch.float32 and scale_b.dtype == torch.float32,
          "scales must be float32")
    _need(d.dtype in (torch.int16, torch.bfloat16, torch.uint16),
          "d must hold bf16 values (bfloat16, or int16/uint16 bit patterns)")
    _dev(a, scale_a, b, scale_b, d)
    st = load().gemm_fp8_pertensor_fmt(_ptr(a), fa, _ptr(scale_a), _ptr(b), fb, _ptr(scale_b),
                                       _ptr(d), M, N, K, _stream(stream))
    _check(st, "gemm_fp8_pertensor_fmt")


def fp8_quantize_delayed(x, fmt, amax_history, slot, q, scale, stream=None):
    """One delayed-scaling step: x float32 [rows][cols] -> q uint8 codes in
    fmt ('e4m3' or 'e5m2') under the scale taken from amax_history (float32
    device tensor, read and written; entry `slot` receives this step's amax);
    scale: float32 device tensor of one element (receives the scale used)."""
    import torch
    f = _fmt(fmt)
    _need(x.dim() == 2 and q.dim() == 2 and x.shape == q.shape, "x and q must be same-shape 2-D")
    _need(x.dtype == torch.float32 and q.dtype == torch.uint8 and scale.dtype == torch.float32
          and scale.numel() == 1 and amax_history.dtype == torch.float32
          and amax_history.dim() == 1, "x float32, q uint8, scale float32 [1], history float32 [H]")
    _dev(x, q, scale, amax_history)
    rows, cols = x.shape
    st = load().fp8_quantize_delayed(_ptr(x), rows, cols, cols, f, _ptr(amax_history),
                                     amax_history.numel(), int(slot), _ptr(q), cols, _ptr(scale),
                                     _stream(stream))
    _check(st, "fp8_quantize_delayed")


def gemm_fp8_blockscaled(a, sa, b, sb, d, stream=None):
    """a uint8 [M][K], sa float32 [K/128][M], b uint8 [N][K], sb float32
    [N/128][K/128], d bf16 (int16/bfloat16) [M][N]."""
    M, K = a.shape
    N = b.shape[0]
    _need(b.shape[1] == K, "a and b disagree on K")
    _need(tuple(sa.shape) == (_nb(K), M), "sa must be [ceil(K/128)][M] (1x128 per-token scales)")
    _need(tuple(sb.shape) == (_nb(N), _nb(K)), "sb must be [ceil(N/128)][ceil(K/128)] (128x128 block scales)")
    _need(tuple(d.shape) == (M, N), "d must be [M][N]")
    _gemm_dtypes(a, sa, b, sb, d)
    _dev(a, sa, b, sb, d)
    st = load().gemm_fp8_blockscaled(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(d), M, N, K,
                                     _stream(stream))
    _check(st, "gemm_fp8_blockscaled")


def _contiguous_args(a, sa, b, sb, d, group_offsets):
    M, K = a.shape
    G, N, K2 = b.shape
    _need(K2 == K, "a and b disagree on K")
    _need(tuple(sa.shape) == (_nb(K), M), "sa must be [ceil(K/128)][M_total]")
    _need(tuple(sb.shape) == (G, _nb(N), _nb(K)), "sb must be [G][ceil(N/128)][ceil(K/128)]")
    _need(tuple(d.shape) == (M, N), "d must be [M_total][N]")
    _need(group_offsets.numel() == G + 1, "group_offsets must be int32 [G+1]")
    _gemm_dtypes(a, sa, b, sb, d, group_offsets)
    _dev(a, sa, b, sb, d, group_offsets)
    return (_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(d), _ptr(group_offsets), G, M, N, K)


def grouped_gemm_fp8_contiguous(a, sa, b, sb, d, group_offsets, stream=None):
    """a uint8 [M_total][K], sa [K/128][M_total], b uint8 [G][N][K],
    sb [G][N/128][K/128], d [M_total][N], group_offsets int32 [G+1] (device)."""
    st = load().grouped_gemm_fp8_contiguous(*_contiguous_args(a, sa, b, sb, d, group_offsets),
                                            _stream(stream))
    _check(st, "grouped_gemm_fp8_contiguous")


def grouped_gemm_fp8_contiguous_workspace_size(G, M_total, N, K):
    """Bytes of workspace grouped_gemm_fp8_contiguous_ws can use (0: none)."""
    out = ctypes.c_size_t(0)
    st = load().grouped_gemm_fp8_contiguous_workspace_size(int(G), int(M_total), int(N), int(K),
                                                           ctypes.byref(out))
    _check(st, "grouped_gemm_fp8_contiguous_workspace_size")
    return int(out.value)


def grouped_gemm_fp8_contiguous_ws(a, sa, b, sb, d, group_offsets, workspace, stream=None):
    """grouped_gemm_fp8_contiguous with a caller-owned workspace (a contiguous
    device tensor of at least grouped_gemm_fp8_contiguous_workspace_size
    bytes, or None)."""
    if workspace is None:
        wp, wb = None, 0
    else:
        _dev(workspace)
        wp, wb = _ptr(workspace), workspace.numel() * workspace.element_size()
    st = load().grouped_gemm_fp8_contiguous_ws(*_contiguous_args(a, sa, b, sb, d, group_offsets),
                                               wp, wb, _stream(stream))
    _check(st, "grouped_gemm_fp8_contiguous_ws")


def grouped_gemm_fp8_contiguous_noalloc(a, sa, b, sb, d, group_offsets, stream=None):
    """grouped_gemm_fp8_contiguous_ws with the library's fixed scratch array
    as the workspace (no allocation; calls on one GPU must not overlap)."""
    st = load().grouped_gemm_fp8_contiguous_noalloc(
        *_contiguous_args(a, sa, b, sb, d, group_offsets), _stream(stream))
    _check(st, "grouped_gemm_fp8_contiguous_noalloc")


def grouped_gemm_fp8_masked(a, sa, b, sb, d, masked_m, expected_m=0, stream=None):
    """a uint8 [G][max_m][K], sa [K/128][G*max_m], b uint8 [G][N][K],
    sb [G][N/128][K/128], d [G][max_m][N], masked_m int32 [G] (device)."""
    import torch
    G, max_m, K = a.shape
    G2, N, K2 = b.shape
    _need(G2 == G and K2 == K, "a and b disagree on G or K")
    _need(tuple(sa.shape) == (_nb(K), G * max_m), "sa must be [ceil(K/128)][G*max_m]")
    _need(tuple(sb.shape) == (G, _nb(N), _nb(K)), "sb must be [G][ceil(N/128)][ceil(K/128)]")
    _need(tuple(d.shape) == (G, max_m, N), "d must be [G][max_m][N]")
    _need(masked_m.numel() == G, "masked_m must be int32 [G]")
    _gemm_dtypes(a, sa, b, sb, d, masked_m)
    _dev(a, sa, b, sb, d, masked_m)
    st = load().grouped_gemm_fp8_masked(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(d),
                                        _ptr(masked_m), G, max_m, N, K, int(expected_m),
                                        _stream(stream))
    _check(st, "grouped_gemm_fp8_masked")


# The training-step calls are short on the GPU, so their checks are written to
# cost little: one attribute each, messages formed only when one fails.
_TYPES = {}


def _torch():
    """torch, with _TYPES (element type -> FP8G_TYPE_*) filled."""
    import torch
    if not _TYPES:
        _TYPES.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    return torch


def _fail(msg):
    raise ValueError(msg)


def _rows(t, what):
    """Pointer, rows, columns and row stride of a GPU matrix whose rows are
    contiguous."""
    if not t.is_cuda or t.dim() != 2:
        _fail(f"{what} must be a matrix on the GPU")
    rows, cols = t.shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        _fail(f"{what}: the elements of a row must be contiguous")
    # (a single row has any stride, and so have empty ones)
    return t.data_ptr(), rows, cols, ld if rows > 1 and cols > 0 else cols


def _out(t, shape, dtype, what):
    """The pointer of a contiguous GPU tensor of this shape and type."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _fail(f"{what} must be {dtype} {list(shape)}, contiguous and on the GPU")
    return t.data_ptr()


def _room(workspace):
    if workspace is None:
        return None, 0
    _dev(workspace)
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def moe_route_workspace_size(T, E):
    """Bytes of workspace moe_route needs for T tokens and E experts (0: none)."""
    out = ctypes.c_size_t(0)
    _check(load().moe_route_workspace_size(int(T), int(E), ctypes.byref(out)),
           "moe_route_workspace_size")
    return int(out.value)


def moe_route(logits, top_k, expert_ids, weights, counts, routed, prob_sum, loss, group_offsets, slots,
              workspace=None, token_mask=None, renormalise=False, loss_coef=1.0, align=128, max_m=0,
              stream=None):
    """Routing of T tokens to top_k of E experts, with the balance loss.

    logits [T][E] (float32, bfloat16 or float16; rows may be strided), token_mask
    bool or uint8 [T] or None. Written: expert_ids int32 [T][top_k] (-1: none),
    weights float32 [T][top_k], counts int32 [E], routed int32 [1], prob_sum
    float32 [E], loss float32 [1], group_offsets int32 [E+1] (contiguous layout,
    multiples of align; with max_m > 0 the masked layout's slabs), slots int32
    [T][top_k] (row of each pair in that layout, -1: none). workspace: a device
    tensor of at least moe_route_workspace_size(T, E) bytes."""
    torch = _torch()
    ptr, T, E, ld = _rows(logits, "logits")
    typ = _TYPES.get(logits.dtype)
    if typ is None:
        _fail("logits must be float32, bfloat16 or float16")
    i32, f32, pairs = torch.int32, torch.float32, (T, top_k)
    ids = _out(expert_ids, pairs, i32, "expert_ids")
    wts = _out(weights, pairs, f32, "weights")
    cnt = _out(counts, (E,), i32, "counts")
    rtd = _out(routed, (1,), i32, "routed")
    psm = _out(prob_sum, (E,), f32, "prob_sum")
    los = _out(loss, (1,), f32, "loss")
    off = _out(group_offsets, (E + 1,), i32, "group_offsets")
    slt = _out(slots, pairs, i32, "slots")
    mask = None
    if token_mask is not None:
        mask = _out(token_mask, (T,), torch.uint8 if token_mask.dtype is torch.uint8 else torch.bool, "token_mask")
    wp, wb = _room(workspace)
    st = load().moe_route(ptr, typ, T, E, ld, mask, top_k, 1 if renormalise else 0, loss_coef,
                          align, max_m, ids, wts, cnt, rtd, psm, los, off, slt, wp, wb, _stream(stream))
    if st:
        _check(st, "moe_route")


def _score(name):
    if name not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}")
    return SCORES[name]


def moe_route_scored(logits, top_k, expert_ids, weights, counts, routed, prob_sum, loss, group_offsets, slots,
                     workspace=None, score="sigmoid", bias=None, groups=1, open_groups=1, group_best=1,
                     token_mask=None, renormalise=False, scale=1.0, loss_coef=1.0, align=128, max_m=0,
                     stream=None):
    """Routing by scores: 'sigmoid' or 'softmax' of the logits, plus bias
    (float32 [E] or None) for the choice alone, inside the open_groups of groups
    equal groups of experts whose group_best (1 or 2) largest values sum to the
    most; weights scale times the scores without the bias, over their sum with
    renormalise. Everything else as for moe_route."""
    torch = _torch()
    ptr, T, E, ld = _rows(logits, "logits")
    typ = _TYPES.get(logits.dtype)
    if typ is None:
        _fail("logits must be float32, bfloat16 or float16")
    i32, f32, pairs = torch.int32, torch.float32, (T, top_k)
    ids = _out(expert_ids, pairs, i32, "expert_ids")
    wts = _out(weights, pairs, f32, "weights")
    cnt = _out(counts, (E,), i32, "counts")
    rtd = _out(routed, (1,), i32, "routed")
    psm = _out(prob_sum, (E,), f32, "prob_sum")
    los = _out(loss, (1,), f32, "loss")
    off = _out(group_offsets, (E + 1,), i32, "group_offsets")
    slt = _out(slots, pairs, i32, "slots")
    bia = None if bias is None else _out(bias, (E,), f32, "bias")
    mask = None
    if token_mask is not None:
        mask = _out(token_mask, (T,), torch.uint8 if token_mask.dtype is torch.uint8 else torch.bool, "token_mask")
    wp, wb = _room(workspace)
    _one_device(logits, expert_ids, weights, counts, routed, prob_sum, loss, group_offsets, slots, bias, token_mask,
                workspace)
    st = load().moe_route_scored(ptr, typ, T, E, ld, bia, _score(score), groups, open_groups, group_best, mask,
                                 top_k, 1 if renormalise else 0, scale, loss_coef, align, max_m, ids, wts, cnt,
                                 rtd, psm, los, off, slt, wp, wb, _stream(stream))
    if st:
        _check(st, "moe_route_scored")


def moe_route_scored_backward(logits, expert_ids, d_weights, d_loss, counts, routed, d_logits, score="sigmoid",
                              renormalise=False, scale=1.0, loss_coef=1.0, stream=None):
    """Gradient of moe_route_scored's weights and loss with respect to the
    logits; score, renormalise, scale and loss_coef as given there, the rest as
    for moe_route_backward."""
    torch = _torch()
    ptr, T, E, ld = _rows(logits, "logits")
    dptr, dT, dE, ldd = _rows(d_logits, "d_logits")
    typ = _TYPES.get(logits.dtype)
    if typ is None or d_logits.dtype is not logits.dtype or dT != T or dE != E:
        _fail("logits and d_logits must be float32, bfloat16 or float16, alike in type and shape")
    top_k = expert_ids.shape[-1]
    ids = _out(expert_ids, (T, top_k), torch.int32, "expert_ids")
    dw = None if d_weights is None else _out(d_weights, (T, top_k), torch.float32, "d_weights")
    dl = None if d_loss is None else _out(d_loss, (1,), torch.float32, "d_loss")
    cnt = _out(counts, (E,), torch.int32, "counts")
    rtd = _out(routed, (1,), torch.int32, "routed")
    _one_device(logits, expert_ids, d_weights, d_loss, counts, routed, d_logits)
    st = load().moe_route_scored_backward(ptr, typ, T, E, ld, _score(score), ids, top_k, 1 if renormalise else 0,
                                          scale, loss_coef, dw, dl, cnt, rtd, dptr, ldd, _stream(stream))
    if st:
        _check(st, "moe_route_scored_backward")


def moe_route_backward(logits, expert_ids, d_weights, d_loss, counts, routed, d_logits,
                       renormalise=False, loss_coef=1.0, stream=None):
    """Gradient of moe_route's weights and loss with respect to the logits.

    logits, expert_ids, counts, routed, renormalise, loss_coef as given to and
    written by moe_route; d_weights float32 [T][top_k] or None, d_loss float32
    [1] or None; d_logits [T][E] of the logits' type (rows may be strided)."""
    torch = _torch()
    ptr, T, E, ld = _rows(logits, "logits")
    dptr, dT, dE, ldd = _rows(d_logits, "d_logits")
    typ = _TYPES.get(logits.dtype)
    if typ is None or d_logits.dtype is not logits.dtype or dT != T or dE != E:
        _fail("logits and d_logits must be float32, bfloat16 or float16, alike in type and shape")
    top_k = expert_ids.shape[-1]
    ids = _out(expert_ids, (T, top_k), torch.int32, "expert_ids")
    dw = None if d_weights is None else _out(d_weights, (T, top_k), torch.float32, "d_weights")
    dl = None if d_loss is None else _out(d_loss, (1,), torch.float32, "d_loss")
    cnt = _out(counts, (E,), torch.int32, "counts")
    rtd = _out(routed, (1,), torch.int32, "routed")
    st = load().moe_route_backward(ptr, typ, T, E, ld, ids, top_k, 1 if renormalise else 0,
                                   loss_coef, dw, dl, cnt, rtd, dptr, ldd, _stream(stream))
    if st:
        _check(st, "moe_route_backward")


def fp8_quantize_transpose(x, fmt, qt, st, stream=None):
    """x [rows][cols] (float32, bfloat16 or float16; rows may be strided) ->
    qt uint8 [cols][R] codes in fmt ('e4m3' or 'e5m2'), R = rows rounded up to
    128, and st uint8 [R/128][cols]: one power-of-two scale per column and 128
    rows, as its exponent + 127. Rows that hold no token must be zero."""
    torch = _torch()
    xp, rows, cols, ldx = _rows(x, "x")
    nb = (rows + 127) // 128
    typ = _TYPES.get(x.dtype)
    if typ is None:
        _fail("x must be float32, bfloat16 or float16")
    qp, qrows, qcols, ldq = _rows(qt, "qt")
    if qt.dtype is not torch.uint8 or qrows != cols or qcols != nb * 128:
        _fail("qt must be uint8 [cols][rows rounded up to 128]")
    scales = _out(st, (nb, cols), torch.uint8, "st (ceil(rows/128), cols)")
    status = load().fp8_quantize_transpose(xp, typ, rows, cols, ldx, _fmt(fmt), qp, ldq, scales,
                                           _stream(stream))
    if status:
        _check(status, "fp8_quantize_transpose")


def grouped_gemm_fp8_wgrad(a, fmt_a, sa, b, fmt_b, sb, d, group_offsets=None, stream=None):
    """Weight gradients of G experts: d bf16 [G][M][N] from a [M][T], sa
    [T/128][M], b [N][T], sb [T/128][N] as fp8_quantize_transpose writes them
    (T a multiple of 128); group_offsets int32 [G+1] (device) or None (G = 1,
    all tokens). Every row of x from one offset up to the next is summed, also
    those past an expert's last token: clear the buffers that tokens are dealt
    into, since whatever such a row holds enters scales and sum."""
    torch = _torch()
    ap, M, T, lda = _rows(a, "a")
    bp, N, Tb, ldb = _rows(b, "b")
    fa, fb = _fmt(fmt_a), _fmt(fmt_b)
    if Tb != T or T % 128:
        _fail("a and b must have the same tokens, a multiple of 128")
    u8 = torch.uint8
    if not ((a.dtype is u8 or _codes_dtype_ok(a, fmt_a)) and (b.dtype is u8 or _codes_dtype_ok(b, fmt_b))):
        _fail("a and b must be codes of their formats (uint8 or the matching float8 dtype)")
    pa = _out(sa, (T // 128, M), u8, "sa (T/128, M)")
    pb = _out(sb, (T // 128, N), u8, "sb (T/128, N)")
    dt = d.dtype
    if d.dim() != 3 or (dt is not torch.bfloat16 and dt is not torch.int16 and dt is not torch.uint16):
        _fail("d must be bf16 [G][M][N]")
    G = len(d)
    pd = _out(d, (G, M, N), dt, "d ([G][M][N])")
    if group_offsets is not None:
        po = _out(group_offsets, (G + 1,), torch.int32, "group_offsets")
    elif G == 1:
        po = None
    else:
        _fail("group_offsets may be None for one expert only")
    st = load().grouped_gemm_fp8_wgrad(ap, fa, lda, pa, bp, fb, ldb, pb, pd, po, G, T, M, N, _stream(stream))
    if st:
        _check(st, "grouped_gemm_fp8_wgrad")


def _grad_list(ts, what):
    """HOST arrays of the tensors' pointers, sizes and types. (Hundreds of
    tensors: every attribute is read in a loop of the interpreter's own.) ts:
    a tuple or list, since it is gone through several times."""
    torch = _torch()
    cls = torch.Tensor
    types = list(map(_TYPES.get, map(operator.attrgetter("dtype"), ts)))
    if None in types:
        _fail(f"{what} must be float32, bfloat16 or float16")
    if not (all(map(operator.attrgetter("is_cuda"), ts)) and all(map(cls.is_contiguous, ts))):
        _fail(f"{what} must be contiguous and on the GPU")
    return (array.array("Q", list(map(cls.data_ptr, ts))), array.array("q", list(map(cls.numel, ts))),
            array.array("i", types))


def _at(a):
    return a.buffer_info()[0] if len(a) else None


def grad_norm_sq_workspace_size(grads):
    """Bytes of workspace grad_norm_sq needs for this list of tensors."""
    out = ctypes.c_size_t(0)
    numels = array.array("q", [t.numel() for t in grads])
    _check(load().grad_norm_sq_workspace_size(_at(numels), len(numels), ctypes.byref(out)),
           "grad_norm_sq_workspace_size")
    return int(out.value)


def grad_norm_sq(grads, sumsq, workspace, stream=None):
    """Sum of squares over a list (or any iterable) of contiguous tensors
    (float32, bfloat16, float16, mixed) into sumsq, a float64 device tensor of
    one element. workspace: at least grad_norm_sq_workspace_size(grads) bytes."""
    torch = _torch()
    ptrs, numels, types = _grad_list(tuple(grads), "grads")
    out = _out(sumsq, (1,), torch.float64, "sumsq")
    wp, wb = _room(workspace)
    _check(load().grad_norm_sq(_at(ptrs), _at(numels), _at(types), len(ptrs), out, wp, wb, _stream(stream)),
           "grad_norm_sq")


def grad_clip(grads, outs, sumsq, max_norm, norm, stream=None):
    """outs[i] = grads[i] * min(1, max_norm / (norm + 1e-6)), norm = sqrt(sumsq)
    (float32 device tensor of one element, written). grads and outs: lists or
    any iterables; outs[i] may be grads[i]."""
    torch = _torch()
    same = outs is grads                              # (also one iterator given twice)
    ptrs, numels, types = _grad_list(tuple(grads), "grads")
    if same:
        optrs = ptrs
    else:
        optrs, onumels, otypes = _grad_list(tuple(outs), "outs")
        if onumels != numels or otypes != types:
            _fail("outs must match grads in number, size and type")
    total = _out(sumsq, (1,), torch.float64, "sumsq")
    nrm = _out(norm, (1,), torch.float32, "norm")
    _check(load().grad_clip(_at(ptrs), _at(optrs), _at(numels), _at(types), len(ptrs), total, max_norm, nrm,
                            _stream(stream)), "grad_clip")


def _overlapping(starts, ends, read):
    """Whether any of the memory ranges starts[i] .. ends[i] overlaps another of
    them or one of `read`, pairs (which may overlap each other). Empty: 0, 0."""
    # (each sorted by itself: where none overlap, the next start is never below the i-th end)
    starts, ends = sorted(starts), sorted(ends)
    if any(map(operator.gt, ends, starts[1:])):
        return True
    for lo, hi in read:
        # (they lie apart: only the last one that starts below hi can reach into it)
        i = bisect.bisect_left(starts, hi) - 1
        if lo < hi and i >= 0 and ends[i] > lo:
            return True
    return False


class AdamwTensors:
    """The tensors of an AdamW step (made by adamw_tensors): their pointers,
    sizes and types as HOST arrays, for a long list as a table in device memory
    too, and their storages, which keeps the memory alive."""

    __slots__ = ("held", "lists", "n", "device", "table", "streams")


def adamw_tensors(params, grads, exp_avgs, exp_avg_sqs, copies=None, m_scales=None, v_scales=None):
    """The list of an AdamW step, for adamw_step: made once and used for many
    steps, as long as the tensors keep their memory (make a new one where a
    gradient or parameter becomes another tensor).

    params, grads: float32, bfloat16 or float16, contiguous, alike in number and
    size. States: exp_avgs and exp_avg_sqs float32 of the same sizes, or, with
    m_scales and v_scales (uint8 [ceil(numel/128)] each), uint8 e4m3 codes of m and
    sqrt(v) (zeros: a fresh state). copies: bfloat16 or float16 tensors that
    receive the parameters, or None; single ones may be None. What the step
    writes may not overlap another tensor of the list."""
    torch = _torch()
    eight = m_scales is not None or v_scales is not None
    if eight and (m_scales is None or v_scales is None):
        _fail("m_scales and v_scales go together")
    lists = [list(ts) for ts in (params, grads, exp_avgs, exp_avg_sqs)]
    n = len(lists[0])
    lists += [list(ts) if ts is not None else [None] * n for ts in (m_scales, v_scales, copies)]
    if any(len(ts) != n for ts in lists):
        _fail("the lists must have as many tensors as params")
    numels = [p.numel() for p in lists[0]]
    state = torch.uint8 if eight else torch.float32
    at = torch._C._cuda_getDevice() if n else -1
    blocks = [(k + 127) // 128 for k in numels]
    cls = torch.Tensor
    # (hundreds of tensors: every attribute is read in a loop of the interpreter's own)
    for ts, kinds, sizes, what in ((lists[0], _TYPES, numels, "params"), (lists[1], _TYPES, numels, "grads"),
                                   (lists[2], (state,), numels, "exp_avgs"), (lists[3], (state,), numels, "exp_avg_sqs"),
                                   (lists[4], (torch.uint8,), blocks, "m_scales"),
                                   (lists[5], (torch.uint8,), blocks, "v_scales"),
                                   (lists[6], (torch.bfloat16, torch.float16), numels, "copies")):
        if any(t is None for t in ts):
            if what == "copies" or not eight and what in ("m_scales", "v_scales"):
                ts, sizes = [t for t in ts if t is not None], [k for t, k in zip(ts, sizes) if t is not None]
            else:
                _fail(f"{what} must not hold None")
        if not set(map(operator.attrgetter("dtype"), ts)) <= set(kinds):
            _fail(f"{what} must be of {list(kinds)}")
        if list(map(cls.numel, ts)) != sizes:
            _fail(f"{what} must match params in size" + (" (a byte for each 128 elements)" if sizes is blocks else ""))
        if not (all(map(cls.is_contiguous, ts)) and set(map(cls.get_device, ts)) <= {at}):
            _fail(f"{what} must be contiguous and on the current device")
    ptr = [array.array("Q", [0 if t is None else t.data_ptr() for t in ts]) for ts in lists]
    typ = [array.array("i", [0 if t is None else _TYPES[t.dtype] for t in lists[i]]) for i in (0, 1, 6)]
    wide = [[4 if k == 0 else 2 for k in ks] for ks in typ[:2]]
    one = 1 if eight else 4
    ends = [list(map(operator.add, ps, map(operator.mul, ks, ws)))
            for ps, ks, ws in ((ptr[0], numels, wide[0]), (ptr[1], numels, wide[1]), (ptr[2], numels, [one] * n),
                               (ptr[3], numels, [one] * n), (ptr[4], blocks, [1 if eight else 0] * n),
                               (ptr[5], blocks, [1 if eight else 0] * n),
                               (ptr[6], numels, [2 if p else 0 for p in ptr[6]]))]
    if _overlapping(itertools.chain(*ptr[:1], *ptr[2:]), itertools.chain(*ends[:1], *ends[2:]), zip(ptr[1], ends[1])):
        _fail("a tensor that the step writes overlaps another tensor of the list")
    out = AdamwTensors()
    # (the memory, whatever becomes of the tensors)
    out.held = [[t.untyped_storage() for t in ts if t is not None] for ts in lists]
    out.lists = (ptr[0], typ[0], ptr[1], typ[1], ptr[2], ptr[3], ptr[4] if eight else (), ptr[5] if eight else (),
                 ptr[6] if copies is not None else (), typ[2], array.array("q", numels))
    out.n = n
    out.device = at
    out.table, out.streams = None, None
    # (a list that one launch takes by value has no use for it; a step that is captured takes that way)
    if n > 52 and not torch.cuda.is_current_stream_capturing():
        size = ctypes.c_size_t(0)
        _check(load().adamw_table_size(n, ctypes.byref(size)), "adamw_table_size")
        table = torch.empty(size.value, dtype=torch.uint8)
        st = load().adamw_table(*map(_at, out.lists), n, table.data_ptr())
        if st == 0:                          # (refused here: the step refuses it too, or does without)
            out.table = table.to(f"cuda:{at}")
            out.streams = {_current_stream()}
    return out


def adamw_step(tensors, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, sumsq=None, max_norm=0.0,
               norm=None, seed=0, stream=None):
    """One AdamW step over `tensors` (adamw_tensors), in place.

    step: the step's number, from 1 on, and lr: numbers, or device tensors of one
    element (int64, float32), which a captured graph reads again at each replay.
    sumsq (float64 device tensor of one element, grad_norm_sq's): the gradients are
    clipped to max_norm within the step, norm (float32, one element, or None) is
    written, and a sum that is infinite or NaN leaves the step out. seed: of the
    8-bit states' rounding. stream: a torch stream or a handle; on one that torch did
    not make (or whose handle alone is given, unless it is the current or default
    stream's) a long list goes by value, so that nothing has to outlive the call."""
    if tensors.n and tensors.device != _torch()._C._cuda_getDevice():
        _fail("the tensors are not on the current device")
    torch = _torch()
    sp = lp = step_at = lr_at = None
    if isinstance(step, torch.Tensor):
        step_at = step
        sp, step = _out(step, (1,) if step.dim() else (), torch.int64, "step"), 1
    if isinstance(lr, torch.Tensor):
        lr_at = lr
        lp, lr = _out(lr, (1,) if lr.dim() else (), torch.float32, "lr"), 0.0
    total = None if sumsq is None else _out(sumsq, (1,), torch.float64, "sumsq")
    nrm = None if norm is None else _out(norm, (1,), torch.float32, "norm")
    _one_device(step_at, lr_at, sumsq, norm)
    on, table = _stream(stream), tensors.table
    if table is not None:
        if on in tensors.streams:
            table = table.data_ptr()
        else:
            own = _torchs_stream(stream, on)
            if own is None:                  # (nothing is kept until a foreign stream is done: the list by value)
                table = None
            else:                            # (its memory is not used again before the steps there are done)
                table.record_stream(own)
                tensors.streams.add(on)
                table = table.data_ptr()
    st = load().adamw_step(*map(_at, tensors.lists), tensors.n, sp, step, lp, lr, beta1, beta2, eps, weight_decay,
                           total, max_norm, nrm, seed & 0xFFFFFFFF, table, on)
    if st:
        _check(st, "adamw_step")


def _one_device(*ts):
    """The calls below launch on the current device, whose memory the tensors
    have to be (None: not given)."""
    at = _torch()._C._cuda_getDevice()
    for t in ts:
        if t is not None and t.get_device() != at:
            _fail(f"tensors must live on the current device (cuda:{at})")


def int8_quantize(x, q, scales, stream=None):
    """x [rows][cols] (float32, bfloat16 or float16; rows may be strided) ->
    q int8 [rows][cols] (rows may be strided) and scales float32 [rows]: one
    scale a row, amax / 127. For activations rows are tokens, for weights
    [N][K] output channels."""
    torch = _torch()
    xp, rows, cols, ldx = _rows(x, "x")
    qp, qrows, qcols, ldq = _rows(q, "q")
    typ = _TYPES.get(x.dtype)
    if typ is None:
        _fail("x must be float32, bfloat16 or float16")
    if q.dtype is not torch.int8 or qrows != rows or qcols != cols:
        _fail("q must be int8 of x's shape")
    sp = _out(scales, (rows,), torch.float32, "scales")
    _one_device(x, q, scales)
    st = load().int8_quantize(xp, typ, rows, cols, ldx, qp, ldq, sp, _stream(stream))
    if st:
        _check(st, "int8_quantize")


def _int8_args(a, sa, b, sb, d, rows, weights, group, groups):
    """Pointers of an integer product's operands: a and d with the row shape
    `rows`, b and sb with the leading shape `weights`."""
    torch = _torch()
    K, N = a.shape[-1], b.shape[-2]
    i8, f32 = torch.int8, torch.float32
    dt = d.dtype
    if dt is not torch.bfloat16 and dt is not torch.int16 and dt is not torch.uint16:
        _fail("d must hold bf16 values (bfloat16, or int16/uint16 bit patterns)")
    ptrs = [_out(a, rows + (K,), i8, "a"), _out(sa, rows, f32, "sa"), _out(b, weights + (N, K), i8, "b"),
            _out(sb, weights + (N,), f32, "sb"), _out(d, rows + (N,), dt, "d")]
    _one_device(a, sa, b, sb, d)
    if group is not None:
        ptrs.append(_out(group, (groups,), torch.int32, "group metadata"))
        _one_device(group)
    return ptrs, N, K


def gemm_int8(a, sa, b, sb, d, stream=None):
    """a int8 [M][K], sa float32 [M], b int8 [N][K], sb float32 [N], d bf16
    (int16/bfloat16) [M][N]: the exact integer product times both scales."""
    if a.dim() != 2 or b.dim() != 2:
        _fail("a and b must be matrices")
    M = a.shape[0]
    ptrs, N, K = _int8_args(a, sa, b, sb, d, (M,), (), None, 0)
    st = load().gemm_int8(*ptrs, M, N, K, _stream(stream))
    if st:
        _check(st, "gemm_int8")


def grouped_gemm_int8_contiguous(a, sa, b, sb, d, group_offsets, stream=None):
    """a int8 [M_total][K], sa float32 [M_total], b int8 [G][N][K], sb float32
    [G][N], d [M_total][N], group_offsets int32 [G+1] (device; any
    non-decreasing rows). Rows of no expert are left as they were."""
    if a.dim() != 2 or b.dim() != 3:
        _fail("a must be [M_total][K] and b [G][N][K]")
    M, G = a.shape[0], b.shape[0]
    ptrs, N, K = _int8_args(a, sa, b, sb, d, (M,), (G,), group_offsets, G + 1)
    st = load().grouped_gemm_int8_contiguous(*ptrs, G, M, N, K, _stream(stream))
    if st:
        _check(st, "grouped_gemm_int8_contiguous")


def grouped_gemm_int8_masked(a, sa, b, sb, d, masked_m, expected_m=0, stream=None):
    """a int8 [G][max_m][K], sa float32 [G][max_m], b int8 [G][N][K], sb
    float32 [G][N], d [G][max_m][N], masked_m int32 [G] (device)."""
    if a.dim() != 3 or b.dim() != 3:
        _fail("a must be [G][max_m][K] and b [G][N][K]")
    G, max_m = a.shape[0], a.shape[1]
    ptrs, N, K = _int8_args(a, sa, b, sb, d, (G, max_m), (G,), masked_m, G)
    st = load().grouped_gemm_int8_masked(*ptrs, G, max_m, N, K, int(expected_m), _stream(stream))
    if st:
        _check(st, "grouped_gemm_int8_masked")


def fp8g_clock_probe(out, ticks=2000, stream=None):
    """Enqueue the clock probe: out is a device int64 tensor of >= 2 elements;
    afterwards out[0] / out[1] * 1e8 is the shader clock in Hz."""
    import torch
    _need(out.dtype == torch.int64 and out.numel() >= 2, "out must be int64 with 2 elements")
    _dev(out)
    _check(load().fp8g_clock_probe(_ptr(out), int(ticks), _stream(stream)), "fp8g_clock_probe")


def fp8g_warmup():
    """Load every kernel's code object onto the current device (host-side,
    synchronous; launches and allocates nothing)."""
    _check(load().fp8g_warmup(), "fp8g_warmup")


def fp8g_set_shape_specialisation(enable):
    """Switch the shape-specialised kernels on (default) or off process-wide;
    results are bit-identical either way."""
    _check(load().fp8g_set_shape_specialisation(1 if enable else 0),
           "fp8g_set_shape_specialisation")


def fp8g_gemm_kernel_name(layout, rows, N, K, G=1, expected_m=0, quant=False):
    """The kernel a GEMM call of this shape launches. layout: 'dense',
    'contiguous', 'masked' or 'pertensor'; rows: M, M_total or max_m."""
    _need(layout in LAYOUTS, f"layout must be one of {sorted(LAYOUTS)}")
    buf = ctypes.create_string_buffer(256)
    _check(load().fp8g_gemm_kernel_name(LAYOUTS[layout], int(rows), int(N), int(K), int(G),
                                        int(expected_m), 1 if quant else 0, buf, len(buf)),
           "fp8g_gemm_kernel_name")
    return buf.value.decode()
