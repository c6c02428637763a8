"""ctypes binding of libnvfp4.so with the C ABI's names (include/nvfp4.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams.  If the library is not
built, importing this module raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import functools
import operator
import os
from dataclasses import dataclass, field

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libnvfp4.so")

# status codes
OK, ERR_INVALID_ARG, ERR_SHAPE, ERR_ALIGN, ERR_ARCH, ERR_WORKSPACE, ERR_CUDA, \
    ERR_DEVICE_TIMEOUT = range(8)
# enums and flags
IN_BF16, IN_FP32 = 0, 1
ROW_1X16, COL_1X16, BLOCK_16X16 = 0, 1, 2
RHT, SR, EMIT_T, AMAX_GIVEN, OFFSET_DEVICE = 1, 2, 4, 8, 32
D_BF16, D_F32_ACCUM, D_BF16_ADD_C = 0, 1, 2
MXFP4, MXFP8 = 0, 1
MX_ROW, MX_COL = 0, 1
(TILE_AUTO, TILE_128X128, TILE_128X256, TILE_PAIR_256X256, TILE_128X256_K128,
 TILE_PAIR_256X384) = 0, 1, 2, 3, 5, 6


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


class Tensor(C.Structure):
    """Mirror of ``nvfp4_tensor``."""
    _fields_ = [("codes", C.c_void_p), ("scales", C.c_void_p), ("codes_t", C.c_void_p),
                ("scales_t", C.c_void_p), ("amax", C.c_void_p), ("s_dec", C.c_void_p),
                ("rows", C.c_int64), ("cols", C.c_int64), ("mode", C.c_int32),
                ("flags", C.c_uint32)]


class NormParams(C.Structure):
    """Mirror of ``nvfp4_norm_params``."""
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("stream_dtype", C.c_int32),
                ("gate_mode", C.c_int32), ("eps", C.c_float), ("x_scale", C.c_float),
                ("z_scale", C.c_float)]


class RouteParams(C.Structure):
    """Mirror of ``nvfp4_route_params``."""
    _fields_ = [("tokens", C.c_int64), ("experts", C.c_int64), ("ld", C.c_int64),
                ("in_dtype", C.c_int32), ("top", C.c_int32), ("score", C.c_int32),
                ("renormalise", C.c_int32), ("groups", C.c_int32), ("groups_kept", C.c_int32),
                ("group_top", C.c_int32), ("scale", C.c_float)]


class MuonParams(C.Structure):
    """Mirror of ``nvfp4_muon_params``."""
    _fields_ = [("batch", C.c_int64), ("rows", C.c_int64), ("cols", C.c_int64),
                ("grad_dtype", C.c_int32), ("nesterov", C.c_int32), ("steps", C.c_int32),
                ("mu", C.c_float), ("eps", C.c_float), ("coefs", C.POINTER(C.c_float))]


class MlpParams(C.Structure):
    """Mirror of ``nvfp4_mlp_params``."""
    _fields_ = [("M", C.c_int64), ("D", C.c_int64), ("F", C.c_int64), ("Wg", C.c_void_p),
                ("Wu", C.c_void_p), ("Wd", C.c_void_p), ("seed", C.c_uint64),
                ("step", C.c_uint64), ("flags", C.c_uint32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -c 'import __graft_entry__ as g; g.build()'`")
    L = C.CDLL(LIB_PATH)
    i32, i64, u32, u64, vp, sz = C.c_int32, C.c_int64, C.c_uint32, C.c_uint64, C.c_void_p, C.c_size_t
    P = C.POINTER
    sigs = {
        "nvfp4_status_string": ([C.c_int], C.c_char_p),
        "nvfp4_version": ([], C.c_int),
        "nvfp4_device_check": ([C.c_int], C.c_int),
        "nvfp4_check_device_errors": ([vp], C.c_int),
        "nvfp4_debug_inject": ([u32, u64], C.c_int),
        "nvfp4_quantize_sizes": ([i64, i64, i32, u32, P(sz), P(sz), P(sz), P(sz)], C.c_int),
        "nvfp4_quantize": ([vp, i32, i64, i64, i64, i32, u32, u64, u64, P(Tensor), vp, sz, vp],
                           C.c_int),
        "nvfp4_quantize_noalloc": ([vp, i32, i64, i64, i64, i32, u32, u64, u64, P(Tensor), vp],
                                   C.c_int),
        "nvfp4_amax": ([vp, i32, i64, i64, i64, u64, vp, vp, vp, sz, vp], C.c_int),
        "nvfp4_quantize_rowcol": ([vp, i32, i64, i64, i64, u32, u32, u64, u64, u64, P(Tensor),
                                   P(Tensor), vp], C.c_int),
        "nvfp4_gemm": ([P(Tensor), i32, P(Tensor), i32, vp, i32, vp, i64, i64, i64, vp, sz, vp],
                       C.c_int),
        "nvfp4_gemm_ex": ([P(Tensor), i32, P(Tensor), i32, vp, i32, vp, i64, i64, i64, i32, vp],
                          C.c_int),
        "nvfp4_mx_sizes": ([i64, i64, i32, i32, P(sz), P(sz), P(sz)], C.c_int),
        "nvfp4_mx_quantize": ([vp, i32, i64, i64, i64, i32, i32, vp, vp, vp, vp], C.c_int),
        "nvfp4_mx_gemm": ([vp, vp, vp, vp, i32, vp, i64, i64, i64, vp], C.c_int),
        "nvfp4_swiglu_workspace_bytes": ([], sz),
        "nvfp4_swiglu_fwd": ([vp, vp, vp, i64, i64, u32, u64, vp, vp, vp, sz, vp], C.c_int),
        "nvfp4_swiglu_bwd": ([vp, vp, vp, vp, vp, i64, i64, u32, u64, vp, vp, vp, vp, vp, sz, vp],
                             C.c_int),
        "nvfp4_mlp_sizes": ([i64, i64, i64, P(sz), P(sz)], C.c_int),
        "nvfp4_mlp_fwd": ([P(MlpParams), vp, vp, vp, sz, vp, sz, vp], C.c_int),
        "nvfp4_mlp_bwd": ([P(MlpParams), vp, vp, vp, vp, vp, vp, vp, sz, vp], C.c_int),
        "nvfp4_mlp_tensor": ([i64, i64, i64, vp, vp, i32, P(vp), P(i64), P(i64)], C.c_int),
        "nvfp4_mlp_operand": ([i64, i64, i64, vp, vp, i32, P(Tensor)], C.c_int),
        "nvfp4_sgd_step": ([vp, vp, i64, C.c_float, u32, vp, vp, sz, vp], C.c_int),
        "nvfp4_muon_sizes": ([i64, i64, i64, P(sz)], C.c_int),
        "nvfp4_muon_update": ([P(MuonParams), vp, vp, vp, u32, vp, sz, vp], C.c_int),
        "nvfp4_muon_apply": ([vp, vp, i64, C.c_float, C.c_float, C.c_float, vp, vp, sz, vp],
                             C.c_int),
        "nvfp4_route_sizes": ([i64, i64, i32, P(i64), P(sz)], C.c_int),
        "nvfp4_route_fwd": ([vp, i32, i64, i64, i64, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp],
                            C.c_int),
        "nvfp4_route_bwd": ([vp, i32, i64, i64, i64, i32, i32, vp, vp, vp, vp, vp], C.c_int),
        "nvfp4_route_scored_fwd": ([P(RouteParams), vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
                                   C.c_int),
        "nvfp4_route_scored_bwd": ([P(RouteParams), vp, vp, vp, vp, vp, vp], C.c_int),
        "nvfp4_route_balance": ([vp, i64, C.c_float, vp, vp], C.c_int),
        "nvfp4_dispatch": ([vp, vp, vp, i64, i64, i32, i64, vp, vp], C.c_int),
        "nvfp4_combine": ([vp, vp, vp, i64, i64, i32, i64, vp, vp], C.c_int),
        "nvfp4_combine_bwd": ([vp, vp, vp, vp, vp, i64, i64, i32, i64, vp, vp, vp], C.c_int),
        "nvfp4_group_gemm": ([P(Tensor), P(Tensor), i32, vp, vp, i32, vp, i32, vp, i64, i64, i64,
                              i32, vp], C.c_int),
        "nvfp4_group_wgrad": ([P(Tensor), P(Tensor), vp, vp, i32, vp, i32, i64, i64, i64, i32, vp],
                              C.c_int),
        "nvfp4_residual_norm_fwd": ([P(NormParams), vp, vp, vp, vp, vp, vp, vp, vp], C.c_int),
        "nvfp4_residual_norm_bwd_sizes": ([i64, i64, P(sz)], C.c_int),
        "nvfp4_residual_norm_bwd": ([P(NormParams), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                     vp, sz, vp], C.c_int),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    return L


lib = _load()


def status_string(s: int) -> str:
    return lib.nvfp4_status_string(s).decode()


def _check(status: int, where: str):
    if status != OK:
        raise NVFP4Error(status, where)


def _stream(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


@dataclass
class QTensor:
    """A quantised operand: the device buffers plus the ABI descriptor."""
    codes: torch.Tensor
    scales: torch.Tensor
    amax: torch.Tensor
    s_dec: torch.Tensor
    codes_t: torch.Tensor | None = None
    scales_t: torch.Tensor | None = None
    desc: Tensor = field(default_factory=Tensor)

    @property
    def rows(self):
        return self.desc.rows

    @property
    def cols(self):
        return self.desc.cols


def quantize_sizes(rows, cols, mode, flags=0):
    c, s, st, w = C.c_size_t(), C.c_size_t(), C.c_size_t(), C.c_size_t()
    _check(lib.nvfp4_quantize_sizes(rows, cols, mode, flags, C.byref(c), C.byref(s), C.byref(st),
                                    C.byref(w)), "nvfp4_quantize_sizes")
    return c.value, s.value, st.value, w.value


def alloc_qtensor(rows, cols, mode, flags=0, device="cuda") -> QTensor:
    """Allocate the output buffers of quantising an input [rows, cols]."""
    cb, sb, stb, _ = quantize_sizes(rows, cols, mode, flags)
    u8 = dict(dtype=torch.uint8, device=device)
    q = QTensor(codes=torch.empty(cb, **u8), scales=torch.empty(sb, **u8),
                amax=torch.zeros(1, dtype=torch.float32, device=device),
                s_dec=torch.zeros(1, dtype=torch.float32, device=device))
    if flags & EMIT_T:
        q.codes_t = torch.empty(cb, **u8)
        q.scales_t = torch.empty(stb, **u8)
    d = q.desc
    d.codes, d.scales = q.codes.data_ptr(), q.scales.data_ptr()
    d.codes_t, d.scales_t = _ptr(q.codes_t), _ptr(q.scales_t)
    d.amax, d.s_dec = q.amax.data_ptr(), q.s_dec.data_ptr()
    return q


_ws_cache: dict = {}


def _workspace(nbytes, device):
    key = (str(device), torch.cuda.current_stream().cuda_stream)
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


def _offset(flags: int, offset: int | torch.Tensor):
    """Flags and offset argument of a quantiser: a number, or a device counter."""
    if not isinstance(offset, torch.Tensor):
        return flags, offset
    if not (offset.is_cuda and offset.dtype is torch.int64 and offset.numel() == 1):
        raise ValueError("a device offset must be a 1-element int64 CUDA tensor")
    return flags | OFFSET_DEVICE, offset.data_ptr()


def nvfp4_quantize(x: torch.Tensor, mode: int, flags: int = 0, seed: int = 0,
                   offset: int | torch.Tensor = 0, out: QTensor | None = None,
                   workspace: torch.Tensor | None = None,
                   amax: float | torch.Tensor | None = None, stream=None) -> QTensor:
    """Quantise a 2-D bf16/fp32 CUDA tensor (see nvfp4_quantize in nvfp4.h).  An
    `offset` on the device (a 1-element int64 tensor) is read when the kernel
    runs, so that replays of a captured graph need not repeat its rounding."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D tensor with unit column stride")
    if x.dtype == torch.bfloat16:
        dt = IN_BF16
    elif x.dtype == torch.float32:
        dt = IN_FP32
    else:
        raise TypeError(f"x must be bf16 or fp32, got {x.dtype}")
    rows, cols = x.shape
    if amax is not None:
        flags |= AMAX_GIVEN
    if out is None:
        out = alloc_qtensor(rows, cols, mode, flags, device=x.device)
    if amax is not None:
        out.amax.copy_(torch.as_tensor(amax, dtype=torch.float32).reshape(1))
    _, _, _, wsb = quantize_sizes(rows, cols, mode, flags)
    if workspace is None and wsb:
        workspace = _workspace(wsb, x.device)
    flags, offset = _offset(flags, offset)
    _check(lib.nvfp4_quantize(x.data_ptr(), dt, rows, cols, x.stride(0), mode, flags, seed, offset,
                              C.byref(out.desc), _ptr(workspace),
                              0 if workspace is None else workspace.numel(), _stream(stream)),
           "nvfp4_quantize")
    return out


def nvfp4_amax(x: torch.Tensor, amax_plain: torch.Tensor | None = None,
               amax_rht: torch.Tensor | None = None, seed: int = 0,
               workspace: torch.Tensor | None = None, stream=None):
    """max |x| and/or max |RHT(x)| along columns from one read (see nvfp4_amax
    in nvfp4.h); the outputs are 1-element float32 CUDA tensors, e.g. the
    `amax` of the QTensors then quantised with NVFP4_AMAX_GIVEN."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D tensor with unit column stride")
    dt = {torch.bfloat16: IN_BF16, torch.float32: IN_FP32}.get(x.dtype)
    if dt is None:
        raise TypeError(f"x must be bf16 or fp32, got {x.dtype}")
    for t in (amax_plain, amax_rht):
        if t is not None and (t.dtype != torch.float32 or t.numel() != 1 or not t.is_cuda):
            raise ValueError("amax outputs must be 1-element float32 CUDA tensors")
    rows, cols = x.shape
    if workspace is None:  # the partial-maxima workspace does not depend on the shape
        workspace = _workspace(quantize_sizes(128, 128, ROW_1X16)[3], x.device)
    _check(lib.nvfp4_amax(x.data_ptr(), dt, rows, cols, x.stride(0), seed, _ptr(amax_plain),
                          _ptr(amax_rht), _ptr(workspace), workspace.numel(), _stream(stream)),
           "nvfp4_amax")


def nvfp4_quantize_rowcol(x: torch.Tensor, row_flags: int = 0, col_flags: int = 0, seed: int = 0,
                          row_offset: int | torch.Tensor = 0,
                          col_offset: int | torch.Tensor = 0,
                          row_out: QTensor | None = None, col_out: QTensor | None = None,
                          amax_row: torch.Tensor | None = None, amax_col: torch.Tensor | None = None,
                          stream=None):
    """Row-wise and column-wise quantisation of a bf16 x from one read (see
    nvfp4_quantize_rowcol in nvfp4.h).  The two amaxes are given: either
    already in row_out.amax / col_out.amax, or as 1-element float32 CUDA
    tensors amax_row / amax_col (copied there).  The offsets may be on the
    device, as nvfp4_quantize's.  Returns (row_out, col_out)."""
    if x.dim() != 2 or x.stride(1) != 1 or x.dtype != torch.bfloat16:
        raise ValueError("x must be a 2-D bf16 tensor with unit column stride")
    rows, cols = x.shape
    row_flags |= AMAX_GIVEN
    col_flags |= AMAX_GIVEN
    if row_out is None:
        row_out = alloc_qtensor(rows, cols, ROW_1X16, device=x.device)
    if col_out is None:
        col_out = alloc_qtensor(rows, cols, COL_1X16, device=x.device)
    if amax_row is not None:
        row_out.amax.copy_(amax_row.reshape(1))
    if amax_col is not None:
        col_out.amax.copy_(amax_col.reshape(1))
    row_flags, row_offset = _offset(row_flags, row_offset)
    col_flags, col_offset = _offset(col_flags, col_offset)
    _check(lib.nvfp4_quantize_rowcol(x.data_ptr(), IN_BF16, rows, cols, x.stride(0), row_flags,
                                     col_flags, seed, row_offset, col_offset, C.byref(row_out.desc),
                                     C.byref(col_out.desc), _stream(stream)),
           "nvfp4_quantize_rowcol")
    return row_out, col_out


def nvfp4_quantize_noalloc(x: torch.Tensor, mode: int, flags: int = 0, seed: int = 0,
                           offset: int | torch.Tensor = 0, out: QTensor | None = None, stream=None) -> QTensor:
    """nvfp4_quantize without a workspace: scratch lives inside the library
    (see nvfp4_quantize_noalloc in nvfp4.h for who needs this and its limits)."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D tensor with unit column stride")
    dt = {torch.bfloat16: IN_BF16, torch.float32: IN_FP32}.get(x.dtype)
    if dt is None:
        raise TypeError(f"x must be bf16 or fp32, got {x.dtype}")
    rows, cols = x.shape
    if out is None:
        out = alloc_qtensor(rows, cols, mode, flags, device=x.device)
    flags, offset = _offset(flags, offset)
    _check(lib.nvfp4_quantize_noalloc(x.data_ptr(), dt, rows, cols, x.stride(0), mode, flags, seed,
                                      offset, C.byref(out.desc), _stream(stream)),
           "nvfp4_quantize_noalloc")
    return out


def mx_sizes(rows, cols, mode, fmt):
    """(codes, scales, scales in the MMA layout) byte sizes."""
    c, s, w = C.c_size_t(), C.c_size_t(), C.c_size_t()
    _check(lib.nvfp4_mx_sizes(rows, cols, mode, fmt, C.byref(c), C.byref(s), C.byref(w)),
           "nvfp4_mx_sizes")
    return c.value, s.value, w.value


def nvfp4_mx_quantize(x: torch.Tensor, mode: int, fmt: int, codes: torch.Tensor | None = None,
                      scales: torch.Tensor | None = None, scales_sw: torch.Tensor | None = None,
                      stream=None):
    """MXFP4 / MXFP8 quantisation of a 2-D bf16/fp32 CUDA tensor (see
    nvfp4_mx_quantize in nvfp4.h); returns (codes, scales) as uint8 tensors
    shaped [out_rows, out_cols/2 or out_cols] and [out_rows, out_cols/32].
    ``scales_sw`` (optional, uint8, mx_sizes()[2] bytes) also receives the
    scales in the MMA layout nvfp4_mx_gemm reads."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D tensor with unit column stride")
    dt = {torch.bfloat16: IN_BF16, torch.float32: IN_FP32}.get(x.dtype)
    if dt is None:
        raise TypeError(f"x must be bf16 or fp32, got {x.dtype}")
    rows, cols = x.shape
    orows, ocols = (cols, rows) if mode == MX_COL else (rows, cols)
    cb, sb, swb = mx_sizes(rows, cols, mode, fmt)
    if codes is None:
        codes = torch.empty(orows, cb // orows, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(orows, sb // orows, dtype=torch.uint8, device=x.device)
    if codes.numel() < cb or scales.numel() < sb or (scales_sw is not None and
                                                     scales_sw.numel() < swb):
        raise ValueError("output buffers are smaller than nvfp4_mx_sizes gives")
    _check(lib.nvfp4_mx_quantize(x.data_ptr(), dt, rows, cols, x.stride(0), mode, fmt,
                                 codes.data_ptr(), scales.data_ptr(), _ptr(scales_sw),
                                 _stream(stream)),
           "nvfp4_mx_quantize")
    return codes, scales


def nvfp4_mx_gemm(a_codes: torch.Tensor, a_scales_sw: torch.Tensor, b_codes: torch.Tensor,
                  b_scales_sw: torch.Tensor, fmt: int, M: int, N: int, K: int,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """D bf16 [M, N] = A . B^T for MX operands (see nvfp4_mx_gemm in nvfp4.h)."""
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a_codes.device)
    _check(lib.nvfp4_mx_gemm(a_codes.data_ptr(), a_scales_sw.data_ptr(), b_codes.data_ptr(),
                             b_scales_sw.data_ptr(), fmt, out.data_ptr(), M, N, K,
                             _stream(stream)), "nvfp4_mx_gemm")
    return out


def nvfp4_gemm(A: QTensor, B: QTensor, a_view: int = 0, b_view: int = 0,
               out: torch.Tensor | None = None, d_mode: int = D_BF16,
               C_add: torch.Tensor | None = None, tile: int = TILE_AUTO, stream=None) -> torch.Tensor:
    """D = alpha * A . B^T (see nvfp4_gemm in nvfp4.h); returns D."""
    M = A.desc.cols if a_view else A.desc.rows
    K = A.desc.rows if a_view else A.desc.cols
    N = B.desc.cols if b_view else B.desc.rows
    if out is None:
        dtype = torch.float32 if d_mode == D_F32_ACCUM else torch.bfloat16
        out = (torch.zeros if d_mode == D_F32_ACCUM else torch.empty)(
            (M, N), dtype=dtype, device=A.codes.device)
    if tile:
        st = lib.nvfp4_gemm_ex(C.byref(A.desc), a_view, C.byref(B.desc), b_view, out.data_ptr(),
                               d_mode, _ptr(C_add), M, N, K, tile, _stream(stream))
    else:
        st = lib.nvfp4_gemm(C.byref(A.desc), a_view, C.byref(B.desc), b_view, out.data_ptr(),
                            d_mode, _ptr(C_add), M, N, K, None, 0, _stream(stream))
    _check(st, "nvfp4_gemm")
    return out


def _bf16_2d(*ts):
    for t in ts:
        if t.dtype != torch.bfloat16 or t.dim() != 2 or not t.is_contiguous() or not t.is_cuda:
            raise ValueError("SwiGLU tensors must be contiguous 2-D bf16 CUDA tensors")
        if t.shape != ts[0].shape:
            raise ValueError("SwiGLU tensors must have one shape")


def _amax_outs(n, device):
    return [torch.zeros(1, dtype=torch.float32, device=device) for _ in range(n)]


def nvfp4_swiglu_fwd(G, U, rht=True, seed=0, H=None, workspace=None, stream=None):
    """H = silu(G) * U with the amaxes of H's row-wise and column-wise (RHT)
    quantisations (see nvfp4_swiglu_fwd in nvfp4.h); returns
    (H, amax_row, amax_col), the amaxes as 1-element float32 CUDA tensors."""
    H = torch.empty_like(G) if H is None else H
    _bf16_2d(G, U, H)
    rows, cols = G.shape
    if workspace is None:
        workspace = _workspace(lib.nvfp4_swiglu_workspace_bytes(), G.device)
    a_row, a_col = _amax_outs(2, G.device)
    _check(lib.nvfp4_swiglu_fwd(G.data_ptr(), U.data_ptr(), H.data_ptr(), rows, cols,
                                RHT if rht else 0, seed, a_row.data_ptr(), a_col.data_ptr(),
                                workspace.data_ptr(), workspace.numel(), _stream(stream)),
           "nvfp4_swiglu_fwd")
    return H, a_row, a_col


def nvfp4_swiglu_bwd(dH, G, U, rht=True, seed=0, workspace=None, stream=None):
    """dG, dU of the SwiGLU with the amaxes of their row-wise and column-wise
    quantisations; returns (dG, dU, amax_dg_row, amax_dg_col, amax_du_row,
    amax_du_col)."""
    dG, dU = torch.empty_like(G), torch.empty_like(G)
    _bf16_2d(dH, G, U, dG, dU)
    rows, cols = G.shape
    if workspace is None:
        workspace = _workspace(lib.nvfp4_swiglu_workspace_bytes(), G.device)
    a = _amax_outs(4, G.device)
    _check(lib.nvfp4_swiglu_bwd(dH.data_ptr(), G.data_ptr(), U.data_ptr(), dG.data_ptr(),
                                dU.data_ptr(), rows, cols, RHT if rht else 0, seed,
                                *(t.data_ptr() for t in a), workspace.data_ptr(),
                                workspace.numel(), _stream(stream)), "nvfp4_swiglu_bwd")
    return (dG, dU, *a)


def mlp_sizes(M, D, F):
    s, w = C.c_size_t(), C.c_size_t()
    _check(lib.nvfp4_mlp_sizes(M, D, F, C.byref(s), C.byref(w)), "nvfp4_mlp_sizes")
    return s.value, w.value


def mlp_params(M, D, F, Wg, Wu, Wd, seed=0, step=0, rht=True,
               weight_amax_given=False) -> MlpParams:
    return MlpParams(M, D, F, Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(), seed, step,
                     (RHT if rht else 0) | (AMAX_GIVEN if weight_amax_given else 0))


def nvfp4_mlp_fwd(p: MlpParams, X, Y, saved, workspace, stream=None):
    _check(lib.nvfp4_mlp_fwd(C.byref(p), X.data_ptr(), Y.data_ptr(), saved.data_ptr(),
                             saved.numel(), workspace.data_ptr(), workspace.numel(),
                             _stream(stream)), "nvfp4_mlp_fwd")
    return Y


def nvfp4_mlp_bwd(p: MlpParams, dY, saved, dX, dWg, dWu, dWd, workspace, stream=None):
    _check(lib.nvfp4_mlp_bwd(C.byref(p), dY.data_ptr(), saved.data_ptr(), dX.data_ptr(),
                             dWg.data_ptr(), dWu.data_ptr(), dWd.data_ptr(), workspace.data_ptr(),
                             workspace.numel(), _stream(stream)), "nvfp4_mlp_bwd")
    return dX


# intermediates of an MLP step inside the saved / workspace buffers
MLP_G, MLP_U, MLP_H, MLP_DH, MLP_DG, MLP_DU, MLP_DX_GATE = range(7)
(MLP_Q_WG, MLP_Q_WU, MLP_Q_WD, MLP_Q_X, MLP_Q_XC, MLP_Q_H, MLP_Q_HC, MLP_Q_DY, MLP_Q_DYC,
 MLP_Q_DG, MLP_Q_DGC, MLP_Q_DU, MLP_Q_DUC) = range(16, 29)


def _slice_of(ptr, nbytes, bufs):
    """The bytes [ptr, ptr + nbytes) as a uint8 view of whichever buffer holds them."""
    for b in bufs:
        if b is not None and b.data_ptr() <= ptr and ptr + nbytes <= b.data_ptr() + b.numel():
            off = ptr - b.data_ptr()
            return b[off:off + nbytes]
    raise ValueError("address outside the given buffers")


def mlp_tensor(M, D, F, saved, workspace, which) -> torch.Tensor:
    """The bf16 intermediate `which` (MLP_G ... MLP_DX_GATE) of the last MLP
    call, as a [rows, cols] view into saved / workspace (nvfp4_mlp_tensor)."""
    p, r, c = C.c_void_p(), C.c_int64(), C.c_int64()
    _check(lib.nvfp4_mlp_tensor(M, D, F, _ptr(saved), _ptr(workspace), which, C.byref(p),
                                C.byref(r), C.byref(c)), "nvfp4_mlp_tensor")
    raw = _slice_of(p.value, r.value * c.value * 2, (saved, workspace))
    return raw.view(torch.bfloat16).view(r.value, c.value)


def mlp_operand(M, D, F, saved, workspace, which) -> QTensor:
    """The quantised operand `which` (MLP_Q_*) of the last MLP call, as a
    QTensor whose tensors are views into saved / workspace (nvfp4_mlp_operand)."""
    d = Tensor()
    _check(lib.nvfp4_mlp_operand(M, D, F, _ptr(saved), _ptr(workspace), which, C.byref(d)),
           "nvfp4_mlp_operand")
    bufs = (saved, workspace)
    rows, cols = d.rows, d.cols
    # the operand's sizes: K-major [rows, cols] (the quantiser's ROW_1X16 form of the same shape)
    cb, sb, _, _ = quantize_sizes(rows, cols, ROW_1X16)
    q = QTensor(codes=_slice_of(d.codes, cb, bufs), scales=_slice_of(d.scales, sb, bufs),
                amax=_slice_of(d.amax, 4, bufs).view(torch.float32),
                s_dec=_slice_of(d.s_dec, 4, bufs).view(torch.float32), desc=d)
    if d.codes_t:
        cbt, sbt, _, _ = quantize_sizes(cols, rows, ROW_1X16)
        q.codes_t = _slice_of(d.codes_t, cbt, bufs)
        q.scales_t = _slice_of(d.scales_t, sbt, bufs)
    return q


ZERO_GRAD = 16


def _changed(*tensors):
    """Tells torch that a call wrote to tensors in place, as its own operations do
    (a weight's known amax goes by it, and autograd's check of what it saved)."""
    for t in tensors:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def nvfp4_sgd_step(W: torch.Tensor, G: torch.Tensor, lr: float, zero_grad: bool = False,
                   amax: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream=None):
    """W -= lr * G on FP32 master weight and gradient (G zeroed with
    zero_grad), writing max |W| of the updated weight into the 1-element
    float32 CUDA tensor `amax` when given (see nvfp4_sgd_step in nvfp4.h)."""
    for t in (W, G):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("W and G must be contiguous float32 CUDA tensors")
    if W.numel() != G.numel():
        raise ValueError("W and G must have the same number of elements")
    if amax is not None and (amax.dtype != torch.float32 or amax.numel() != 1 or not amax.is_cuda):
        raise ValueError("amax must be a 1-element float32 CUDA tensor")
    if amax is not None and workspace is None:
        workspace = _workspace(quantize_sizes(128, 128, ROW_1X16)[3], W.device)
    _check(lib.nvfp4_sgd_step(W.data_ptr(), G.data_ptr(), W.numel(), float(lr),
                              ZERO_GRAD if zero_grad else 0, _ptr(amax), _ptr(workspace),
                              workspace.numel() if workspace is not None else 0,
                              _stream(stream)), "nvfp4_sgd_step")
    _changed(W, G if zero_grad else None, amax)
    return W


# ---- mixture of experts ------------------------------------------------------
# These calls are made once per layer and token at a server, so their checks
# are kept to a few attribute reads, and messages are only built to be raised.
ROUTE_ALL, ROUTE_CHOSEN = 0, 1
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
GATE_NONE, GATE_CHANNEL, GATE_ROW = 0, 1, 2
_DTYPES = {torch.bfloat16: IN_BF16, torch.float32: IN_FP32}
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _cuda(t, dtype, name, shape=None):
    """Refuses what is not a contiguous CUDA tensor of one type (and shape)."""
    if not (t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor"
                         + ("" if shape is None else f" of shape {tuple(shape)}"))


def _current(t) -> int:
    """The current stream of a tensor's device, as a handle."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _on_stream(call):
    """Runs a call with its `stream` as the current one, so that what it
    allocates (outputs, a workspace) belongs to the stream that uses it."""
    @functools.wraps(call)
    def run(*args, stream=None, **kwargs):
        if stream is None:
            return call(*args, **kwargs)
        with torch.cuda.stream(stream):
            return call(*args, **kwargs)
    return run


def _scratch(nbytes, t):
    """A workspace of the current stream for one call.  It comes from the
    allocator each time: one that a later, larger call replaced would still be
    written by the graphs that captured it."""
    return torch.empty(max(nbytes, 16), dtype=_U8, device=t.device)


def _on_device(call):
    """As _on_stream, for a call whose first tensor may lie on another device
    than the current one: the call then runs there, on that device's current
    stream."""
    name = call.__code__.co_varnames[0]

    @functools.wraps(call)
    def run(*args, stream=None, **kwargs):
        first = args[0] if args else kwargs.get(name)
        if not (isinstance(first, torch.Tensor) and first.is_cuda):
            raise ValueError(f"{call.__name__}: {name} must be a CUDA tensor")
        if first.get_device() != torch._C._cuda_getDevice():
            with torch.cuda.device(first.device):
                return run(*args, stream=stream, **kwargs)
        if stream is None:
            return call(*args, **kwargs)
        with torch.cuda.stream(stream):
            return call(*args, **kwargs)
    return run


def _together(first, *others):
    """Refuses tensors of several devices."""
    for t in others:
        if t is not None and t.get_device() != first.get_device():
            raise ValueError("tensors of one call must lie on one device")


# ---- orthogonalised momentum ---------------------------------------------------
MUON_COEFS = (3.4445, -4.7750, 2.0315)
MUON_MAX_STEPS = 32


def muon_sizes(batch, rows, cols) -> int:
    """Workspace bytes of nvfp4_muon_update."""
    w = C.c_size_t()
    _check(lib.nvfp4_muon_sizes(batch, rows, cols, w), "nvfp4_muon_sizes")
    return w.value


def _floats(v):
    """A number, or the numbers of a sequence, as floats."""
    if isinstance(v, (list, tuple)) or getattr(v, "ndim", 0):
        return tuple([_floats(x) for x in v])
    return float(v)


# What is kept goes by the arguments' values: plain numbers alone, for a tensor stays the
# same object when its value changes.
@functools.lru_cache(maxsize=64)
def _coefs(coefs, steps):
    """[steps][3] for the library: one triple for every step, or one for each."""
    if not 1 <= steps <= MUON_MAX_STEPS:
        raise ValueError(f"steps must be 1 to {MUON_MAX_STEPS}")

    def triple(r):
        return isinstance(r, tuple) and len(r) == 3 and all(isinstance(v, float) for v in r)

    rows = (coefs,) * steps if triple(coefs) else coefs
    if not (isinstance(rows, tuple) and len(rows) == steps and all(map(triple, rows))):
        raise ValueError("coefs must be one triple, or one for each step")
    flat = [v for r in rows for v in r]
    return (C.c_float * len(flat))(*flat)


@_on_device
def nvfp4_muon_update(grad: torch.Tensor, momentum: torch.Tensor, mu: float = 0.95,
                      nesterov: bool = True, steps: int = 5, coefs=MUON_COEFS, eps: float = 1e-7,
                      out: torch.Tensor | None = None, zero_grad: bool = False,
                      workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The orthogonalised momentum of a matrix, or of each of a stack of them:
    grad [..., rows, cols] (bf16 or fp32) is taken into the fp32 `momentum`, in
    place; returns the update in bf16 (see nvfp4_muon_update in nvfp4.h).  `coefs`:
    the polynomial's (a, b, c), or one such triple for each step."""
    kind = _DTYPES.get(grad.dtype)
    if kind is None:
        raise TypeError(f"grad must be bf16 or fp32, got {grad.dtype}")
    given = out
    shape = grad.shape
    if len(shape) < 2 or grad.numel() == 0:
        raise ValueError("grad must be a matrix or a stack of matrices, not empty")
    _cuda(grad, grad.dtype, "grad")
    _cuda(momentum, _F32, "momentum", shape)
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=grad.device)
    else:
        _cuda(out, _BF16, "out", shape)
    rows, cols = shape[-2], shape[-1]
    batch = grad.numel() // (rows * cols)
    if workspace is None:
        workspace = _scratch(muon_sizes(batch, rows, cols), grad)
    else:
        _cuda(workspace, _U8, "workspace")
    _together(grad, momentum, out, workspace)
    steps = operator.index(steps)
    if coefs is not MUON_COEFS:  # lists and arrays as well
        coefs = _floats(coefs)
    p = MuonParams(batch, rows, cols, kind, 1 if nesterov else 0, steps, mu, eps,
                   _coefs(coefs, steps))
    st = lib.nvfp4_muon_update(p, grad.data_ptr(), momentum.data_ptr(), out.data_ptr(),
                               ZERO_GRAD if zero_grad else 0, workspace.data_ptr(),
                               workspace.numel(), _current(grad))
    if st:
        raise NVFP4Error(st, "nvfp4_muon_update")
    _changed(momentum, grad if zero_grad else None, given)
    return out


_APPLY_BYTES = quantize_sizes(128, 128, ROW_1X16)[3]


@_on_device
def nvfp4_muon_apply(W: torch.Tensor, update: torch.Tensor, lr: float, scale: float = 1.0,
                     decay: float = 0.0, amax: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None) -> torch.Tensor:
    """W = (1 - lr decay) W - lr scale update on an fp32 master weight, in place
    (see nvfp4_muon_apply in nvfp4.h); returns max |W| of the result, a 1-element
    tensor that its quantisation takes."""
    _cuda(W, _F32, "W")
    _cuda(update, _BF16, "update", W.shape)
    given = amax
    if amax is None:
        amax = torch.empty(1, dtype=_F32, device=W.device)
    else:
        _cuda(amax, _F32, "amax", (1,))
    if workspace is None:
        workspace = _scratch(_APPLY_BYTES, W)
    else:
        _cuda(workspace, _U8, "workspace")
    _together(W, update, amax, workspace)
    st = lib.nvfp4_muon_apply(W.data_ptr(), update.data_ptr(), W.numel(), lr, scale, decay,
                              amax.data_ptr(), workspace.data_ptr(), workspace.numel(),
                              _current(W))
    if st:
        raise NVFP4Error(st, "nvfp4_muon_apply")
    _changed(W, given)
    return amax


def operand(codes: torch.Tensor, scales: torch.Tensor, s_dec: torch.Tensor, rows: int,
            cols: int) -> QTensor:
    """A QTensor over buffers that hold a K-major operand [rows, cols] already:
    codes and scales (MMA layout) as uint8, s_dec one float32."""
    _cuda(codes, _U8, "codes")
    _cuda(scales, _U8, "scales")
    _cuda(s_dec, _F32, "s_dec")
    if (rows <= 0 or cols <= 0 or cols % 16 or codes.numel() < rows * cols // 2
            or scales.numel() < (rows + 127) // 128 * ((cols + 63) // 64) * 512
            or s_dec.numel() < 1):
        raise ValueError("buffers smaller than the operand, or cols not a multiple of 16")
    return QTensor(codes, scales, None, s_dec, None, None,
                   Tensor(codes.data_ptr(), scales.data_ptr(), None, None, None,
                          s_dec.data_ptr(), rows, cols, ROW_1X16, 0))


def operand_t(codes_t: torch.Tensor, scales_t: torch.Tensor, s_dec: torch.Tensor, rows: int,
              cols: int) -> QTensor:
    """A QTensor over the transposed view alone (codes_t / scales_t hold the
    K-major operand [cols, rows]) of a 16x16 quantisation of [rows, cols]: what
    b_view 1 of the products reads."""
    q = operand(codes_t, scales_t, s_dec, cols, rows)
    q.codes_t, q.scales_t, q.codes, q.scales = codes_t, scales_t, None, None
    q.desc = Tensor(None, None, codes_t.data_ptr(), scales_t.data_ptr(), None, s_dec.data_ptr(),
                    rows, cols, BLOCK_16X16, EMIT_T)
    return q


def route_sizes(tokens, experts, top):
    """(rows of a plan, workspace bytes of nvfp4_route_fwd)."""
    r, w = C.c_int64(), C.c_size_t()
    _check(lib.nvfp4_route_sizes(tokens, experts, top, r, w), "nvfp4_route_sizes")
    return r.value, w.value


@dataclass
class RoutePlan:
    """The outputs of nvfp4_route_fwd (see nvfp4.h)."""
    expert: torch.Tensor   # int32 [tokens, top]
    weight: torch.Tensor   # float32 [tokens, top]
    sizes: torch.Tensor    # int32 [experts]
    offsets: torch.Tensor  # int32 [experts + 1]
    row: torch.Tensor      # int32 [tokens, top]
    source: torch.Tensor   # int32 [rows]

    @property
    def rows(self):
        return self.source.numel()


def alloc_plan(tokens, experts, top, device="cuda") -> RoutePlan:
    """Buffers of a plan, e.g. for a server to route into at every step."""
    return _alloc_plan(tokens, experts, top, route_sizes(tokens, experts, top)[0], device)


def _alloc_plan(tokens, experts, top, rows, device):
    empty = torch.empty
    return RoutePlan(empty((tokens, top), dtype=_I32, device=device),
                     empty((tokens, top), dtype=_F32, device=device),
                     empty(experts, dtype=_I32, device=device),
                     empty(experts + 1, dtype=_I32, device=device),
                     empty((tokens, top), dtype=_I32, device=device),
                     empty(rows, dtype=_I32, device=device))


def _logits(logits):
    if not (logits.is_cuda and logits.dim() == 2 and logits.stride(1) == 1):
        raise ValueError("logits must be a 2-D CUDA tensor with unit column stride")
    kind = _DTYPES.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be bf16 or fp32, got {logits.dtype}")
    tokens, experts = logits.shape
    return kind, tokens, experts, logits.stride(0) if tokens > 1 else experts


_route_sizes = functools.lru_cache(maxsize=256)(route_sizes)


def _plan_buffers(tokens, experts, top, plan, workspace, logits):
    """The plan and the workspace of a routing call, checked or new."""
    rows, nbytes = _route_sizes(tokens, experts, top)
    if plan is None:
        plan = _alloc_plan(tokens, experts, top, rows, logits.device)
    else:
        _cuda(plan.expert, _I32, "expert", (tokens, top))
        _cuda(plan.weight, _F32, "weight", (tokens, top))
        _cuda(plan.sizes, _I32, "sizes", (experts,))
        _cuda(plan.offsets, _I32, "offsets", (experts + 1,))
        _cuda(plan.row, _I32, "row", (tokens, top))
        _cuda(plan.source, _I32, "source", (rows,))
    if workspace is None:
        workspace = _scratch(nbytes, logits)
    else:
        _cuda(workspace, _U8, "workspace")
    return plan, workspace


@_on_stream
def nvfp4_route_fwd(logits: torch.Tensor, top: int, mode: int = ROUTE_CHOSEN,
                    plan: RoutePlan | None = None,
                    workspace: torch.Tensor | None = None) -> RoutePlan:
    """Choose each token's `top` experts and order the rows by expert (see
    nvfp4_route_fwd in nvfp4.h)."""
    kind, tokens, experts, ld = _logits(logits)
    top = operator.index(top)
    plan, workspace = _plan_buffers(tokens, experts, top, plan, workspace, logits)
    st = lib.nvfp4_route_fwd(logits.data_ptr(), kind, tokens, experts, ld, top, mode,
                             plan.expert.data_ptr(), plan.weight.data_ptr(),
                             plan.sizes.data_ptr(), plan.offsets.data_ptr(), plan.row.data_ptr(),
                             plan.source.data_ptr(), workspace.data_ptr(), workspace.numel(),
                             _current(logits))
    if st:
        raise NVFP4Error(st, "nvfp4_route_fwd")
    return plan


@_on_stream
def nvfp4_route_bwd(logits: torch.Tensor, plan: RoutePlan, dweight: torch.Tensor,
                    mode: int = ROUTE_CHOSEN,
                    dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """The logits' gradient from that of the plan's weights."""
    kind, tokens, experts, ld = _logits(logits)
    top = plan.expert.shape[1]
    _cuda(plan.expert, _I32, "expert", (tokens, top))
    _cuda(plan.weight, _F32, "weight", (tokens, top))
    _cuda(dweight, _F32, "dweight", (tokens, top))
    if dlogits is None:
        dlogits = torch.empty((tokens, experts), dtype=logits.dtype, device=logits.device)
    else:
        _cuda(dlogits, logits.dtype, "dlogits", (tokens, experts))
    st = lib.nvfp4_route_bwd(logits.data_ptr(), kind, tokens, experts, ld, top, mode,
                             plan.expert.data_ptr(), plan.weight.data_ptr(), dweight.data_ptr(),
                             dlogits.data_ptr(), _current(logits))
    if st:
        raise NVFP4Error(st, "nvfp4_route_bwd")
    return dlogits


_small_workspace: dict = {}


def _untouched(t):
    """The workspace of a device's routing calls of up to 64 tokens, whose kernel does
    not touch it: one for all of them, on any stream and in any graph."""
    device = t.get_device()
    if device not in _small_workspace:
        _small_workspace[device] = torch.empty(route_sizes(1, 512, 1)[1], dtype=_U8,
                                               device=t.device)
    return _small_workspace[device]


_route_params = functools.lru_cache(maxsize=256)(RouteParams)


def _scored(tokens, experts, ld, kind, top, score, renormalise, groups, kept, group_top, scale):
    """The parameters of a scored routing, kept by their values: plain numbers alone, for
    a tensor stays the same object when its value changes."""
    index = operator.index
    return _route_params(tokens, experts, ld, kind, top, index(score), 1 if renormalise else 0,
                         index(groups), index(groups if kept is None else kept),
                         index(group_top), float(scale))


@_on_device
def nvfp4_route_scored_fwd(logits: torch.Tensor, top: int, score: int = SCORE_SIGMOID,
                           bias: torch.Tensor | None = None, groups: int = 1,
                           groups_kept: int | None = None, group_top: int = 2,
                           renormalise: bool = True, scale: float = 1.0,
                           plan: RoutePlan | None = None,
                           workspace: torch.Tensor | None = None) -> RoutePlan:
    """Choose each token's `top` experts by their scores plus a bias, among the best
    groups of experts, and order the rows by expert (see nvfp4_route_scored_fwd in
    nvfp4.h).  groups_kept None: all of them."""
    kind, tokens, experts, ld = _logits(logits)
    top = operator.index(top)
    if workspace is None and tokens <= 64:
        workspace = _untouched(logits)
    given = plan
    if plan is not None:
        _together(logits, plan.expert, plan.weight, plan.sizes, plan.offsets, plan.row,
                  plan.source)
    plan, workspace = _plan_buffers(tokens, experts, top, plan, workspace, logits)
    if bias is not None:
        _cuda(bias, _F32, "bias", (experts,))
    _together(logits, bias, workspace)
    p = _scored(tokens, experts, ld, kind, top, score, renormalise, groups, groups_kept, group_top,
                scale)
    st = lib.nvfp4_route_scored_fwd(p, logits.data_ptr(), _ptr(bias), plan.expert.data_ptr(),
                                    plan.weight.data_ptr(), plan.sizes.data_ptr(),
                                    plan.offsets.data_ptr(), plan.row.data_ptr(),
                                    plan.source.data_ptr(), workspace.data_ptr(),
                                    workspace.numel(), _current(logits))
    if st:
        raise NVFP4Error(st, "nvfp4_route_scored_fwd")
    if given is not None:
        _changed(plan.expert, plan.weight, plan.sizes, plan.offsets, plan.row, plan.source)
    return plan


@_on_device
def nvfp4_route_scored_bwd(logits: torch.Tensor, plan: RoutePlan, dweight: torch.Tensor,
                           score: int = SCORE_SIGMOID, renormalise: bool = True,
                           scale: float = 1.0,
                           dlogits: torch.Tensor | None = None) -> torch.Tensor:
    """The logits' gradient from that of the weights of nvfp4_route_scored_fwd."""
    kind, tokens, experts, ld = _logits(logits)
    top = plan.expert.shape[1]
    _cuda(plan.expert, _I32, "expert", (tokens, top))
    _cuda(plan.weight, _F32, "weight", (tokens, top))
    _cuda(dweight, _F32, "dweight", (tokens, top))
    given = dlogits
    if dlogits is None:
        dlogits = torch.empty((tokens, experts), dtype=logits.dtype, device=logits.device)
    else:
        _cuda(dlogits, logits.dtype, "dlogits", (tokens, experts))
    _together(logits, plan.expert, plan.weight, dweight, dlogits)
    p = _scored(tokens, experts, ld, kind, top, score, renormalise, 1, 1, 1, scale)
    st = lib.nvfp4_route_scored_bwd(p, logits.data_ptr(), plan.expert.data_ptr(),
                                    plan.weight.data_ptr(), dweight.data_ptr(), dlogits.data_ptr(),
                                    _current(logits))
    if st:
        raise NVFP4Error(st, "nvfp4_route_scored_bwd")
    _changed(given)
    return dlogits


@_on_device
def nvfp4_route_balance(sizes: torch.Tensor, bias: torch.Tensor, rate: float) -> torch.Tensor:
    """bias += rate sign(mean load - load) in place, from the loads of a plan (or
    the sum of several plans'): see nvfp4_route_balance in nvfp4.h; returns bias."""
    experts = sizes.numel()
    _cuda(sizes, _I32, "sizes", (experts,))
    _cuda(bias, _F32, "bias", (experts,))
    _together(sizes, bias)
    st = lib.nvfp4_route_balance(sizes.data_ptr(), experts, rate, bias.data_ptr(),
                                 _current(sizes))
    if st:
        raise NVFP4Error(st, "nvfp4_route_balance")
    _changed(bias)
    return bias


def _rows2d(t, name):
    _cuda(t, _BF16, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return t.shape


def _slots(row):
    _cuda(row, _I32, "row")
    if row.dim() != 2:
        raise ValueError("row must be [tokens, top]")
    return row.shape


@_on_stream
def nvfp4_dispatch(x: torch.Tensor, row: torch.Tensor, source: torch.Tensor,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """x's rows in the order of a plan's groups (`row`, `source` of a
    RoutePlan), padding rows zero (see nvfp4_dispatch in nvfp4.h)."""
    tokens, top = _slots(row)
    n, cols = _rows2d(x, "x")
    if n != tokens:
        raise ValueError("x must have one row per token")
    _cuda(source, _I32, "source")
    rows = source.numel()
    if out is None:
        out = torch.empty((rows, cols), dtype=_BF16, device=x.device)
    else:
        _cuda(out, _BF16, "out", (rows, cols))
    st = lib.nvfp4_dispatch(x.data_ptr(), row.data_ptr(), source.data_ptr(), tokens, cols, top,
                            rows, out.data_ptr(), _current(x))
    if st:
        raise NVFP4Error(st, "nvfp4_dispatch")
    return out


@_on_stream
def nvfp4_combine(o: torch.Tensor, row: torch.Tensor, weight: torch.Tensor | None = None,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """Each token's weighted sum of its rows of `o`; without weights, the
    gradient of nvfp4_dispatch (see nvfp4_combine in nvfp4.h)."""
    tokens, top = _slots(row)
    rows, cols = _rows2d(o, "o")
    if weight is not None:
        _cuda(weight, _F32, "weight", (tokens, top))
    if out is None:
        out = torch.empty((tokens, cols), dtype=_BF16, device=o.device)
    else:
        _cuda(out, _BF16, "out", (tokens, cols))
    st = lib.nvfp4_combine(o.data_ptr(), row.data_ptr(),
                           None if weight is None else weight.data_ptr(), tokens, cols, top, rows,
                           out.data_ptr(), _current(o))
    if st:
        raise NVFP4Error(st, "nvfp4_combine")
    return out


@_on_stream
def nvfp4_combine_bwd(dy: torch.Tensor, o: torch.Tensor, row: torch.Tensor, source: torch.Tensor,
                      weight: torch.Tensor, d_o: torch.Tensor | None = None,
                      dweight: torch.Tensor | None = None):
    """(d_o, dweight) of nvfp4_combine (see nvfp4_combine_bwd in nvfp4.h)."""
    tokens, top = _slots(row)
    rows, cols = _rows2d(o, "o")
    _cuda(dy, _BF16, "dy", (tokens, cols))
    _cuda(source, _I32, "source", (rows,))
    _cuda(weight, _F32, "weight", (tokens, top))
    if d_o is None:
        d_o = torch.empty_like(o)
    else:
        _cuda(d_o, _BF16, "d_o", (rows, cols))
    if dweight is None:
        dweight = torch.empty_like(weight)
    else:
        _cuda(dweight, _F32, "dweight", (tokens, top))
    st = lib.nvfp4_combine_bwd(dy.data_ptr(), o.data_ptr(), row.data_ptr(), source.data_ptr(),
                               weight.data_ptr(), tokens, cols, top, rows, d_o.data_ptr(),
                               dweight.data_ptr(), _current(o))
    if st:
        raise NVFP4Error(st, "nvfp4_combine_bwd")
    return d_o, dweight


def _groups(sizes, offsets):
    groups = sizes.numel()
    _cuda(sizes, _I32, "sizes", (groups,))
    _cuda(offsets, _I32, "offsets", (groups + 1,))
    if groups < 1:
        raise ValueError("there must be a group")
    return groups


@_on_stream
def nvfp4_group_gemm(A: QTensor, B: QTensor, sizes: torch.Tensor, offsets: torch.Tensor,
                     b_view: int = 0, out: torch.Tensor | None = None, d_mode: int = D_BF16,
                     C_add: torch.Tensor | None = None, tile: int = TILE_AUTO) -> torch.Tensor:
    """D[r] = alpha A[r] . B_e^T for the rows r of each group e (see
    nvfp4_group_gemm in nvfp4.h); returns D bf16 [rows, N]."""
    groups = _groups(sizes, offsets)
    a, b = A.desc, B.desc
    rows, K = a.rows, a.cols
    N = b.cols if b_view else b.rows // groups
    if out is None:
        out = torch.empty((rows, N), dtype=_BF16, device=sizes.device)
    else:
        _cuda(out, _BF16, "out", (rows, N))
    if C_add is not None:
        _cuda(C_add, _BF16, "C_add", (rows, N))
    st = lib.nvfp4_group_gemm(a, b, b_view, sizes.data_ptr(), offsets.data_ptr(), groups,
                              out.data_ptr(), d_mode,
                              None if C_add is None else C_add.data_ptr(), rows, N, K, tile,
                              _current(sizes))
    if st:
        raise NVFP4Error(st, "nvfp4_group_gemm")
    return out


@_on_stream
def nvfp4_group_wgrad(A: QTensor, B: QTensor, sizes: torch.Tensor, offsets: torch.Tensor,
                      out: torch.Tensor | None = None, d_mode: int = D_BF16,
                      tile: int = TILE_AUTO) -> torch.Tensor:
    """D_e = alpha A[:, rows of e] . B[:, rows of e]^T (see nvfp4_group_wgrad in
    nvfp4.h); returns D [groups, M, N], bf16 or (D_F32_ACCUM: folded into) fp32."""
    groups = _groups(sizes, offsets)
    a, b = A.desc, B.desc
    M, rows, N = a.rows, a.cols, b.rows
    dtype = _F32 if d_mode == D_F32_ACCUM else _BF16
    if out is None:
        out = (torch.zeros if d_mode == D_F32_ACCUM else torch.empty)(
            (groups, M, N), dtype=dtype, device=sizes.device)
    else:
        _cuda(out, dtype, "out", (groups, M, N))
    st = lib.nvfp4_group_wgrad(a, b, sizes.data_ptr(), offsets.data_ptr(), groups, out.data_ptr(),
                               d_mode, M, N, rows, tile, _current(sizes))
    if st:
        raise NVFP4Error(st, "nvfp4_group_wgrad")
    return out


def _norm_args(x, z, w_post, gate, w_pre, eps, x_scale, z_scale):
    """The call's parameters, and the five inputs' addresses."""
    if not (x.is_cuda and x.dim() == 2 and x.is_contiguous()):
        raise ValueError("x must be a contiguous 2-D CUDA tensor")
    kind = _DTYPES.get(x.dtype)
    if kind is None:
        raise TypeError(f"x must be bf16 or fp32, got {x.dtype}")
    rows, cols = x.shape
    mode, pz, pw, pg, pp = GATE_NONE, None, None, None, None
    if z is not None:
        _cuda(z, _BF16, "z", (rows, cols))
        pz = z.data_ptr()
    if w_post is not None:
        _cuda(w_post, _F32, "w_post", (cols,))
        pw = w_post.data_ptr()
    if gate is not None:
        mode = GATE_CHANNEL if gate.dim() == 1 else GATE_ROW
        _cuda(gate, _F32, "gate", (cols,) if mode == GATE_CHANNEL else (rows, 1))
        pg = gate.data_ptr()
    if w_pre is not None:
        _cuda(w_pre, _F32, "w_pre", (cols,))
        pp = w_pre.data_ptr()
    return NormParams(rows, cols, kind, mode, eps, x_scale, z_scale), (x.data_ptr(), pz, pw, pg, pp)


@_on_stream
def nvfp4_residual_norm_fwd(x: torch.Tensor, z: torch.Tensor | None = None,
                            w_post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                            w_pre: torch.Tensor | None = None, eps: float = 1e-5,
                            x_scale: float = 1.0, z_scale: float = 1.0,
                            y: torch.Tensor | None = None, h: torch.Tensor | None = None):
    """y = x_scale x + z_scale gate (.) norm(z) w_post and h = norm(y) w_pre in
    one pass (see nvfp4_residual_norm_fwd in nvfp4.h); returns (y, h).  Without
    z, y is only written when given or x_scale is not 1 (and is x otherwise);
    without w_pre, h is None.  A gate [rows, 1] is per row, one of [cols] per
    channel."""
    p, ins = _norm_args(x, z, w_post, gate, w_pre, eps, x_scale, z_scale)
    if y is not None:
        _cuda(y, x.dtype, "y", x.shape)
    elif z is not None or x_scale != 1.0:
        y = torch.empty_like(x)
    if h is not None:
        _cuda(h, _BF16, "h", x.shape)
    elif w_pre is not None:
        h = torch.empty_like(x) if x.dtype is _BF16 else torch.empty_like(x, dtype=_BF16)
    st = lib.nvfp4_residual_norm_fwd(p, *ins, None if y is None else y.data_ptr(),
                                     None if h is None else h.data_ptr(), _current(x))
    if st:
        raise NVFP4Error(st, "nvfp4_residual_norm_fwd")
    return (x if y is None else y), h


@_on_stream
def nvfp4_residual_norm_bwd(dy: torch.Tensor | None, dh: torch.Tensor | None, x: torch.Tensor,
                            z: torch.Tensor | None = None, w_post: torch.Tensor | None = None,
                            gate: torch.Tensor | None = None, w_pre: torch.Tensor | None = None,
                            eps: float = 1e-5, x_scale: float = 1.0, z_scale: float = 1.0,
                            workspace: torch.Tensor | None = None):
    """(dx, dz, dw_post, dgate, dw_pre) of nvfp4_residual_norm_fwd from the
    gradients of y and h (None: zero); an entry is None where its input is."""
    p, ins = _norm_args(x, z, w_post, gate, w_pre, eps, x_scale, z_scale)
    if dy is not None:
        _cuda(dy, x.dtype, "dy", x.shape)
    if dh is not None:
        _cuda(dh, _BF16, "dh", x.shape)
    if workspace is None:
        n = C.c_size_t()
        _check(lib.nvfp4_residual_norm_bwd_sizes(p.rows, p.cols, n),
               "nvfp4_residual_norm_bwd_sizes")
        workspace = _scratch(n.value, x)
    else:
        _cuda(workspace, _U8, "workspace")
    outs = [None if t is None else torch.empty_like(t) for t in (x, z, w_post, gate, w_pre)]
    st = lib.nvfp4_residual_norm_bwd(p, _ptr(dy), _ptr(dh), *ins, *[_ptr(t) for t in outs],
                                     workspace.data_ptr(), workspace.numel(), _current(x))
    if st:
        raise NVFP4Error(st, "nvfp4_residual_norm_bwd")
    return tuple(outs)


STALL_QUANTIZE, STALL_GEMM, LOSE_NORM, QUIT_GEMM = 1, 2, 16, 32


def debug_inject(stall_mask: int = 0, wait_limit_ns: int = 0):
    """Failure injection for tests of the bounded waits (nvfp4_debug_inject)."""
    _check(lib.nvfp4_debug_inject(stall_mask, wait_limit_ns), "nvfp4_debug_inject")


def check_device_errors(stream=None):
    _check(lib.nvfp4_check_device_errors(_stream(stream)), "nvfp4_check_device_errors")
