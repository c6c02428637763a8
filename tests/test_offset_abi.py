"""The quantisers refuse a device offset that cannot be one, on the host, before
any CUDA call: the stand-in addresses below are never dereferenced."""
import ctypes as C

import pytest

vp, i32, i64, u32, u64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_uint32, C.c_uint64, C.c_size_t
INVALID, ALIGN = 1, 3
A = 1 << 40
SR, GIVEN, DEVICE = 2, 8, 32


class Desc(C.Structure):
    _fields_ = [("codes", vp), ("scales", vp), ("codes_t", vp), ("scales_t", vp), ("amax", vp),
                ("s_dec", vp), ("rows", i64), ("cols", i64), ("mode", i32), ("flags", u32)]


@pytest.fixture(scope="module")
def lib():
    from nvfp4_block_scaled_03_gb300 import build
    return C.CDLL(build.build())


def test_device_offsets(lib):
    out = Desc(A, A, None, None, A, A, 0, 0, 0, 0)
    one = lib.nvfp4_quantize
    one.argtypes = [vp, i32, i64, i64, i64, i32, u32, u64, u64, C.POINTER(Desc), vp, sz, vp]
    two = lib.nvfp4_quantize_rowcol
    two.argtypes = [vp, i32, i64, i64, i64, u32, u32, u64, u64, u64, C.POINTER(Desc),
                    C.POINTER(Desc), vp]

    def quantize(flags, offset):
        return one(A, 0, 128, 128, 128, 0, flags | GIVEN, 0, offset, out, None, 0, None)

    def rowcol(row, col, at_row, at_col):
        return two(A, 0, 128, 128, 128, row | GIVEN, col | GIVEN, 0, at_row, at_col, out, out, None)

    assert quantize(DEVICE, A) == INVALID            # no stochastic rounding
    assert quantize(SR | DEVICE, 0) == INVALID       # no address
    assert quantize(SR | DEVICE, A + 4) == ALIGN
    assert rowcol(DEVICE, SR, A, 0) == INVALID and rowcol(SR, DEVICE, 0, A) == INVALID
    assert rowcol(SR | DEVICE, SR, 0, 0) == INVALID and rowcol(SR, SR | DEVICE, 0, 0) == INVALID
    assert rowcol(SR | DEVICE, SR, A + 4, 0) == ALIGN and rowcol(SR, SR | DEVICE, 0, A + 4) == ALIGN
