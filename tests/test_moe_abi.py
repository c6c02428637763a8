"""The mixture-of-experts entry points refuse bad arguments on the host, before
any CUDA call: the stand-in addresses below are never dereferenced."""
import ctypes as C

import pytest

vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5
A = 1 << 40  # an aligned stand-in


@pytest.fixture(scope="module")
def lib():
    from nvfp4_block_scaled_03_gb300 import build
    return C.CDLL(build.build())


class Desc(C.Structure):
    _fields_ = [("codes", vp), ("scales", vp), ("codes_t", vp), ("scales_t", vp), ("amax", vp),
                ("s_dec", vp), ("rows", i64), ("cols", i64), ("mode", i32), ("flags", C.c_uint32)]


class Norm(C.Structure):
    _fields_ = [("rows", i64), ("cols", i64), ("stream_dtype", i32), ("gate_mode", i32),
                ("eps", C.c_float), ("x_scale", C.c_float), ("z_scale", C.c_float)]


def test_route_sizes(lib):
    f = lib.nvfp4_route_sizes
    f.argtypes = [i64, i64, i32, C.POINTER(i64), C.POINTER(sz)]
    rows, ws = i64(), sz()

    def call(t, e, k):
        return f(t, e, k, C.byref(rows), C.byref(ws))

    for t, e, k in ((1, 8, 2), (5, 3, 3), (1000, 64, 8), (7, 512, 16), (1, 1, 1)):
        assert call(t, e, k) == 0
        n = t * k
        assert rows.value == (n + 127 * min(e, n)) // 128 * 128
        # the worst spread of n rows over e experts fits: each partial block filled
        full, left = divmod(n, 1)
        worst = min(e, n) * 128 + max(0, n - min(e, n)) // 128 * 128
        assert rows.value >= min(worst, -(-n // 128) * 128) and rows.value % 128 == 0
    assert f(1, 8, 2, None, None) == 0
    for t, e, k in ((0, 8, 2), (-1, 8, 2), (4, 0, 1), (4, 513, 1), (4, 8, 0), (4, 8, 9), (4, 64, 17),
                    (1 << 31, 8, 2), ((1 << 31) - 1, 8, 8)):
        assert call(t, e, k) == SHAPE, (t, e, k)


def test_rows_bound_holds_every_spread(lib):
    """For small numbers, every way to spread n rows over e experts fits."""
    from itertools import product
    f = lib.nvfp4_route_sizes
    f.argtypes = [i64, i64, i32, C.POINTER(i64), C.POINTER(sz)]
    rows = i64()
    for t in (1, 2, 127, 128, 129, 257):
        for e in (1, 2, 3):
            assert f(t, e, 1, C.byref(rows), None) == 0
            step = range(0, t + 1, max(1, t // 16))
            for part in product(step, repeat=e - 1):
                last = t - sum(part)
                if last >= 0:
                    assert sum(-(-s // 128) * 128 for s in (*part, last)) <= rows.value


def test_route_refusals(lib):
    f = lib.nvfp4_route_fwd
    f.argtypes = [vp, i32, i64, i64, i64, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]

    def call(logits=A, dt=1, T=8, E=8, ld=8, top=2, mode=1, out=(A,) * 6, ws=A, wsb=1 << 20):
        return f(logits, dt, T, E, ld, top, mode, *out, ws, wsb, None)

    assert call(logits=None) == INVALID and call(dt=2) == INVALID and call(mode=2) == INVALID
    for k in range(6):
        assert call(out=tuple(None if i == k else A for i in range(6))) == INVALID
        assert call(out=tuple(A + 2 if i == k else A for i in range(6))) == ALIGN
    assert call(T=0) == SHAPE and call(E=1) == SHAPE and call(ld=7) == SHAPE
    assert call(logits=A + 2) == ALIGN and call(logits=A + 1, dt=0) == ALIGN
    assert call(ws=None) == WORKSPACE and call(wsb=64) == WORKSPACE
    b = lib.nvfp4_route_bwd
    b.argtypes = [vp, i32, i64, i64, i64, i32, i32, vp, vp, vp, vp, vp]
    args = [A, 1, 8, 8, 8, 2, 1, A, A, A, A, None]
    for k in (0, 7, 8, 9, 10):
        assert b(*[None if i == k else v for i, v in enumerate(args)]) == INVALID
    assert b(*[A + 2 if i == 10 else v for i, v in enumerate(args)]) == ALIGN
    assert b(*[3 if i == 6 else v for i, v in enumerate(args)]) == INVALID


def test_move_refusals(lib):
    lib.nvfp4_dispatch.argtypes = [vp, vp, vp, i64, i64, i32, i64, vp, vp]
    lib.nvfp4_combine.argtypes = [vp, vp, vp, i64, i64, i32, i64, vp, vp]
    lib.nvfp4_combine_bwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i32, i64, vp, vp, vp]
    calls = [(lib.nvfp4_dispatch, [A, A, A, 4, 64, 2, 256, A, None], (0, 1, 2, 7), 3),
             (lib.nvfp4_combine, [A, A, A, 4, 64, 2, 256, A, None], (0, 1, 7), 3),
             (lib.nvfp4_combine_bwd, [A, A, A, A, A, 4, 64, 2, 256, A, A, None],
              (0, 1, 2, 3, 4, 9, 10), 5)]
    for f, args, pointers, n in calls:
        def call(k, v):
            return f(*[v if i == k else a for i, a in enumerate(args)])
        for k in pointers:
            assert call(k, None) == INVALID and call(k, A + 2) == ALIGN
        assert call(n, 0) == SHAPE and call(n + 1, 60) == SHAPE and call(n + 2, 17) == SHAPE
        assert call(n + 2, 0) == SHAPE and call(n + 3, 0) == SHAPE and call(n, 1 << 31) == SHAPE


def _operand(rows, cols, transposed=False):
    d = Desc()
    d.codes, d.scales, d.amax, d.s_dec = A, A, A, A
    if transposed:
        d.codes_t, d.scales_t = A, A
    d.rows, d.cols = rows, cols
    return d


def test_group_gemm_refusals(lib):
    f = lib.nvfp4_group_gemm
    P = C.POINTER(Desc)
    f.argtypes = [P, P, i32, vp, vp, i32, vp, i32, vp, i64, i64, i64, i32, vp]

    def call(a=None, b=None, view=0, sizes=A, offsets=A, groups=4, D=A, mode=0, c=None, rows=512,
             N=128, K=256, tile=0):
        a = a or _operand(512, 256)
        b = b or (_operand(4 * 256, 128, True) if view else _operand(4 * 128, 256))
        return f(a, b, view, sizes, offsets, groups, D, mode, c, rows, N, K, tile, None)

    assert call(sizes=None) == INVALID and call(offsets=None) == INVALID and call(D=None) == INVALID
    assert call(view=2) == INVALID and call(mode=1) == INVALID
    assert call(mode=2) == INVALID and call(c=A) == INVALID       # C and its mode go together
    assert call(tile=1) == INVALID and call(tile=99) == INVALID
    assert call(view=1, b=_operand(1024, 128)) == INVALID         # no transposed codes
    assert call(groups=0) == SHAPE and call(groups=513) == SHAPE and call(groups=3) == SHAPE
    assert call(rows=500) == SHAPE and call(N=64) == SHAPE and call(K=96) == SHAPE
    assert call(a=_operand(512, 128)) == SHAPE and call(b=_operand(512, 512)) == SHAPE
    assert call(view=1, b=_operand(128, 1024, True)) == SHAPE
    assert call(D=A + 8) == ALIGN and call(sizes=A + 2) == ALIGN and call(c=A + 8, mode=2) == ALIGN
    no_codes = _operand(512, 256)
    no_codes.codes = None
    assert call(a=no_codes) == INVALID


def test_group_wgrad_refusals(lib):
    f = lib.nvfp4_group_wgrad
    P = C.POINTER(Desc)
    f.argtypes = [P, P, vp, vp, i32, vp, i32, i64, i64, i64, i32, vp]

    def call(a=None, b=None, sizes=A, offsets=A, groups=4, D=A, mode=0, M=256, N=128, rows=512,
             tile=0):
        return f(a or _operand(256, 512), b or _operand(128, 512), sizes, offsets, groups, D, mode,
                 M, N, rows, tile, None)

    assert call(sizes=None) == INVALID and call(D=None) == INVALID and call(mode=2) == INVALID
    assert call(mode=1, tile=6) == INVALID                        # the wide tile has no fold
    assert call(groups=0) == SHAPE and call(M=200) == SHAPE and call(N=64) == SHAPE
    assert call(rows=500) == SHAPE and call(a=_operand(128, 512)) == SHAPE
    assert call(b=_operand(128, 256)) == SHAPE and call(D=A + 4) == ALIGN


def test_norm_refusals(lib):
    fwd, bwd, size = (lib.nvfp4_residual_norm_fwd, lib.nvfp4_residual_norm_bwd,
                      lib.nvfp4_residual_norm_bwd_sizes)
    P = C.POINTER(Norm)
    fwd.argtypes = [P] + [vp] * 8
    bwd.argtypes = [P] + [vp] * 13 + [sz, vp]
    size.argtypes = [i64, i64, C.POINTER(sz)]
    n = sz()
    assert size(1000, 4096, C.byref(n)) == 0 and n.value % 16 == 0 and n.value > 0
    assert size(0, 64, C.byref(n)) == SHAPE and size(4, 60, C.byref(n)) == SHAPE
    assert size(4, 65544, C.byref(n)) == SHAPE and size(4, 64, None) == INVALID

    def params(rows=4, cols=64, dt=0, gate=0, eps=1e-5, a=1.0, b=1.0):
        return Norm(rows, cols, dt, gate, eps, a, b)

    def f(p=None, x=A, z=A, wp=A, g=None, wq=A, y=A, h=A):
        return fwd(p or params(), x, z, wp, g, wq, y, h, None)

    inf, nan = float("inf"), float("nan")
    for bad in (params(dt=2), params(gate=3), params(eps=0.0), params(eps=-1.0), params(eps=nan),
                params(eps=inf), params(a=inf), params(b=nan)):
        assert f(bad) == INVALID
    assert f(x=None) == INVALID and f(wp=None) == INVALID and f(z=None) == INVALID
    assert f(z=None, wp=None, wq=None, h=None) == INVALID          # nothing to do
    assert f(g=A) == INVALID and f(params(gate=1)) == INVALID      # the gate and its mode
    assert f(y=None) == INVALID and f(h=None) == INVALID and f(wq=None) == INVALID
    assert f(params(rows=0)) == SHAPE and f(params(cols=60)) == SHAPE
    assert f(x=A + 8) == ALIGN and f(y=A + 8) == ALIGN and f(params(gate=1), g=A + 4) == ALIGN
    assert f(params(gate=2), g=A + 2) == ALIGN

    def b(p=None, dy=A, dh=A, x=A, z=A, wp=A, g=None, wq=A, dx=A, dz=A, dwp=A, dg=None, dwq=A, ws=A,
          wsb=1 << 30):
        return bwd(p or params(), dy, dh, x, z, wp, g, wq, dx, dz, dwp, dg, dwq, ws, wsb, None)

    assert b(dx=None) == INVALID and b(dz=None) == INVALID and b(dwp=None) == INVALID
    assert b(dwq=None) == INVALID and b(dh=None) == INVALID and b(dg=A) == INVALID
    assert b(dy=None, dh=None, wq=None, dwq=None) == INVALID       # no gradient at all
    assert b(dx=A + 8) == ALIGN and b(dwp=A + 2) == ALIGN
