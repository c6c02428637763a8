"""The scored routing, the balance bias and the orthogonalised momentum refuse bad
arguments on the host, before any CUDA call: the stand-in addresses below are
never dereferenced."""
import ctypes as C

import pytest

vp, i32, i64, sz, f32 = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t, C.c_float
INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5
A, B, D = 1 << 40, 1 << 41, 1 << 42  # aligned stand-ins, far apart
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from nvfp4_block_scaled_03_gb300 import build
    return C.CDLL(build.build())


class Route(C.Structure):
    _fields_ = [("tokens", i64), ("experts", i64), ("ld", i64), ("in_dtype", i32), ("top", i32),
                ("score", i32), ("renormalise", i32), ("groups", i32), ("groups_kept", i32),
                ("group_top", i32), ("scale", f32)]


class Muon(C.Structure):
    _fields_ = [("batch", i64), ("rows", i64), ("cols", i64), ("grad_dtype", i32),
                ("nesterov", i32), ("steps", i32), ("mu", f32), ("eps", f32),
                ("coefs", C.POINTER(f32))]


def route(**kw):
    d = dict(tokens=8, experts=64, ld=64, in_dtype=1, top=4, score=1, renormalise=1, groups=8,
             groups_kept=3, group_top=2, scale=1.0) | kw
    return Route(*[d[n] for n, _ in Route._fields_])


BAD_ROUTES = [(INVALID, dict(score=2)), (INVALID, dict(score=-1)), (INVALID, dict(renormalise=2)),
              (INVALID, dict(scale=0.0)), (INVALID, dict(scale=-1.0)), (INVALID, dict(scale=NAN)),
              (INVALID, dict(scale=INF)), (INVALID, dict(in_dtype=2)), (SHAPE, dict(tokens=0)),
              (SHAPE, dict(experts=513, ld=513)), (SHAPE, dict(ld=63)), (SHAPE, dict(top=0)),
              (SHAPE, dict(top=17)), (SHAPE, dict(groups=0)), (SHAPE, dict(groups=3)),
              (SHAPE, dict(groups=64)), (SHAPE, dict(experts=60, ld=60)),
              (SHAPE, dict(groups_kept=0)), (SHAPE, dict(groups_kept=9)),
              (SHAPE, dict(group_top=0)), (SHAPE, dict(group_top=3)),
              (SHAPE, dict(top=9, groups_kept=1)), (SHAPE, dict(tokens=1 << 31))]


def test_scored_routing_refusals(lib):
    f = lib.nvfp4_route_scored_fwd
    f.argtypes = [C.POINTER(Route), vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]

    def call(p=None, logits=A, bias=None, out=(A,) * 6, ws=A, wsb=1 << 20):
        return f(C.byref(p or route()), logits, bias, *out, ws, wsb, None)

    assert f(None, A, None, *(A,) * 6, A, 1 << 20, None) == INVALID
    for status, kw in BAD_ROUTES:
        assert call(route(**kw)) == status, kw
    assert call(logits=None) == INVALID and call(bias=A + 2) == ALIGN
    for k in range(6):
        assert call(out=tuple(None if i == k else A for i in range(6))) == INVALID
        assert call(out=tuple(A + 2 if i == k else A for i in range(6))) == ALIGN
    assert call(logits=A + 2) == ALIGN and call(route(in_dtype=0), logits=A + 1) == ALIGN
    assert call(ws=None) == WORKSPACE and call(wsb=64) == WORKSPACE and call(ws=A + 2) == WORKSPACE
    b = lib.nvfp4_route_scored_bwd
    b.argtypes = [C.POINTER(Route), vp, vp, vp, vp, vp, vp]

    def back(p=None, ptrs=(A,) * 5):
        return b(C.byref(p or route()), *ptrs, None)

    for status, kw in BAD_ROUTES:
        assert back(route(**kw)) == status, kw
    for k in range(5):
        assert back(ptrs=tuple(None if i == k else A for i in range(5))) == INVALID
        assert back(ptrs=tuple(A + 1 if i == k else A for i in range(5))) == ALIGN


def test_balance_refusals(lib):
    f = lib.nvfp4_route_balance
    f.argtypes = [vp, i64, f32, vp, vp]
    assert f(None, 8, 0.1, A, None) == INVALID and f(A, 8, 0.1, None, None) == INVALID
    assert f(A, 8, NAN, A, None) == INVALID and f(A, 8, INF, A, None) == INVALID
    assert f(A, 0, 0.1, A, None) == SHAPE and f(A, 513, 0.1, A, None) == SHAPE
    assert f(A + 2, 8, 0.1, A, None) == ALIGN and f(A, 8, 0.1, A + 2, None) == ALIGN


def test_muon_sizes(lib):
    f = lib.nvfp4_muon_sizes
    f.argtypes = [i64, i64, i64, C.POINTER(sz)]
    n = sz()
    for batch, rows, cols in ((1, 1, 1), (1, 64, 4096), (64, 1024, 2048), (3, 777, 1290)):
        assert f(batch, rows, cols, C.byref(n)) == 0
        # X's halves and the two square matrices at least
        assert n.value >= batch * (4 * rows * cols + 4 * min(rows, cols) ** 2)
        assert f(batch, rows, cols, None) == 0
    for shape in ((0, 8, 8), (1, 0, 8), (1, 8, 0), (-1, 8, 8), (65536, 8, 8), (1, 1 << 21, 8),
                  (1, 1 << 16, 1 << 15), (1, 40000, 40000)):
        assert f(*shape, C.byref(n)) == SHAPE, shape


def test_muon_update_refusals(lib):
    f = lib.nvfp4_muon_update
    f.argtypes = [C.POINTER(Muon), vp, vp, vp, C.c_uint32, vp, sz, vp]
    good = (f32 * 6)(3.4445, -4.7750, 2.0315, 3.4445, -4.7750, 2.0315)

    def call(grad=A, momentum=B, update=D, flags=0, ws=A + (1 << 38), wsb=1 << 30, **kw):
        d = dict(batch=2, rows=64, cols=128, grad_dtype=1, nesterov=1, steps=2, mu=0.9, eps=1e-7,
                 coefs=good) | kw
        return f(C.byref(Muon(*[d[n] for n, _ in Muon._fields_])), grad, momentum, update, flags,
                 ws, wsb, None)

    assert f(None, A, B, D, 0, A, 1 << 30, None) == INVALID
    for kw in (dict(grad=None), dict(momentum=None), dict(update=None), dict(flags=1),
               dict(flags=32), dict(grad_dtype=2), dict(nesterov=2), dict(nesterov=-1),
               dict(steps=0), dict(steps=33), dict(mu=NAN), dict(mu=INF), dict(eps=0.0),
               dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(coefs=None),
               dict(coefs=(f32 * 6)(1, 2, 3, 4, NAN, 6))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(batch=0), dict(rows=0), dict(cols=0), dict(batch=70000),
               dict(rows=1 << 16, cols=1 << 15)):
        assert call(**kw) == SHAPE, kw
    count = 2 * 64 * 128
    # overlaps, at either end
    assert call(momentum=A + 4 * count - 16) == INVALID and call(update=A + 16) == INVALID
    assert call(update=B + 4 * count - 16) == INVALID
    assert call(grad=B, grad_dtype=0) == INVALID
    for kw in (dict(grad=A + 8), dict(momentum=B + 4), dict(update=D + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(ws=None) == WORKSPACE and call(wsb=1000) == WORKSPACE
    assert call(ws=A + (1 << 38) + 8) == WORKSPACE


def test_muon_apply_refusals(lib):
    f = lib.nvfp4_muon_apply
    f.argtypes = [vp, vp, i64, f32, f32, f32, vp, vp, sz, vp]

    def call(W=A, update=B, n=100, lr=0.1, scale=1.0, decay=0.0, amax=D, ws=D + 64, wsb=8192):
        return f(W, update, n, lr, scale, decay, amax, ws, wsb, None)

    for kw in (dict(W=None), dict(update=None), dict(lr=NAN), dict(scale=INF), dict(decay=NAN),
               dict(update=A), dict(update=A + 384)):
        assert call(**kw) == INVALID, kw
    assert call(n=0) == SHAPE and call(n=-4) == SHAPE
    assert call(W=A + 4) == ALIGN and call(update=B + 2) == ALIGN and call(amax=D + 2) == ALIGN
    assert call(ws=None) == WORKSPACE and call(wsb=16) == WORKSPACE
