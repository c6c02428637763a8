"""GPU parity of the mixture-of-experts operators against their 64-bit forms
(moe_reference), whose docstring derives the tolerances of the norms.

* Norms: every output within E_NORM times the size of its terms, plus half a
  bf16 unit where it is rounded to bf16.
* Routing: experts and plan exact.  Weights: expf (2 ulp) of a difference, at
  most 16 + 5 additions and a division, below 2^-18 relative; the logit
  difference itself is rounded, |difference| 2^-24 <= 2^-18 for logits whose
  spread is below 64 (the tests').  Gradients 2^-17 of the terms' size.
* Rows: dispatch exact; combine and its gradient r 2^-24 of the terms' size
  with r the additions in a row, plus half a bf16 unit.
* Products: bf16 outputs by the rule of the other GEMM tests (assert_gemm_close);
  the FP32 fold within (K / 64 + 64) 2^-22 sum |a b|: one rounding (or
  truncation) of the accumulator for each of the K / 64 steps, and of each of
  the 64 aligned products inside a step.
"""
import ctypes as C

import numpy as np
import pytest

import gpu_helpers as H
import moe_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding
    return binding


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _close(got, ref, size, e, name, rounded):
    got = _f64(got)
    assert got.shape == ref.shape, name
    bound = e * size + (R.half_ulp_bf16(np.abs(ref) + e * size) if rounded else 0.0)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.size} off, first "
                           f"{np.argwhere(bad)[:4].tolist()}: {got[bad][:4]} for {ref[bad][:4]}, "
                           f"bound {np.broadcast_to(bound, bad.shape)[bad][:4]}")


# ---- norms -------------------------------------------------------------------
def _norm_case(T, D, wide, gate, seed, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    kind = torch.float32 if wide else torch.bfloat16
    t = dict(x=(torch.randn(T, D, generator=g) * 2 * scale).to(kind),
             z=(torch.randn(T, D, generator=g) * 0.3 * scale).bfloat16(),
             w_post=1 + 0.3 * torch.randn(D, generator=g), w_pre=1 + 0.3 * torch.randn(D, generator=g),
             gate={"none": None, "channel": torch.randn(D, generator=g),
                   "row": torch.randn(T, 1, generator=g)}[gate],
             dy=torch.randn(T, D, generator=g).to(kind), dh=torch.randn(T, D, generator=g).bfloat16())
    return t


NORM_SHAPES = [(1, 8), (3, 64), (2, 256), (5, 264), (700, 520), (1, 4096), (17, 4104), (3, 8192),
               (2, 16384), (2, 65536), (1000, 1032)]


@pytest.mark.parametrize("T,D", NORM_SHAPES)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("gate,parts", [("none", "both"), ("channel", "both"), ("row", "both"),
                                        ("none", "first"), ("row", "last"), ("channel", "last")])
def test_residual_norm(nv, T, D, wide, gate, parts):
    import torch
    t = _norm_case(T, D, wide, gate, seed=T + D)
    if parts == "first":
        t["z"] = t["w_post"] = t["gate"] = None
    if parts == "last":
        t["w_pre"] = t["dh"] = None
    c = {k: None if v is None else v.cuda() for k, v in t.items()}
    n = {k: None if v is None else _f64(v) for k, v in t.items()}
    eps, a, b = 1e-5, np.float32(0.9), np.float32(0.7)
    # the binding passes eps and the scales as FP32
    ra = (np.float64(np.float32(eps)), np.float64(a), np.float64(b))
    args = dict(w_post=c["w_post"], gate=c["gate"], w_pre=c["w_pre"], eps=eps, x_scale=float(a),
                z_scale=float(b))
    y, h = nv.nvfp4_residual_norm_fwd(c["x"], c["z"], **args)
    ry, rh, my, mh = R.norm_fwd(n["x"], n["z"], n["w_post"], n["gate"], n["w_pre"], *ra)
    assert y.dtype == c["x"].dtype and (h is None) == (parts == "last")
    _close(y, ry, my, R.E_NORM, "y", not wide)
    if h is not None:
        _close(h, rh, mh, R.E_NORM, "h", True)
    for dy in (c["dy"], None) if parts != "last" else (c["dy"],):
        got = dict(zip(("dx", "dz", "dw_post", "dgate", "dw_pre"),
                       nv.nvfp4_residual_norm_bwd(dy, c["dh"], c["x"], c["z"], **args)))
        ref = R.norm_bwd(None if dy is None else n["dy"], n["dh"], n["x"], n["z"], n["w_post"],
                         n["gate"], n["w_pre"], *ra)
        assert {k for k, v in got.items() if v is not None} == set(ref)
        for k, (v, size) in ref.items():
            # column sums add up to rows / CTAs and CTAs / 8 + 8 further terms in a row
            e = R.E_NORM + (2.0 ** -24 * (T + 64) if k.startswith("dw") or k == "dgate" else 0.0)
            _close(got[k], v, size, e, k, k == "dz" or (k == "dx" and not wide))
    torch.cuda.synchronize()


def test_residual_norm_in_place_and_zero_rows(nv):
    import torch
    t = {k: v.cuda() for k, v in _norm_case(37, 512, True, "row", seed=9).items()}
    t["x"][5] = 0
    t["z"][5] = 0
    args = dict(w_post=t["w_post"], gate=t["gate"], w_pre=t["w_pre"])
    y, h = nv.nvfp4_residual_norm_fwd(t["x"], t["z"], **args)
    assert (y[5] == 0).all() and (h[5] == 0).all()
    x = t["x"].clone()
    y2, h2 = nv.nvfp4_residual_norm_fwd(x, t["z"], y=x, **args)
    assert y2.data_ptr() == x.data_ptr()
    assert torch.equal(y2, y) and torch.equal(h2, h)
    grads = nv.nvfp4_residual_norm_bwd(t["dy"], t["dh"], t["x"], t["z"], **args)
    assert all(torch.isfinite(v.float()).all() for v in grads)
    again = nv.nvfp4_residual_norm_bwd(t["dy"], t["dh"], t["x"], t["z"], **args)
    assert all(torch.equal(u, v) for u, v in zip(grads, again))  # fixed order of every sum


@pytest.mark.parametrize("T,D,wide", [(37, 512, True), (700, 4096, False), (9, 16384, False)])
def test_residual_norm_gradients_in_place(nv, T, D, wide):
    """dx may be dy, and dz may be dh or z (the library's own call: the binding
    allocates its outputs)."""
    import ctypes as C
    import torch
    t = {k: v.cuda() for k, v in _norm_case(T, D, wide, "channel", seed=3).items()}
    want = nv.nvfp4_residual_norm_bwd(t["dy"], t["dh"], t["x"], t["z"], t["w_post"], t["gate"],
                                      t["w_pre"])
    p = nv.NormParams(T, D, int(wide), nv.GATE_CHANNEL, 1e-5, 1.0, 1.0)
    n = C.c_size_t()
    nv.lib.nvfp4_residual_norm_bwd_sizes(T, D, n)
    ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    for dz in ("dh", "z"):
        c = {k: v.clone() for k, v in t.items()}
        dw, dg, dp = (torch.empty(D, device="cuda") for _ in range(3))
        st = nv.lib.nvfp4_residual_norm_bwd(
            p, *[c[k].data_ptr() for k in ("dy", "dh", "x", "z", "w_post", "gate", "w_pre")],
            c["dy"].data_ptr(), c[dz].data_ptr(), dw.data_ptr(), dg.data_ptr(), dp.data_ptr(),
            ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert st == nv.OK
        for got, ref in zip((c["dy"], c[dz], dw, dg, dp), want):
            assert torch.equal(got, ref)


def test_residual_norm_keeps_a_bad_row_to_itself(nv):
    import torch
    t = {k: None if v is None else v.cuda() for k, v in _norm_case(6, 256, False, "none", 2).items()}
    args = dict(w_post=t["w_post"], w_pre=t["w_pre"])
    good = nv.nvfp4_residual_norm_fwd(t["x"], t["z"], **args)
    z = t["z"].clone()
    z[3, 7] = float("nan")
    z[4, 9] = float("inf")
    bad = nv.nvfp4_residual_norm_fwd(t["x"], z, **args)
    keep = [0, 1, 2, 5]
    for u, v in zip(good, bad):
        assert torch.equal(u[keep], v[keep]) and torch.isnan(v[3].float()).all()


def test_residual_norm_weight_gradient_against_differences(nv):
    """y is linear in w_post and in the gate: its differences are exact but for
    the FP32 stream's rounding."""
    import torch
    t = {k: v.cuda() for k, v in _norm_case(9, 64, True, "channel", 5).items()}
    dw, dg = nv.nvfp4_residual_norm_bwd(t["dy"], None, t["x"], t["z"], t["w_post"], t["gate"])[2:4]
    for name, got in (("w_post", dw), ("gate", dg)):
        d = torch.randn(64, generator=torch.Generator().manual_seed(1)).cuda()
        value = []
        for s in (1.0, -1.0):
            u = dict(t)
            u[name] = t[name] + s * d
            y, _ = nv.nvfp4_residual_norm_fwd(t["x"], t["z"], u["w_post"], u["gate"])
            value.append((y.double() * t["dy"].double()).sum().item())
        diff = (value[0] - value[1]) / 2
        size = (t["dy"].double().abs() * t["x"].double().abs()).sum().item()
        assert abs(diff - (got.double() * d.double()).sum().item()) <= 2.0 ** -20 * size


# ---- routing -----------------------------------------------------------------
ROUTE_SHAPES = [(1, 1, 1), (1, 8, 2), (7, 3, 3), (128, 64, 8), (129, 64, 8), (1000, 33, 5),
                (2049, 128, 8), (300, 512, 16), (5000, 8, 2), (3001, 256, 1)]


def _route_logits(T, E, wide, seed):
    import torch
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, E)).astype(np.float32) * 2
    x[rng.random((T, E)) < 0.1] = -np.inf
    x[rng.random(T) < 0.05] = -np.inf            # padding tokens
    x[rng.random((T, E)) < 0.02] = np.nan
    x[rng.random((T, E)) < 0.05] = 1.5           # ties
    x[rng.random((T, E)) < 0.02] = -0.0
    x[rng.random((T, E)) < 0.02] = 0.0
    t = torch.from_numpy(x)
    return t if wide else t.bfloat16()


@pytest.mark.parametrize("T,E,top", ROUTE_SHAPES)
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("chosen", [False, True])
def test_route(nv, T, E, top, wide, chosen):
    import torch
    x = _route_logits(T, E, wide, seed=T * E + top)
    mode = nv.ROUTE_CHOSEN if chosen else nv.ROUTE_ALL
    r = R.route(x.float().numpy(), top, chosen)
    p = nv.nvfp4_route_fwd(x.cuda(), top, mode)
    for k in ("expert", "sizes", "offsets", "row", "source"):
        assert np.array_equal(getattr(p, k).cpu().numpy(), r[k]), k
    assert p.rows == r["source"].size
    _close(p.weight, r["weight"], r["weight"], 2.0 ** -18, "weight", False)
    dw = np.random.default_rng(1).normal(size=(T, top)).astype(np.float32)
    got = nv.nvfp4_route_bwd(x.cuda(), p, torch.from_numpy(dw).cuda(), mode)
    assert got.dtype == x.dtype
    ref, size = R.route_bwd(r, dw.astype(np.float64), chosen)
    _close(got, ref, size, 2.0 ** -17, "dlogits", not wide)
    # strided logits give the same
    wide_x = torch.zeros(T, E + 5, dtype=x.dtype)
    wide_x[:, 3:3 + E] = x
    view = wide_x.cuda()[:, 3:3 + E]
    q = nv.nvfp4_route_fwd(view, top, mode)
    assert all(torch.equal(getattr(p, k), getattr(q, k))
               for k in ("expert", "weight", "sizes", "offsets", "row", "source"))
    assert torch.equal(nv.nvfp4_route_bwd(view, q, torch.from_numpy(dw).cuda(), mode), got)


def test_route_extremes(nv):
    import torch
    inf = float("inf")
    x = torch.tensor([[inf, 1., inf, -3.], [3.4e38, -3.4e38, 0., 1.], [-inf, -inf, -3.4e38, -inf]])
    p = nv.nvfp4_route_fwd(x.cuda(), 2, nv.ROUTE_ALL)
    assert p.expert.cpu().tolist() == [[0, 2], [0, 3], [2, -1]]
    assert p.weight.cpu().tolist() == [[0.5, 0.5], [1.0, 0.0], [1.0, 0.0]]


# ---- rows to the experts and back ----------------------------------------------
@pytest.mark.parametrize("T,E,top,D", [(1, 4, 2, 8), (5, 3, 3, 264), (129, 16, 4, 1024),
                                       (300, 64, 16, 72), (1000, 8, 1, 4096), (33, 5, 2, 8200)])
def test_rows_to_the_experts_and_back(nv, T, E, top, D):
    import torch
    g = torch.Generator().manual_seed(T + D)
    p = nv.nvfp4_route_fwd(_route_logits(T, E, True, seed=D).cuda(), top)
    row, source = p.row.cpu().numpy(), p.source.cpu().numpy()
    x = torch.randn(T, D, generator=g).bfloat16()
    o = torch.randn(p.rows, D, generator=g).bfloat16()  # padding rows hold values too
    dy = torch.randn(T, D, generator=g).bfloat16()
    w = torch.randn(T, top, generator=g)

    xe = torch.full((p.rows, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_dispatch(x.cuda(), p.row, p.source, out=xe)
    want = np.where(source[:, None] >= 0, _f64(x)[np.maximum(source, 0) // top], 0.0)
    assert np.array_equal(_f64(xe), want)

    some = row >= 0
    picked = np.where(some[:, :, None], _f64(o)[np.maximum(row, 0)], 0.0)
    e = (top + 1) * 2.0 ** -24
    for weight in (w, None):
        wn = np.ones((T, top)) if weight is None else _f64(w)
        y = nv.nvfp4_combine(o.cuda(), p.row, None if weight is None else w.cuda())
        terms = wn[:, :, None] * picked
        _close(y, terms.sum(1), np.abs(terms).sum(1), e, "combine", True)

    do = torch.full((p.rows, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    do, dw = nv.nvfp4_combine_bwd(dy.cuda(), o.cuda(), p.row, p.source, w.cuda(), d_o=do)
    src = np.maximum(source, 0)
    want = _f64(w).reshape(-1)[src][:, None] * _f64(dy)[src // top]
    want = np.where(source[:, None] >= 0, want, 0.0)
    _close(do, want, np.abs(want), 2.0 ** -24, "do", True)
    terms = picked * _f64(dy)[:, None, :]
    _close(dw, terms.sum(2), np.abs(terms).sum(2), (D / 32 + 16) * 2.0 ** -24, "dweight", False)


# ---- grouped products ------------------------------------------------------------
def _groups(sizes):
    """sizes, offsets as CUDA tensors and the rows that hold them."""
    import torch
    off = np.concatenate([[0], np.cumsum([(s + 127) // 128 * 128 for s in sizes])])
    return (torch.tensor(sizes, dtype=torch.int32, device="cuda"),
            torch.tensor(off, dtype=torch.int32, device="cuda"), off)


def _decode(q, rows, cols, view=0):
    codes, scales = (q.codes_t, q.scales_t) if view else (q.codes, q.scales)
    return R.decode(codes.cpu().numpy(), scales.cpu().numpy(), q.s_dec.item(), rows, cols)


GROUP_SIZES = [[1], [0, 3, 0], [127, 128, 129], [300, 0, 1, 64, 255, 0], [5, 700], [0, 0],
               [256, 512, 1024]]
GROUP_DIMS = [(128, 64), (384, 320), (256, 512), (640, 1024)]


@pytest.mark.parametrize("sizes", GROUP_SIZES, ids=str)
@pytest.mark.parametrize("N,K", GROUP_DIMS)
@pytest.mark.parametrize("view,spare", [(0, 0), (1, 384)])
@pytest.mark.parametrize("tile", [0, 3, 6])
def test_group_gemm(nv, sizes, N, K, view, spare, tile):
    import torch
    E = len(sizes)
    s, o, off = _groups(sizes)
    rows = max(128, int(off[-1]) + spare)
    g = torch.Generator(device="cuda").manual_seed(N + K)
    # padding rows of A hold values: the product's must be zero all the same
    A = nv.nvfp4_quantize(torch.randn(rows, K, generator=g, device="cuda").bfloat16(), nv.ROW_1X16)
    shape = (E * K, N) if view else (E * N, K)
    W = torch.randn(*shape, generator=g, device="cuda") * 0.05
    B = nv.nvfp4_quantize(W, nv.BLOCK_16X16, nv.EMIT_T)
    C = torch.randn(rows, N, generator=g, device="cuda").bfloat16()
    a = _decode(A, rows, K)
    b = _decode(B, N, E * K, 1) if view else _decode(B, E * N, K)
    ref, live = np.zeros((rows, N)), np.zeros(rows, dtype=bool)
    for e, n in enumerate(sizes):
        be = b[:, e * K:(e + 1) * K] if view else b[e * N:(e + 1) * N]
        ref[off[e]:off[e] + n] = a[off[e]:off[e] + n] @ be.T
        live[off[e]:off[e] + n] = True
    for c in (None, C):
        out = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        nv.nvfp4_group_gemm(A, B, s, o, b_view=view, out=out, C_add=c, tile=tile,
                            d_mode=nv.D_BF16 if c is None else nv.D_BF16_ADD_C)
        got = _f64(out)
        assert (got[~live] == 0).all()
        if live.any():
            want = ref[live] + (0.0 if c is None else _f64(C)[live])
            H.assert_gemm_close(got[live], want, f"{sizes} {N} {K}", rms=np.sqrt(np.mean(ref[live] ** 2)))
    nv.check_device_errors()


@pytest.mark.parametrize("sizes", [[1], [0, 2], [1, 0, 1], [40], [33, 1], [128], [0], [129], [250]],
                         ids=str)
@pytest.mark.parametrize("N,K", [(128, 2048), (384, 2112), (1024, 4096), (1280, 14336), (2048, 4160)])
@pytest.mark.parametrize("view", [0, 1])
def test_group_gemm_of_few_tiles(nv, sizes, N, K, view):
    """Few tiles with a long contraction: pairs of a cluster share a tile (two or
    four, by the tiles there can be), and hand over the rows of the group."""
    import torch
    E = len(sizes)
    s, o, off = _groups(sizes)
    rows = max(128, int(off[-1]))
    g = torch.Generator(device="cuda").manual_seed(N + K)
    A = nv.nvfp4_quantize(torch.randn(rows, K, generator=g, device="cuda").bfloat16(), nv.ROW_1X16)
    shape = (E * K, N) if view else (E * N, K)
    B = nv.nvfp4_quantize(torch.randn(*shape, generator=g, device="cuda") * 0.05, nv.BLOCK_16X16,
                          nv.EMIT_T)
    C = torch.randn(rows, N, generator=g, device="cuda").bfloat16()
    a = _decode(A, rows, K)
    b = _decode(B, N, E * K, 1) if view else _decode(B, E * N, K)
    out = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_group_gemm(A, B, s, o, b_view=view, out=out)
    again = nv.nvfp4_group_gemm(A, B, s, o, b_view=view)
    plus = nv.nvfp4_group_gemm(A, B, s, o, b_view=view, C_add=C, d_mode=nv.D_BF16_ADD_C)
    assert torch.equal(out, again)
    live = np.zeros(rows, dtype=bool)
    for e, n in enumerate(sizes):
        r = slice(off[e], off[e] + n)
        live[r] = True
        if n:
            ref = a[r] @ (b[:, e * K:(e + 1) * K] if view else b[e * N:(e + 1) * N]).T
            H.assert_gemm_close(_f64(out)[r], ref, f"group {e}")
            H.assert_gemm_close(_f64(plus)[r], ref + _f64(C)[r], f"group {e} + C",
                                rms=np.sqrt(np.mean(ref ** 2)))
    assert (_f64(out)[~live] == 0).all() and (_f64(plus)[~live] == 0).all()
    nv.check_device_errors()


@pytest.mark.parametrize("sizes", GROUP_SIZES, ids=str)
@pytest.mark.parametrize("M,N", [(128, 128), (384, 256), (256, 640)])
@pytest.mark.parametrize("spare,tile", [(0, 0), (256, 3), (0, 6)])
def test_group_wgrad(nv, sizes, M, N, spare, tile):
    import torch
    E = len(sizes)
    s, o, off = _groups(sizes)
    rows = max(128, int(off[-1]) + spare)
    g = torch.Generator(device="cuda").manual_seed(M + N)
    live = torch.zeros(rows, 1, device="cuda")
    for e, n in enumerate(sizes):
        live[off[e]:off[e] + n] = 1
    x = (torch.randn(rows, M, generator=g, device="cuda") * live).bfloat16()
    y = (torch.randn(rows, N, generator=g, device="cuda") * live).bfloat16()
    A = nv.nvfp4_quantize(x, nv.COL_1X16, nv.RHT, seed=3)
    B = nv.nvfp4_quantize(y, nv.COL_1X16, nv.RHT, seed=3)
    a, b = _decode(A, M, rows), _decode(B, N, rows)
    ref, size = np.zeros((E, M, N)), np.zeros((E, M, N))
    for e, n in enumerate(sizes):
        w = slice(off[e], off[e] + (n + 63) // 64 * 64)
        ref[e] = a[:, w] @ b[:, w].T
        size[e] = np.abs(a[:, w]) @ np.abs(b[:, w]).T
    out = torch.full((E, M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_group_wgrad(A, B, s, o, out=out, tile=tile)
    got = _f64(out)
    for e, n in enumerate(sizes):
        if n:
            H.assert_gemm_close(got[e], ref[e], f"group {e}")
        else:
            assert (got[e] == 0).all()
    start = torch.randn(E, M, N, generator=g, device="cuda")
    fold = start.clone()
    nv.nvfp4_group_wgrad(A, B, s, o, out=fold, d_mode=nv.D_F32_ACCUM, tile=tile if tile < 6 else 0)
    bound = (np.array(sizes)[:, None, None] / 64 + 64) * 2.0 ** -22 * size \
        + 2.0 ** -23 * (np.abs(_f64(start)) + np.abs(ref))
    assert (np.abs(_f64(fold) - (_f64(start) + ref)) <= bound).all()
    for e, n in enumerate(sizes):
        if not n:
            assert torch.equal(fold[e], start[e])
    nv.check_device_errors()


@pytest.mark.parametrize("tile", [3, 6])
def test_group_outside_the_rows_counts_as_empty(nv, tile):
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    A = nv.nvfp4_quantize(torch.randn(384, 128, generator=g, device="cuda"), nv.ROW_1X16)
    B = nv.nvfp4_quantize(torch.randn(5 * 128, 128, generator=g, device="cuda"), nv.BLOCK_16X16)
    i = dict(dtype=torch.int32, device="cuda")
    sizes = torch.tensor([100, 500, -3, 40, 128], **i)
    offsets = torch.tensor([0, 128, 128, 72, 256, 1 << 30], **i)
    out = torch.full((384, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_group_gemm(A, B, sizes, offsets, out=out, tile=tile)
    a, b = _decode(A, 384, 128), _decode(B, 640, 128)
    got = _f64(out)
    H.assert_gemm_close(got[:100], a[:100] @ b[:128].T, "group 0")
    H.assert_gemm_close(got[256:], a[256:] @ b[512:].T, "group 4")
    assert (got[100:128] == 0).all() and (got[128:256] == 7).all()  # no group's rows
    nv.check_device_errors()


@pytest.mark.parametrize("tile", [3, 6])
def test_group_wait_expires_then_recovers(nv, tile):
    """The grouped kernels' bounded waits: with the injected stall nothing
    arrives, the error word is set, and the next call is whole again."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    A = nv.nvfp4_quantize(torch.randn(256, 256, generator=g, device="cuda"), nv.ROW_1X16)
    B = nv.nvfp4_quantize(torch.randn(512, 256, generator=g, device="cuda"), nv.BLOCK_16X16)
    s, o, off = _groups([100, 128])
    want = nv.nvfp4_group_gemm(A, B, s, o, tile=tile)
    nv.check_device_errors()
    nv.debug_inject(nv.STALL_GEMM, 1_000_000)
    try:
        nv.nvfp4_group_gemm(A, B, s, o, tile=tile)
        with pytest.raises(nv.NVFP4Error) as e:
            nv.check_device_errors()
        assert e.value.status == nv.ERR_DEVICE_TIMEOUT
    finally:
        nv.debug_inject(0, 0)
    nv.check_device_errors()
    assert torch.equal(nv.nvfp4_group_gemm(A, B, s, o, tile=tile), want)
    nv.check_device_errors()


def test_shared_tile_wait_expires_then_recovers(nv):
    """The same with pairs that share a tile: all of them give up and meet at
    their barriers."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    A = nv.nvfp4_quantize(torch.randn(128, 4096, generator=g, device="cuda"), nv.ROW_1X16)
    B = nv.nvfp4_quantize(torch.randn(1024, 4096, generator=g, device="cuda"), nv.BLOCK_16X16)
    s, o, _ = _groups([3])
    want = nv.nvfp4_group_gemm(A, B, s, o)
    nv.check_device_errors()
    nv.debug_inject(nv.STALL_GEMM, 1_000_000)
    try:
        nv.nvfp4_group_gemm(A, B, s, o)
        with pytest.raises(nv.NVFP4Error) as e:
            nv.check_device_errors()
        assert e.value.status == nv.ERR_DEVICE_TIMEOUT
    finally:
        nv.debug_inject(0, 0)
    nv.check_device_errors()
    assert torch.equal(nv.nvfp4_group_gemm(A, B, s, o), want)
    nv.check_device_errors()


def test_norm_wait_expires_then_recovers(nv):
    """The norms' ring of rows: injected, no row arrives; the error word says so
    and the next call is whole."""
    import torch
    t = {k: v.cuda() for k, v in _norm_case(40, 512, False, "channel", 4).items()}
    args = (t["x"], t["z"], t["w_post"], t["gate"], t["w_pre"])
    calls = (lambda: nv.nvfp4_residual_norm_fwd(*args),
             lambda: nv.nvfp4_residual_norm_bwd(t["dy"], t["dh"], *args))
    for call in calls:
        want = call()
        nv.check_device_errors()
        nv.debug_inject(nv.STALL_QUANTIZE, 1_000_000)
        try:
            call()
            with pytest.raises(nv.NVFP4Error) as e:
                nv.check_device_errors()
            assert e.value.status == nv.ERR_DEVICE_TIMEOUT
        finally:
            nv.debug_inject(0, 0)
        nv.check_device_errors()
        assert all(torch.equal(u, v) for u, v in zip(call(), want))
    nv.check_device_errors()


def test_calls_on_another_stream(nv):
    """Outputs and workspaces of a call belong to the stream it is given."""
    import torch
    side = torch.cuda.Stream()
    x = _route_logits(3000, 64, True, seed=8).cuda()
    t = {k: v.cuda() for k, v in _norm_case(900, 1024, False, "channel", 4).items()}
    args = (t["dy"], t["dh"], t["x"], t["z"], t["w_post"], t["gate"], t["w_pre"])
    plan, grads = nv.nvfp4_route_fwd(x, 8), nv.nvfp4_residual_norm_bwd(*args)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        p = nv.nvfp4_route_fwd(x, 8, stream=side)
        q = nv.nvfp4_residual_norm_bwd(*args, stream=side)
        nv.nvfp4_residual_norm_bwd(*args)  # meanwhile, the same call here
    torch.cuda.synchronize()
    assert all(torch.equal(getattr(plan, k), getattr(p, k)) for k in ("row", "source", "weight"))
    assert all(torch.equal(u, v) for u, v in zip(grads, q))


def test_binding_refuses_what_does_not_fit(nv):
    import torch
    c = dict(device="cuda")
    x, z, w = torch.randn(4, 64, **c), torch.randn(4, 64, **c).bfloat16(), torch.ones(64, **c)
    for bad in (dict(x=x.t()), dict(z=z.float()), dict(z=z[:2]), dict(w_post=w[:8]),
                dict(gate=torch.ones(4, **c)), dict(gate=torch.ones(3, 1, **c)), dict(w_pre=w.double())):
        with pytest.raises(ValueError):
            nv.nvfp4_residual_norm_fwd(**{**dict(x=x, z=z, w_post=w, w_pre=w), **bad})
    with pytest.raises(nv.NVFP4Error) as e:
        nv.nvfp4_residual_norm_fwd(torch.randn(4, 60, **c), w_pre=torch.ones(60, **c))
    assert e.value.status == nv.ERR_SHAPE
    with pytest.raises(nv.NVFP4Error) as e:
        nv.nvfp4_residual_norm_fwd(x, z, w, w_pre=w, eps=0.0)
    assert e.value.status == nv.ERR_INVALID_ARG
    for top, E in ((0, 8), (9, 8), (17, 64), (1, 513)):
        with pytest.raises(nv.NVFP4Error) as e:
            nv.nvfp4_route_fwd(torch.randn(3, E, **c), top)
        assert e.value.status == nv.ERR_SHAPE
    with pytest.raises(TypeError):
        nv.nvfp4_route_fwd(torch.randn(3, 8, **c).half(), 2)
    p = nv.nvfp4_route_fwd(torch.randn(3, 8, **c), 2)
    with pytest.raises(ValueError):
        nv.nvfp4_dispatch(z, p.row, p.source)  # four rows for three tokens
    A = nv.nvfp4_quantize(torch.randn(256, 256, **c), nv.ROW_1X16)
    B = nv.nvfp4_quantize(torch.randn(512, 256, **c), nv.BLOCK_16X16)
    s, o, _ = _groups([100, 128])
    with pytest.raises(ValueError):
        nv.nvfp4_group_gemm(A, B, s, o[:2])
    with pytest.raises(ValueError):
        nv.nvfp4_group_gemm(A, B, s[:0], o[:1])
    with pytest.raises(nv.NVFP4Error) as e:
        nv.nvfp4_group_gemm(A, B, s, o, d_mode=nv.D_F32_ACCUM)
    assert e.value.status == nv.ERR_INVALID_ARG
    with pytest.raises(nv.NVFP4Error) as e:
        nv.nvfp4_group_gemm(A, B, s, o, b_view=1)  # B has no transposed codes
    assert e.value.status == nv.ERR_INVALID_ARG


def test_a_graph_keeps_its_scratch_to_itself(nv):
    """A captured call is replayed after a larger one on the same stream: what
    was allocated since is not written, and the replay gives what the call gave."""
    import torch
    stream = torch.cuda.Stream()
    small = [torch.randn(640, 128, device="cuda") for _ in range(2)]
    large = [torch.randn(640, 8192, device="cuda") for _ in range(2)]
    w = [torch.ones(n, device="cuda") for n in (128, 8192)]
    torch.cuda.synchronize()

    def call(t, w):
        return nv.nvfp4_residual_norm_bwd(t[0], None, t[0], t[1].bfloat16(), w_post=w)

    with torch.cuda.stream(stream):
        want = call(small, w[0])
        n = C.c_size_t()
        nv._check(nv.lib.nvfp4_residual_norm_bwd_sizes(640, 128, n), "sizes")
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = call(small, w[0])
        call(large, w[1])
        since = [torch.full((n.value,), 7, dtype=torch.uint8, device="cuda") for _ in range(64)]
        graph.replay()
        stream.synchronize()
    assert all((t == 7).all() for t in since)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    nv.check_device_errors()


@pytest.mark.parametrize("tile", [0, 3, 6])
@pytest.mark.parametrize("view,N,K", [(0, 1280, 192), (1, 1408, 512)])
def test_group_gemm_of_many_tiles_plus_c(nv, tile, view, N, K):
    """Several tiles for each pair of SMs, C fetched for one while another leaves;
    C holds NaN outside the groups, and may be the output."""
    import torch
    sizes = [(37 * e) % 300 for e in range(40)]
    E = len(sizes)
    s, o, off = _groups(sizes)
    rows = int(off[-1]) + 128
    g = torch.Generator(device="cuda").manual_seed(N + K)
    A = nv.nvfp4_quantize(torch.randn(rows, K, generator=g, device="cuda").bfloat16(), nv.ROW_1X16)
    shape = (E * K, N) if view else (E * N, K)
    B = nv.nvfp4_quantize(torch.randn(*shape, generator=g, device="cuda") * 0.05, nv.BLOCK_16X16,
                          nv.EMIT_T)
    C = torch.randn(rows, N, generator=g, device="cuda").bfloat16()
    a = _decode(A, rows, K)
    b = _decode(B, N, E * K, 1) if view else _decode(B, E * N, K)
    ref, live = np.zeros((rows, N)), np.zeros(rows, dtype=bool)
    for e, n in enumerate(sizes):
        be = b[:, e * K:(e + 1) * K] if view else b[e * N:(e + 1) * N]
        ref[off[e]:off[e] + n] = a[off[e]:off[e] + n] @ be.T
        live[off[e]:off[e] + n] = True
    C[torch.from_numpy(~live).cuda()] = float("nan")
    rms = np.sqrt(np.mean(ref[live] ** 2))
    for c, out in ((None, torch.empty_like(C)), (C, torch.empty_like(C)), (C, C)):
        want = ref if c is None else ref + _f64(c)
        nv.nvfp4_group_gemm(A, B, s, o, b_view=view, out=out, C_add=c, tile=tile,
                            d_mode=nv.D_BF16 if c is None else nv.D_BF16_ADD_C)
        got = _f64(out)
        assert (got[~live] == 0).all()
        H.assert_gemm_close(got[live], want[live], f"{N} {K}", rms=rms)
    nv.check_device_errors()


@pytest.mark.parametrize("tile", [3, 6])
def test_group_plus_c_wait_expires_then_recovers(nv, tile):
    """The bounded waits of the calls that add C, whose own copies are in flight."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    A = nv.nvfp4_quantize(torch.randn(256, 256, generator=g, device="cuda"), nv.ROW_1X16)
    B = nv.nvfp4_quantize(torch.randn(512, 256, generator=g, device="cuda"), nv.BLOCK_16X16)
    C = torch.randn(256, 256, generator=g, device="cuda").bfloat16()
    s, o, _ = _groups([100, 128])
    call = lambda: nv.nvfp4_group_gemm(A, B, s, o, C_add=C, d_mode=nv.D_BF16_ADD_C,  # noqa: E731
                                       tile=tile)
    want = call()
    nv.check_device_errors()
    nv.debug_inject(nv.STALL_GEMM, 1_000_000)
    try:
        call()
        with pytest.raises(nv.NVFP4Error) as e:
            nv.check_device_errors()
        assert e.value.status == nv.ERR_DEVICE_TIMEOUT
    finally:
        nv.debug_inject(0, 0)
    nv.check_device_errors()
    assert torch.equal(call(), want)
    nv.check_device_errors()


def test_given_workspaces(nv):
    """A caller's own scratch: bytes on the device, as many as the sizes say."""
    import torch
    logits = torch.randn(100, 16, device="cuda")
    x, z = torch.randn(100, 256, device="cuda"), torch.randn(100, 256, device="cuda").bfloat16()
    w = torch.randn(256, device="cuda")
    n = C.c_size_t()
    nv._check(nv.lib.nvfp4_residual_norm_bwd_sizes(100, 256, n), "sizes")
    calls = [(lambda ws: [getattr(nv.nvfp4_route_fwd(logits, 4, workspace=ws), f)
                          for f in ("expert", "weight", "sizes", "offsets", "row", "source")],
              nv.route_sizes(100, 16, 4)[1]),
             (lambda ws: [t for t in nv.nvfp4_residual_norm_bwd(x, None, x, z, w_post=w,
                                                                 workspace=ws) if t is not None],
              n.value)]
    for call, nbytes in calls:
        want = call(None)
        got = call(torch.empty(nbytes, dtype=torch.uint8, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        with pytest.raises(nv.NVFP4Error) as e:
            call(torch.empty(64, dtype=torch.uint8, device="cuda"))
        assert e.value.status == nv.ERR_WORKSPACE
        for bad in (torch.empty(nbytes, dtype=torch.uint8),
                    torch.empty(nbytes, dtype=torch.float32, device="cuda"),
                    torch.empty(2 * nbytes, dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(ValueError):
                call(bad)
    nv.check_device_errors()
