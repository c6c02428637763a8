"""The mixture-of-experts block end to end on the GPU: its forward stage by
stage against 64 bits, its gradients' direction against the block without
quantisation, captured as a graph, and trained.

Stages are compared on the block's own inputs to them, with the tolerances of
the operators' own tests.  Gradients: a product of two 4-bit operands is off by
about 0.16 of its size, a stochastically rounded one by 0.26; through the
gated product, up to three products in a row and the weight gradients' own two
operands that adds up to less than 0.75, so the angle to the exact gradient
has a cosine above 1 / sqrt(1 + 0.75^2) = 0.8 (a wrong sign, a wrong operand
or a missing term would not)."""
import numpy as np
import pytest

import gpu_helpers as H
import moe_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import moe
    return moe


def _reference(block, x, expert):
    """y and z of the block in 64 bits, with the experts chosen."""
    import torch
    p = {k: v.double().requires_grad_() for k, v in block.params.items()}
    x = x.double().requires_grad_()
    norm = lambda v, w: v / torch.sqrt((v * v).mean(1, keepdim=True) + block.eps) * w  # noqa: E731
    h = norm(x, p["w_in"])
    logits = h @ p["router"].t()
    weight = torch.softmax(torch.gather(logits, 1, expert), 1)
    E, F, D = block.experts, block.ffn, block.hidden
    wg, wu = p["gate_proj"].view(E, F, D), p["up_proj"].view(E, F, D)
    wd = p["down_proj"].view(E, D, F)
    z = torch.zeros_like(x)
    for e in range(E):
        t, j = torch.nonzero(expert == e, as_tuple=True)
        a = torch.nn.functional.silu(h[t] @ wg[e].t()) * (h[t] @ wu[e].t())
        z = z.index_add(0, t, weight[t, j][:, None] * (a @ wd[e].t()))
    return x + block.z_scale * p["gate"] * norm(z, p["w_out"]), z, x, p


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _within(got, ref, size, e, name):
    d = np.abs(_f64(got) - ref)
    bad = d > e * size + R.half_ulp_bf16(np.abs(ref) + e * size)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.size} off"


def _decode(q, view=0):
    r, c = (q.cols, q.rows) if view else (q.rows, q.cols)
    codes, scales = (q.codes_t, q.scales_t) if view else (q.codes, q.scales)
    return R.decode(codes.cpu().numpy(), scales.cpu().numpy(), q.s_dec.item(), r, c)


def _grouped(a, b, plan, n):
    """a [rows, K] times each group's [n, K] of b, rows outside the groups zero."""
    out = np.zeros((a.shape[0], n))
    for e, (size, off) in enumerate(zip(plan.sizes.tolist(), plan.offsets.tolist())):
        out[off:off + size] = a[off:off + size] @ b[e * n:(e + 1) * n].T
    return out


@pytest.mark.parametrize("tokens,wide", [(1, True), (200, False), (333, True)])
def test_forward_stages(moe, tokens, wide):
    import torch
    nv = moe.nv
    block = moe.MoEBlock(256, 512, 8, 2, z_scale=0.5)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(tokens, 256, generator=g, device="cuda")
    x = x if wide else x.bfloat16()
    y = block.forward(x)
    nv.check_device_errors()
    s, p = block.saved, {k: _f64(v) for k, v in block.params.items()}
    plan, eps = s["plan"], float(np.float32(block.eps))
    _, rh, _, mh = R.norm_fwd(_f64(x), None, None, None, p["w_in"], eps, 1.0, 1.0)
    _within(s["h"], rh, mh, R.E_NORM, "h")
    r = R.route(s["logits"].float().cpu().numpy(), 2, True)
    for k in ("expert", "sizes", "offsets", "row", "source"):
        assert np.array_equal(getattr(plan, k).cpu().numpy(), r[k]), k
    src = np.maximum(r["source"], 0)
    xe = torch.from_numpy(np.where(r["source"][:, None] >= 0, _f64(s["h"])[src // 2], 0.0))
    qx = nv.nvfp4_quantize(xe.bfloat16().cuda(), nv.ROW_1X16)
    for name, got, n in (("gate_proj", s["G"], 512), ("up_proj", s["U"], 512)):
        H.assert_gemm_close(_f64(got), _grouped(_decode(qx), _decode(s[name]), plan, n), name)
    hh, _, _ = nv.nvfp4_swiglu_fwd(s["G"], s["U"])
    qh = nv.nvfp4_quantize(hh, nv.ROW_1X16)
    H.assert_gemm_close(_f64(s["o"]), _grouped(_decode(qh), _decode(s["down_proj"]), plan, 256),
                        "down_proj")
    picked = np.where(r["row"][:, :, None] >= 0, _f64(s["o"])[np.maximum(r["row"], 0)], 0.0)
    terms = picked * _f64(plan.weight)[:, :, None]
    _within(s["z"], terms.sum(1), np.abs(terms).sum(1), 2.0 ** -22, "z")
    ry, _, my, _ = R.norm_fwd(_f64(x), _f64(s["z"]), p["w_out"], p["gate"], None, eps, 1.0, 0.5)
    _within(y, ry, my, R.E_NORM, "y")


@pytest.mark.parametrize("tokens,wide", [(200, False), (777, True)])
def test_gradients_point_the_right_way(moe, tokens, wide):
    import torch
    block = moe.MoEBlock(256, 512, 8, 2, z_scale=0.5)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(tokens, 256, generator=g, device="cuda")
    x = x if wide else x.bfloat16()
    dy = torch.randn(tokens, 256, generator=g, device="cuda").to(x.dtype)
    block.forward(x)
    dx = block.backward(dy)
    moe.nv.check_device_errors()
    ry, rz, rx, p = _reference(block, x, block.saved["plan"].expert.long())
    ry.backward(dy.double())
    cos = lambda a, b: torch.nn.functional.cosine_similarity(  # noqa: E731
        a.double().flatten(), b.flatten(), 0).item()
    assert cos(dx.double() - dy.double(), rx.grad - dy.double()) > 0.8
    for k in block.params:
        assert cos(block.grads[k], p[k].grad) > 0.8, k


def test_block_step_as_a_graph(moe):
    """Forward and backward captured once and replayed on new inputs give what
    the calls give one by one: nothing of a plan reaches the host."""
    import torch
    block = moe.MoEBlock(256, 256, 16, 4)
    x, dy = (torch.randn(300, 256, device="cuda") for _ in range(2))
    zero = lambda: [v.zero_() for v in block.grads.values()]  # noqa: E731
    block.forward(x)
    block.backward(dy)   # kernels are configured by an uncaptured call
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.forward(x)
        dx = block.backward(dy)
    for seed in (1, 2):
        x.copy_(torch.randn(300, 256, generator=torch.Generator().manual_seed(seed)))
        zero()
        graph.replay()
        got = [y.clone(), dx.clone()] + [v.clone() for v in block.grads.values()]
        zero()
        want = [block.forward(x), block.backward(dy)] + list(block.grads.values())
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    moe.nv.check_device_errors()


def test_block_learns(moe):
    losses = moe.main(steps=20, tokens=200, hidden=256, ffn=256)
    assert losses[-1] < 0.8 * losses[0]
