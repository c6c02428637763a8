"""The gradient of scored routing at the ends of the range of its scale."""
import pytest
import torch

import route_reference as R

pytestmark = pytest.mark.gpu
nv = None


@pytest.fixture(scope="module", autouse=True)
def _binding():
    global nv
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding
    nv = binding


@pytest.mark.parametrize("scale", [1e-39, 1e-30, 1.0, 2.5, 1e30, 3e38])
@pytest.mark.parametrize("score,renormalise", [(0, True), (0, False), (1, True), (1, False)])
def test_scales(scale, score, renormalise):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(100, 24, generator=g, device="cuda")
    # gradients that leave the logits' around 1e-2 and none infinite
    dw = torch.randn(100, 4, generator=g, device="cuda") * min(1 / scale, 1e37) * 1e-2
    p = nv.nvfp4_route_scored_fwd(x, 4, score, renormalise=renormalise, scale=scale)
    got = nv.nvfp4_route_scored_bwd(x, p, dw, score, renormalise, scale).double()
    x64 = x.double().requires_grad_()
    want = R.choose(x, 4, score)
    assert torch.equal(p.expert.long(), want)
    c = float(torch.tensor(scale))
    w = R.weights(x64, want, score, renormalise, c)
    (w * dw.double()).sum().backward()
    # a weight is off by a step of 2^-149 at most where it is that small, its share by as
    # much of the scale; else all by 2^-16 of the terms that add up
    step, w, d = 2.0 ** -149, w.detach(), dw.double().abs()
    spread = (d.amax(1, keepdim=True) + d)
    off = (step + 2.0 ** -17 * w) * spread * 4 + w * (step / c + 2.0 ** -17) * spread * 4
    bound = off.sum(1, keepdim=True).expand_as(got)
    assert torch.isfinite(got).all()
    assert ((got - x64.grad).abs() <= bound + step).all()
