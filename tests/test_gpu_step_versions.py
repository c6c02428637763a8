"""What the calls of a training step tell torch about the tensors that they write in
place."""
import pytest
import torch

pytestmark = pytest.mark.gpu
nv = None


@pytest.fixture(scope="module", autouse=True)
def _binding():
    global nv
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding
    nv = binding


def moved(call, *tensors):
    """Which tensors' versions a call moves."""
    before = [t._version for t in tensors]
    call()
    return [t._version != v for t, v in zip(tensors, before)]


def test_momentum_and_gradient_are_written():
    g, m = torch.randn(32, 48, device="cuda"), torch.randn(32, 48, device="cuda")
    out = torch.empty(32, 48, dtype=torch.bfloat16, device="cuda")
    assert moved(lambda: nv.nvfp4_muon_update(g, m), g, m) == [False, True]
    assert moved(lambda: nv.nvfp4_muon_update(g, m, out=out, zero_grad=True),
                 g, m, out) == [True, True, True]
    # autograd's check of what it saved
    w = torch.ones(32, 48, device="cuda", requires_grad=True)
    y = (w * m).sum()
    nv.nvfp4_muon_update(g, m)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_steps_are_written():
    w, g = torch.randn(3000000, device="cuda"), torch.randn(3000000, device="cuda")
    u, amax = g.bfloat16(), torch.zeros(1, device="cuda")
    assert moved(lambda: nv.nvfp4_sgd_step(w, g, 0.1), w, g) == [True, False]
    assert moved(lambda: nv.nvfp4_sgd_step(w, g, 0.1, zero_grad=True, amax=amax),
                 w, g, amax) == [True, True, True]
    assert moved(lambda: nv.nvfp4_muon_apply(w, u, 0.1, amax=amax),
                 w, u, amax) == [True, False, True]


def test_routing_is_written():
    x, bias = torch.randn(100, 16, device="cuda"), torch.zeros(16, device="cuda")
    p = nv.nvfp4_route_scored_fwd(x, 2, bias=bias)
    fields = (p.expert, p.weight, p.sizes, p.offsets, p.row, p.source)
    assert moved(lambda: nv.nvfp4_route_scored_fwd(x, 2, bias=bias, plan=p), x, bias,
                 *fields) == [False, False] + [True] * 6
    assert moved(lambda: nv.nvfp4_route_balance(p.sizes, bias, 0.1), p.sizes,
                 bias) == [False, True]
    dw, dl = torch.randn(100, 2, device="cuda"), torch.empty_like(x)
    assert moved(lambda: nv.nvfp4_route_scored_bwd(x, p, dw, dlogits=dl), x, dw,
                 dl) == [False, False, True]


def test_inference_tensors_have_no_version():
    with torch.inference_mode():
        g, m = torch.randn(32, 48, device="cuda"), torch.randn(32, 48, device="cuda")
        nv.nvfp4_muon_update(g, m, zero_grad=True)
        nv.nvfp4_route_balance(torch.ones(4, dtype=torch.int32, device="cuda"),
                               torch.zeros(4, device="cuda"), 0.1)
        nv.nvfp4_sgd_step(m, g, 0.1, zero_grad=True)
    nv.check_device_errors()
