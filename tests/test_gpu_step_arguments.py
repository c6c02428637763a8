"""Arguments of a training step's calls that are tensors, whose value changes between the
calls while they stay the same objects."""
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


def test_a_scale_that_changes():
    """The arguments' values count, not which objects hold them."""
    x = torch.randn(100, 16, device="cuda")
    scale, top = torch.tensor(2.0), torch.tensor(3)
    a = nv.nvfp4_route_scored_fwd(x, 4, scale=scale)
    dw = torch.randn(100, 4, device="cuda")
    da = nv.nvfp4_route_scored_bwd(x, a, dw, scale=scale)
    scale.fill_(4.0)
    b = nv.nvfp4_route_scored_fwd(x, 4, scale=scale)
    assert torch.equal(b.weight, 2 * a.weight)
    assert torch.equal(nv.nvfp4_route_scored_bwd(x, b, dw, scale=scale), 2 * da)
    for call in (nv.nvfp4_route_scored_fwd, nv.nvfp4_route_fwd):
        for k in (3, 2, 5):
            top.fill_(k)
            p, q = call(x, top), call(x, k)
            assert torch.equal(p.expert, q.expert) and torch.equal(p.source, q.source)


def test_coefficients_that_change():
    g, m = torch.randn(32, 48, device="cuda"), torch.randn(32, 48, device="cuda")
    a = torch.tensor(3.4445)
    coefs = ((a, -4.775, 2.0315),) * 2
    nv.nvfp4_muon_update(g, m.clone(), steps=2, coefs=coefs)
    a.fill_(2.5)
    got = nv.nvfp4_muon_update(g, m.clone(), steps=2, coefs=coefs)
    want = nv.nvfp4_muon_update(g, m.clone(), steps=2, coefs=(2.5, -4.775, 2.0315))
    assert torch.equal(got, want)


def test_forms_of_coefficients():
    """One triple or one for each step, as tuples, lists, arrays or tensors."""
    g, m = torch.randn(32, 48, device="cuda"), torch.randn(32, 48, device="cuda")
    want = nv.nvfp4_muon_update(g, m.clone(), steps=3)
    c = nv.MUON_COEFS
    for coefs in (list(c), (c,) * 3, [list(c)] * 3, torch.tensor(c), torch.tensor([c] * 3),
                  torch.tensor(c).numpy(), [torch.tensor(c)] * 3):
        assert torch.equal(nv.nvfp4_muon_update(g, m.clone(), steps=3, coefs=coefs), want)
    for coefs in ((1.0, 2.0), (c,) * 2, 1.0, (1.0, c, c), ((1.0,) * 4,) * 3, torch.tensor(1.0)):
        with pytest.raises(ValueError):
            nv.nvfp4_muon_update(g, m.clone(), steps=3, coefs=coefs)
