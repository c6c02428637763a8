"""Orthogonalised momentum where the norm or eps is below what FP32 squares hold."""
import pytest
import torch

pytestmark = pytest.mark.gpu
nv = None
# on chip, one launch for all products, a launch each
SHAPES = [(40, 72), (100, 3001), (200, 328), (300, 1001), (40, 264, 520)]


@pytest.fixture(scope="module", autouse=True)
def _binding():
    global nv
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding
    nv = binding


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("eps", [1e-45, 1e-37, 1e-30, 1e-7])
def test_zeros(shape, eps):
    z = torch.zeros(shape, device="cuda")
    got = nv.nvfp4_muon_update(z, z.clone(), eps=eps)
    nv.check_device_errors()
    assert not got.any()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_norms_below_the_smallest(shape):
    """A norm below 1e-18 counts as 1e-18: U's entries are about 1e-24 here, its matrix
    far from orthogonal after one step of X <- a X + (b A + c A A) X, X = U / 1e-18."""
    g = torch.Generator(device="cuda").manual_seed(1)
    u = torch.randn(shape, generator=g, device="cuda") * 1e-24
    coefs = (3.4445, -4.7750, 2.0315)
    got = nv.nvfp4_muon_update(u, torch.zeros_like(u), mu=0.0, steps=1, eps=1e-37, coefs=coefs)
    nv.check_device_errors()
    # A's terms are below 2e-6 of X: X <- a X, 2^-8 of a value for bf16; X's halves are
    # whole multiples of 2^-24 / 4096, half of one off at most, times a
    want = coefs[0] * (u.double() / 1e-18)
    assert ((got.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -18) * want.abs() + 2.0 ** -35).all()
