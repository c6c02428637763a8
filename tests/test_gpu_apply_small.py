"""The step on small masters, whose maxima one CTA of a cluster gathers from the others':
weights with less to do than there are CTAs, many times over."""
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


@pytest.mark.parametrize("n", [1, 3, 5, 4097, 65536, 65541, 262144])
def test_every_maximum_arrives(n):
    """The largest weight wherever it lies, first CTA to last: the maximum of each launch."""
    u = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    places = sorted({0, n // 3, n // 2, n - 1})
    weights = []
    for k, at in enumerate(places * 25):
        w = torch.full((n,), 0.5, device="cuda")
        w[at] = -(2.0 + k)
        weights.append(w)
    torch.cuda.synchronize()
    got = [nv.nvfp4_muon_apply(w, u, 0.1) for w in weights]  # one launch right behind another
    assert torch.cat(got).tolist() == [2.0 + k for k in range(len(weights))]
    nv.check_device_errors()
