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


def test_without_a_maximum():
    """The same step through the library's entry without an amax, at both sizes of it."""
    for n in (1, 5, 65541, 1000003):
        g = torch.Generator(device="cuda").manual_seed(n)
        w = torch.randn(n, generator=g, device="cuda")
        u = torch.randn(n, generator=g, device="cuda").bfloat16()
        a, b = w.clone(), w.clone()
        nv.nvfp4_muon_apply(a, u, 0.02, 3.0, 0.1)
        stream = torch.cuda.current_stream().cuda_stream
        assert nv.lib.nvfp4_muon_apply(b.data_ptr(), u.data_ptr(), n, 0.02, 3.0, 0.1, None, None, 0,
                                       stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(a, b)
