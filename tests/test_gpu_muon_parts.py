"""Orthogonalised momentum of matrices with a side of at most 128, shared by CTAs that
hand each other their parts of X X^T: a step's parts stay while the next one's are
written, and the result does not depend on when a CTA comes to read them."""
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


def inputs(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda"),
            torch.randn(*shape, generator=g, device="cuda"))


# parts that every CTA adds by itself, in a cluster and (16 x 60000) in a team that meets
# by a counter
@pytest.mark.parametrize("shape", [(64, 4096), (4096, 64), (16, 2000), (128, 128), (33, 700),
                                   (16, 60000)], ids=lambda s: "x".join(map(str, s)))
def test_a_step_leaves_the_parts_of_the_one_before(shape):
    """What the first step wrote to the workspace is there after the second: a CTA that is
    late reads its own step's."""
    grad, momentum = inputs(shape, 1)
    left = []
    for steps in (1, 2):
        ws = torch.full((nv.muon_sizes(1, *shape),), 0xAB, dtype=torch.uint8, device="cuda")
        nv.nvfp4_muon_update(grad, momentum.clone(), steps=steps, workspace=ws)
        left.append(ws.view(torch.int32))
    nv.check_device_errors()
    written = left[0] != torch.full((4,), 0xAB, dtype=torch.uint8, device="cuda").view(torch.int32)
    assert int(written.sum()) >= min(shape) ** 2
    # a counter of barriers goes on
    assert int((left[0] != left[1])[written].sum()) <= 1


@pytest.mark.parametrize("shape,steps", [((64, 4096), 5), ((16, 2000), 4), ((128, 128), 5),
                                         ((40, 64, 4096), 3), ((30, 33, 3000), 5),
                                         ((200, 20, 7000), 2), ((16, 60000), 5)],
                         ids=lambda s: "x".join(map(str, s)) if isinstance(s, tuple) else str(s))
def test_repeats_beside_a_busy_memory(shape, steps):
    """The same bits alone and while another stream moves memory, over stacks whose teams
    take several matrices with odd and even numbers of steps."""
    grad, momentum = inputs(shape, 2)
    want_buf = momentum.clone()
    want = nv.nvfp4_muon_update(grad, want_buf, steps=steps)
    load = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    other = torch.empty_like(load)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(side):
            other.copy_(load)
        buf = momentum.clone()
        got = nv.nvfp4_muon_update(grad, buf, steps=steps)
        assert torch.equal(got, want) and torch.equal(buf, want_buf)
    torch.cuda.synchronize()
    nv.check_device_errors()
