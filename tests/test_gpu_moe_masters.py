"""Masters that change between forwards in ways that torch does not see: a forward
quantises them by what they are, unless its caller says that only the block's own
steps have touched them."""
import pytest
import torch

pytestmark = pytest.mark.gpu
nv = moe = None
WEIGHTS = ("gate_proj", "up_proj", "down_proj")


@pytest.fixture(scope="module", autouse=True)
def _modules():
    global nv, moe
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding, moe as m
    nv, moe = binding, m


def stepped_block(seed=0):
    """A block with one step of its matrices behind it, and a batch."""
    block = moe.MoEBlock(256, 384, 16, 3, seed=3, score=1)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(200, 256, generator=g, device="cuda")
    block.forward(x)
    block.backward(torch.randn(200, 256, generator=g, device="cuda"))
    block.muon(0.02, 0.01)
    return block, x


def fresh(block, x):
    """The same forward by a block that has made no step."""
    other = moe.MoEBlock(256, 384, 16, 3, seed=3, score=1)
    for k, w in block.params.items():
        other.params[k].copy_(w)
    other.bias.copy_(block.bias)
    return other.forward(x)


def captured(call):
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


@pytest.mark.parametrize("how", ["copy", "data", "sgd", "scale"])
def test_captured_forward_of_changed_masters(how):
    block, x = stepped_block()
    graph, y = captured(lambda: block.forward(x))
    if how == "sgd":
        for k in block.grads:
            block.grads[k].fill_(1.0)
        block.sgd(0.5)
    for k in WEIGHTS:
        w = block.params[k]
        if how == "copy":
            w.copy_(w * 3)
        elif how == "data":
            w.data.mul_(3)
        elif how == "scale":
            w.mul_(0.3)
    graph.replay()
    assert torch.equal(y, fresh(block, x))
    nv.check_device_errors()


def test_forward_after_a_captured_change():
    """A replay changes the masters without torch's knowing."""
    block, x = stepped_block()
    for k in block.grads:
        block.grads[k].fill_(1.0)
    graph, _ = captured(lambda: block.sgd(0.5))
    block.muon(0.02, 0.01)
    for k in block.grads:
        block.grads[k].fill_(1.0)
    graph.replay()
    assert torch.equal(block.forward(x), fresh(block, x))


def test_forward_after_a_change_of_the_data():
    block, x = stepped_block()
    for k in WEIGHTS:
        block.params[k].data.mul_(3)
    assert torch.equal(block.forward(x), fresh(block, x))


def test_told_so_a_forward_takes_the_step_s_amaxes():
    block, x = stepped_block()
    want = block.forward(x)
    assert torch.equal(block.forward(x, after_muon=True), want)
    own = block.amax["up_proj"].clone()
    block.amax["up_proj"].mul_(8)  # not the weight's own any more
    block.forward(x, after_muon=True)
    assert torch.equal(block.saved["up_proj"].amax, 8 * own)
    assert torch.equal(block.forward(x), want)
    assert torch.equal(block.saved["up_proj"].amax, own)
    # what torch sees ends it
    block.params["up_proj"].mul_(0.3)
    assert torch.equal(block.forward(x, after_muon=True), fresh(block, x))


def test_a_whole_step_captured_with_its_amaxes():
    """Replays against eager steps that read the weights."""
    (block, x), (eager, _) = stepped_block(), stepped_block()
    dy = torch.randn(200, 256, device="cuda")
    count = torch.zeros(1, dtype=torch.int64, device="cuda")

    def whole(b, step, told):
        y = b.forward(x, after_muon=told)
        b.backward(dy, step)
        b.muon(0.02, 0.01)
        return y

    def both():
        y = whole(block, count, True)
        count.add_(1)
        return y

    graph, y = captured(both)
    for k in range(3):
        graph.replay()
        assert torch.equal(y, whole(eager, torch.full_like(count, k), False))
        for name, w in block.params.items():
            assert torch.equal(w, eager.params[name]), name
    nv.check_device_errors()


def test_a_step_that_was_only_captured():
    """It has not run: a change of the weights before it has still ended their amaxes."""
    block, x = stepped_block()
    for k in WEIGHTS:
        block.params[k].mul_(3)
    graph, _ = captured(lambda: block.muon(0.02, 0.01))
    assert torch.equal(block.forward(x, after_muon=True), fresh(block, x))
    graph.replay()
    assert torch.equal(block.forward(x, after_muon=True), fresh(block, x))
