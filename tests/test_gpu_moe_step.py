"""A training step of the mixture-of-experts block with the scored router, its bias and
the orthogonalised momentum together: the router's part against 64 bits on the block's
own tensors, the masters' step against the iteration in 64 bits, and the whole step
captured as a graph.  Tolerances: those of the operators' own tests (route: 2^-17 of a
weight, muon: 2^-7 of an update in the 2-norm)."""
import math

import pytest
import torch

import route_reference as R

pytestmark = pytest.mark.gpu
nv = moe = None


@pytest.fixture(scope="module", autouse=True)
def _modules():
    global nv, moe
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding, moe as m
    nv, moe = binding, m


def make(score=1, **kw):
    args = dict(score=score, groups=4, groups_kept=2, route_scale=2.0) | kw
    return moe.MoEBlock(256, 384, 16, 3, seed=3, **args)


def data(seed, tokens=200):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(tokens, 256, generator=g, device="cuda"),
            torch.randn(tokens, 256, generator=g, device="cuda"))


@pytest.mark.parametrize("score,renormalise", [(1, True), (1, False), (0, True)])
def test_router_in_the_block(score, renormalise):
    block = make(score, renormalise=renormalise)
    block.bias.copy_(torch.randn(16, device="cuda") * 0.05)
    x, dy = data(1)
    block.forward(x)
    plan, logits = block.saved["plan"], block.saved["logits"]
    want = R.choose(logits, 3, score, block.bias, 4, 2)
    assert torch.equal(plan.expert.long(), want)
    w = R.weights(logits.double(), want, score, renormalise, 2.0)
    assert ((plan.weight.double() - w).abs() <= 2.0 ** -17 * w).all()
    before = block.grads["router"].clone()
    block.backward(dy)
    # the router's gradient: its logits' (rounded to bf16) times h
    dweight = nv.nvfp4_combine_bwd(
        nv.nvfp4_residual_norm_bwd(dy, None, x, block.saved["z"], block.params["w_out"],
                                   block.params["gate"], eps=block.eps)[1],
        block.saved["o"], plan.row, plan.source, plan.weight)[1]
    l64 = logits.double().requires_grad_()
    (R.weights(l64, want, score, renormalise, 2.0) * dweight.double()).sum().backward()
    ref = l64.grad.t() @ block.saved["h"].double()
    got = (block.grads["router"] - before).double()
    # each logit's gradient is rounded to bf16 once, 2^-8 of it at most
    size = l64.grad.abs().t() @ block.saved["h"].double().abs()
    assert ((got - ref).abs() <= 2.0 ** -7 * size + 1e-12).all()
    nv.check_device_errors()


def test_masters_step():
    block = make()
    x, dy = data(2)
    block.forward(x)
    block.backward(dy)
    lr, vector_lr, mu, decay = 0.02, 0.01, 0.9, 0.1
    old = {k: v.clone() for k, v in block.params.items()}
    grads = {k: v.clone() for k, v in block.grads.items()}
    for _ in range(2):  # the second with a momentum
        block.muon(lr, vector_lr, mu, decay)
        assert all(not g.any() for g in block.grads.values())
        for k in block.grads:
            block.grads[k].copy_(grads[k])
    for name, w in block.params.items():
        shape, g = block.matrices.get(name), grads[name].double()
        if shape is None:
            want = old[name].double() - 2 * vector_lr * g
            assert torch.allclose(w.double(), want, rtol=1e-6, atol=1e-9)
            continue
        want, v = old[name].double().view(shape), torch.zeros(shape, device="cuda").double()
        bound = 0.0
        for _ in range(2):
            v = mu * v + g.view(shape)
            u = g.view(shape) + mu * v
            o = u / u.square().sum((-2, -1), keepdim=True).sqrt().clamp(min=1e-7)
            a, b, c = nv.MUON_COEFS
            for _ in range(5):
                p = o @ o.transpose(-1, -2)
                o = a * o + (b * p + c * p @ p) @ o
            step = lr * 0.2 * math.sqrt(max(shape[-2:]))
            want = (1 - lr * decay) * want - step * o
            bound = bound + 2.0 ** -7 * step * o.square().sum((-2, -1)).sqrt()
        off = (w.double().view(shape) - want).square().sum((-2, -1)).sqrt()
        assert (off <= bound + 1e-5 * want.square().sum((-2, -1)).sqrt()).all(), name
    assert torch.equal(block._known_amax("up_proj"), block.params["up_proj"].abs().max().view(1))
    nv.check_device_errors()


def test_given_amax_and_its_end():
    """The amaxes of the last step stand for the weights until one is changed."""
    block, plain = make(), make()
    x, dy = data(3)
    for b in (block, plain):
        b.forward(x)
        b.backward(dy)
        b.muon(0.02, 0.01)
    plain.stepped.clear()
    assert torch.equal(block.forward(x), plain.forward(x))
    for b in (block, plain):
        b.params["up_proj"].mul_(0.5)
    assert block._known_amax("up_proj") is None and block._known_amax("down_proj") is not None
    assert torch.equal(block.forward(x), plain.forward(x))
    # a step past the block, and another tensor in the weight's place
    for b in (block, plain):
        nv.nvfp4_sgd_step(b.params["down_proj"], torch.ones_like(b.params["down_proj"]), 0.5)
        b.params["gate_proj"] = b.params["gate_proj"] * 2
    assert block._known_amax("down_proj") is None and block._known_amax("gate_proj") is None
    assert torch.equal(block.forward(x), plain.forward(x))


def test_balance():
    block = make()
    x, _ = data(4)
    block.forward(x)
    sizes = block.saved["plan"].sizes.double()
    block.balance(0.25)
    assert torch.equal(block.bias.double(), 0.25 * torch.sign(sizes.mean() - sizes))
    with pytest.raises(ValueError):
        moe.MoEBlock(256, 384, 16, 3).balance(0.1)


def test_captured_step():
    """Forward, backward, update and balance as one graph, against the same calls."""
    block, eager = make(), make()
    x, dy = data(5)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def whole(b, s):
        y = b.forward(x)
        b.backward(dy, s)
        b.muon(0.02, 0.01, decay=0.05)
        b.balance(1e-2)
        return y

    for b in (block, eager):  # the momenta exist, every kernel has run
        whole(b, torch.zeros(1, dtype=torch.int64, device="cuda"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = whole(block, step)
        step += 1
    for k in range(3):
        graph.replay()
        want = whole(eager, torch.full((1,), k, dtype=torch.int64, device="cuda"))
        assert torch.equal(y, want)
        for name in block.params:
            assert torch.equal(block.params[name], eager.params[name]), name
        assert torch.equal(block.bias, eager.bias)
    nv.check_device_errors()


def test_the_first_step_is_not_captured():
    """A graph would make the momenta anew in every replay."""
    block = make()
    x, dy = data(7)
    block.forward(x)
    block.backward(dy)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="momenta"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            block.muon(0.02, 0.01)
    torch.cuda.synchronize()
    block.muon(0.02, 0.01)
    nv.check_device_errors()


def test_plain_block_is_unchanged():
    """Without a score the block routes by the logits as before."""
    block = moe.MoEBlock(256, 384, 16, 3, seed=3)
    x, dy = data(6)
    block.forward(x)
    plan = nv.nvfp4_route_fwd(block.saved["logits"], 3, nv.ROUTE_CHOSEN)
    assert torch.equal(plan.expert, block.saved["plan"].expert)
    assert torch.equal(plan.weight, block.saved["plan"].weight)
    block.backward(dy)
    block.sgd(0.01)
    assert not block.stepped


def test_trains():
    losses = moe.main(steps=3, tokens=100, hidden=256, ffn=256, muon_lr=0.02)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
