"""A training step's operators where offsets pass 32 bits, and the update's error against
what the header promises.

That: products within 1.5e-3 of the result in the 2-norm, and one rounding to bf16.  The
rounding's errors of N elements are independent of the products' and of one another, so
the squares add up, but for a chance of some 1 / sqrt(N) of each term, five of which are
allowed."""
import math

import pytest
import torch

import route_reference as R

pytestmark = pytest.mark.gpu
nv = None
COEFS = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module", autouse=True)
def _binding():
    global nv
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding
    nv = binding
    yield
    torch.cuda.empty_cache()


def reference(grad, momentum, mu=0.95, steps=5):
    """(update, momentum) of one matrix in 64 bits."""
    v = mu * momentum.double() + grad.double()
    x = grad.double() + mu * v
    x = x / x.square().sum().sqrt()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    a, b, c = COEFS
    for _ in range(steps):
        p = x @ x.t()
        x = a * x + (b * p + c * p @ p) @ x
    return (x.t() if tall else x), v


def promised(got, want):
    n = want.numel()
    size = float(want.square().sum())
    err = float((got.double() - want).square().sum()) / size
    half = float((want.bfloat16().double() - want).square().sum()) / size
    few = 5 / math.sqrt(n)
    most = 1.5e-3 ** 2 + half * (1 + few) + 2 * 1.5e-3 * math.sqrt(half) * few
    assert err <= most, (math.sqrt(err), math.sqrt(most))


@pytest.mark.parametrize("shape,rank", [((64, 4096), None), ((4096, 64), None), ((100, 9001), None),
                                        ((1024, 1024), None), ((777, 1290), None),
                                        ((256, 8192), None), ((2048, 2048), None),
                                        ((3000, 1500), None), ((512, 1024), 64), ((300, 600), 8)])
def test_error_of_the_update(shape, rank):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    if rank is None:
        grad, mom = (torch.randn(*shape, generator=g, device="cuda") for _ in range(2))
    else:
        grad = (torch.randn(shape[0], rank, generator=g, device="cuda")
                @ torch.randn(rank, shape[1], generator=g, device="cuda"))
        mom = 2 * grad
    want, _ = reference(grad, mom)
    promised(nv.nvfp4_muon_update(grad, mom.clone()), want)


# the products' kernel in pairs of CTAs, and the one on chip with rows of ragged width
@pytest.mark.parametrize("batch,rows,cols", [(515, 2048, 2048), (2400, 101, 9001)])
def test_stacks_beyond_32_bits(batch, rows, cols):
    assert batch * rows * cols > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(batch)
    grad = torch.empty(batch, rows, cols, dtype=torch.bfloat16, device="cuda")
    mom = torch.empty(batch, rows, cols, device="cuda")
    for i in range(batch):
        grad[i] = torch.randn(rows, cols, generator=g, device="cuda")
        mom[i] = torch.randn(rows, cols, generator=g, device="cuda")
    looked_at = (0, 1, batch // 2, batch - 2, batch - 1)
    before = {i: (grad[i].clone(), mom[i].clone()) for i in looked_at}
    got = nv.nvfp4_muon_update(grad, mom, zero_grad=True)
    nv.check_device_errors()
    assert not any(bool(grad[i].any()) for i in range(batch))
    for i in looked_at:
        want, v = reference(*before[i])
        promised(got[i], want)
        assert (mom[i].double() - v).abs().le(
            2.0 ** -23 * (v.abs() + before[i][1].abs())).all()


def test_a_master_beyond_32_bits():
    n = 2 ** 31 + 4099
    w = torch.full((n,), 0.5, device="cuda")
    u = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    w[-1], u[-2] = -3.0, -8.0
    amax = nv.nvfp4_muon_apply(w, u, 0.125, 2.0)
    assert float(amax) == 3.25
    assert w[-2:].tolist() == [2.5, -3.25]
    for part in w[:-2].split(1 << 28):
        assert (part == 0.25).all()


def test_logits_beyond_32_bits():
    tokens, experts = 2 ** 22 + 77, 512
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.empty(tokens, experts, dtype=torch.bfloat16, device="cuda")
    for part in x.split(1 << 18):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    bias = torch.randn(experts, generator=g, device="cuda") * 0.1
    p = nv.nvfp4_route_scored_fwd(x, 2, nv.SCORE_SIGMOID, bias, 8, 4, 2)
    dw = torch.randn(tokens, 2, generator=g, device="cuda")
    dl = nv.nvfp4_route_scored_bwd(x, p, dw)
    for at in (slice(0, 500), slice(tokens // 2, tokens // 2 + 500), slice(tokens - 500, tokens)):
        want = R.choose(x[at], 2, 1, bias, 8, 4, 2)
        assert torch.equal(p.expert[at].long(), want)
        x64 = x[at].double().requires_grad_()
        w = R.weights(x64, want, 1, True, 1.0)
        assert ((p.weight[at].double() - w).abs() <= 2.0 ** -17 * w).all()
        (w * dw[at].double()).sum().backward()
        # w_i (1 - s_i) sum_j w_j (dw_i - dw_j): 2^-16 of its terms, one rounding to bf16
        terms = w * (dw[at].double().abs() + (w * dw[at].double().abs()).sum(1, keepdim=True))
        size = torch.zeros_like(x64).scatter_add(1, want, terms)
        grad = x64.grad
        bound = 2.0 ** -16 * size + 2.0 ** -8 * grad.abs() + 1e-38
        assert ((dl[at].double() - grad).abs() <= bound.detach()).all()
    assert int(p.sizes.sum()) == 2 * tokens
    rows = p.row.reshape(-1).long()
    assert torch.equal(p.source[rows].long(), torch.arange(2 * tokens, device="cuda"))
