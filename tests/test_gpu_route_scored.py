"""Routing by scores on the GPU against 64 bits: the choice exactly, the weights
and gradients within FP32's rounding.

Tolerances.  A weight is scale u_i / sum u with u from expf (2 units in the last
place, and the argument's rounding, |x| 2^-24 of the value for an argument x,
here below 40), one reciprocal, a sum of at most 16 terms and a division: below
(2 (4 + 40) + 16 + 4) 2^-24 < 2^-17 of its value.  A gradient adds a sum of at
most 16 products of those, and one more factor: 2^-16 of the sum of its terms'
magnitudes, plus half a step of the output's type.
"""
import pytest
import torch

import route_reference as R

pytestmark = pytest.mark.gpu
INF = float("inf")
nv = None


@pytest.fixture(scope="module", autouse=True)
def _binding():
    global nv
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding
    nv = binding


def make(tokens, experts, seed, dtype=torch.float32, masked=0.05):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, experts, generator=g, device="cuda") * 2
    x[torch.rand(tokens, experts, generator=g, device="cuda") < masked] = -INF
    x[torch.rand(tokens, generator=g, device="cuda") < masked] = -INF
    return x.to(dtype), torch.randn(experts, generator=g, device="cuda") * 0.1


def check_plan(p, experts):
    sizes, offsets, row, source = R.plan(p.expert.cpu(), experts, p.rows)
    assert p.sizes.tolist() == sizes and p.offsets.tolist() == offsets
    assert p.row.reshape(-1).tolist() == row and p.source.tolist() == source


def check(logits, top, score, bias=None, groups=1, kept=None, group_top=2, renormalise=True,
          scale=1.0, seed=0):
    p = nv.nvfp4_route_scored_fwd(logits, top, score, bias, groups, kept, group_top, renormalise,
                                  scale)
    want = R.choose(logits, top, score, bias, groups, kept, group_top)
    assert torch.equal(p.expert.long(), want)
    check_plan(p, logits.shape[1])
    _, open_, x = R.scores(logits, score)
    x = torch.where(open_, x, -1e300 if score == 0 else -1e3).requires_grad_()
    w = R.weights(x, want, score, renormalise, scale)
    assert ((p.weight.double() - w).abs() <= 2.0 ** -17 * w + 1e-38).all()
    assert (p.weight[want < 0] == 0).all()
    # gradient: against autograd of the formula in 64 bits
    g = torch.Generator(device="cuda").manual_seed(seed)
    dw = torch.randn(logits.shape[0], top, generator=g, device="cuda")
    dl = nv.nvfp4_route_scored_bwd(logits, p, dw, score, renormalise, scale)
    (w * dw.double()).sum().backward()
    grad = torch.where(open_, x.grad, 0.0)
    terms = (w * (dw.double().abs() + (w / scale * dw.double().abs()).sum(1, keepdim=True))).sum(
        1, keepdim=True).expand_as(grad)
    if score == 1:  # of its own slot alone, times 1 - s
        size = torch.zeros_like(grad).scatter_add(
            1, want.clamp(min=0),
            w * (dw.double().abs() + (w / scale * dw.double().abs()).sum(1, keepdim=True)))
    else:
        size = terms
    eps = torch.finfo(logits.dtype).eps / 2
    assert dl.dtype is logits.dtype
    bound = 2.0 ** -16 * size + eps * grad.abs() + 1e-38
    assert ((dl.double() - grad).abs() <= bound.detach()).all()
    return p


CASES = [  # tokens, experts, top, groups, kept, group_top
    (1, 256, 8, 8, 4, 2), (1, 1, 1, 1, 1, 1), (3, 8, 2, 1, 1, 2), (64, 60, 4, 1, 1, 1),
    (65, 160, 6, 8, 3, 1), (500, 96, 16, 16, 4, 2), (777, 384, 8, 1, 1, 2), (300, 512, 8, 32, 5, 2),
    (129, 40, 3, 4, 1, 2), (200, 64, 5, 32, 31, 2), (1000, 33, 7, 1, 1, 2), (90, 24, 2, 8, 2, 2),
    (2000, 128, 8, 2, 1, 1), (31, 510, 10, 2, 2, 2), (64, 512, 16, 1, 1, 2)]


@pytest.mark.parametrize("tokens,experts,top,groups,kept,group_top", CASES)
@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True], ids=["plain", "bias"])
def test_choice_weights_gradient(tokens, experts, top, groups, kept, group_top, score, with_bias):
    for dtype in (torch.float32, torch.bfloat16):
        x, bias = make(tokens, experts, tokens + experts, dtype)
        for renormalise in (True, False):
            check(x, top, score, bias * (1.0 if score else 0.05) if with_bias else None, groups,
                  kept, group_top, renormalise, 1.0 if renormalise else 2.5)


@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3)])
def test_scores_closer_than_fp32(score, groups, kept):
    """Logits a unit in the last place apart: FP32 scores tie, 64 bits order them."""
    t, e = 200, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    order = torch.argsort(torch.rand(t, e, generator=g, device="cuda"), dim=1)
    x = 2.0 + order.float() * 2.0 ** -22
    check(x, 8, score, torch.zeros(e, device="cuda"), groups, kept)
    check(x, 8, score, torch.full((e,), 0.25, device="cuda"), groups, kept)
    check(x, 8, score, None, groups, kept)
    # near ties between different logits, through the bias
    bias = (torch.rand(e, generator=g, device="cuda") * 0.2).float()
    s = 0.6 - bias.double()
    x = torch.log(s / (1 - s)).float().repeat(t, 1) if score else x
    x = x + (order % 3 - 1).float() * 2.0 ** -23
    check(x, 8, score, bias, groups, kept)


@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(score):
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.zeros(70, 64, device="cuda", dtype=dtype)
        for bias in (None, torch.zeros(64, device="cuda")):
            p = check(x, 4, score, bias)
            assert (p.expert == torch.arange(4, device="cuda", dtype=torch.int32)).all()
            check(x, 4, score, bias, groups=8, kept=2)
            x2 = x.clone()
            x2[:, ::2] = -0.0
            x2[:, 40:44] = 1.0
            check(x2, 6, score, bias, groups=4, kept=2)


@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_closer_than_fp32(group_top):
    """Groups whose worths FP32 cannot tell apart, some of them with their second and
    third experts alike or as close."""
    t, e = 400, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(t, 8, 8, generator=g, device="cuda") - 3
    # every group's two best: nearly the same two logits, in other places
    place = torch.argsort(torch.rand(t, 8, 8, generator=g, device="cuda"), dim=2)
    ulp = (torch.rand(t, 8, 2, generator=g, device="cuda") * 4).floor() * 2.0 ** -22
    x.scatter_(2, place[:, :, :2], torch.tensor([2.5, 1.5], device="cuda") + ulp)
    third = x[100:].gather(2, place[100:, :, 1:2]) - (torch.arange(300, device="cuda") % 3).view(
        -1, 1, 1) * 2.0 ** -23
    x[100:].scatter_(2, place[100:, :, 2:3], third)  # as good as the second, or just below
    x = x.view(t, e)
    for bias in (torch.zeros(e, device="cuda"), torch.full((e,), -0.125, device="cuda")):
        check(x, 4, 1, bias, 8, 3, group_top)
        check(torch.zeros_like(x), 4, 1, bias, 8, 3, group_top)
    check(x, 4, 1, torch.randn(e, generator=g, device="cuda") * 1e-7, 8, 3, group_top)


@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
def test_masks(score):
    x, bias = make(100, 64, 5, masked=0.0)
    x[0] = -INF
    x[1] = float("nan")
    x[2, 1:] = -INF
    x[3, 5] = INF
    x[4, 3:60] = float("nan")
    x[5, :56] = -INF  # one group of eight
    x[6, ::8] = -INF
    x[7] = torch.where(torch.arange(64, device="cuda") % 8 == 3, x[7], -INF)  # one of each
    x[8, 5] = x[8, 9] = INF
    for b in (None, bias):
        for groups, kept in ((1, 1), (8, 3)):
            p = nv.nvfp4_route_scored_fwd(x, 6, score, b, groups, kept)
            assert torch.equal(p.expert.long(), R.choose(x, 6, score, b, groups, kept))
            assert (p.weight[p.expert < 0] == 0).all() and torch.isfinite(p.weight).all()
            assert (p.expert[:2] == -1).all()
            live = p.expert[:, 0] >= 0
            assert torch.allclose(p.weight[live].sum(1), torch.ones(int(live.sum()), device="cuda"),
                                  atol=2e-6)
            dl = nv.nvfp4_route_scored_bwd(x, p, torch.ones_like(p.weight), score)
            assert torch.isfinite(dl).all() and (dl[~(x > -INF)] == 0).all()


@pytest.mark.parametrize("shift", [-200.0, -90.0, -30.0, 30.0, 80.0])
def test_far_logits(shift):
    """Where a sigmoid leaves FP32's range its share of a row does not."""
    x, bias = make(200, 32, 6, masked=0.0)
    x = x + shift
    p = nv.nvfp4_route_scored_fwd(x, 4, 1, None)
    want = R.choose(x, 4, 1)
    assert torch.equal(p.expert.long(), want)
    w = R.weights(x.double(), want, 1, True, 1.0)
    assert ((p.weight.double() - w).abs() <= 2.0 ** -16 * w).all()
    if shift < 0:
        p = nv.nvfp4_route_scored_fwd(x, 4, 1, bias)
        assert torch.equal(p.expert.long(), R.choose(x, 4, 1, bias))


def test_bias_only_chooses():
    x, bias = make(300, 64, 7, masked=0.0)
    p = nv.nvfp4_route_scored_fwd(x, 4, 1, bias * 5)
    q = nv.nvfp4_route_scored_fwd(x, 4, 1, None)
    assert not torch.equal(p.expert, q.expert)
    w = R.weights(x.double(), p.expert.long(), 1, True, 1.0)
    assert ((p.weight.double() - w).abs() <= 2.0 ** -17 * w).all()


def test_softmax_modes_agree_with_the_plain_routing():
    for dtype in (torch.float32, torch.bfloat16):
        x, _ = make(700, 100, 8, dtype)
        dw = torch.randn(700, 5, device="cuda")
        for mode, renormalise in ((nv.ROUTE_CHOSEN, True), (nv.ROUTE_ALL, False)):
            a = nv.nvfp4_route_fwd(x, 5, mode)
            b = nv.nvfp4_route_scored_fwd(x, 5, nv.SCORE_SOFTMAX, renormalise=renormalise)
            for k in ("expert", "sizes", "offsets", "row", "source"):
                assert torch.equal(getattr(a, k), getattr(b, k))
            assert torch.allclose(a.weight, b.weight, rtol=2.0 ** -17, atol=0)
            da = nv.nvfp4_route_bwd(x, a, dw, mode)
            db = nv.nvfp4_route_scored_bwd(x, a, dw, nv.SCORE_SOFTMAX, renormalise)
            assert torch.equal(da, db)


def test_leading_dimension_and_alignment():
    for dtype in (torch.float32, torch.bfloat16):
        x, bias = make(100, 64, 9, dtype)
        wide = torch.full((100, 97), 5.0, dtype=dtype, device="cuda")
        for at in (0, 1, 3, 8):
            wide[:, at:at + 64] = x
            p = nv.nvfp4_route_scored_fwd(wide[:, at:at + 64], 6, 1, bias, 8, 4)
            q = nv.nvfp4_route_scored_fwd(x, 6, 1, bias, 8, 4)
            assert torch.equal(p.expert, q.expert) and torch.equal(p.weight, q.weight)
            dw = torch.randn(100, 6, device="cuda")
            assert torch.equal(nv.nvfp4_route_scored_bwd(wide[:, at:at + 64], p, dw),
                               nv.nvfp4_route_scored_bwd(x, q, dw))


def test_finite_differences():
    x, _ = make(40, 24, 10, masked=0.0)
    for score in (0, 1):
        for renormalise in (True, False):
            p = nv.nvfp4_route_scored_fwd(x, 3, score, renormalise=renormalise, scale=2.0)
            dw = torch.randn(40, 3, device="cuda")
            dl = nv.nvfp4_route_scored_bwd(x, p, dw, score, renormalise, 2.0)
            d = torch.randn_like(x).double()
            h = 1e-6
            f = [(R.weights(x.double() + k * h * d, p.expert.long(), score, renormalise, 2.0)
                  * dw.double()).sum() for k in (1, -1)]
            want = (f[0] - f[1]) / (2 * h)
            got = (dl.double() * d).sum()
            assert abs(got - want) <= 1e-4 * (dl.double() * d).abs().sum()


def test_balance():
    for experts in (1, 7, 64, 512):
        g = torch.Generator(device="cuda").manual_seed(experts)
        sizes = torch.randint(0, 50, (experts,), generator=g, device="cuda", dtype=torch.int32)
        bias = torch.randn(experts, generator=g, device="cuda")
        total = int(sizes.sum())
        sign = torch.sign(total - sizes.long() * experts)
        want = bias + 1e-3 * sign.float()
        got = nv.nvfp4_route_balance(sizes, bias, 1e-3)
        assert got is bias and torch.equal(got, want)
    big = torch.full((512,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    big[3] = 0
    bias = torch.zeros(512, device="cuda")
    nv.nvfp4_route_balance(big, bias, 0.5)
    assert bias[3] == 0.5 and (bias[:3] == -0.5).all() and (bias[4:] == -0.5).all()


def test_balance_evens_the_loads():
    x, bias = make(4000, 32, 11, masked=0.0)
    x = x + torch.linspace(-1.5, 1.5, 32, device="cuda")
    bias.zero_()
    first = None
    for _ in range(300):
        p = nv.nvfp4_route_scored_fwd(x, 4, 1, bias)
        first = first if first is not None else int(p.sizes.max())
        nv.nvfp4_route_balance(p.sizes, bias, 3e-3)
    assert int(p.sizes.max()) < 1.2 * 500 < first


def test_graph_and_stream():
    x, bias = make(500, 128, 12)
    y, _ = make(500, 128, 13)
    src = x.clone()
    nv.nvfp4_route_scored_fwd(src, 8, 1, bias, 8, 4)
    b2, b3 = bias.clone(), bias.clone()
    dw = torch.randn(500, 8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p = nv.nvfp4_route_scored_fwd(src, 8, 1, b2, 8, 4)
        dl = nv.nvfp4_route_scored_bwd(src, p, dw)
        nv.nvfp4_route_balance(p.sizes, b2, 1e-2)
    for t in (x, y, x):
        src.copy_(t)
        graph.replay()
        q = nv.nvfp4_route_scored_fwd(t, 8, 1, b3, 8, 4)
        assert torch.equal(p.expert, q.expert) and torch.equal(p.source, q.source)
        assert torch.equal(dl, nv.nvfp4_route_scored_bwd(t, q, dw))
        nv.nvfp4_route_balance(q.sizes, b3, 1e-2)
        assert torch.equal(b2, b3)
    p = nv.nvfp4_route_scored_fwd(x, 8, 1, b3, 8, 4, stream=side)
    side.synchronize()
    assert torch.equal(p.expert, nv.nvfp4_route_scored_fwd(x, 8, 1, b3, 8, 4).expert)


def test_given_plan_and_refusals():
    x, bias = make(50, 32, 14)
    plan = nv.alloc_plan(50, 32, 4)
    assert nv.nvfp4_route_scored_fwd(x, 4, 1, bias, plan=plan) is plan
    bad = [(ValueError, dict(bias=bias[:16])), (ValueError, dict(bias=bias.double())),
           (ValueError, dict(bias=bias.cpu())), (ValueError, dict(plan=nv.alloc_plan(50, 32, 3))),
           (nv.NVFP4Error, dict(groups=3)), (nv.NVFP4Error, dict(groups=64)),
           (nv.NVFP4Error, dict(groups=8, groups_kept=9)), (nv.NVFP4Error, dict(group_top=3)),
           (nv.NVFP4Error, dict(groups=16, groups_kept=1)), (nv.NVFP4Error, dict(scale=0.0)),
           (nv.NVFP4Error, dict(scale=INF)), (nv.NVFP4Error, dict(score=2)),
           (nv.NVFP4Error, dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")))]
    for error, kw in bad:
        with pytest.raises(error):
            nv.nvfp4_route_scored_fwd(x, 4, **kw)
    by_name = nv.nvfp4_route_scored_fwd(logits=x, top=4, bias=bias)
    assert torch.equal(by_name.expert, plan.expert)
    with pytest.raises(TypeError):
        nv.nvfp4_route_scored_fwd(x.half(), 4)
    with pytest.raises(ValueError):
        nv.nvfp4_route_scored_fwd(x.cpu(), 4)
    with pytest.raises(ValueError):
        nv.nvfp4_route_scored_bwd(x, plan, torch.zeros(50, 3, device="cuda"))
    with pytest.raises(nv.NVFP4Error):
        nv.nvfp4_route_balance(plan.sizes, bias, INF)


def test_a_small_call_leaves_its_workspace_alone():
    """Up to 64 tokens: the binding lets all such calls share one."""
    for tokens, experts in ((1, 512), (64, 512), (64, 7)):
        x, bias = make(tokens, experts, 16)
        ws = torch.full((nv.route_sizes(tokens, experts, 4)[1],), 0xAB, dtype=torch.uint8,
                        device="cuda")
        p = nv.nvfp4_route_scored_fwd(x, 4, 1, bias, workspace=ws)
        assert (ws == 0xAB).all()
        assert torch.equal(p.source, nv.nvfp4_route_scored_fwd(x, 4, 1, bias).source)


def test_many_tokens():
    for dtype, groups in ((torch.float32, 8), (torch.bfloat16, 1)):
        x, bias = make(40000, 256, 15, dtype)
        p = nv.nvfp4_route_scored_fwd(x, 8, 1, bias, groups, max(1, groups // 2))
        assert torch.equal(p.expert.long(), R.choose(x, 8, 1, bias, groups, max(1, groups // 2)))
        assert int(p.sizes.sum()) == int((p.expert >= 0).sum())
