"""The choice of groups by worths that FP32 does not order: far below a token's largest
logit, where exponentials lose their bits, and beside biases that swallow a score's."""
import math

import pytest
import torch

import route_reference as R

pytestmark = pytest.mark.gpu
nv = None
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _binding():
    global nv
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding
    nv = binding


def same(x, top, score, bias, groups, kept, group_top=2):
    p = nv.nvfp4_route_scored_fwd(x, top, score, bias, groups, kept, group_top)
    want = R.choose(x, top, score, bias, groups, kept, group_top)
    wrong = (p.expert.long() != want).any(1)
    assert not wrong.any(), f"{int(wrong.sum())} of {x.shape[0]} tokens"
    return p


def close_pairs(tokens, groups, size, centre, spread, seed):
    """Logits of groups whose two best have nearly the same sum of exponentials."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = centre + spread * torch.rand(tokens, 1, 1, generator=g, device="cuda").double()
    share = 0.1 + 0.8 * torch.rand(tokens, groups, 1, generator=g, device="cuda").double()
    sure = 1e-3 * torch.randn(tokens, groups, 1, generator=g, device="cuda").double()
    x = (c - 8).repeat(1, groups, size)
    x[:, :, :1] = c + torch.log(share) + sure
    x[:, :, 1:2] = c + torch.log1p(-share) + sure
    return x.reshape(tokens, groups * size).float()


@pytest.mark.parametrize("centre", [-103.0, -98.0, -90.0, -60.0, -10.0])
def test_softmax_groups_far_below_the_maximum(centre):
    """One group near the maximum, three kept: the others' order is by sums of
    exponentials that FP32 holds in a few bits or not at all."""
    x = close_pairs(20000, 8, 4, centre, 5.0, 1)
    x[:, 4:8] = torch.tensor([0.0, -1.0, -3.0, -2.0], device="cuda")
    same(x, 10, 0, None, 8, 3)


@pytest.mark.parametrize("centre", [-88.9, -88.0, -60.0, -10.0])
def test_sigmoid_groups_at_the_end_of_the_range(centre):
    """e^-l is infinite in FP32 from 88.73 on: the sum of a group's two scores is one
    score then, whatever the other."""
    same(close_pairs(20000, 8, 4, centre, 1.0, 2), 10, 1, None, 8, 3)


def test_groups_by_one_or_by_two_and_none_open():
    """Groups of a single open expert, of none and of several side by side, each with
    and without a bias."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(3000, 64, generator=g, device="cuda") * 2
    x[torch.rand(3000, 64, generator=g, device="cuda") < 0.75] = -INF
    bias = torch.randn(64, generator=g, device="cuda") * 0.1
    for score in (0, 1):
        for b in (None, bias * (1.0 if score else 0.1)):
            for group_top in (1, 2):
                same(x, 5, score, b, 16, 4, group_top)
                same(x, 5, score, b, 32, 7, group_top)


@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
def test_groups_of_one_expert_are_as_clear_as_by_one(score):
    """The same choice whether one or two experts count where a group has one, and not
    token by token in 64 bits (eight times as long): at most three times the time."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(65536, 32, generator=g, device="cuda") * 1.5
    bias = torch.randn(32, generator=g, device="cuda") * (0.05 if score else 0.01)

    def call(group_top):
        p = nv.nvfp4_route_scored_fwd(x, 4, score, bias, 32, 8, group_top)
        best = INF
        for _ in range(20):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            nv.nvfp4_route_scored_fwd(x, 4, score, bias, 32, 8, group_top, plan=p)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return p, best

    (p, one), (q, two) = call(1), call(2)
    assert torch.equal(p.expert, q.expert) and torch.equal(p.weight, q.weight)
    assert two <= 3 * one, (two, one)


@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
def test_a_large_bias_beside_its_opposite(score):
    """Groups whose two best have biases that cancel: their worth is known less well than
    that of the groups next to the last kept, and can lie behind theirs."""
    t, groups = 40000, 8
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(t, 2 * groups, generator=g, device="cuda") * 1e-4
    bias = torch.zeros(2 * groups, device="cuda")
    bias[::4], bias[1::4] = 1000.0, -1000.0  # every other group
    same(x, 2, score, bias, groups, 4)
