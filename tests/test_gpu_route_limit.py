"""Routing at the largest number of tokens that it accepts, where the ends of the
blocks' and warps' shares of the tokens pass 2^31: each token gets its slot."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [(1 << 31) - 128, (1 << 31) - 135])
def test_route_takes_every_token(tokens):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding as nv
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("less than 60 GB free")
    assert nv.route_sizes(tokens, 1, 1)[0] == (1 << 31) - 128
    with pytest.raises(nv.NVFP4Error):
        nv.route_sizes((1 << 31) - 127, 1, 1)
    logits = torch.zeros(tokens, 1, dtype=torch.bfloat16, device="cuda")
    plan = nv.alloc_plan(tokens, 1, 1)
    for t in (plan.expert, plan.row, plan.source):
        t.fill_(-7)
    plan.weight.zero_()
    nv.nvfp4_route_fwd(logits, 1, plan=plan)
    assert plan.sizes.item() == tokens and plan.offsets.tolist() == [0, (1 << 31) - 128]
    step = 1 << 27
    for at in range(0, tokens, step):
        n = min(step, tokens - at)
        want = torch.arange(at, at + n, dtype=torch.int32, device="cuda")
        assert (plan.expert[at:at + n] == 0).all() and (plan.weight[at:at + n] == 1).all()
        assert torch.equal(plan.row[at:at + n, 0], want)
        assert torch.equal(plan.source[at:at + n], want)
    assert (plan.source[tokens:] == -1).all()
    nv.check_device_errors()
    del logits, plan
    torch.cuda.empty_cache()
