"""Stochastic rounding in a captured graph: with the counter on the device each
replay rounds with the random numbers of the step that the counter names, as
the calls with that number do one by one; the call's own number stays the same
in every replay."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding
    return binding


def _same(a, b):
    import torch
    return all(torch.equal(getattr(a, k), getattr(b, k)) for k in ("codes", "scales", "s_dec"))


@pytest.mark.parametrize("mode,flags", [("ROW_1X16", "SR"), ("COL_1X16", "SR"),
                                        ("COL_1X16", "SR RHT"), ("BLOCK_16X16", "SR EMIT_T")])
@pytest.mark.parametrize("wide", [False, True])
def test_offset_on_the_device(nv, mode, flags, wide):
    import torch
    m, f = getattr(nv, mode), sum(getattr(nv, k) for k in flags.split())
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(272, 320, generator=g, device="cuda")
    x = x if wide else x.bfloat16()
    # beyond 32 bits too: the low word counts
    for n in (0, 7, (1 << 32) + 9):
        want = nv.nvfp4_quantize(x, m, f, seed=5, offset=n)
        at = torch.tensor([n], device="cuda")
        assert _same(nv.nvfp4_quantize(x, m, f, seed=5, offset=at), want)
        assert _same(nv.nvfp4_quantize_noalloc(x, m, f, seed=5, offset=at), want)
    nv.check_device_errors()


@pytest.mark.parametrize("row,col", [("SR", "SR RHT"), ("", "SR RHT"), ("SR", "RHT"), ("SR", "SR")])
def test_both_offsets_on_the_device(nv, row, col):
    import torch
    rf, cf = (sum(getattr(nv, k) for k in s.split()) for s in (row, col))
    x = torch.randn(272, 320, generator=torch.Generator(device="cuda").manual_seed(3),
                    device="cuda").bfloat16()
    amax = [torch.zeros(1, device="cuda") for _ in range(2)]
    nv.nvfp4_amax(x, *amax, seed=5)
    if "RHT" not in col:
        amax[1] = amax[0]
    args = dict(seed=5, amax_row=amax[0], amax_col=amax[1])
    want = nv.nvfp4_quantize_rowcol(x, rf, cf, row_offset=3, col_offset=4, **args)
    at = torch.tensor([3, 4], device="cuda").split(1)
    got = nv.nvfp4_quantize_rowcol(x, rf, cf, row_offset=at[0] if "SR" in row else 3,
                                   col_offset=at[1] if "SR" in col else 4, **args)
    assert _same(got[0], want[0]) and _same(got[1], want[1])
    nv.check_device_errors()


def test_replays_of_a_step_round_anew(nv):
    import torch
    from nvfp4_block_scaled_03_gb300.moe import MoEBlock
    block = MoEBlock(256, 256, 8, 2)
    x, dy = (torch.randn(300, 256, device="cuda") for _ in range(2))
    zero = lambda: [v.zero_() for v in block.grads.values()]  # noqa: E731
    grads = lambda: [v.clone() for v in block.grads.values()]  # noqa: E731

    def eager(step):
        zero()
        return [block.forward(x).clone(), block.backward(dy, step)] + grads()

    want = [eager(n) for n in range(4)]
    assert not torch.equal(want[0][1], want[1][1])  # another step rounds otherwise
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.forward(x)
        dx = block.backward(dy, step)
        step += 1
    for n in range(4):
        zero()
        graph.replay()
        assert step.item() == n + 1
        assert all(torch.equal(a, b) for a, b in zip([y, dx] + grads(), want[n])), n
    nv.check_device_errors()


def test_device_offset_refusals(nv):
    import torch
    x = torch.randn(128, 128, device="cuda").bfloat16()
    at = torch.zeros(2, dtype=torch.int64, device="cuda")
    for bad in (at, at[:1].int(), at[:1].cpu()):
        with pytest.raises(ValueError):
            nv.nvfp4_quantize(x, nv.ROW_1X16, nv.SR, offset=bad)
    with pytest.raises(nv.NVFP4Error) as e:
        nv.nvfp4_quantize(x, nv.ROW_1X16, 0, offset=at[:1])  # nothing to round
    assert e.value.status == nv.ERR_INVALID_ARG
