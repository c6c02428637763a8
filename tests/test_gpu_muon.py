"""Orthogonalised momentum on the GPU against the iteration in 64 bits, and the
step that applies it.

Tolerance of the update, in the 2-norm of the difference over that of the
result: 2^-8 for its rounding to bf16 (half a step is at most 2^-8 of a value),
and as much again for the products' f16 operands.  Those: a step rounds E, F and
X's first half, each by at most 2^-11 of a value and by 2^-11 / sqrt(3) in the
mean square; E's error reaches X times |b| = 4.8 at most, F's times 1, X's times
the norm of F, below 2.8, so a step adds at most sqrt(4.8^2 + 1 + 2.8^2) 2^-11 /
sqrt(3) = 1.6e-3, five of them, independent, 3.6e-3 < 2^-8; later steps do not
enlarge what belongs to singular values near 1, and the small ones, which they
do, are carried in 22 bits.
"""
import itertools

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


COEFS = (3.4445, -4.7750, 2.0315)
TOL = 2 * 2.0 ** -8


def reference(grad, momentum, mu, nesterov, steps, coefs, eps):
    """(update, momentum) in 64 bits."""
    g = grad.double()
    v = mu * momentum.double() + g
    u = g + mu * v if nesterov else v
    x = u / u.square().sum((-2, -1), keepdim=True).sqrt().clamp(min=eps)
    per = [coefs] * steps if not hasattr(coefs[0], "__len__") else coefs
    for a, b, c in per:
        if x.shape[-2] <= x.shape[-1]:
            p = x @ x.transpose(-1, -2)
            x = a * x + (b * p + c * p @ p) @ x
        else:
            p = x.transpose(-1, -2) @ x
            x = a * x + x @ (b * p + c * p @ p)
    return x, v


def inputs(shape, seed, dtype=torch.float32, rank=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m = torch.randn(*shape, generator=g, device="cuda")
    if rank is not None:
        a = torch.randn(*shape[:-1], rank, generator=g, device="cuda")
        b = torch.randn(*shape[:-2], rank, shape[-1], generator=g, device="cuda")
        return (a @ b).to(dtype), 2 * (a @ b)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype), m


def off(got, want):
    """2-norm of the difference over that of the result, the worst matrix."""
    d = (got.double() - want).square().sum((-2, -1)).sqrt()
    return float((d / want.square().sum((-2, -1)).sqrt()).max())


def run(grad, momentum, tol=TOL, **kw):
    args = dict(mu=0.95, nesterov=True, steps=5, coefs=COEFS, eps=1e-7) | kw
    want, v = reference(grad, momentum, **args)
    buf = momentum.clone()
    got = nv.nvfp4_muon_update(grad, buf, **args)
    nv.check_device_errors()
    assert got.dtype is torch.bfloat16 and got.shape == grad.shape
    # an FMA a value: half a step of fp32, and the product's before it
    assert (buf.double() - v).abs().le(2.0 ** -23 * (v.abs() + momentum.abs())).all()
    assert off(got, want) <= tol, (tuple(grad.shape), off(got, want))
    return got


SHAPES = [(1, 1), (1, 7), (7, 1), (8, 8), (16, 48), (31, 33), (33, 31), (64, 4096), (4096, 64),
          (100, 260), (260, 100), (127, 129), (128, 128), (256, 256), (257, 255), (256, 512),
          (512, 256), (300, 1000), (777, 1290), (1290, 777), (1024, 1024)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_update(shape):
    run(*inputs(shape, sum(shape)))


@pytest.mark.parametrize("shape", [(3, 40, 72), (5, 257, 130), (2, 3, 128, 264), (9, 130, 257),
                                   (17, 64, 64)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_stacks(shape, dtype):
    run(*inputs(shape, 3, dtype))


@pytest.mark.parametrize("nesterov,mu,steps", [(False, 0.9, 5), (True, 0.0, 3), (False, 0.95, 1),
                                               (True, 0.95, 2), (True, 0.95, 6)])
def test_variants(nesterov, mu, steps):
    run(*inputs((200, 328), 7), nesterov=nesterov, mu=mu, steps=steps)


@pytest.mark.parametrize("shape", [(200, 5000), (5000, 200), (2, 300, 6001), (140, 20000),
                                   (1, 129, 2048)], ids=lambda s: "x".join(map(str, s)))
def test_long_contractions(shape):
    """Few tiles, whose contraction several CTAs share; twice the same."""
    g, m = inputs(shape, 6)
    a = run(g, m)
    for _ in range(3):
        assert torch.equal(a, nv.nvfp4_muon_update(g, m.clone()))


@pytest.mark.parametrize("shape", [(3, 348, 14268), (8192, 512), (12, 200, 4001), (18, 256, 2312),
                                   (20, 256, 2312)], ids=lambda s: "x".join(map(str, s)))
def test_few_products_of_many_rounds(shape):
    """One launch whose updates have more rounds of tiles than two, and the first that has not."""
    g, m = inputs(shape, 16)
    a = run(g, m)
    for _ in range(3):
        assert torch.equal(a, nv.nvfp4_muon_update(g, m.clone()))


@pytest.mark.parametrize("shape", [(2, 78, 8723), (1, 37, 11654), (5, 101, 2137), (300, 20, 35),
                                   (2, 128, 4001)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_ragged_widths(shape, dtype):
    """Small rows whose width eight does not divide, over several CTAs and rounds."""
    g, m = inputs(shape, 17, dtype)
    want = run(g, m)
    grad, buf = g.clone(), m.clone()
    assert torch.equal(nv.nvfp4_muon_update(grad, buf, zero_grad=True), want)
    assert not grad.any()


def test_coefficients_of_each_step():
    coefs = ((3.9, -6.0, 2.9), (3.4445, -4.7750, 2.0315), (2.8, -2.9, 1.1))
    a = run(*inputs((136, 520), 8), steps=3, coefs=coefs)
    g, m = inputs((136, 520), 8)
    assert torch.equal(a, nv.nvfp4_muon_update(g, m, steps=3, coefs=[list(c) for c in coefs]))


@pytest.mark.parametrize("shape,rank", [((256, 512), 1), ((512, 264), 2), ((300, 300), 8),
                                        ((512, 1024), 64)])
def test_deficient_rank(shape, rank):
    """The null space stays empty: its rounding errors would grow by 3.4 a step."""
    run(*inputs(shape, 9, rank=rank))


@pytest.mark.parametrize("scale", [1e-12, 1e-3, 1e12])
def test_scales(scale):
    g, m = inputs((96, 200), 10)
    run(g * scale, m * scale, eps=1e-30)


def test_eps_bounds_the_start():
    g, m = inputs((64, 64), 11)
    run(g * 1e-9, m * 1e-9, eps=1e-3)


def test_zeros_in_a_stack():
    g, m = inputs((4, 72, 136), 12)
    g[1] = 0
    m[1] = 0
    buf = m.clone()
    got = nv.nvfp4_muon_update(g, buf)
    want, _ = reference(g, m, 0.95, True, 5, COEFS, 1e-7)
    assert torch.equal(got[1], torch.zeros_like(got[1]))
    keep = [0, 2, 3]
    assert off(got[keep], want[keep]) <= TOL


def test_nan_stays_in_its_matrix():
    g, m = inputs((3, 264, 300), 13)
    clean = nv.nvfp4_muon_update(g, m.clone())
    g[1, 5, 7] = float("nan")
    got = nv.nvfp4_muon_update(g, m.clone())
    nv.check_device_errors()
    assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])


@pytest.mark.parametrize("shape", [(400, 40, 72), (200, 130, 33), (90, 300, 264)],
                         ids=lambda s: "x".join(map(str, s)))
def test_nan_does_not_reach_what_follows_on_the_same_unit(shape):
    """More matrices than there are units: those behind one with NaN take its place."""
    g, m = inputs(shape, 33)
    clean = nv.nvfp4_muon_update(g, m.clone())
    g[0, 3, 5] = float("nan")
    g[1, 0, 0] = float("inf")
    got = nv.nvfp4_muon_update(g, m.clone())
    nv.check_device_errors()
    assert torch.equal(got[2:], clean[2:])


def test_zero_grad_and_repeats():
    g, m = inputs((2, 300, 520), 14)
    a = nv.nvfp4_muon_update(g.clone(), m.clone())
    for t in (g, g.bfloat16()):
        b, c = t.clone(), t.clone()
        buf, buf2 = m.clone(), m.clone()
        x = nv.nvfp4_muon_update(b, buf, zero_grad=True)
        y = nv.nvfp4_muon_update(c, buf2)
        assert not b.any() and torch.equal(c, t)
        assert torch.equal(x, y) and torch.equal(buf, buf2)
    assert torch.equal(a, nv.nvfp4_muon_update(g, m.clone()))


def test_given_buffers_and_stream():
    g, m = inputs((264, 136), 15)
    want = nv.nvfp4_muon_update(g, m.clone())
    ws = torch.full((nv.muon_sizes(1, 264, 136),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty(264, 136, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    buf = m.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = nv.nvfp4_muon_update(g, buf, out=out, workspace=ws, stream=side)
    side.synchronize()
    assert got is out and torch.equal(out, want)


def test_graph():
    g, m = inputs((2, 264, 520), 16)
    buf, want_buf = m.clone(), m.clone()
    nv.nvfp4_muon_update(g, m.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nv.nvfp4_muon_update(g, buf)
    for k in range(3):
        g.copy_(inputs((2, 264, 520), 20 + k)[0])
        graph.replay()
        want = nv.nvfp4_muon_update(g, want_buf)
        assert torch.equal(out, want) and torch.equal(buf, want_buf)


def test_rows_behind_the_end_are_left():
    """Neither the update nor what follows it in memory is written beyond it."""
    for shape in ((33, 31), (130, 264)):
        n = shape[0] * shape[1]
        room = torch.full((n + 4096,), 7.0, dtype=torch.bfloat16, device="cuda")
        g, m = inputs(shape, 17)
        nv.nvfp4_muon_update(g, m, out=room[:n].view(shape))
        assert (room[n:] == 7).all() and not (room[:n] == 7).all()


# ---- the step ------------------------------------------------------------------
@pytest.mark.parametrize("n", [1, 7, 8, 9, 255, 2048, 4100, 262144, 3000001])
@pytest.mark.parametrize("decay", [0.0, 0.1])
def test_apply(n, decay):
    g = torch.Generator(device="cuda").manual_seed(n)
    w = torch.randn(n, generator=g, device="cuda")
    u = torch.randn(n, generator=g, device="cuda").bfloat16()
    lr, scale = 0.02, 3.0
    keep = (1 - w.new_tensor(lr).double() * w.new_tensor(decay).double()).float()
    step = (w.new_tensor(lr).double() * scale).float()
    want = w.double() * keep.double() - step.double() * u.double()
    got = w.clone()
    amax = nv.nvfp4_muon_apply(got, u, lr, scale, decay)
    # the product's rounding and the sum's, half a step each
    bound = 2.0 ** -24 * ((w * keep).abs().double() + want.abs()) * (1 + 2.0 ** -20)
    assert ((got.double() - want).abs() <= bound).all()
    assert torch.equal(amax, got.abs().max().reshape(1))


def test_apply_matches_the_quantiser():
    g, m = inputs((128, 256), 18)
    w = torch.randn(128, 256, device="cuda")
    amax = nv.nvfp4_muon_apply(w, nv.nvfp4_muon_update(g, m), 0.02, 0.2 * 16)
    plain = torch.zeros(1, device="cuda")
    nv.nvfp4_amax(w, plain)
    assert torch.equal(amax, plain)
    given = nv.nvfp4_quantize(w, nv.BLOCK_16X16, nv.EMIT_T, amax=amax)
    own = nv.nvfp4_quantize(w, nv.BLOCK_16X16, nv.EMIT_T)
    assert torch.equal(given.codes, own.codes) and torch.equal(given.scales, own.scales)


def test_refusals():
    g, m = inputs((64, 72), 19)
    out = torch.empty(64, 72, dtype=torch.bfloat16, device="cuda")
    bad = [(ValueError, dict(momentum=m.bfloat16())), (ValueError, dict(momentum=m[:, :64])),
           (ValueError, dict(out=out.float())), (ValueError, dict(steps=0)),
           (ValueError, dict(steps=33)), (ValueError, dict(coefs=((1.0, 2.0, 3.0),) * 4)),
           (nv.NVFP4Error, dict(eps=0.0)), (nv.NVFP4Error, dict(mu=float("nan"))),
           (nv.NVFP4Error, dict(coefs=(1.0, float("inf"), 0.0))),
           (nv.NVFP4Error, dict(workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))),
           (nv.NVFP4Error, dict(out=g.view(-1).view(torch.bfloat16)[:64 * 72].view(64, 72)))]
    for error, kw in bad:
        with pytest.raises(error):
            nv.nvfp4_muon_update(**(dict(grad=g, momentum=m) | kw)) if "grad" in kw else \
                nv.nvfp4_muon_update(g, **(dict(momentum=m) | kw))
    for error, args in ((TypeError, (g.half(), m)), (ValueError, (g[0], m[0])),
                        (ValueError, (g.t(), m.t())), (ValueError, (g.cpu(), m))):
        with pytest.raises(error):
            nv.nvfp4_muon_update(*args)
    w = torch.randn(64, 72, device="cuda")
    for error, args in ((ValueError, (w.bfloat16(), out)), (ValueError, (w, out.float())),
                        (nv.NVFP4Error, (w, out, float("inf")))):
        with pytest.raises(error):
            nv.nvfp4_muon_apply(*(args if len(args) == 3 else args + (0.1,)))


def test_large_layer():
    """The sides of this repository's layer, wide and tall; sampled against 64 bits."""
    for shape in ((4096, 14336), (14336, 4096)):
        g, m = inputs(shape, 21)
        run(g, m)
        torch.cuda.empty_cache()


def test_many_matrices():
    for shape in itertools.chain([(300, 24, 40)], [(40, 264, 520)]):
        run(*inputs(shape, 22))


# one launch a product on pairs; one launch for all; a team of CTAs by counters
@pytest.mark.parametrize("shape", [(40, 264, 520), (300, 400), (128, 14336)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("quit", [False, True], ids=["stall", "quit"])
def test_a_kernel_that_gives_up_recovers(shape, quit):
    """Injected: no loads come (a CTA does not count itself in), or the MMA threads give
    up with the loads in flight.  The error is reported, and the calls after it give what
    they gave before."""
    if quit and shape == (128, 14336):
        pytest.skip("that kernel has no loads in flight")
    g, m = inputs(shape, 23)
    want = nv.nvfp4_muon_update(g, m.clone())
    nv.check_device_errors()
    nv.debug_inject(nv.QUIT_GEMM if quit else nv.STALL_GEMM, 1_000_000)
    try:
        nv.nvfp4_muon_update(g, m.clone())
        with pytest.raises(nv.NVFP4Error) as e:
            nv.check_device_errors()
        assert e.value.status == nv.ERR_DEVICE_TIMEOUT
    finally:
        nv.debug_inject(0, 0)
    nv.check_device_errors()
    for _ in range(2):
        assert torch.equal(nv.nvfp4_muon_update(g, m.clone()), want)
    nv.check_device_errors()


def test_two_streams_at_once():
    """Calls of every kind side by side, each with its own workspace."""
    shapes = [(64, 512), (300, 400), (128, 14336), (40, 264, 520)]
    ins = [inputs(s, 24 + i) for i, s in enumerate(shapes)]
    want = [nv.nvfp4_muon_update(g, m.clone()) for g, m in ins]
    streams = [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    for _ in range(5):
        bufs, got = [m.clone() for _, m in ins], []
        torch.cuda.synchronize()
        for (g, _), b, s in zip(ins, bufs, streams):
            got.append(nv.nvfp4_muon_update(g, b, stream=s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    nv.check_device_errors()
