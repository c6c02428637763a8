"""A kernel that gives up at a wait while copies that it issued are in flight sees
them land before it ends: its shared memory goes to the next block on the SM.
Injected, each block waits at first for more bytes than come, with the loads of
its other stages issued behind them; the error is reported, and the calls after
it, which take the same shared memory, give what they gave before.  (A block
gives up after the injected limit, and its last look at the copies, of which one
is never complete, has the library's own limit of 2 s.)"""
import pytest

pytestmark = pytest.mark.gpu
LIMIT_NS = 1_000


@pytest.fixture(scope="module")
def nv():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding
    return binding


def _gives_up_then_recovers(nv, bit, call):
    import torch
    want = call()
    nv.check_device_errors()
    nv.debug_inject(bit, LIMIT_NS)
    try:
        call()
        with pytest.raises(nv.NVFP4Error) as e:
            nv.check_device_errors()
        assert e.value.status == nv.ERR_DEVICE_TIMEOUT
    finally:
        nv.debug_inject(0, 0)
    nv.check_device_errors()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
    nv.check_device_errors()


# one row; rows for every stage of the ring, several and one to a block
@pytest.mark.parametrize("rows,cols,wide", [(1, 8, False), (9000, 512, False), (2000, 4096, True)])
def test_norm_that_gives_up_waits_for_its_rows(nv, rows, cols, wide):
    import torch
    g = torch.Generator(device="cuda").manual_seed(rows)
    kind = torch.float32 if wide else torch.bfloat16
    x, dy = (torch.randn(rows, cols, generator=g, device="cuda").to(kind) for _ in range(2))
    z, dh = (torch.randn(rows, cols, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = [torch.randn(cols, generator=g, device="cuda") for _ in range(3)]
    _gives_up_then_recovers(nv, nv.LOSE_NORM, lambda: nv.nvfp4_residual_norm_fwd(x, z, *w))
    _gives_up_then_recovers(nv, nv.LOSE_NORM, lambda: nv.nvfp4_residual_norm_bwd(dy, dh, x, z, *w))
    _gives_up_then_recovers(nv, nv.LOSE_NORM,
                            lambda: nv.nvfp4_residual_norm_fwd(x, w_pre=w[0])[1:])


def _groups(sizes):
    import torch
    off = [0]
    for n in sizes:
        off.append(off[-1] + (n + 127) // 128 * 128)
    i = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(sizes, **i), torch.tensor(off, **i), off[-1]


# fewer fills than stages; more, over several tiles; a tile shared by two and by four pairs
@pytest.mark.parametrize("sizes,N,K,tile", [([100, 128], 256, 256, 3), ([100, 128], 384, 256, 6),
                                            ([700, 0, 900, 300] * 6, 1280, 2048, 3),
                                            ([700, 0, 900, 300] * 6, 1280, 2048, 6),
                                            ([3], 1024, 4096, 0), ([3], 4096, 8192, 0),
                                            ([3, 200], 4096, 8192, 0)])
@pytest.mark.parametrize("plus_c", [False, True])
def test_grouped_product_that_gives_up_waits_for_its_copies(nv, sizes, N, K, tile, plus_c):
    import torch
    g = torch.Generator(device="cuda").manual_seed(N)
    s, o, rows = _groups(sizes)
    A = nv.nvfp4_quantize(torch.randn(rows, K, generator=g, device="cuda"), nv.ROW_1X16)
    B = nv.nvfp4_quantize(torch.randn(len(sizes) * N, K, generator=g, device="cuda"), nv.BLOCK_16X16)
    C = torch.randn(rows, N, generator=g, device="cuda").bfloat16() if plus_c else None
    _gives_up_then_recovers(nv, nv.QUIT_GEMM, lambda: [nv.nvfp4_group_gemm(
        A, B, s, o, C_add=C, d_mode=nv.D_BF16_ADD_C if plus_c else nv.D_BF16, tile=tile)])


@pytest.mark.parametrize("tile,fold", [(3, False), (6, False), (3, True)])
def test_grouped_weight_gradient_that_gives_up_waits_for_its_copies(nv, tile, fold):
    import torch
    g = torch.Generator(device="cuda").manual_seed(tile)
    s, o, rows = _groups([700, 0, 900, 64] * 6)
    a, b = (nv.nvfp4_quantize(torch.randn(rows, n, generator=g, device="cuda"), nv.COL_1X16)
            for n in (512, 1280))
    mode = nv.D_F32_ACCUM if fold else nv.D_BF16
    _gives_up_then_recovers(nv, nv.QUIT_GEMM,
                            lambda: [nv.nvfp4_group_wgrad(a, b, s, o, d_mode=mode, tile=tile)])


# the single-SM tiles, then the pairs; fewer fills than stages, and several tiles
@pytest.mark.parametrize("tile", [1, 2, 5, 3, 6])
@pytest.mark.parametrize("M,N,K", [(128, 256, 512), (4096, 8192, 2048)])
@pytest.mark.parametrize("fold", [False, True])
def test_gemm_that_gives_up_waits_for_its_copies(nv, tile, M, N, K, fold):
    import torch
    g = torch.Generator(device="cuda").manual_seed(tile)
    A = nv.nvfp4_quantize(torch.randn(M, K, generator=g, device="cuda"), nv.ROW_1X16)
    B = nv.nvfp4_quantize(torch.randn(N, K, generator=g, device="cuda"), nv.BLOCK_16X16)
    mode = nv.D_F32_ACCUM if fold else nv.D_BF16

    def call():
        out = torch.zeros(M, N, device="cuda") if fold else None
        return [nv.nvfp4_gemm(A, B, tile=tile, d_mode=mode, out=out)]

    _gives_up_then_recovers(nv, nv.QUIT_GEMM, call)


@pytest.mark.parametrize("fmt", ["MXFP4", "MXFP8"])
@pytest.mark.parametrize("M,N,K", [(256, 256, 512), (2048, 8192, 2048)])
def test_mx_gemm_that_gives_up_waits_for_its_copies(nv, fmt, M, N, K):
    import torch
    f = getattr(nv, fmt)
    g = torch.Generator(device="cuda").manual_seed(K)
    ops = []
    for n in (M, N):
        sw = torch.zeros(n // 128 * (K // 128) * 512, dtype=torch.uint8, device="cuda")
        x = torch.randn(n, K, generator=g, device="cuda").bfloat16()
        ops += [nv.nvfp4_mx_quantize(x, nv.MX_ROW, f, scales_sw=sw)[0], sw]
    _gives_up_then_recovers(nv, nv.QUIT_GEMM, lambda: [nv.nvfp4_mx_gemm(*ops, f, M, N, K)])
