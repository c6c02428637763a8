"""Grouped products at a training batch's sizes, where rows, strides and output
offsets are widest: eight experts of 4096 x 14336, 16384 rows.  Sampled rows --
the first and last of each group and of its 256-row tiles, and some between --
are compared over all columns with the operands' values multiplied in 64 bits;
the rule is the other GEMM tests' (4 bf16 units + 1e-3 of the root mean square).
The FP32 fold is held to the accumulator's rounding instead, as in the tests of
small sizes: (K / 64 + 64) 2^-22 sum |a b|."""
import numpy as np
import pytest

import gpu_helpers as H

pytestmark = pytest.mark.gpu

SIZES = [2301, 0, 1, 4096, 255, 3000, 2731, 4000]


@pytest.fixture(scope="module")
def nv():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import binding
    return binding


def _groups():
    import torch
    off = [0]
    for n in SIZES:
        off.append(off[-1] + (n + 127) // 128 * 128)
    i = dict(dtype=torch.int32, device="cuda")
    return torch.tensor(SIZES, **i), torch.tensor(off, **i), off


def _values(q, rows, first, n, view=0):
    """Values in 64 bits, on the device: `rows` (indices), columns first .. + n."""
    import torch
    codes, scales = (q.codes_t, q.scales_t) if view else (q.codes, q.scales)
    cols = q.rows if view else q.cols
    r = torch.as_tensor(rows, device="cuda").long().unsqueeze(1)
    c = torch.arange(first, first + n, device="cuda").unsqueeze(0)
    code = (codes[r * (cols // 2) + c // 2].int() >> (4 * (c % 2))) & 15
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    v = grid[code & 7] * torch.where(code >= 8, -1.0, 1.0)
    b = c // 16
    at = ((r // 128) * (cols // 64) + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4
    return v * scales[at].view(torch.float8_e4m3fn).double()


def _sample(n, rng):
    edge = [i for i in (0, 127, 128, 255, 256, n - 257, n - 1) if 0 <= i < n]
    return sorted(set(edge) | set(rng.integers(0, max(n, 1), 4).tolist() if n else []))


@pytest.mark.parametrize("view,N,K", [(0, 14336, 4096), (1, 4096, 14336)])
def test_rows_product(nv, view, N, K):
    import torch
    E, (s, o, off) = len(SIZES), _groups()
    rows = off[-1] + 256
    g = torch.Generator(device="cuda").manual_seed(N)
    A = nv.nvfp4_quantize(torch.randn(rows, K, generator=g, device="cuda").bfloat16(), nv.ROW_1X16)
    W = torch.randn(*((E * K, N) if view else (E * N, K)), generator=g, device="cuda") * 0.02
    B = nv.nvfp4_quantize(W, nv.BLOCK_16X16, nv.EMIT_T if view else 0)
    del W
    out = nv.nvfp4_group_gemm(A, B, s, o, b_view=view,
                              out=torch.full((rows, N), 3.0, dtype=torch.bfloat16, device="cuda"))
    nv.check_device_errors()
    alpha, rng = A.s_dec.double() * B.s_dec.double(), np.random.default_rng(1)
    live = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e, n in enumerate(SIZES):
        live[off[e]:off[e] + n] = True
        at = [off[e] + i for i in _sample(n, rng)]
        if at:
            b = (_values(B, range(N), e * K, K, 1) if view
                 else _values(B, range(e * N, e * N + N), 0, K))
            ref = (_values(A, at, 0, K) @ b.t()) * alpha
            H.assert_gemm_close(out[at].double().cpu().numpy(), ref.cpu().numpy(), f"group {e}")
    assert (out[~live] == 0).all()


@pytest.mark.parametrize("fold", [False, True])
def test_weight_gradient(nv, fold):
    import torch
    M, N, (s, o, off) = 14336, 4096, _groups()
    rows = off[-1] + 256
    g = torch.Generator(device="cuda").manual_seed(M)
    live = torch.zeros(rows, 1, device="cuda")
    for e, n in enumerate(SIZES):
        live[off[e]:off[e] + n] = 1
    q = [nv.nvfp4_quantize((torch.randn(rows, n, generator=g, device="cuda") * live).bfloat16(),
                           nv.COL_1X16, nv.RHT) for n in (M, N)]
    out = nv.nvfp4_group_wgrad(*q, s, o, d_mode=nv.D_F32_ACCUM if fold else nv.D_BF16)
    nv.check_device_errors()
    alpha, rng = q[0].s_dec.double() * q[1].s_dec.double(), np.random.default_rng(1)
    for e, n in enumerate(SIZES):
        if not n:
            assert (out[e] == 0).all()
            continue
        k = (n + 63) // 64 * 64
        at = _sample(M, rng)
        a, b = _values(q[0], at, off[e], k), _values(q[1], range(N), off[e], k)
        ref = a @ b.t() * alpha
        if fold:
            size = a.abs() @ b.abs().t() * alpha
            assert ((out[e][at].double() - ref).abs() <= (k / 64 + 64) * 2.0 ** -22 * size).all()
        else:
            H.assert_gemm_close(out[e][at].double().cpu().numpy(), ref.cpu().numpy(), f"group {e}")
