"""The router inside the mixture-of-experts block: its logits, its weights'
gradient and its share of the input's gradient, each by itself against 64 bits
on the block's own operands.  (Together with the experts' share, whose 4-bit
products are off by more, a missing share of the router would go unnoticed.)

A product of bf16 operands with n terms taken in FP32, in any order, is off by at
most n 2^-24 sum|terms| and the last rounding of the FP32 result; a result in
bf16 by half a unit more."""
import numpy as np
import pytest

import moe_reference as R

pytestmark = pytest.mark.gpu


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.fixture(params=[(200, False, "ROUTE_CHOSEN"), (777, True, "ROUTE_ALL")])
def block(request, monkeypatch):
    """A block after one forward and backward, and what its calls returned or took."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from nvfp4_block_scaled_03_gb300 import moe
    tokens, wide, mode = request.param
    nv, seen = moe.nv, {}

    def watch(name, pick):
        call = getattr(nv, name)

        def run(*args, **kwargs):
            out = call(*args, **kwargs)
            pick(args, kwargs, out)
            return out
        monkeypatch.setattr(nv, name, run)

    # the last of each kind in a backward
    watch("nvfp4_route_bwd", lambda a, k, out: seen.update(dlogits=out.clone()))
    watch("nvfp4_combine", lambda a, k, out: seen.update(share=out.clone()))
    watch("nvfp4_residual_norm_bwd", lambda a, k, out: seen.update(dh=a[1]))
    b = moe.MoEBlock(256, 512, 8, 2, z_scale=0.5, mode=getattr(nv, mode))
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(tokens, 256, generator=g, device="cuda")
    x = x if wide else x.bfloat16()
    b.forward(x)
    b.backward(torch.randn(tokens, 256, generator=g, device="cuda").to(x.dtype))
    nv.check_device_errors()
    return b, seen


def test_logits(block):
    b, _ = block
    h, w = _f64(b.saved["h"]), R.bf16(b.params["router"].cpu().numpy())
    size = np.abs(h) @ np.abs(w).T
    assert (np.abs(_f64(b.saved["logits"]) - h @ w.T) <= (256 + 2) * 2.0 ** -24 * size).all()


def test_weight_gradient(block):
    b, seen = block
    d, h = R.bf16(seen["dlogits"].float().cpu().numpy()), _f64(b.saved["h"])
    size = np.abs(d).T @ np.abs(h)
    assert (np.abs(_f64(b.grads["router"]) - d.T @ h)
            <= (len(h) + 2) * 2.0 ** -24 * size).all()


def test_share_of_the_input_gradient(block):
    b, seen = block
    d, w = R.bf16(seen["dlogits"].float().cpu().numpy()), R.bf16(b.params["router"].cpu().numpy())
    share, size = d @ w, np.abs(d) @ np.abs(w)
    want = _f64(seen["share"]) + share
    off = np.abs(_f64(seen["dh"]) - want)
    e = (8 + 3) * 2.0 ** -24 * (size + np.abs(want))
    assert (off <= e + R.half_ulp_bf16(np.abs(want) + e)).all()
    # and it is one that counts here: without it most elements would be off by more
    assert (np.abs(share) > R.half_ulp_bf16(np.abs(want))).mean() > 0.5
