"""A mixture-of-experts MLP block on the library's calls, forward and backward:

    h      = norm(x) w_in                               the block's input
    plan   = top-k of softmax(h Wr^T)                   the router
    o      = experts' SwiGLU MLPs over the plan's rows  (NVFP4 products)
    z      = sum over a token's experts of weight * o
    y      = x + z_scale gate (.) norm(z) w_out         the next block's stream

Every projection of every expert is one grouped product; quantisation follows
the dense MLP (activations and weights to nearest, gradients stochastically,
the random Hadamard transform on the weight gradients' operands).  The router's
products take bf16 operands (h is one; its weights and the logits' gradient are
rounded to it) and give FP32 logits and an FP32 weight gradient; what it adds to
h's gradient is added in FP32 to the experts' share, which the combination has
rounded to bf16, and the sum is rounded to bf16 again, the type in which the
norm takes it.  Weight gradients are folded into FP32 masters.  Nothing synchronises with the host,
so a step can be captured as a CUDA graph; its backward then takes the step's
number from the device, since a captured number, and with it the stochastic
rounding's random words, would be the same in every replay.

``python -m nvfp4_block_scaled_03_gb300.moe`` trains a small block for a few
steps on a GB300 and prints the loss.
"""
from __future__ import annotations

import torch

from . import binding as nv


class MoEBlock:
    """`experts` SwiGLU experts of width `ffn` behind a top-`top` router, with
    FP32 masters and their gradients (`grads`, by the parameters' names)."""

    def __init__(self, hidden: int, ffn: int, experts: int, top: int, *, seed: int = 0,
                 z_scale: float = 1.0, eps: float = 1e-5, mode: int = nv.ROUTE_CHOSEN,
                 device: str = "cuda"):
        if hidden % 128 or ffn % 128:
            raise ValueError("hidden and ffn must be multiples of 128")
        self.experts, self.top, self.mode = experts, top, mode
        self.eps, self.z_scale, self.seed = eps, z_scale, seed
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(*shape, generator=g, device=device) * scale

        self.params = {
            "w_in": torch.ones(hidden, device=device),
            "w_out": torch.ones(hidden, device=device),
            "gate": torch.ones(hidden, device=device),
            "router": normal(experts, hidden, scale=hidden ** -0.5),
            "gate_proj": normal(experts * ffn, hidden, scale=hidden ** -0.5),
            "up_proj": normal(experts * ffn, hidden, scale=hidden ** -0.5),
            "down_proj": normal(experts * hidden, ffn, scale=ffn ** -0.5),
        }
        self.grads = {k: torch.zeros_like(v) for k, v in self.params.items()}
        self.hidden, self.ffn = hidden, ffn
        self.operand_ids = torch.arange(6, device=device)

    def _both(self, x, flags=0, offsets=(0, 0)):
        """Row-wise and column-wise operands of x from one read (after its amaxes)."""
        row, col = self._amax(x)
        return nv.nvfp4_quantize_rowcol(x, flags, flags | nv.RHT, seed=self.seed,
                                        row_offset=offsets[0], col_offset=offsets[1],
                                        amax_row=row, amax_col=col)

    def _amax(self, x):
        row = torch.zeros(1, device=x.device)
        col = torch.zeros(1, device=x.device)
        nv.nvfp4_amax(x, row, col, seed=self.seed)
        return row, col

    def forward(self, x: torch.Tensor):
        """y [tokens, hidden] of x (bf16 or FP32); what the backward reads is
        kept in `self.saved`."""
        p, s = self.params, {}
        s["x"] = x
        _, s["h"] = nv.nvfp4_residual_norm_fwd(x, w_pre=p["w_in"], eps=self.eps)
        s["router"] = p["router"].bfloat16()
        s["logits"] = torch.mm(s["h"], s["router"].t(), out_dtype=torch.float32)
        plan = s["plan"] = nv.nvfp4_route_fwd(s["logits"], self.top, self.mode)
        groups = (plan.sizes, plan.offsets)
        xe = nv.nvfp4_dispatch(s["h"], plan.row, plan.source)
        qx, s["qx_col"] = self._both(xe)
        for name in ("gate_proj", "up_proj", "down_proj"):
            s[name] = nv.nvfp4_quantize(p[name], nv.BLOCK_16X16, nv.EMIT_T)
        s["G"] = nv.nvfp4_group_gemm(qx, s["gate_proj"], *groups)
        s["U"] = nv.nvfp4_group_gemm(qx, s["up_proj"], *groups)
        H, row, col = nv.nvfp4_swiglu_fwd(s["G"], s["U"], seed=self.seed)
        qh, s["qh_col"] = nv.nvfp4_quantize_rowcol(H, 0, nv.RHT, seed=self.seed, amax_row=row,
                                                   amax_col=col)
        s["o"] = nv.nvfp4_group_gemm(qh, s["down_proj"], *groups)
        s["z"] = nv.nvfp4_combine(s["o"], plan.row, plan.weight)
        y, _ = nv.nvfp4_residual_norm_fwd(x, s["z"], p["w_out"], p["gate"], eps=self.eps,
                                          z_scale=self.z_scale)
        self.saved = s
        return y

    def backward(self, dy: torch.Tensor, step: int | torch.Tensor = 0) -> torch.Tensor:
        """dx from dy; the parameters' gradients are added to `self.grads`.
        `step` picks the random numbers of the stochastic rounding: a number,
        or, where the call is captured into a graph that is replayed, a
        1-element int64 tensor on the device that each step advances."""
        p, g, s = self.params, self.grads, self.saved
        plan = s["plan"]
        if isinstance(step, torch.Tensor):
            at = (8 * step.reshape(1) + self.operand_ids).split(1)
        else:
            at = [8 * step + k for k in range(6)]
        groups = (plan.sizes, plan.offsets)
        E, F, D = self.experts, self.ffn, self.hidden
        dx, dz, dw_out, dgate, _ = nv.nvfp4_residual_norm_bwd(
            dy, None, s["x"], s["z"], p["w_out"], p["gate"], eps=self.eps, z_scale=self.z_scale)
        g["w_out"] += dw_out
        g["gate"] += dgate
        do, dweight = nv.nvfp4_combine_bwd(dz, s["o"], plan.row, plan.source, plan.weight)
        qdo, qdo_col = self._both(do, nv.SR, at[0:2])
        dH = nv.nvfp4_group_gemm(qdo, s["down_proj"], *groups, b_view=1)
        nv.nvfp4_group_wgrad(qdo_col, s["qh_col"], *groups, out=g["down_proj"].view(E, D, F),
                             d_mode=nv.D_F32_ACCUM)
        dG, dU, g_row, g_col, u_row, u_col = nv.nvfp4_swiglu_bwd(dH, s["G"], s["U"], seed=self.seed)
        dxe = None
        for name, d, row, col, k in (("gate_proj", dG, g_row, g_col, 2),
                                     ("up_proj", dU, u_row, u_col, 4)):
            qd, qd_col = nv.nvfp4_quantize_rowcol(
                d, nv.SR, nv.SR | nv.RHT, seed=self.seed, row_offset=at[k], col_offset=at[k + 1],
                amax_row=row, amax_col=col)
            dxe = nv.nvfp4_group_gemm(qd, s[name], *groups, b_view=1, C_add=dxe,
                                      d_mode=nv.D_BF16 if dxe is None else nv.D_BF16_ADD_C)
            nv.nvfp4_group_wgrad(qd_col, s["qx_col"], *groups, out=g[name].view(E, F, D),
                                 d_mode=nv.D_F32_ACCUM)
        dh = nv.nvfp4_combine(dxe, plan.row)
        dlogits = nv.nvfp4_route_bwd(s["logits"], plan, dweight, self.mode).bfloat16()
        g["router"] += torch.mm(dlogits.t(), s["h"], out_dtype=torch.float32)
        dh = torch.mm(dlogits, s["router"], out_dtype=torch.float32).add_(dh).bfloat16()
        dx, _, _, _, dw_in = nv.nvfp4_residual_norm_bwd(dx, dh, s["x"], w_pre=p["w_in"],
                                                        eps=self.eps)
        g["w_in"] += dw_in
        return dx

    def sgd(self, lr: float):
        """One step on every FP32 master; the gradients are cleared."""
        for name, w in self.params.items():
            nv.nvfp4_sgd_step(w, self.grads[name], lr, zero_grad=True)


def main(steps: int = 30, tokens: int = 500, hidden: int = 512, ffn: int = 1024, experts: int = 8,
         top: int = 2, lr: float = 5.0):
    """Fits a block to a fixed random map and prints the loss as it falls."""
    torch.manual_seed(0)
    block = MoEBlock(hidden, ffn, experts, top)
    x = torch.randn(tokens, hidden, device="cuda")
    target = x + torch.randn(tokens, hidden, device="cuda")
    losses = []
    for step in range(steps):
        diff = block.forward(x) - target
        losses.append((diff * diff).mean().item())
        block.backward(diff * (2.0 / diff.numel() * hidden), step)
        block.sgd(lr / tokens)
        if step % 5 == 0 or step == steps - 1:
            print(f"step {step}: loss {losses[-1]:.4f}", flush=True)
    nv.check_device_errors()
    return losses


if __name__ == "__main__":
    main()
