"""A training step of one transformer block over packed documents, on the framework's operators.

    x, y0   residual stream and its normalised form (the block's input)
    qkv   = y0 @ w_qkv                                  one matrix product
    o     = causal attention inside each document       mha_packed_forward
    f     = o @ w_out
    h, y  = x + scale * gate * norm(f), norm(h)         residual_rmsnorm_forward
    loss  = mean (y - target)^2
and back again: residual_rmsnorm_backward, two products, mha_packed_backward, two products.  The documents lie one
after another in one buffer, so the step has no padding but the buffer's unused tail; q, k and v are read as slices
of the fused projection, without a copy.

    python examples/packed_block_step.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import conv2d_backward_implicit_gb300 as dg  # noqa: E402

EPS = 1e-5


class Block:
    """Weights (float32 masters, bf16 copies for the step), the workspaces and one step of SGD."""

    def __init__(self, width=512, heads=8, kv_heads=2, dim=64, scale=0.5, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.width, self.heads, self.kv_heads, self.dim, self.scale = width, heads, kv_heads, dim, scale
        n = (heads + 2 * kv_heads) * dim

        def normal(*shape, std):
            return torch.randn(shape, generator=g, device=device) * std

        self.weights = {"w_qkv": normal(width, n, std=width ** -0.5), "w_out": normal(heads * dim, width, std=width ** -0.5),
                        "gate": torch.ones(width, device=device), "w_post": torch.ones(width, device=device),
                        "w_pre": torch.ones(width, device=device)}
        self.workspace = torch.empty(0, dtype=torch.uint8, device=device)

    def _space(self, nbytes):
        if self.workspace.numel() < nbytes:
            self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.workspace.device)
        return self.workspace

    def step(self, x, y0, offsets, target):
        """x, y0, target [tokens, width] bf16, offsets int32 [documents + 1]; returns (loss, gradients of the weights,
        gradients of x and y0)."""
        T, H, G, D, code, stream = x.shape[0], self.heads, self.kv_heads, self.dim, dg.DGRAD_BF16, torch.cuda.current_stream()
        w = {k: v.to(torch.bfloat16) for k, v in self.weights.items()}
        new = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=x.device)  # noqa: E731

        qkv = (y0 @ w["w_qkv"]).view(T, H + 2 * G, D)
        q, k, v = qkv.split([H, G, G], dim=1)
        ap = dg.MhaPackedParams(T, offsets.numel() - 1, H, G, D, 0, q.stride(0), k.stride(0), v.stride(0))
        o, lse = new(T, H, D), new(T, H, 2, dtype=torch.float32)
        dg.mha_packed_forward(q, k, v, offsets, o, lse, ap, code, stream)
        f = o.view(T, H * D) @ w["w_out"]
        np_ = dg.ResidualRmsnormParams(T, self.width, dg.RESIDUAL_GATE_CHANNEL, EPS, self.scale)
        h, y, rstd = new(T, self.width), new(T, self.width), new(T, 2, dtype=torch.float32)
        dg.residual_rmsnorm_forward(f, x, w["gate"], w["w_post"], w["w_pre"], h, y, rstd, np_, code, stream)

        diff = y.float() - target.float()
        loss = diff.square().mean()
        dy = (diff * (2.0 / diff.numel())).to(torch.bfloat16)

        df, dx = new(T, self.width), new(T, self.width)
        small = {n: new(self.width, dtype=torch.float32) for n in ("gate", "w_post", "w_pre")}
        size = dg.residual_rmsnorm_workspace_size(np_, code)
        dg.residual_rmsnorm_backward(f, h, w["gate"], w["w_post"], w["w_pre"], rstd, dy, None, df, dx, small["gate"],
                                     small["w_post"], small["w_pre"], self._space(size), size, np_, code, stream)
        d_o = (df @ w["w_out"].T).view(T, H, D)
        dq, dk, dv = new(T, H, D), new(T, G, D), new(T, G, D)
        size = dg.mha_packed_workspace_size(ap, code)
        dg.mha_packed_backward(q, k, v, o, d_o, lse, offsets, dq, dk, dv, self._space(size), size, ap, code, stream)
        d_qkv = torch.cat([dq, dk, dv], dim=1).view(T, -1)
        grads = dict(small, w_out=(o.view(T, H * D).T @ df).float(), w_qkv=(y0.T @ d_qkv).float())
        return loss, grads, dx, d_qkv @ w["w_qkv"].T

    def update(self, grads, rate):
        for k, g in grads.items():
            self.weights[k] -= rate * g


def documents(lens, tail, width, seed, device="cuda"):
    """A packed batch: (x, y0, offsets, target), with `tail` unused rows behind the last document."""
    g = torch.Generator(device=device).manual_seed(seed)
    offsets = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=device)
    x, target = (torch.randn((sum(lens) + tail, width), generator=g, device=device).to(torch.bfloat16) for _ in range(2))
    y0 = torch.nn.functional.rms_norm(x.float(), (width,), eps=EPS).to(torch.bfloat16)
    return x, y0, offsets, target


def main(steps=10):
    block = Block()
    batch = documents([700, 33, 1, 250], 40, block.width, 1)
    for i in range(steps):
        loss, grads, _, _ = block.step(*batch)
        block.update(grads, 50.0)
        print(f"step {i}: loss {loss.item():.4f}")
    for check in (dg.mha_packed_check_errors,):
        rc = check(torch.cuda.current_stream())
        if rc:
            raise RuntimeError(dg.STATUS.get(rc, rc))


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 10)
