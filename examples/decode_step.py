"""One decode step of a mixture-of-experts block for a few tokens, on random weights.

    residual + norm (bf16 for the router and the experts, e4m3 for the dense projection)
    router logits -> experts and gate weights
    the gated expert layer, once with bf16 experts and once with 4-bit experts
    a dense 4-bit projection of the 8-bit rows beside it

Run from the repository's root: python examples/decode_step.py [tokens]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from consumer_movement_gemm_gb300 import build, tovl  # noqa: E402


class Block:
    """Weights, buffers and the handle that a serving program keeps between steps."""

    def __init__(self, handle, tokens, H=1024, I=512, E=16, k=4, N=2048, group=128, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(0)
        bf16 = lambda *shape, scale=1.0: (torch.randn(*shape, generator=g, device=device) * scale).to(torch.bfloat16)  # noqa: E731
        self.h, self.group = handle, group
        self.norm_w = bf16(H, scale=0.1) + 1
        self.router = bf16(H, E, scale=H ** -0.5)
        self.w13, self.w2 = bf16(E, H, 2 * I, scale=H ** -0.5), bf16(E, I, H, scale=I ** -0.5)
        self.proj = bf16(H, N, scale=H ** -0.5)
        # 4-bit copies, laid out once
        self.w13_q, self.w2_q = handle.quantize_q4(self.w13, group), handle.quantize_q4(self.w2, group)
        self.proj_q = handle.quantize_q4(self.proj, group, zeros=True)
        self.y = torch.empty(tokens, H, dtype=torch.bfloat16, device=device)
        self.y8 = torch.empty(tokens, H, dtype=torch.float8_e4m3fn, device=device)
        self.y8_scale = torch.empty(tokens, -(-H // 128), device=device)
        self.topk = torch.empty(tokens, k, dtype=torch.int32, device=device)
        self.gate = torch.empty(tokens, k, device=device)
        self.out, self.out_q = torch.empty_like(self.y), torch.empty_like(self.y)
        self.side = torch.empty(tokens, N, dtype=torch.bfloat16, device=device)
        self.ws = torch.empty(max(handle.moe_decode_workspace(tokens, k, H, I), handle.matvec_q4_workspace(tokens, N)),
                              dtype=torch.uint8, device=device)

    def step(self, x, residual):
        """The block's outputs for rows x; residual (fp32) is updated in place."""
        h = self.h
        h.add_rmsnorm(x, self.norm_w, 1e-5, residual=residual, residual_out=residual, out=self.y, q=self.y8,
                      q_scale=self.y8_scale)
        h.route_topk(self.y @ self.router, self.topk, self.gate)
        h.moe_decode(self.y, self.topk, self.gate, self.w13, self.w2, self.out, self.ws)
        h.moe_decode_q4(self.y, self.topk, self.gate, self.w13_q, self.w2_q, self.group, self.out_q, self.ws)
        q, scale, zero = self.proj_q
        h.matvec_q4(self.y8, q, scale, self.group, self.side, self.ws, zero=zero, x_scale=self.y8_scale)
        return self.out, self.out_q, self.side


def main(tokens=8):
    build.build()
    with tovl.Handle(0) as handle:
        block = Block(handle, tokens)
        H = block.y.shape[1]
        x = torch.randn(tokens, H, device="cuda").to(torch.bfloat16)
        residual = torch.zeros(tokens, H, device="cuda")
        for _ in range(3):
            out, out_q, side = block.step(x, residual)
            x = out.clone()
        status = handle.sync_status()
        if status:
            raise SystemExit(f"device status {status}: {tovl.error_string(status)}")
        near = float((out_q.float() - out.float()).norm() / out.float().norm())
        exact = block.y.float() @ block.proj.float()
        print(f"{tokens} tokens, 3 steps; 4-bit experts differ from bf16 ones by {near:.3f}, the 4-bit projection of 8-bit "
              f"rows from the exact one by {float((side.float() - exact).norm() / exact.norm()):.3f} (relative)")
        return near


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
