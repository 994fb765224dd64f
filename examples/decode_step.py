"""Decode steps of an attention and a mixture-of-experts block for a few requests, on random weights.

    pages, cache slots and positions of the step's tokens, one a request
    residual + norm, projection, rotary embedding with the cache writes, attention over the request's pages, projection
    residual + norm (bf16 for the router and the experts, e4m3 for the dense projection)
    router logits -> experts and gate weights
    the gated expert layer, once with bf16 experts and once with 4-bit experts
    a dense 4-bit projection of the 8-bit rows beside it

Run from the repository's root: python examples/decode_step.py [requests]
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


class Pages:
    """The requests' pages: block table, lengths and the ring of free pages, updated in place by every step."""

    def __init__(self, handle, requests, longest, page=16, device="cuda"):
        i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=device)  # noqa: E731
        self.h, self.page, width = handle, page, -(-longest // page)
        self.pages = requests * width
        self.length, self.table = i32(requests), i32(requests, width)
        self.ring = torch.arange(self.pages, dtype=torch.int32, device=device)
        self.state = torch.tensor([0, self.pages, 0, 0], dtype=torch.int32, device=device)
        self.one = torch.ones(requests, dtype=torch.int32, device=device)
        self.slots, self.positions, self.starts = i32(requests), i32(requests), i32(requests + 1)

    def step(self):
        """One more token for every request."""
        self.h.page_plan(self.length, self.one, self.table, self.ring, self.state, self.page, self.length, self.state, self.slots,
                         self.positions, self.starts)


class Attention:
    """Weights, cache and buffers of an attention block."""

    def __init__(self, handle, pages, H=1024, Hq=16, heads=4, D=64, longest=64, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(1)
        bf16 = lambda *shape, scale=1.0: (torch.randn(*shape, generator=g, device=device) * scale).to(torch.bfloat16)  # noqa: E731
        self.h, self.pages, self.shape = handle, pages, (Hq, heads, D)
        B = len(pages.length)
        self.norm_w = bf16(H, scale=0.1) + 1
        self.qkv, self.proj = bf16(H, (Hq + 2 * heads) * D, scale=H ** -0.5), bf16(Hq * D, H, scale=(Hq * D) ** -0.5)
        angle = torch.arange(longest, device=device, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(D // 2, device=device, dtype=torch.float64) * 2 / D)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float()
        k, v = (torch.zeros(pages.pages, pages.page, heads, D, dtype=torch.bfloat16, device=device) for _ in range(2))
        self.cache = tovl.KVCache(k, v)
        self.y = torch.empty(B, H, dtype=torch.bfloat16, device=device)
        self.q, self.out = (torch.empty(B, Hq, D, dtype=torch.bfloat16, device=device) for _ in range(2))
        self.ws = torch.empty(handle.attn_decode_workspace(Hq, heads, D), dtype=torch.uint8, device=device)

    def step(self, x, residual):
        """The block's outputs for rows x, whose pages.step() has been; residual (fp32) is updated in place."""
        h, p, (Hq, heads, D) = self.h, self.pages, self.shape
        h.add_rmsnorm(x, self.norm_w, 1e-5, residual=residual, residual_out=residual, out=self.y)
        rows = self.y @ self.qkv
        q, k, v = (t.unflatten(1, (-1, D)) for t in rows.split([Hq * D, heads * D, heads * D], 1))
        h.rope_append(q, k, v, p.positions, p.slots, self.cos_sin, self.cache, self.q)
        h.attn_decode(self.q, self.cache, p.table, p.length, D ** -0.5, self.out, self.ws)
        return self.out.flatten(1) @ self.proj


def main(tokens=8):
    build.build()
    with tovl.Handle(0) as handle:
        block, pages = Block(handle, tokens), Pages(handle, tokens, 64)
        attention = Attention(handle, pages)
        H = block.y.shape[1]
        x = torch.randn(tokens, H, device="cuda").to(torch.bfloat16)
        residual = torch.zeros(tokens, H, device="cuda")
        for _ in range(3):
            pages.step()
            out, out_q, side = block.step(attention.step(x, residual), residual)
            x = out.clone()
        status = handle.sync_status()
        if status:
            raise SystemExit(f"device status {status}: {tovl.error_string(status)}")
        near = float((out_q.float() - out.float()).norm() / out.float().norm())
        exact = block.y.float() @ block.proj.float()
        print(f"{tokens} requests, 3 steps; 4-bit experts differ from bf16 ones by {near:.3f}, the 4-bit projection of 8-bit "
              f"rows from the exact one by {float((side.float() - exact).norm() / exact.norm()):.3f} (relative)")
        return near


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
