"""A block of experts with 4-bit weights, from the residual stream back to it.

    python examples/moe_block.py [tokens]

One step as a decode or verify loop runs it, every operator through the C ABI:
norm before the block -> router projection (fp32 weights) -> choice and sort by
expert -> gather -> the experts' up and down products on 4-bit weights ->
weighted combine -> norm after the block, gate, residual and the next block's
norm.  Weights are random; sizes are the router's (hidden 8192, 256 experts)
with small experts.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from gemv_projection_layers_gb300 import binding as B  # noqa: E402

HIDDEN, EXPERTS = 8192, 256


def quantise(w: torch.Tensor, group: int):
    """4-bit codes and group scales of w [E, N, K] (symmetric, largest value at 7)."""
    E, N, K = w.shape
    g = w.view(E, N, K // group, group).float()
    scale = (g.abs().amax(-1, keepdim=True) / 7.0).clamp(min=1e-8).bfloat16()
    q = (torch.round(g / scale.float()).clamp(-8, 7) + 8).to(torch.uint8).view(E, N, K)
    return (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous(), scale.view(E, N, K // group).contiguous()


class MoeBlock:
    """The block's weights and the buffers for up to `tokens` tokens."""

    def __init__(self, tokens: int, inner: int = 256, k: int = 8, group: int = 128, seed: int = 0):
        gen = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.tokens, self.k, self.inner, self.group = tokens, k, inner, group
        self.w_router = rand(EXPERTS, HIDDEN) / HIDDEN ** 0.5
        up = rand(EXPERTS, 2 * inner, HIDDEN) / HIDDEN ** 0.5
        down = rand(EXPERTS, HIDDEN, inner) / inner ** 0.5
        self.up_codes, self.up_scales = quantise(up, group)
        self.down_codes, self.down_scales = quantise(down, group)
        self.w_in, self.w_post, self.w_next = ((1 + 0.1 * rand(HIDDEN)).bfloat16() for _ in range(3))
        self.gate = rand(HIDDEN).bfloat16()
        self.router = B.proj_prepare_ex(B.PROJ_ROUTER, self.w_router, EXPERTS, HIDDEN, B.PROJ_FP32, 0, tokens)
        self.up = B.proj_w4_prepare(self.up_codes, self.up_scales, None, EXPERTS, 2 * inner, HIDDEN, group, B.PROJ_BF16)
        self.down = B.proj_w4_prepare(self.down_codes, self.down_scales, None, EXPERTS, HIDDEN, inner, group, B.PROJ_BF16)
        rows = tokens * k
        bf16 = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        i32 = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.int32)  # noqa: E731
        self.h, self.y, self.out, self.next = (bf16(tokens, HIDDEN) for _ in range(4))
        self.logits, self.weight = torch.zeros(tokens, EXPERTS, device="cuda"), torch.zeros(tokens, k, device="cuda")
        self.expert, self.slot, self.order, self.offsets = i32(tokens, k), i32(tokens, k), i32(rows), i32(EXPERTS + 1)
        self.xs, self.ys = bf16(rows, HIDDEN), bf16(rows, HIDDEN)
        self.mid, self.act = bf16(rows, 2 * inner), bf16(rows, inner)
        self.room = torch.zeros(max(16, B.proj_moe_workspace(tokens, EXPERTS, k)), device="cuda", dtype=torch.uint8)

    def __call__(self, residual: torch.Tensor, stream=None):
        """(new residual, input of the next block), views of the block's buffers.  Everything runs on `stream`
        (a torch stream; left out: torch's current one), the gated unit between the products included."""
        if residual.shape[0] > self.tokens or residual.shape[1:] != (HIDDEN,) or not residual.is_contiguous():
            raise ValueError(f"residual: at most {self.tokens} contiguous rows of {HIDDEN}, not {tuple(residual.shape)}")
        stream = stream or torch.cuda.current_stream()
        with torch.cuda.stream(stream):
            return self._steps(residual, stream)

    def _steps(self, residual: torch.Tensor, stream):
        m, k, D, F = residual.shape[0], self.k, HIDDEN, self.inner
        common = dict(m=m, D=D, dtype=B.PROJ_BF16, eps=1e-6, residual=residual, ldr=D)
        B.proj_norm(B.norm_args(**common, w_pre=self.w_in, normed=self.h, ldn=D), stream)
        B.proj_run(self.router, self.h, m, self.logits, stream)
        B.proj_moe_route(self.logits, EXPERTS, m, EXPERTS, k, B.PROJ_ROUTE_CHOSEN, self.expert, self.weight, self.offsets, self.order,
                         self.slot, self.room, self.room.numel(), stream)
        B.proj_moe_gather(self.h, D, self.slot, m, D, k, B.PROJ_BF16, self.xs, D, stream)
        B.proj_w4_run_experts(self.up, self.xs, D, m * k, self.offsets, self.mid, 2 * F, stream)
        torch.mul(torch.nn.functional.silu(self.mid[:m * k, :F]), self.mid[:m * k, F:], out=self.act[:m * k])
        B.proj_w4_run_experts(self.down, self.act, F, m * k, self.offsets, self.ys, D, stream)
        B.proj_moe_combine(self.ys, D, self.slot, self.weight, m, D, k, B.PROJ_BF16, self.y, D, stream)
        B.proj_norm(B.norm_args(**common, y=self.y, ldy=D, gate=self.gate, gate_mode=B.PROJ_GATE_CHANNEL,
                                gate_act=B.PROJ_GATE_SIGMOID, w_post=self.w_post, w_pre=self.w_next, out=self.out, ldo=D,
                                normed=self.next, ldn=D), stream)
        return self.out[:m], self.next[:m]

    def close(self):
        B.proj_destroy(self.router)
        B.proj_w4_destroy(self.up)
        B.proj_w4_destroy(self.down)


def main() -> None:
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 16
    block = MoeBlock(tokens)
    try:
        residual = torch.randn(tokens, HIDDEN, device="cuda").bfloat16()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(2):
                block(residual, side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            block(residual, side)
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(50):
            graph.replay()
        stop.record()
        torch.cuda.synchronize()
        busy = int((block.offsets[1:] > block.offsets[:-1]).sum())
        print(f"{tokens} tokens, {busy} of {EXPERTS} experts with rows: {start.elapsed_time(stop) * 20:.1f} us a block "
              f"(graph replay); up: {B.proj_w4_describe(block.up, tokens * block.k)}")
    finally:
        block.close()


if __name__ == "__main__":
    main()
