"""The operators together, as examples/moe_block.py runs them, against the same block in 64 bits.

Each step rounds its output to bf16 (2^-8) and the next reads it; a reference that takes the
kernels' own choice of experts then differs by the roundings only: seven of them between the
residual stream and the block's output, each within 2^-8 of its vector's size, amplified by at most
the product's two factors in the gated unit -- in the norm, (7 + 2) 2^-8 with a margin of 2.
"""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 5, 300])
def test_block(m):
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    block = ex.MoeBlock(m, inner=128, k=4, group=64, seed=m)
    try:
        residual = torch.randn(m, ex.HIDDEN, device="cuda").bfloat16()
        out, nxt = block(residual)
        torch.cuda.synchronize()
        d = lambda t: t.double()  # noqa: E731
        r = d(residual)
        norm = lambda v: v * (v.pow(2).mean(1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
        h = norm(r) * d(block.w_in)
        assert (d(block.h) - h).norm() <= 2.0 ** -8 * h.norm()
        logits = d(block.h) @ d(block.w_router).t()
        assert (d(block.logits) - logits).abs().max() <= 1e-4 * logits.abs().max()
        chosen = block.expert.long()
        assert torch.equal(chosen.sort(1).values, block.logits.topk(4, 1).indices.sort(1).values)
        weight = torch.softmax(torch.gather(d(block.logits), 1, chosen), 1)

        def w64(codes, scales, e):
            q = torch.stack((codes[e] & 15, codes[e] >> 4), -1).flatten(-2).double() - 8
            return q * d(scales[e]).repeat_interleave(block.group, -1)

        y = torch.zeros_like(h)
        F = block.inner
        for e in chosen.unique().tolist():
            t, j = (chosen == e).nonzero(as_tuple=True)
            mid = h[t] @ w64(block.up_codes, block.up_scales, e).t()
            act = torch.nn.functional.silu(mid[:, :F]) * mid[:, F:]
            y.index_add_(0, t, (act @ w64(block.down_codes, block.down_scales, e).t()) * weight[t, j][:, None])
        bound = 2 * 9 * 2.0 ** -8
        assert (d(block.y) - y).norm() <= bound * y.norm()
        u = r + torch.sigmoid(d(block.gate)) * norm(y) * d(block.w_post)
        assert (d(out) - u).norm() <= bound * u.norm()
        z = norm(u) * d(block.w_next)
        assert (d(nxt) - z).norm() <= bound * z.norm()
        assert B.proj_w4_device_status(block.up) == 0 and B.proj_w4_device_status(block.down) == 0
    finally:
        block.close()
