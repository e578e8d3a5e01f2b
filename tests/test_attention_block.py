"""The cache's operators between two projections, as examples/attention_block.py runs them, against the same in 64 bits.

The block's row of qkv_gate and what stands in its cache are taken as the kernels left them; from there to the output
come a probability's rounding to fp16 (2^-11) and its sums, the attention's rounding to bf16, and the o projection's sum
and rounding (2^-8 each): in the norm within 2 2^-8, with a margin of 2.
"""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B

from kv_plain import words_of

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")


def example():
    spec = importlib.util.spec_from_file_location("attention_block", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


def cached(block, name, b, n):
    page = block.page
    at = torch.arange(n, device="cuda")
    ids = block.table[b].long()[at // page]
    code = getattr(block, name).view(torch.float8_e4m3fn).float().double()[ids, 0, at % page]
    return code * getattr(block, name + "_scale").double()[ids, 0, at % page][:, None]


@pytest.mark.gpu
@pytest.mark.parametrize("sequences,drafts,graph", [(1, 1, False), (3, 4, True), (2, 9, True), (1, 40, False)])
def test_block(sequences, drafts, graph):
    ex = example()
    block = ex.AttentionBlock(sequences, drafts, 300, page=16, seed=drafts)
    rng = np.random.default_rng(drafts)
    try:
        m = sequences * drafts
        h = torch.randn(m, ex.HIDDEN, device="cuda").bfloat16()
        mask = torch.zeros(m, block.words, dtype=torch.int32, device="cuda")
        side = torch.cuda.Stream()
        captured = None
        for step in range(4):
            h.copy_(torch.randn(m, ex.HIDDEN, device="cuda"))
            sees = np.zeros((sequences, drafts, drafts), bool)
            for b in range(sequences):
                for i in range(drafts):
                    parent = i - 1 - int(rng.integers(0, 3))
                    if parent >= 0:
                        sees[b, i] = sees[b, parent]
                    sees[b, i, i] = True
            mask.copy_(words_of(sees.reshape(m, drafts)))
            torch.cuda.synchronize()
            if graph and captured is None:
                with torch.cuda.stream(side):
                    block(h, mask, side)
                torch.cuda.synchronize()
                captured = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured, stream=side):
                    block(h, mask, side)
            if captured is not None:
                captured.replay()
                out = block.out
            else:
                out = block(h, mask)
            torch.cuda.synchronize()
            d = lambda t: t.double()  # noqa: E731
            row = d(block.row)
            ref = d(h) @ d(block.w_in).t()
            assert (row - ref).norm() <= 1.1 * 2.0 ** -8 * ref.norm()
            y = torch.zeros(m, ex.HEADS * ex.HEAD, device="cuda", dtype=torch.float64)
            start = block.start.tolist()
            for b in range(sequences):
                n = start[b]
                rows = slice(b * drafts, (b + 1) * drafts)
                k, v = cached(block, "k", b, n + drafts), cached(block, "v", b, n + drafts)
                q = row[rows, :1024].reshape(drafts, ex.HEADS, ex.HEAD)
                s = torch.einsum("thd,kd->thk", q, k) / ex.HEAD ** 0.5
                hidden = torch.ones(drafts, n + drafts, dtype=torch.bool, device="cuda")
                hidden[:, :n] = False
                hidden[:, n:] = torch.from_numpy(~sees[b]).cuda()
                p = torch.softmax(s.masked_fill(hidden[:, None, :], -torch.inf), -1)
                y[rows] = torch.einsum("thk,kd->thd", p, v).reshape(drafts, -1)
            y = y * torch.sigmoid(row[:, 1280:])
            ref = y @ d(block.w_out).t()
            assert (d(out) - ref).norm() <= 4 * 2.0 ** -8 * ref.norm()
            path = np.full((sequences, drafts), -1, np.int32)
            for b in range(sequences):
                taken = np.flatnonzero(sees[b, int(rng.integers(0, drafts))])
                path[b, :len(taken)] = taken
                start[b] += len(taken)
            block.accept(torch.from_numpy(path).cuda())
            torch.cuda.synchronize()
            assert block.start.tolist() == start
        assert B.proj_attn_device_status() == 0
    finally:
        block.close()


def test_shapes_are_checked():
    ex = example()
    block = object.__new__(ex.AttentionBlock)
    block.sequences, block.drafts, block.words = 2, 3, 1
    with pytest.raises(ValueError):
        block(torch.zeros(5, ex.HIDDEN))
    with pytest.raises(ValueError):
        block(torch.zeros(6, ex.HIDDEN), torch.zeros(6, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        block.accept(torch.zeros(3, 3, dtype=torch.int32))
