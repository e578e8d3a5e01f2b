"""Attention between the qkv_gate and o projections, over a quantised cache, for trees of drafted tokens.

    python examples/attention_block.py [sequences] [drafts] [context]

One verify step, every operator through the C ABI: qkv_gate projection -> the
drafts' keys and values to the cache, quantised -> attention of the drafts over
the cache, with the row's gate -> o projection; and, when a path of the tree is
accepted, its entries to their places.  Everything that says how long sequences
are stays on the device, so a step can be captured in a graph and replayed while
they grow.  Weights are random; the widths are the projections' (a row of
qkv_gate is eight query heads of 128, one head of keys and one of values, and a
gate of 1024).
"""
from __future__ import annotations

import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from gemv_projection_layers_gb300 import binding as B  # noqa: E402

HIDDEN, HEADS, HEAD, ROW = 8192, 8, 128, 2304


class AttentionBlock:
    """The projections' weights, and a cache with room for `context` tokens of each sequence and `drafts` more."""

    def __init__(self, sequences: int, drafts: int, context: int, page: int = 64, seed: int = 0):
        gen = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.sequences, self.drafts, self.room_for, self.page = sequences, drafts, context, page
        self.w_in = (rand(ROW, HIDDEN) / HIDDEN ** 0.5).bfloat16()
        self.w_out = (rand(HIDDEN, HEADS * HEAD) / (HEADS * HEAD) ** 0.5).bfloat16()
        m = sequences * drafts
        self.qkv_gate = B.proj_prepare_ex(B.PROJ_QKV_GATE, self.w_in, ROW, HIDDEN, B.PROJ_BF16, 0, m)
        self.o = B.proj_prepare_ex(B.PROJ_O, self.w_out, HIDDEN, HEADS * HEAD, B.PROJ_BF16, 0, m)
        width = -(-(context + drafts) // page)
        pages = sequences * width
        self.k, self.v = (torch.zeros(pages, 1, page, HEAD, device="cuda", dtype=torch.uint8) for _ in range(2))
        self.k_scale, self.v_scale = (torch.zeros(pages, 1, page, device="cuda") for _ in range(2))
        self.table = torch.arange(pages, device="cuda", dtype=torch.int32).view(sequences, width)
        self.cache = B.kv_cache(format=B.PROJ_KV_E4M3, dtype=B.PROJ_BF16, pages=pages, page=page, heads=1, D=HEAD, k=self.k, v=self.v,
                                k_scale=self.k_scale, v_scale=self.v_scale, page_stride=page * HEAD, head_stride=page * HEAD,
                                token_stride=HEAD, table=self.table, ldt=width, width=width, sequences=sequences)
        i32 = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.int32)  # noqa: E731
        self.start, self.next = i32(sequences), i32(sequences)  # tokens of each sequence, before and after a move
        self.offsets = torch.arange(sequences + 1, device="cuda", dtype=torch.int32) * drafts
        self.words = -(-drafts // 32)
        bf16 = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
        self.row, self.mid, self.out = bf16(m, ROW), bf16(m, HEADS * HEAD), bf16(m, HIDDEN)
        self.room = torch.zeros(B.proj_attn_workspace(self.cache, m, HEADS), device="cuda", dtype=torch.uint8)

    def __call__(self, h: torch.Tensor, mask: torch.Tensor | None = None, stream=None):
        """The block's output for h [sequences drafts, HIDDEN], a view of its buffer.  mask [sequences drafts, words]: which
        drafts each row sees, 32 to a word (left out: a chain, each its predecessors and itself).  Everything runs on `stream`
        (a torch stream; left out: torch's current one)."""
        m = self.sequences * self.drafts
        if tuple(h.shape) != (m, HIDDEN) or not h.is_contiguous():
            raise ValueError(f"h: {m} contiguous rows of {HIDDEN}, not {tuple(h.shape)}")
        if mask is not None and (tuple(mask.shape) != (m, self.words) or mask.dtype != torch.int32 or not mask.is_contiguous()):
            raise ValueError(f"mask: int32 [{m}, {self.words}]")
        stream = stream or torch.cuda.current_stream()
        q, k, v, gate = torch.split(self.row, [HEADS * HEAD, HEAD, HEAD, HEADS * HEAD], 1)
        B.proj_run(self.qkv_gate, h, m, self.row, stream)
        B.proj_kv_write(self.cache, self.offsets, self.start, m, k, ROW, v, ROW, stream)
        B.proj_attn(B.attn_args(self.cache, m=m, heads=HEADS, q=q, ldq=ROW, offsets=self.offsets, start=self.start, mask=mask,
                                ldm=self.words, words=self.words, scale=1 / math.sqrt(HEAD), gate=gate, ldg=ROW,
                                gate_act=B.PROJ_GATE_SIGMOID, out=self.mid, ldo=HEADS * HEAD, workspace=self.room,
                                workspace_bytes=self.room.numel()), stream)
        B.proj_run(self.o, self.mid, m, self.out, stream)
        return self.out

    def accept(self, path: torch.Tensor, stream=None):
        """The drafts that stay: path int32 [sequences, depth], ascending, -1 behind its end."""
        if path.shape[0] != self.sequences or path.dtype != torch.int32 or not path.is_contiguous():
            raise ValueError(f"path: int32 [{self.sequences}, depth]")
        stream = stream or torch.cuda.current_stream()
        depth = path.shape[1]
        B.proj_kv_move(self.cache, self.start, path, depth, depth, self.next, stream)
        with torch.cuda.stream(stream):
            self.start.copy_(self.next)

    def close(self):
        B.proj_destroy(self.qkv_gate)
        B.proj_destroy(self.o)


def main() -> None:
    sequences, drafts, context = (int(a) for a in (sys.argv[1:] + ["16", "8", "8192"][len(sys.argv) - 1:])[:3])
    block = AttentionBlock(sequences, drafts, context)
    try:
        # a filled cache: keys and values of some size, uniform scales
        block.k.random_(0, 120)
        block.v.random_(0, 120)
        block.k_scale.fill_(1 / 200)
        block.v_scale.fill_(1 / 200)
        block.start.fill_(context)
        h = torch.randn(sequences * drafts, HIDDEN, device="cuda").bfloat16()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(2):
                block(h, None, side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            block(h, None, side)
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(50):
            graph.replay()
        stop.record()
        torch.cuda.synchronize()
        print(f"{sequences} sequences of {drafts} drafts over {context} tokens: {start.elapsed_time(stop) * 20:.1f} us a step "
              f"(graph replay); {B.proj_attn_describe(block.cache, sequences * drafts, HEADS)}")
    finally:
        block.close()


if __name__ == "__main__":
    main()
