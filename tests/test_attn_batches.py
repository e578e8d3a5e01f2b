"""Attention of batches: more than three items to two SMs, which are streamed by warps with a share each.  Bounds as in test_attn.py."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B

import test_attn as A
from kv_plain import DT, int32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def lib():
    A.libbuild.build()


def batch(fmt, dtype, T, G, D, seed, n=44, kv=8, page=16, **more):
    """Sequences without rows, without context, of a page's length, some long ones that several warps share."""
    rng = np.random.default_rng(seed)
    counts = [T if b % 3 else int(rng.integers(0, T + 1)) for b in range(n)]
    starts = [[0, 1, 15, 16, 31, 33, 64][b % 7] if b % 5 else int(rng.integers(0, 200)) for b in range(n)]
    starts[n // 2] = 1500
    starts[-1] = 700
    c = A.Call(fmt, dtype, counts, starts, kv, G, D, page, seed=seed, **more)
    assert "warps" in B.proj_attn_describe(c.cache.c, c.m, c.heads)
    return c


CASES = [("e4m3", "bf16", 1, 8, 128), ("rows", "bf16", 1, 5, 128), ("int8", "fp16", 2, 4, 64), ("rows", "fp16", 4, 4, 64),
         ("e4m3", "fp16", 3, 8, 64), ("int8", "bf16", 4, 3, 128)]


@pytest.mark.parametrize("fmt,dtype,T,G,D", CASES)
def test_batches(fmt, dtype, T, G, D):
    c = batch(fmt, dtype, T, G, D, seed=T * G + D, masks=[A.tree] * 44, gate=B.PROJ_GATE_SIGMOID if D == 128 else None, more=8)
    c.run()
    c.check()
    assert B.proj_attn_device_status() == 0


@pytest.mark.parametrize("fmt,dtype", [("rows", "bf16"), ("e4m3", "bf16")])
def test_rows_that_see_nothing_and_no_finite_numbers(fmt, dtype):
    T, D = 3, 64
    c = batch(fmt, dtype, T, 2, D, seed=41, masks=[A.EMPTY if b % 4 == 0 else A.tree for b in range(44)])
    for b in range(44):
        if c.counts[b] < 2 or b % 2:
            continue
        k, v = torch.ones(1, 8, D), torch.ones(1, 8, D)
        k[0, 1, 3] = math.nan
        v[0, 2, 5] = math.nan
        c.cache.put(b, c.starts[b] + c.counts[b] - 1, k.to(DT[dtype][0]), v.to(DT[dtype][0]))
    c.run()
    c.check()


def test_in_place_two_streams_and_the_same_bits():
    a = batch("e4m3", "bf16", 2, 4, 64, seed=42, gate=B.PROJ_GATE_SIGMOID)
    b = batch("rows", "fp16", 1, 4, 64, seed=43)
    a.run()
    b.run()
    torch.cuda.synchronize()
    a.check()
    b.check()
    want = [a.out.clone(), b.out.clone()]
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        q = a.q.clone()
        b.out.fill_(A.GUARD)
        for c in (a, b):
            c.room.fill_(255)
        torch.cuda.synchronize()
        a.run(one, q=q, out=q, lse=None)
        b.run(two)
        torch.cuda.synchronize()
        rows = sum(a.counts)
        assert torch.equal(q[:rows], want[0][:rows]) and torch.equal(b.out, want[1])


def test_graph_of_sequences_that_change():
    c = batch("int8", "bf16", 2, 8, 64, seed=44)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.run(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.run(side)
    for _ in range(3):
        c.out.fill_(A.GUARD)
        c.lse.fill_(A.GUARD)
        graph.replay()
        torch.cuda.synchronize()
        c.check()
        c.starts = [max(0, s - 29) for s in c.starts]
        c.start.copy_(int32(c.starts))
        torch.cuda.synchronize()


@pytest.mark.parametrize("T", [1, 3])
def test_many_short_sequences(T):
    """More sequences than a warp looks at by itself; several shares begin in one sequence, and sequences in one share."""
    n = 400
    counts = [T - (b % 4 == 0) for b in range(n)]
    starts = [(5 * b) % 40 for b in range(n)]
    starts[17], starts[399] = 3000, 900
    c = A.Call("int8", "fp16", counts, starts, 1, 4, 64, 16, None, seed=45)
    assert "warps" in B.proj_attn_describe(c.cache.c, c.m, c.heads)
    c.run()
    c.check()


def test_workspace_never_shrinks_with_more_rows():
    for sequences, kv, width in ((1, 1, 64), (40, 8, 4), (64, 1, 300), (700, 1, 2), (16, 1, 2100)):
        cache = B.kv_cache(format=B.PROJ_KV_ROWS, dtype=B.PROJ_FP16, pages=1, page=16, heads=kv, D=128, k=4096, v=8192, page_stride=1 << 20,
                           head_stride=2048, token_stride=128, table=4096, ldt=width, width=width, sequences=sequences)
        sizes = [B.proj_attn_workspace(cache, m, 4 * kv) for m in range(0, 40 * sequences, max(1, sequences // 2))]
        assert sizes == sorted(sizes)
