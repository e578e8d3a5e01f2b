"""Offsets and starts beyond their range, a table that is full to its last place, and queries of very different size: values against
attention in 64 bits under the bounds of test_attn.py, on either kernel."""
import copy
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B

import test_attn as A
from kv_plain import Cache, int32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def lib():
    A.libbuild.build()


@pytest.fixture(params=["narrow", "wide"])
def table(request, monkeypatch):
    if request.param == "wide":
        monkeypatch.setattr(Cache, "more", 1 << 20)
    return request.param


class One:
    """A cache's sequence b as the first."""

    def __init__(self, cache, b):
        self.cache, self.b = cache, b

    def get(self, n, b, first, count):
        return self.cache.get(n, self.b, first, count)


def part(c, b, lo, hi, start, keys, sees):
    """The rows lo .. hi - 1 of a call as one of their own: sequence b's, over `keys` positions of which row i sees sees[i]."""
    d = copy.copy(c)
    d.cache, d.counts, d.starts = One(c.cache, b), [hi - lo], [start]
    d.q, d.out, d.lse = c.q[lo:hi], c.out[lo:hi], c.lse[lo:hi]
    d.lens, d.sees = lambda: [keys], lambda _: sees.copy()
    return d


def chain(rows, start, keys):
    return np.arange(keys)[None, :] <= start + np.arange(rows)[:, None]


@pytest.mark.parametrize("n,G", [(8, 4), (7, 1), (40, 4), (90, 2)])
@pytest.mark.parametrize("fmt,dtype", [("rows", "fp16"), ("e4m3", "bf16")])
def test_offsets(n, G, fmt, dtype, table):
    for off in ([-3, n, 400 + 2 * n], [2, n - 1, 2 * n - 3], [0, n, 2], [n + 1, 3, n], [-5, -3, n], [2 * n, 2 * n, 2 * n],
                [3 * n, 0, n], [-2 ** 31, n, 2 ** 31 - 1]):
        c = A.Call(fmt, dtype, [n, n], [40, 71], 1, G, 64, 16, None, more=8, seed=81)
        c.run(offsets=int32(off))
        torch.cuda.synchronize()
        owned = np.zeros(2 * n, bool)
        for b, start in enumerate(c.starts):
            lo = min(max(off[b], 0), 2 * n)
            hi = min(max(off[b + 1], lo), 2 * n)
            if hi > lo:
                part(c, b, lo, hi, start, start + hi - lo, chain(hi - lo, start, start + hi - lo)).check()
            assert not owned[lo:hi].any()
            owned[lo:hi] = True
        left = torch.from_numpy(~owned).cuda()
        assert bool((c.out[left] == A.GUARD).all()) and bool((c.lse[left] == A.GUARD).all())
    assert B.proj_attn_device_status() == 0


@pytest.mark.parametrize("T,G", [(2, 4), (9, 4), (40, 2)])
def test_negative_starts(T, G, table):
    """A negative start counts as 0."""
    for s in (-1, -7, -2 ** 31):
        c = A.Call("e4m3", "bf16", [T, T], [0, 30], 1, G, 64, 16, [A.tree] * 2, seed=82)
        c.start.copy_(int32([s, 30]))
        c.run()
        c.check()


@pytest.mark.parametrize("T,G,kv", [(2, 4, 1), (9, 4, 1), (64, 8, 8)])
@pytest.mark.parametrize("fmt,dtype,page", [("e4m3", "bf16", 16), ("rows", "fp16", 24)])
def test_to_the_last_place_of_a_table(T, G, kv, fmt, dtype, page):
    """Every place of the table is a page; drafts behind its end have no place and are not seen."""
    for past in (-T, -T // 2, -1, 0, 5, 2 ** 31):
        c = A.Call(fmt, dtype, [T], [520 - T], kv, G, 64, page, None, seed=83)
        if T == 64:
            assert "tcgen05" in B.proj_attn_describe(c.cache.c, c.m, c.heads)
        free = c.cache.table[0] < 0
        c.cache.table[0, free] = c.cache.table[0, 0]
        c.cache.d_table.copy_(c.cache.table)
        last = c.cache.width * page
        # the part of the last page that was never written
        fill = -(-520 // page) * page - 520
        if fill:
            c.cache.put(0, 520, torch.randn(fill, kv, 64), torch.randn(fill, kv, 64))
        start = min(last + past, 2 ** 31 - 1)
        c.start.copy_(int32([start]))
        c.run()
        part(c, 0, 0, T, start, last, chain(T, start, last)).check()
    assert B.proj_attn_device_status() == 0


@pytest.mark.parametrize("T,G", [(6, 2), (12, 4), (12, 8), (16, 12)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("scale", [0.125, -0.125])
def test_extreme_queries(T, G, fmt, scale, table):
    """Rows of queries of very different size (bf16's range, numbers below its normal ones among them), zeros, and one with an infinity."""
    c = A.Call(fmt, "bf16", [T], [50], 1, G, 64, 16, None, seed=84, scale=scale)
    sizes = [2.0 ** -126, 2.0 ** -60, 0.0, 1.0, 2.0 ** 8]
    sizes = torch.tensor([sizes[i % 5] for i in range(T - 1)] + [1.0], dtype=torch.bfloat16)
    c.q.mul_(sizes.cuda()[:, None])
    c.q[T - 1, 3] = math.inf
    c.run()
    assert c.out[T - 1, :64].isnan().all()
    # the infinity is the first head's alone
    assert c.out[T - 1, 64:].isfinite().all()
    part(c, 0, 0, T - 1, 50, 50 + T, chain(T - 1, 50, 50 + T)).check()


@pytest.mark.parametrize("T,G", [(2, 4), (9, 8), (40, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scores_of_minus_infinity(T, G, dtype, table):
    """A row of which every score is -infinity gets zeros, as one that sees nothing; beside other keys such a score counts for nothing."""
    c = A.Call("rows", dtype, [T, T], [0, 20], 1, G, 64, 16, None, seed=85)
    for b, s in enumerate(c.starts):
        k, v = torch.zeros(1, 1, 64), torch.ones(1, 1, 64)
        k[0, 0, 0] = -math.inf
        c.cache.put(b, s, k.to(c.q.dtype), v.to(c.q.dtype))
    c.q[:, 0::64] = 1.0  # each head's first dimension: the key's score is -infinity for every row
    c.run()
    torch.cuda.synchronize()
    assert bool((c.out[0] == 0).all()) and bool((c.lse[0] == -math.inf).all())
    # without that key
    for b, (s, at) in enumerate(zip(c.starts, (0, T))):
        sees = chain(T, s, s + T)
        sees[:, s] = False
        d = part(c, b, at, at + T, s, s + T, sees)
        k = c.cache.get("k", b, 0, s + T)
        k[s] = 0
        d.cache = type("Kept", (), {"get": staticmethod(lambda n, _, first, count, k=k, b=b: k if n == "k" else c.cache.get(n, b, first, count))})
        d.check()
