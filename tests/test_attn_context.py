"""Values that are no finite numbers at positions before the drafts, which every row sees: each of their columns is none either,
wherever the position stands in a kernel's tile of keys.  Bounds as in test_attn.py."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B

import test_attn as A
from kv_plain import DT, Cache

pytestmark = pytest.mark.gpu
STARTS = [21, 64, 129, 190]  # drafts begin within a tile of 64 keys, at one, just behind one, and at the end of one


@pytest.fixture(autouse=True)
def lib():
    A.libbuild.build()


@pytest.fixture(params=["narrow", "wide"])
def table(request, monkeypatch):
    """Wide tables take the tcgen05 kernel from 33 rows on."""
    if request.param == "wide":
        monkeypatch.setattr(Cache, "more", 1 << 20)
    return request.param


def call(fmt, dtype, T, G, mask, table, seed, starts=STARTS):
    masks = None if mask is None else [mask] * len(starts)
    c = A.Call(fmt, dtype, [T] * len(starts), starts, 2, G, 64, 16, masks, seed=seed)
    if T * G > 32 and table == "wide":
        assert "tcgen05" in B.proj_attn_describe(c.cache.c, c.m, c.heads)
    if T * G <= 16:
        assert "stream" in B.proj_attn_describe(c.cache.c, c.m, c.heads)
    return c


def spots(c):
    """A sequence's last position before its drafts, the first one of that tile of 64, and one of a tile before."""
    for b, s in enumerate(c.starts):
        yield b, sorted({s - 1, (s - 1) // 64 * 64, (s - 1) // 64 * 32})


@pytest.mark.parametrize("mask", [None, A.tree, A.EMPTY], ids=["chain", "tree", "empty"])
@pytest.mark.parametrize("fmt,dtype,T,G", [("rows", "bf16", 9, 7), ("rows", "fp16", 9, 8), ("e4m3", "bf16", 12, 4), ("int8", "fp16", 40, 4),
                                           ("e4m3", "fp16", 70, 2), ("rows", "bf16", 3, 2), ("int8", "bf16", 2, 4)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_rows_of_values(fmt, dtype, T, G, mask, value, table):
    c = call(fmt, dtype, T, G, mask, table, seed=51)
    for b, at in spots(c):
        for i, p in enumerate(at):
            k, v = c.cache.get("k", b, p, 1).to(DT[dtype][0]), c.cache.get("v", b, p, 1).to(DT[dtype][0])
            v[0, (b + i) % 2, 5 + 20 * i] = value
            c.cache.put(b, p, k, v)
    c.run()
    c.check()
    assert not torch.isfinite(c.out.float()).all()
    assert B.proj_attn_device_status() == 0


@pytest.mark.parametrize("mask", [None, A.tree], ids=["chain", "tree"])
@pytest.mark.parametrize("what", ["code", "scale inf", "scale nan"])
@pytest.mark.parametrize("fmt,T,G", [("e4m3", 10, 4), ("e4m3", 40, 4), ("int8", 40, 4), ("int8", 5, 8), ("e4m3", 2, 2)])
def test_codes_and_scales(fmt, T, G, mask, what, table):
    """The e4m3 code that is no number under a finite scale, and scales that are none."""
    if what == "code" and fmt == "int8":
        pytest.skip("every int8 code is a number")
    c = call(fmt, "bf16", T, G, mask, table, seed=52)
    for b, at in spots(c):
        for i, p in enumerate(at[-2:]):
            page, spot = (int(x[0]) for x in c.cache.spots(b, p, 1))
            if what == "code":
                c.cache.t["v"].view(torch.uint8)[page, (b + i) % 2, spot, 17 + i] = 0x7F + 0x80 * i
            else:
                c.cache.t["v_scale"][page, (b + i) % 2, spot] = math.inf if what == "scale inf" else math.nan
    c.run()
    c.check()
    assert not torch.isfinite(c.out.float()).all()


@pytest.mark.parametrize("T,G", [(8, 8), (70, 2)])
@pytest.mark.parametrize("fmt,dtype", [("rows", "fp16"), ("e4m3", "bf16")])
def test_of_a_long_sequence(fmt, dtype, T, G, table):
    """Shares of one sequence end anywhere: the position's part is joined with others."""
    for start in (4000, 4095, 4097):
        c = call(fmt, dtype, T, G, A.tree, table, seed=53, starts=[start])
        k, v = (c.cache.get(i, 0, start - 1, 1).to(DT[dtype][0]) for i in ("k", "v"))
        v[0, 1, 9] = math.inf
        c.cache.put(0, start - 1, k, v)
        c.run()
        c.check()
        rows = c.out.float().reshape(T, 2, G, 64)
        assert torch.isfinite(rows[:, 0]).all() and not torch.isfinite(rows[:, 1, :, 9]).any()


@pytest.mark.parametrize("T,G", [(9, 8), (70, 2)])
def test_an_accepted_row_stays(T, G, monkeypatch):
    """A row of no finite numbers that was written as a draft and accepted: no later draft gets a number for its head, step after step
    through the tile."""
    monkeypatch.setattr(Cache, "more", 1 << 20)
    for start in range(61, 132, 10):
        c = A.Call("e4m3", "bf16", [T], [start], 1, G, 64, 16, None, seed=start)
        v = torch.ones(1, 1, 64)
        v[0, 0, 7] = math.nan
        c.cache.put(0, 60, torch.ones(1, 1, 64).bfloat16(), v.bfloat16())
        c.run()
        c.check()
        assert not torch.isfinite(c.out.float()).any()
