"""Values of drafts that a row does not see, however large: what the row gets is as good as without them.

Bounds as in test_attn.py, but for the absolute term.  A key's probability times its scale of V is a number of fp16, whose steps end
at 2^-24: off by half of that, 2^-25, where the largest product of a row is 2^4 (or up to 2^14, by how far a reference lags: then it
is less) and stands for a value of its code times the reference scale, which is at most the largest scale among the keys that the
row sees.  So n keys are off by n 2^-29 max |v|, the maximum over what the row sees.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B

import test_attn as A
from kv_plain import DT, Cache, attention

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def lib():
    A.libbuild.build()


@pytest.fixture(params=["narrow", "wide"])
def table(request, monkeypatch):
    if request.param == "wide":
        monkeypatch.setattr(Cache, "more", 1 << 20)
    return request.param


def check(c):
    """As Call.check for finite values, with the maximum of |v| over what a row sees."""
    out, lse = c.out.cpu().double().numpy(), c.lse.cpu().double().numpy()
    u, r, D, at = DT[c.dtype][2], 2.0 ** -8 if c.fmt == "rows" and c.dtype == "bf16" else 2.0 ** -11, c.D, 0
    for b, n in enumerate(c.counts):
        rows, total = slice(at, at + n), c.lens()[b]
        q = c.q[rows, :c.heads * D].reshape(n, c.heads, D).cpu().double().numpy()
        k, v = (c.cache.get(i, b, 0, total).numpy() for i in ("k", "v"))
        sees = c.sees(b)
        ref, ref_lse, mag, spread = attention(q, k, v, sees, float(np.float32(c.scale)))
        assert np.isfinite(ref).all()
        d = ((D + 8) * 2.0 ** -23 + 2.0 ** -20) * spread
        grow = np.expm1(2 * d)[..., None] + r + 2.0 ** -18 + (total + 64) * 2.0 ** -23
        by_key = np.abs(v).max(-1)  # [keys, kv]
        top = np.stack([by_key[sees[i]].max(0) if sees[i].any() else np.zeros(by_key.shape[1]) for i in range(n)])
        top = np.repeat(top, c.G, 1)[..., None]
        bound = grow * mag + 2.0 ** -29 * total * top
        # no less than half a step of the smallest numbers of the output
        bound = bound + u * (np.abs(ref) + bound) + (2.0 ** -25 if c.dtype == "fp16" else 2.0 ** -133)
        got = out[rows, :c.heads * D].reshape(n, c.heads, D)
        assert np.isfinite(got).all()
        far = np.abs(got - ref)
        assert (far <= bound).all(), (b, np.argwhere(far > bound)[:5], (far / bound).max())
        empty = ~sees.any(1)
        assert (lse[rows][empty] == -np.inf).all() and (got[empty] == 0).all()
        assert (np.abs(lse[rows] - ref_lse)[~empty] <= (d + 2.0 ** -20 * (1 + np.abs(ref_lse)))[~empty]).all()
        at += n


def call(fmt, dtype, T, G, starts, table, seed, masks=A.tree, size=0, times=24, drafts=None):
    """Every third draft (or those named) has values 2^times as large as the others, which are some 2^size."""
    c = A.Call(fmt, dtype, [T] * len(starts), starts, 2, G, 64, 16, None if masks is None else [masks] * len(starts), seed=seed)
    if T * G > 32 and table == "wide":
        assert "tcgen05" in B.proj_attn_describe(c.cache.c, c.m, c.heads)
    gen = torch.Generator().manual_seed(seed)
    for b, s in enumerate(starts):
        k, v = torch.randn(s + T, 2, 64, generator=gen), torch.randn(s + T, 2, 64, generator=gen) * 2.0 ** size
        big = torch.zeros(s + T, dtype=torch.bool)
        big[[s + d for d in (range(1, T, 3) if drafts is None else drafts)]] = True
        v[big] *= 2.0 ** times
        c.cache.put(b, 0, k.to(DT[dtype][0]), v.to(DT[dtype][0]))
    return c


STARTS = [0, 21, 64, 190, 700]


@pytest.mark.parametrize("fmt,dtype,size,times", [("e4m3", "bf16", 0, 24), ("int8", "bf16", -20, 40), ("e4m3", "bf16", -90, 60),
                                                  ("int8", "fp16", -10, 20), ("e4m3", "bf16", 30, 60), ("rows", "bf16", 0, 60)])
@pytest.mark.parametrize("T,G", [(9, 8), (70, 2), (4, 4), (3, 2), (40, 1)])
def test_large_drafts(fmt, dtype, size, times, T, G, table):
    c = call(fmt, dtype, T, G, STARTS, table, seed=61, size=size, times=times)
    c.run()
    check(c)
    assert B.proj_attn_device_status() == 0


@pytest.mark.parametrize("T,G", [(9, 8), (100, 2), (4, 4), (2, 2), (40, 1)])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_chain_before_a_large_draft(T, G, fmt, table):
    """Without a mask a row sees no draft behind its own: the last one's size reaches its own row alone."""
    c = call(fmt, "bf16", T, G, STARTS, table, seed=62, masks=None, drafts=[T - 1], times=50)
    c.run()
    check(c)


@pytest.mark.parametrize("T,G", [(9, 8), (100, 2), (4, 4), (2, 2)])
def test_drafts_in_steps(T, G, table):
    """Each draft 2^5 times the one before it: every row sees a larger one than the rows before."""
    c = A.Call("e4m3", "bf16", [T] * 3, [0, 33, 640], 2, G, 64, 16, None, seed=63)
    gen = torch.Generator().manual_seed(63)
    for b, s in enumerate(c.starts):
        grow = torch.exp2(torch.clamp(torch.arange(s + T) - s, 0, 11) * 5.0)[:, None, None]
        k, v = torch.randn(s + T, 2, 64, generator=gen), torch.randn(s + T, 2, 64, generator=gen) * grow
        c.cache.put(b, 0, k.bfloat16(), v.bfloat16())
    c.run()
    check(c)


@pytest.mark.parametrize("T,G", [(9, 8), (70, 2), (4, 4), (3, 2)])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_context_of_zeros(T, G, fmt, table):
    """Rows of zeros have the smallest scale there is; the drafts behind them ordinary ones, and some large."""
    c = call(fmt, "bf16", T, G, STARTS, table, seed=64, times=20)
    for b, s in enumerate(STARTS):
        if s:
            c.cache.put(b, 0, torch.randn(s, 2, 64).bfloat16(), torch.zeros(s, 2, 64).bfloat16())
    c.run()
    check(c)


@pytest.mark.parametrize("T,G", [(9, 8), (70, 2), (4, 4), (3, 2)])
@pytest.mark.parametrize("up", [True, False])
def test_unseen_drafts_beside_references_that_move(T, G, up, table):
    """Scores that rise or fall by hundreds along the keys, values whose scales do by 2^12, and large drafts that some rows do not see."""
    c = call("int8", "bf16", T, G, [0, 45, 700], table, seed=65)
    for b, s in enumerate(c.starts):
        n = s + T
        rise = torch.linspace(0, 1, n) if up else torch.linspace(1, 0, n)
        gen = torch.Generator().manual_seed(b)
        k = torch.randn(n, 2, 64, generator=gen) * 0.05
        k[:, :, 0] = 300.0 * rise[:, None]
        v = torch.randn(n, 2, 64, generator=gen) * torch.exp2(12.0 * rise)[:, None, None]
        v[s + 1::3] *= 2.0 ** 20
        c.cache.put(b, 0, k.bfloat16(), v.bfloat16())
    c.q[:, 0::64] = 1.0
    c.scale = 1.0
    c.run()
    check(c)


def test_no_other_row_changes(table):
    """The rows that do not see a draft have the same numbers whatever its size, up to the rounding of their own keys' products."""
    for T, G in ((9, 8), (4, 4)):
        outs = []
        for times in (0, 24):
            c = call("e4m3", "bf16", T, G, [100], table, seed=66, drafts=[2], times=times)
            c.run()
            check(c)
            outs.append(c.out[~torch.from_numpy(c.sees(0)[:, 102]).cuda()].double())
        assert outs[0].shape[0] and (outs[0] - outs[1]).abs().max() <= 2 * (2.0 ** -8 + 2.0 ** -11) * outs[0].abs().max()
