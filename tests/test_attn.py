"""Attention of drafted tokens over the cache against plain attention in 64 bits, on the values that the cache stands for.

Bounds, with u the rounding of the output's type (half a step) and w the probabilities of a row:
  score:  its fp32 sum of D products is off by (D + 8) 2^-23 of a = scale sum |q k| (terms of one sum, either order, chopped
          or rounded), the factors and the subtraction of the reference by 2^-20 of |score| <= a;  d = ((D + 8) 2^-23 + 2^-20) a.
  output: each probability is off by its score's error, exp2's 2^-21, its rounding to 16 bits (r = 2^-8 in a bf16 cache, 2^-11 else),
          the product with V's scale (2^-22) and an absolute 2^-30 where it falls below fp16's range; the sums of n terms by
          (n + 64) 2^-24 each:  (r + 2 d + 2^-18 + (n + 64) 2^-23) sum w |v|  +  2^-30 n max |v|, and u of the result;  a gate
          multiplies all that by itself and adds 2^-20 of the result (sigmoid by exp and a quotient).
  lse:    d + 2^-20 (1 + |lse|).
"""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B
from gemv_projection_layers_gb300 import build as libbuild

from kv_plain import DT, Cache, attention, int32, offsets_of, words_of

GUARD = 7.0


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return B.load()


def tree(n, rng):
    """A random tree of n drafts: what each sees."""
    sees = np.zeros((n, n), bool)
    for i in range(n):
        parent = i - 1 - int(rng.integers(0, 3))
        if parent >= 0:
            sees[i] = sees[parent]
        sees[i, i] = True
    return sees


class Call:
    """A filled cache, queries, and a call over them."""

    def __init__(self, fmt, dtype, counts, starts, kv, G, D, page, masks=None, gate=None, layout="head", more=0, behind=0, seed=0, scale=None,
                 spread=1.0):
        self.fmt, self.dtype, self.counts, self.starts, self.kv, self.G, self.D = fmt, dtype, counts, starts, kv, G, D
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        T = DT[dtype][0]
        self.cache = Cache(fmt, dtype, [s + n for s, n in zip(starts, counts)], kv, D, page, layout, seed)
        for b, n in enumerate(self.lens()):
            k = torch.randn(n, kv, D, generator=gen) * torch.exp(spread * torch.randn(n, 1, 1, generator=gen) / 3)
            v = torch.randn(n, kv, D, generator=gen) * torch.exp(spread * torch.randn(n, 1, 1, generator=gen))
            self.cache.put(b, 0, k.to(T), v.to(T))
        self.m, self.heads = sum(counts) + behind, kv * G
        width = self.heads * D
        wide = lambda: (torch.randn(self.m, width + more, generator=gen)).to(T).cuda()  # noqa: E731
        self.q = wide()
        self.gate, self.act = (None, B.PROJ_GATE_SIGMOID) if gate is None else (wide(), gate)
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale
        self.masks = masks if masks is None or masks == [] else [m(n, rng) if callable(m) else m for m, n in zip(masks, counts)]
        self.mask = None
        if self.masks is not None:
            most = max(m.shape[1] for m in self.masks)
            full = np.ones((self.m, max(most, 1)), bool)
            at = 0
            for m, n in zip(self.masks, counts):
                full[at:at + n, :m.shape[1]] = m
                full[at:at + n, m.shape[1]:] = False
                at += n
            self.mask = words_of(full)
        self.more = more
        self.out = torch.full((self.m, width + more), GUARD, device="cuda", dtype=T)
        self.lse = torch.full((self.m, self.heads), GUARD, device="cuda")
        self.offsets, self.start = offsets_of(counts), int32(starts)
        self.room = self.workspace()

    def lens(self):
        return [s + n for s, n in zip(self.starts, self.counts)]

    def workspace(self):
        return torch.full((B.proj_attn_workspace(self.cache.c, self.m, self.heads),), 255, device="cuda", dtype=torch.uint8)

    def args(self, **change):
        words = 0 if self.mask is None else self.mask.shape[1]
        f = dict(m=self.m, heads=self.heads, q=self.q, ldq=self.q.stride(0), offsets=self.offsets, start=self.start, mask=self.mask, ldm=words,
                 words=words, scale=self.scale, gate=self.gate, ldg=self.q.stride(0), gate_act=self.act, out=self.out, ldo=self.out.stride(0),
                 lse=self.lse, workspace=self.room, workspace_bytes=self.room.numel())
        return B.attn_args(self.cache.c, **{**f, **change})

    def run(self, stream=None, **change):
        B.proj_attn(self.args(**change), stream)

    def sees(self, b):
        n, s = self.counts[b], self.starts[b]
        if self.masks is None:
            own = np.tril(np.ones((n, n), bool))
        else:
            own = np.zeros((n, n), bool)
            w = min(n, self.masks[b].shape[1])
            own[:, :w] = self.masks[b][:, :w]
        return np.concatenate([np.ones((n, s), bool), own], 1)

    def check(self, hidden=None, out=None, lse=None):
        """`hidden`: positions (sequence, position) without a page."""
        out = (self.out if out is None else out).cpu().double().numpy()
        lse = (self.lse if lse is None else lse).cpu().double().numpy()
        width, D = self.heads * self.D, self.D
        u = DT[self.dtype][2]
        r = 2.0 ** -8 if self.fmt == "rows" and self.dtype == "bf16" else 2.0 ** -11
        r = getattr(self, "r", r)
        at = 0
        for b, n in enumerate(self.counts):
            if n == 0:
                continue
            rows = slice(at, at + n)
            total = self.lens()[b]
            q = self.q[rows, :width].reshape(n, self.heads, D).cpu().double().numpy()
            k, v = (self.cache.get(i, b, 0, total).numpy() for i in ("k", "v"))
            sees = self.sees(b)
            for (hb, p) in hidden or []:
                if hb == b:
                    sees[:, p] = False
            ref, ref_lse, mag, spread = attention(q, k, v, sees, float(np.float32(self.scale)))
            d = ((D + 8) * 2.0 ** -23 + 2.0 ** -20) * spread
            # exp of a score that is off by d is off by exp(d) - 1
            grow = np.expm1(2 * d)[..., None] + r + 2.0 ** -18 + (total + 64) * 2.0 ** -23
            top = np.abs(np.where(np.isfinite(v), v, 0)).max() if total else 0.0
            bound = grow * mag + 2.0 ** -30 * total * top
            if self.gate is not None:
                x = self.gate[rows, :width].reshape(n, self.heads, D).cpu().double().numpy()
                x = x if self.act == B.PROJ_GATE_LINEAR else 1 / (1 + np.exp(-x))
                ref, bound = ref * x, bound * np.abs(x) + 2.0 ** -20 * np.abs(ref * x)
            bound = bound + u * (np.abs(ref) + bound) + 2.0 ** -25
            got = out[rows, :width].reshape(n, self.heads, D)
            fine = np.isfinite(ref)
            assert (np.isfinite(got) == fine).all(), (b, np.argwhere(np.isfinite(got) != fine)[:5])
            with np.errstate(invalid="ignore"):  # infinities: `fine` leaves them out
                far, far_lse = np.abs(got - ref), np.abs(lse[rows] - ref_lse)
            bad = np.where(fine, far, 0) > np.where(fine, bound, 1)
            assert not bad.any(), (b, np.argwhere(bad)[:5], far[bad][:5], bound[bad][:5])
            got_lse = lse[rows]
            empty = ~sees.any(1)
            assert (got_lse[empty] == -np.inf).all() and (got[empty] == 0).all()
            fine = np.isfinite(ref_lse)
            assert (np.isfinite(got_lse[~empty]) == fine[~empty]).all()
            off = np.where(fine, far_lse, 0) > np.where(fine, d + 2.0 ** -20 * (1 + np.abs(ref_lse)), 1)
            assert not off.any(), (b, np.argwhere(off)[:5])
            at += n
        assert (out[at:] == GUARD).all() and (out[:, width:] == GUARD).all() and (lse[at:] == GUARD).all()


EMPTY = lambda n, rng: np.zeros((n, n), bool)  # noqa: E731
CASES = [
    # fmt, dtype, counts, starts, kv, G, D, page, masks, gate, layout
    ("e4m3", "bf16", [1], [0], 1, 1, 64, 16, None, None, "head"),
    ("e4m3", "bf16", [1], [1], 1, 8, 128, 64, None, B.PROJ_GATE_SIGMOID, "head"),
    ("rows", "bf16", [1, 1, 1], [0, 16, 333], 2, 7, 128, 7, None, B.PROJ_GATE_LINEAR, "token"),
    ("rows", "fp16", [1] * 5, [15, 127, 128, 129, 1000], 1, 8, 64, 1, None, None, "head"),
    ("int8", "fp16", [1, 0, 1], [700, 5, 63], 3, 5, 64, 48, None, None, "token"),
    ("int8", "bf16", [2, 3], [31, 250], 1, 8, 128, 16, [tree] * 2, B.PROJ_GATE_SIGMOID, "head"),
    ("e4m3", "fp16", [4, 1, 0, 2], [0, 0, 9, 600], 5, 3, 64, 100, [tree] * 4, None, "head"),
    ("e4m3", "bf16", [8, 8], [257, 2000], 1, 8, 128, 128, [tree] * 2, B.PROJ_GATE_SIGMOID, "head"),
    ("rows", "bf16", [13, 5], [40, 511], 2, 4, 128, 32, None, None, "token"),
    ("rows", "fp16", [33, 64, 1], [100, 3, 0], 2, 3, 64, 24, [tree] * 3, None, "head"),
    ("int8", "bf16", [70, 129], [90, 1], 1, 2, 128, 16, [tree] * 2, B.PROJ_GATE_LINEAR, "token"),
    ("e4m3", "fp16", [64, 17, 0, 40], [300, 0, 8, 77], 1, 8, 128, 64, [tree] * 4, None, "head"),
    ("rows", "bf16", [40], [5000], 1, 16, 128, 64, [tree], None, "head"),
    ("e4m3", "bf16", [150], [37], 2, 1, 64, 64, None, None, "head"),
    ("rows", "fp16", [200, 31], [0, 64], 1, 4, 128, 128, None, B.PROJ_GATE_SIGMOID, "head"),
    # rows that see nothing: no context and an empty mask, beside others
    ("e4m3", "bf16", [3, 2], [0, 20], 1, 8, 128, 16, [EMPTY] * 2, B.PROJ_GATE_SIGMOID, "head"),
    ("rows", "fp16", [40, 9], [0, 0], 1, 8, 128, 16, [EMPTY, tree], None, "head"),
    ("int8", "fp16", [20], [0], 2, 4, 64, 16, [EMPTY], None, "head"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case):
    fmt, dtype, counts, starts, kv, G, D, page, masks, gate, layout = CASES[case]
    c = Call(fmt, dtype, counts, starts, kv, G, D, page, masks, gate, layout, more=8 * (case % 3), behind=case % 2 * 3, seed=case)
    c.run()
    c.check()
    assert B.proj_attn_device_status() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 9, 16, 17, 31, 33])
@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("rows", "bf16"), ("int8", "fp16")])
def test_numbers_of_drafts(T, fmt, dtype):
    """Every number of rows of an item, lengths around the units' ends, many sequences on few CTAs."""
    counts = [T - (b % 2 if T > 1 else 0) for b in range(9)]
    starts = [0, 1, 15, 16, 63, 64, 65, 127, 128]
    c = Call(fmt, dtype, counts, starts, 1, 8, 64, 16, [tree] * 9, seed=T)
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 8, 64])
def test_split_over_all_ctas(T):
    """One long sequence: every CTA has a part, and the parts are joined."""
    c = Call("e4m3", "bf16", [T], [40000], 1, 8, 64, 64, [tree], B.PROJ_GATE_SIGMOID, seed=3)
    c.run()
    c.check()


@pytest.mark.gpu
def test_many_sequences():
    """More sequences than threads look at in one go, some without rows."""
    n = 700
    counts = [(3 * b) % 4 for b in range(n)]
    starts = [(7 * b) % 50 for b in range(n)]
    c = Call("int8", "fp16", counts, starts, 1, 4, 64, 16, None, seed=4)
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("spread,scale", [(4.0, 0.125), (0.0, 20.0), (1.0, -0.3), (1.0, 0.0)])
@pytest.mark.parametrize("T", [1, 2, 12])
def test_scores_and_scales_that_differ(spread, scale, T):
    """References that move often: scores far apart, scales of V over many powers of two, either sign of scale."""
    c = Call("int8", "bf16", [T, T], [600, 90], 1, 8, 64, 16, [tree] * 2, seed=5, scale=scale, spread=spread)
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dtype,T,G", [("rows", "bf16", 5, 1), ("rows", "fp16", 3, 8), ("e4m3", "bf16", 2, 4), ("int8", "fp16", 4, 3),
                                           ("rows", "fp16", 40, 4), ("e4m3", "bf16", 70, 2), ("rows", "bf16", 12, 12), ("int8", "bf16", 90, 2)])
def test_no_finite_number_in_unseen_drafts(fmt, dtype, T, G):
    """NaN and infinities in keys and values of drafts reach the rows that see them and no others."""
    c = Call(fmt, dtype, [T, T], [21, 64], 2, G, 64, 16, [tree] * 2, seed=6)
    T16 = DT[dtype][0]
    for b, s in enumerate(c.starts):
        for d, value in ((1, math.nan), (T - 1, math.inf)):
            k, v = torch.ones(1, 2, 64), torch.ones(1, 2, 64)
            if d == 1:
                k[0, 0, 3] = value
            v[0, 1, 5] = value
            if b == 1:
                v[0, 1, 9] = -value
            c.cache.put(b, s + d, k.to(T16), v.to(T16))
    c.run()
    c.check()


@pytest.mark.gpu
def test_no_finite_number_in_codes():
    """8-bit NaN codes under a finite scale, and scales that are infinite, in drafts that some rows do not see."""
    for fmt in ("e4m3", "int8"):
        for T, G in ((4, 4), (40, 4)):
            c = Call(fmt, "bf16", [T], [30], 1, G, 64, 16, [tree], seed=7)
            (p1, s1), (p2, s2) = c.cache.spots(0, 31, 1), c.cache.spots(0, 30 + T - 1, 1)
            if fmt == "e4m3":
                c.cache.t["v"].view(torch.uint8)[int(p1[0]), 0, int(s1[0]), 17] = 0x7F
            c.cache.t["v_scale"][int(p2[0]), 0, int(s2[0])] = math.inf
            c.run()
            c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 6, 40])
def test_pages_that_do_not_exist(T):
    """Keys without a page are not seen; rows with no other key get zeros."""
    c = Call("e4m3", "bf16", [T, T, T], [100, 0, 40], 1, 8, 64, 16, [tree] * 3, seed=8)
    hidden = [(0, p) for p in range(16, 48)] + [(1, p) for p in range(T) if p < 16] + [(2, p) for p in range(16)]
    c.cache.d_table[0, 1], c.cache.d_table[0, 2], c.cache.d_table[1, 0], c.cache.d_table[2, 0] = -1, c.cache.pages, -7, 2 ** 31 - 1
    c.run()
    c.check(hidden)


@pytest.mark.gpu
def test_extreme_queries():
    """Rows of queries of very different size (bf16's range), zeros, and one with an infinity."""
    c = Call("int8", "bf16", [6], [50], 1, 2, 64, 16, None, seed=9, scale=0.125)
    sizes = torch.tensor([2.0 ** -120, 2.0 ** -60, 0.0, 1.0, 2.0 ** 8, 1.0])
    c.q.mul_(sizes.to(torch.bfloat16).cuda()[:, None])
    c.q[5, 3] = math.inf
    c.run()
    assert c.out[5, :64].isnan().all()
    c.q[5], c.out[5] = 0, 0
    width = c.heads * c.D
    c.out[5, :width] = 0
    out, lse = c.out[:5], c.lse[:5]
    c.counts, c.m = [5], 5
    c.masks = [np.tril(np.ones((5, 6), bool))]
    # the cache keeps six positions of drafts: the last is seen by the row that was left out alone
    c.check(out=out, lse=lse)


@pytest.mark.gpu
def test_masks_shorter_than_the_drafts():
    """Drafts beyond the mask's words are not seen."""
    sees = np.ones((40, 40), bool)
    c = Call("rows", "bf16", [40], [33], 1, 1, 64, 16, [sees], seed=10)
    c.mask = c.mask[:, :1].contiguous()
    c.masks = [np.concatenate([np.ones((40, 32), bool), np.zeros((40, 8), bool)], 1)]
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 24])
def test_in_place_and_without_lse(T):
    c = Call("e4m3", "bf16", [T, T], [900, 77], 2, 4, 64, 16, None, B.PROJ_GATE_SIGMOID, seed=11)
    c.run()
    c.check()
    q, gate = c.q.clone(), c.gate.clone()
    c.run(q=q, out=q, lse=None)
    assert torch.equal(q, c.out)
    c.run(gate=gate, out=gate, lse=None)
    assert torch.equal(gate, c.out)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 12])
def test_same_bits_and_two_streams(T):
    """Two calls at once with a workspace each, again and again: the same bits."""
    a = Call("e4m3", "bf16", [T] * 4, [3000, 10, 800, 0], 1, 8, 128, 64, [tree] * 4, seed=12)
    b = Call("rows", "fp16", [T] * 3, [100, 4000, 5], 2, 4, 64, 16, None, seed=13)
    a.run()
    b.run()
    torch.cuda.synchronize()
    want = [t.clone() for t in (a.out, a.lse, b.out, b.lse)]
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        for c in (a, b):
            c.out.fill_(GUARD)
            c.lse.fill_(GUARD)
            c.room.fill_(255)
        torch.cuda.synchronize()
        a.run(one)
        b.run(two)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, (a.out, a.lse, b.out, b.lse)))


@pytest.mark.gpu
def test_graphs_that_share_a_workspace():
    """Two captured calls, replayed in turn on one workspace, with lengths that change between replays."""
    a = Call("e4m3", "bf16", [4, 4], [2000, 300], 1, 8, 64, 64, None, seed=14)
    b = Call("e4m3", "bf16", [1, 1], [900, 1500], 1, 8, 64, 64, None, seed=15)
    room = torch.full((max(a.room.numel(), b.room.numel()),), 255, device="cuda", dtype=torch.uint8)
    side = torch.cuda.Stream()
    graphs = []
    for c in (a, b):
        with torch.cuda.stream(side):
            c.run(side, workspace=room, workspace_bytes=room.numel())
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            c.run(side, workspace=room, workspace_bytes=room.numel())
    for turn in range(3):
        for g, c in zip(graphs, (a, b)):
            c.out.fill_(GUARD)
            c.lse.fill_(GUARD)
            g.replay()
        torch.cuda.synchronize()
        a.check()
        b.check()
        # shorter contexts: what was behind them is now a draft's place
        for c in (a, b):
            c.starts = [max(0, s - 37) for s in c.starts]
            c.start.copy_(int32(c.starts))


@pytest.mark.gpu
def test_loop_of_verify_steps():
    """Write drafts, attend, accept a path, write the next: against attention over all that was accepted."""
    kv, G, D, T, page = 2, 4, 64, 6, 16
    rng, gen = np.random.default_rng(16), torch.Generator().manual_seed(16)
    first = [20, 0, 45]
    n = len(first)
    c = Cache("e4m3", "bf16", [s + 40 for s in first], kv, D, page, seed=16)
    held = [[] for _ in range(n)]  # values as the cache stands for them
    start, after = int32(first), int32([0] * n)
    for b, s in enumerate(first):
        x = torch.randn(s, kv, D, generator=gen).bfloat16()
        c.put(b, 0, x, -x)
    offsets = offsets_of([T] * n)
    m, width = n * T, (2 * G + 2) * kv * D
    room = torch.zeros(B.proj_attn_workspace(c.c, m, kv * G), device="cuda", dtype=torch.uint8)
    out, lse = torch.zeros(m, kv * G * D, device="cuda", dtype=torch.bfloat16), torch.zeros(m, kv * G, device="cuda")
    at = list(first)
    for step in range(4):
        row = torch.randn(m, width, generator=gen).bfloat16().cuda()  # q, k, v, gate side by side
        q, k, v, gate = torch.split(row, [kv * G * D, kv * D, kv * D, kv * G * D], 1)
        masks = [tree(T, rng) for _ in range(n)]
        mask = words_of(np.concatenate(masks))
        B.proj_kv_write(c.c, offsets, start, m, k, width, v, width)
        B.proj_attn(B.attn_args(c.c, m=m, heads=kv * G, q=q, ldq=width, offsets=offsets, start=start, mask=mask, ldm=1, words=1,
                                scale=0.125, gate=gate, ldg=width, gate_act=B.PROJ_GATE_SIGMOID, out=out, ldo=out.shape[1], lse=lse,
                                workspace=room, workspace_bytes=room.numel()))
        for b in range(n):
            rows = slice(b * T, (b + 1) * T)
            kk, vv = (c.get(i, b, 0, at[b] + T).numpy() for i in ("k", "v"))
            for i, old in enumerate(held[b]):  # what was accepted stands where it belongs
                assert np.array_equal(kk[first[b] + i], old)
            sees = np.concatenate([np.ones((T, at[b]), bool), masks[b]], 1)
            ref, ref_lse, mag, spread = attention(q[rows].reshape(T, kv * G, D).cpu().double().numpy(), kk, vv, sees, 0.125)
            x = 1 / (1 + np.exp(-gate[rows].reshape(T, kv * G, D).cpu().double().numpy()))
            d = ((D + 8) * 2.0 ** -23 + 2.0 ** -20) * spread
            bound = (np.expm1(2 * d)[..., None] + 2.0 ** -11 + 2.0 ** -16) * mag * x + 2.0 ** -8 * np.abs(ref * x) * (1 + 2.0 ** -8) + 2.0 ** -20
            got = out[rows].reshape(T, kv * G, D).cpu().double().numpy()
            assert (np.abs(got - ref * x) <= bound * 1.01).all()
            path = [i for i in range(T) if masks[b][T - 1, i]]
            held[b] += [kk[at[b] + i] for i in path]
        path = np.full((n, T), -1, np.int32)
        for b in range(n):
            p = np.flatnonzero(masks[b][T - 1])
            path[b, :len(p)] = p
        B.proj_kv_move(c.c, start, torch.from_numpy(path).cuda(), T, T, after)
        start, after = after, start
        at = [a + int((path[b] >= 0).sum()) for b, a in enumerate(at)]
        assert start.tolist() == at


def _args(**change):
    cache = B.kv_cache(format=B.PROJ_KV_E4M3, dtype=B.PROJ_BF16, pages=4, page=16, heads=2, D=64, k=1 << 20, v=1 << 21, k_scale=1 << 22,
                       v_scale=1 << 23, page_stride=2048, head_stride=1024, token_stride=64, table=1 << 24, ldt=3, width=3, sequences=2)
    f = dict(m=3, heads=4, q=1 << 20, ldq=256, offsets=16, start=16, mask=16, ldm=1, words=1, scale=1.0, gate_act=B.PROJ_GATE_SIGMOID,
             gate=1 << 21, ldg=256, out=1 << 22, ldo=256, lse=16, workspace=1 << 24, workspace_bytes=1 << 30)
    return B.attn_args(cache, **{**f, **change})


@pytest.mark.parametrize("change,status", [
    (dict(m=-1), B.PROJ_EINVAL), (dict(heads=3), B.PROJ_EINVAL), (dict(heads=0), B.PROJ_EINVAL), (dict(q=None), B.PROJ_EINVAL),
    (dict(out=None), B.PROJ_EINVAL), (dict(offsets=None), B.PROJ_EINVAL), (dict(start=None), B.PROJ_EINVAL), (dict(ldq=255), B.PROJ_EINVAL),
    (dict(ldo=248), B.PROJ_EINVAL), (dict(ldg=248), B.PROJ_EINVAL), (dict(words=0), B.PROJ_EINVAL), (dict(ldm=1, words=2), B.PROJ_EINVAL),
    (dict(scale=math.inf), B.PROJ_EINVAL), (dict(scale=math.nan), B.PROJ_EINVAL), (dict(gate_act=2), B.PROJ_EINVAL),
    (dict(out=1 << 20, ldo=264), B.PROJ_EINVAL), (dict(out=1 << 21, ldo=264), B.PROJ_EINVAL), (dict(workspace=None), B.PROJ_EINVAL),
    (dict(workspace_bytes=16), B.PROJ_EINVAL), (dict(heads=1026), B.PROJ_EUNSUPPORTED), (dict(m=(1 << 20) + 1), B.PROJ_EUNSUPPORTED),
    (dict(words=1025, ldm=1025), B.PROJ_EUNSUPPORTED), (dict(ldq=1 << 31), B.PROJ_EUNSUPPORTED), (dict(q=(1 << 20) + 8), B.PROJ_EALIGN),
    (dict(ldq=260), B.PROJ_EALIGN), (dict(out=(1 << 22) + 2), B.PROJ_EALIGN), (dict(gate=(1 << 21) + 8), B.PROJ_EALIGN),
    (dict(mask=18), B.PROJ_EALIGN), (dict(lse=18), B.PROJ_EALIGN), (dict(workspace=(1 << 24) + 8), B.PROJ_EALIGN), (dict(cache=None), B.PROJ_EINVAL),
])
def test_refused(lib, change, status):
    a = _args(**change) if "cache" not in change else _args()
    if "cache" in change:
        a.cache = None
    assert lib.proj_attn(ctypes.byref(a), None) == status
    assert B.last_cuda_error()


def test_nothing_to_do(lib):
    assert lib.proj_attn(None, None) == B.PROJ_EINVAL
    assert lib.proj_attn(ctypes.byref(_args(m=0, q=None, out=None, workspace=None)), None) == B.PROJ_OK
    assert lib.proj_attn_describe(None, 1, 1, None, 0) == B.PROJ_EINVAL
