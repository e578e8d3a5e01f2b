"""Tokens to their experts and back against plain definitions: whole numbers exactly, weights and
rows within bounds from the arithmetic.

weight:  64 2^-24 of its size (exp and the quotient within a few units, a sum of at most 1024 terms
         in a tree whose leaves add up at most 32), and 2^-149, the spacing of fp32 below its
         normal range (likewise 2^-146 for dlogits, a few such roundings).
combine: u |ref| + (k + 2) 2^-24 sum |w y|;  dys: u |ref| + 2^-24 |ref|.
dweight: (D / 128 + 32) 2^-24 sum |dout y|: at most D / 256 terms a thread, then a tree.
dlogits: 128 2^-24 of p (|dw| + sum |w dw|), for the same reasons as the weights.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B
from gemv_projection_layers_gb300 import build as libbuild

DT = {"bf16": (torch.bfloat16, B.PROJ_BF16, 2.0 ** -8), "fp16": (torch.float16, B.PROJ_FP16, 2.0 ** -11),
      "fp32": (torch.float32, B.PROJ_FP32, 2.0 ** -24)}
INF, LOWEST = math.inf, float(np.finfo(np.float32).min)


def choose64(logits, k, mode):
    """One row at a time: sort by (-value, index) what may be chosen."""
    lg = logits.astype(np.float64)
    m = lg.shape[0]
    expert = np.full((m, k), -1, np.int64)
    weight = np.zeros((m, k))
    prob = np.zeros(lg.shape)
    for t in range(m):
        can = [e for e in range(lg.shape[1]) if lg[t, e] > -INF]  # false for NaN too
        if not can:
            continue
        top = max(lg[t, e] for e in can)
        part = {e: 1.0 if lg[t, e] == top else math.exp(lg[t, e] - top) for e in can}
        pick = sorted(can, key=lambda e: (-lg[t, e], e))[:k]
        all_ = sum(part.values())
        for e in can:
            prob[t, e] = part[e] / all_
        total = all_ if mode == B.PROJ_ROUTE_ALL else sum(part[e] for e in pick)
        expert[t, :len(pick)] = pick
        weight[t, :len(pick)] = [part[e] / total for e in pick]
    return expert, weight, prob


def sort64(expert, E):
    flat = expert.reshape(-1)
    order = [i for e in range(E) for i in np.flatnonzero(flat == e)]
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    slot = np.full(flat.shape, -1, np.int64)
    slot[order] = np.arange(len(order))
    full = np.full(flat.shape, -1, np.int64)
    full[:len(order)] = order
    return offsets, full, slot.reshape(expert.shape)


def make_logits(m, E, kind, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, E)).astype(np.float32) * 2
    if kind == "ties":
        x = np.round(x)
        x[::2] = np.where(x[::2] == 0, np.float32(-0.0), x[::2])  # both zeros are one value
    elif kind == "masked":
        x[:, rng.random(E) < 0.4] = -INF
        x[rng.random((m, E)) < 0.1] = np.nan
        x[::5] = -INF
        x[1::5, 1:] = -INF
    elif kind == "lowest":
        x[rng.random((m, E)) < 0.7] = LOWEST
        x[::3] = LOWEST
    elif kind == "infinite":
        x[rng.random((m, E)) < 0.2] = INF
        x[rng.random((m, E)) < 0.2] = -LOWEST
    elif kind == "one":
        x[:, E // 2] = 100.0
    return x


def run_route(logits, k, mode, ld_extra=0, sort=True):
    m, E = logits.shape
    buf = torch.full((max(m, 1), E + ld_extra), float("nan"), device="cuda")
    buf[:m, :E] = torch.from_numpy(logits).cuda()
    new = lambda *s: torch.full(s, -99, device="cuda", dtype=torch.int32)  # noqa: E731
    expert, weight = new(m, k), torch.full((m, k), -99.0, device="cuda")
    room = torch.empty(max(16, B.proj_moe_workspace(m, E, k)), dtype=torch.uint8, device="cuda")
    if sort:
        offsets, order, slot = new(E + 2), new(m * k + 1), new(m, k)
        B.proj_moe_route(buf, E + ld_extra, m, E, k, mode, expert, weight, offsets, order, slot, room, room.numel())
        torch.cuda.synchronize()
        assert offsets[-1] == -99 and order[-1] == -99
        return expert, weight, offsets[:-1], order[:-1], slot
    B.proj_moe_route(buf, E + ld_extra, m, E, k, mode, expert, weight)
    torch.cuda.synchronize()
    return expert, weight


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [B.PROJ_ROUTE_CHOSEN, B.PROJ_ROUTE_ALL])
@pytest.mark.parametrize("kind", ["plain", "ties", "masked", "lowest", "infinite", "one"])
@pytest.mark.parametrize("m,E,k", [(1, 1, 1), (1, 256, 8), (3, 7, 7), (64, 60, 4), (65, 64, 6), (130, 257, 3), (333, 128, 8),
                                   (97, 1024, 32), (700, 8, 2)])
def test_route(m, E, k, kind, mode):
    logits = make_logits(m, E, kind, m + E)
    expert, weight, offsets, order, slot = run_route(logits, k, mode, ld_extra=m % 2)
    e64, w64, _ = choose64(logits, k, mode)
    assert np.array_equal(expert.cpu().numpy(), e64)
    err = np.abs(weight.cpu().numpy() - w64)
    assert (err <= 64 * 2.0 ** -24 * w64 + 2.0 ** -149).all(), err.max()
    o64, r64, s64 = sort64(e64, E)
    assert np.array_equal(offsets.cpu().numpy(), o64)
    assert np.array_equal(order.cpu().numpy(), r64)
    assert np.array_equal(slot.cpu().numpy(), s64)
    only = run_route(logits, k, mode, sort=False)
    assert torch.equal(only[0], expert) and torch.equal(only[1], weight)


@pytest.mark.gpu
@pytest.mark.parametrize("m,E,k", [(1, 1, 1), (20, 4, 3), (5000, 256, 8), (20000, 32, 2), (40000, 1, 1), (3000, 1024, 32)])
def test_sort_of_given_choices(m, E, k):
    rng = np.random.default_rng(m)
    ids = rng.integers(-1, E, (m, k)).astype(np.int32)
    ids[rng.random((m, k)) < 0.02] = E + 5  # not an expert
    ids[rng.random((m, k)) < 0.02] = -(2 ** 31)
    d = torch.from_numpy(ids).cuda()
    new = lambda *s: torch.full(s, -99, device="cuda", dtype=torch.int32)  # noqa: E731
    room = torch.empty(max(16, B.proj_moe_workspace(m, E, k)), dtype=torch.uint8, device="cuda")
    got = [new(E + 1), new(m * k), new(m, k)]
    B.proj_moe_sort(d, m, E, k, *got, room, room.numel())
    torch.cuda.synchronize()
    flat = np.where((ids >= 0) & (ids < E), ids, E).reshape(-1)
    ranked = np.argsort(flat, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E + 1)[:E])])
    order = ranked.copy()
    order[offsets[-1]:] = -1
    slot = np.empty(m * k, np.int64)
    slot[ranked] = np.arange(m * k)
    slot[flat == E] = -1
    assert np.array_equal(got[0].cpu().numpy(), offsets)
    assert np.array_equal(got[1].cpu().numpy(), order)
    assert np.array_equal(got[2].cpu().numpy().reshape(-1), slot)


def plan(m, E, k, seed, drop=0.2):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(m)]).astype(np.int32)
    ids[rng.random((m, k)) < drop] = -1
    if m > 1:
        ids[0] = -1  # a token that goes nowhere
    _, _, slot = sort64(ids, E)
    w = rng.random((m, k)).astype(np.float32)
    return (torch.from_numpy(slot.astype(np.int32)).cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(slot).cuda())


def rows(n, D, dtype, seed, ld):
    gen = torch.Generator("cuda").manual_seed(seed)
    buf = torch.full((n + 1, ld), float("nan"), device="cuda", dtype=DT[dtype][0])
    buf[:n, :D] = torch.randn(n, D, device="cuda", generator=gen).to(buf.dtype)
    return buf


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,E,k,D,extra", [(1, 8, 8, 8192, 0), (1, 1, 1, 1, 0), (5, 16, 3, 7, 1), (33, 32, 9, 264, 8), (40, 60, 20, 1000, 0),
                                           (7, 256, 32, 4100, 0), (100, 8, 2, 2048, 3)])
def test_gather_and_combine_and_gradients(m, E, k, D, extra, dtype):
    t, kind, u = DT[dtype]
    slot, w, s64 = plan(m, E, k, m + D)
    ld, n = D + extra, m * k
    valid = s64 >= 0
    # gather
    x = rows(m, D, dtype, 1, ld)
    xs = torch.full((n, ld), -7.0, device="cuda", dtype=t)
    B.proj_moe_gather(x, ld, slot, m, D, k, kind, xs, ld)
    torch.cuda.synchronize()
    want = torch.full_like(xs, -7.0)
    want[s64[valid], :D] = x[:m, :D].unsqueeze(1).expand(m, k, D)[valid]
    assert torch.equal(xs, want)
    # combine; rows of ys that no entry names are NaN and never read
    ys = rows(n, D, dtype, 2, ld)
    named = torch.zeros(n, dtype=torch.bool, device="cuda")
    named[s64[valid]] = True
    ys[:n][~named] = float("nan")
    y64 = torch.where(valid[..., None], ys[:n, :D].double()[s64.clamp(min=0)], torch.zeros((), device="cuda", dtype=torch.float64))
    for weight, w64 in ((w, w.double()), (None, torch.ones_like(w, dtype=torch.float64))):
        out = torch.full((m + 1, ld), -7.0, device="cuda", dtype=t)
        B.proj_moe_combine(ys, ld, slot, weight, m, D, k, kind, out, ld)
        torch.cuda.synchronize()
        ref = (w64[..., None] * y64).sum(1)
        tol = u * ref.abs() + (k + 2) * 2.0 ** -24 * (w64[..., None] * y64).abs().sum(1) + (2.0 ** -25 if dtype == "fp16" else 0)
        assert ((out[:m, :D].double() - ref).abs() <= tol).all()
        assert (out[m:] == -7.0).all() and (out[:, D:] == -7.0).all()
    # gradient of combine
    dout = rows(m, D, dtype, 3, ld)
    dys = torch.full((n, ld), -7.0, device="cuda", dtype=t)
    dw = torch.full((m, k), -7.0, device="cuda")
    B.proj_moe_combine_backward(dout, ld, ys, ld, slot, w, m, D, k, kind, dys, ld, dw)
    torch.cuda.synchronize()
    d64 = dout[:m, :D].double()
    ref = w.double()[..., None] * d64[:, None, :]
    want = torch.full((n, D), -7.0, device="cuda", dtype=torch.float64)
    want[s64[valid]] = ref[valid]
    assert ((dys[:, :D].double() - want).abs() <= (u + 2.0 ** -24) * want.abs() + (2.0 ** -25 if dtype == "fp16" else 0)).all()
    assert (dys[~named] == -7.0).all() and (dys[:, D:] == -7.0).all()
    S = (d64[:, None, :] * y64).abs().sum(-1)
    assert ((dw.double() - (d64[:, None, :] * y64).sum(-1)).abs() <= (D / 128 + 32) * 2.0 ** -24 * S).all()
    # either half alone gives the same
    dys2, dw2 = torch.full_like(dys, -7.0), torch.full_like(dw, -7.0)
    B.proj_moe_combine_backward(dout, ld, None, 0, slot, w, m, D, k, kind, dys2, ld, None)
    B.proj_moe_combine_backward(dout, ld, ys, ld, slot, w, m, D, k, kind, None, 0, dw2)
    torch.cuda.synchronize()
    assert torch.equal(dys2, dys) and torch.equal(dw2, dw)


@pytest.mark.gpu
def test_slots_out_of_range_are_skipped():
    m, k, D = 4, 2, 64
    x = torch.randn(m, D, device="cuda")
    slot = torch.tensor([[0, 8], [-1, 3], [2 ** 31 - 1, -(2 ** 31)], [5, 7]], dtype=torch.int32, device="cuda")
    xs = torch.zeros(m * k + 2, D, device="cuda")
    B.proj_moe_gather(x, D, slot, m, D, k, B.PROJ_FP32, xs, D)
    out = torch.full((m, D), -7.0, device="cuda")
    B.proj_moe_combine(xs, D, slot, None, m, D, k, B.PROJ_FP32, out, D)
    torch.cuda.synchronize()
    want = torch.zeros_like(xs)
    want[0], want[3], want[5], want[7] = x[0], x[1], x[3], x[3]
    assert torch.equal(xs, want)
    assert torch.equal(out, torch.stack([x[0], x[1], torch.zeros_like(x[0]), x[3] * 2]))


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [B.PROJ_ROUTE_CHOSEN, B.PROJ_ROUTE_ALL])
@pytest.mark.parametrize("kind", ["plain", "masked", "lowest"])
@pytest.mark.parametrize("m,E,k", [(1, 8, 2), (70, 60, 4), (33, 256, 8), (9, 1000, 32), (10, 5, 5)])
def test_route_gradient(m, E, k, kind, mode):
    logits = make_logits(m, E, kind, m + k)
    expert, weight = run_route(logits, k, mode, sort=False)
    e64, w64, p64 = choose64(logits, k, mode)
    rng = np.random.default_rng(1)
    dw = rng.standard_normal((m, k)).astype(np.float32)
    dl = torch.full((m, E + 1), -7.0, device="cuda")
    lg = torch.from_numpy(logits).cuda()
    B.proj_moe_route_backward(lg, E, m, E, k, mode, expert, weight, torch.from_numpy(dw).cuda(), dl, E + 1)
    torch.cuda.synchronize()
    assert (dl[:, E] == -7.0).all()
    got = dl[:, :E].double().cpu().numpy()
    d64 = np.where(e64 >= 0, dw.astype(np.float64), 0.0)
    inner, size = (w64 * d64).sum(1), np.abs(w64 * d64).sum(1)
    ref, tol = np.zeros((m, E)), np.zeros((m, E))
    if mode == B.PROJ_ROUTE_ALL:
        ref, tol = -p64 * inner[:, None], p64 * size[:, None]
    for t in range(m):
        for j in range(k):
            e = e64[t, j]
            if e < 0:
                continue
            if mode == B.PROJ_ROUTE_ALL:
                ref[t, e] += p64[t, e] * d64[t, j]
                tol[t, e] += p64[t, e] * abs(d64[t, j])
            else:
                ref[t, e] = w64[t, j] * (d64[t, j] - inner[t])
                tol[t, e] = w64[t, j] * (abs(d64[t, j]) + size[t])
    assert (np.abs(got - ref) <= 128 * 2.0 ** -24 * tol + 2.0 ** -146).all()
    if kind != "plain" or E == k:
        return
    # Differences of the definition, the choice held fixed (steps too small to change it).
    v = rng.standard_normal((m, E))
    h = 1e-6

    def loss(x):
        x = x - x.max(1, keepdims=True)
        full = np.exp(x)
        part = np.take_along_axis(full, e64, 1)
        total = full.sum(1, keepdims=True) if mode == B.PROJ_ROUTE_ALL else part.sum(1, keepdims=True)
        return (part / total * dw).sum()

    x = logits.astype(np.float64)
    diff = (loss(x + h * v) - loss(x - h * v)) / (2 * h)
    # truncation h^2, rounding 2^-52 / h of the loss's terms, and the gradient's own bound
    bound = np.abs(128 * 2.0 ** -24 * tol * v).sum() + (1e-9 + 1e-11) * m * (1 + np.abs(v).max() ** 3) * k
    assert abs((got * v).sum() - diff) <= bound


@pytest.mark.gpu
def test_nothing_to_do():
    off = torch.full((5,), -9, device="cuda", dtype=torch.int32)
    lib = B.load()
    assert lib.proj_moe_route(None, 4, 0, 4, 2, 0, None, None, off.data_ptr(), off.data_ptr(), off.data_ptr(), None, 0, None) == B.PROJ_OK
    torch.cuda.synchronize()
    assert (off == 0).all()
    assert lib.proj_moe_gather(None, 8, None, 0, 8, 2, B.PROJ_BF16, None, 8, None) == B.PROJ_OK
    assert lib.proj_moe_combine(None, 8, None, None, 0, 8, 2, B.PROJ_BF16, None, 8, None) == B.PROJ_OK


def test_refusals_before_any_device_call():
    libbuild.build()
    lib = B.load()

    def route(logits=16, ldl=8, m=4, E=8, k=2, mode=0, expert=16, weight=16, offsets=16, order=16, slot=16, ws=None, wb=0):
        return lib.proj_moe_route(logits, ldl, m, E, k, mode, expert, weight, offsets, order, slot, ws, wb, None)

    assert route(logits=None) == B.PROJ_EINVAL
    assert route(expert=None) == B.PROJ_EINVAL
    assert route(weight=None) == B.PROJ_EINVAL
    assert route(offsets=None) == B.PROJ_EINVAL
    assert route(slot=None) == B.PROJ_EINVAL
    assert route(ldl=7) == B.PROJ_EINVAL
    assert route(m=-1) == B.PROJ_EINVAL
    assert route(k=0) == B.PROJ_EINVAL
    assert route(k=9) == B.PROJ_EINVAL
    assert route(mode=2) == B.PROJ_EINVAL
    assert route(E=1025, ldl=1025) == B.PROJ_EUNSUPPORTED
    assert route(E=64, ldl=64, k=33) == B.PROJ_EUNSUPPORTED
    assert route(m=2 ** 30) == B.PROJ_EUNSUPPORTED
    assert route(logits=18) == B.PROJ_EALIGN
    assert route(m=100000, ws=None) == B.PROJ_EINVAL  # wants a workspace
    assert route(m=100000, ws=16, wb=16) == B.PROJ_EINVAL
    assert route(m=100000, ws=8, wb=1 << 30) == B.PROJ_EALIGN
    assert lib.proj_moe_workspace(-1, 8, 2) == -1
    assert lib.proj_moe_workspace(1, 8, 2) == 0
    assert lib.proj_moe_workspace(100000, 8, 2) > 0
    assert lib.proj_moe_sort(None, 4, 8, 2, 16, 16, 16, None, 0, None) == B.PROJ_EINVAL
    assert lib.proj_moe_sort(16, 4, 8, 2, None, 16, 16, None, 0, None) == B.PROJ_EINVAL
    assert lib.proj_moe_sort(16, 4, 8, 2, 16, 18, 16, None, 0, None) == B.PROJ_EALIGN

    def rows(fn, a=16, lda=8, slot=16, m=4, D=8, k=2, dtype=0, out=16, ldo=8):
        mid = (None,) if fn is lib.proj_moe_combine else ()
        return fn(a, lda, slot, *mid, m, D, k, dtype, out, ldo, None)

    for fn in (lib.proj_moe_gather, lib.proj_moe_combine):
        assert rows(fn, a=None) == B.PROJ_EINVAL
        assert rows(fn, slot=None) == B.PROJ_EINVAL
        assert rows(fn, out=None) == B.PROJ_EINVAL
        assert rows(fn, lda=7) == B.PROJ_EINVAL
        assert rows(fn, ldo=7) == B.PROJ_EINVAL
        assert rows(fn, D=0) == B.PROJ_EINVAL
        assert rows(fn, k=0) == B.PROJ_EINVAL
        assert rows(fn, dtype=3) == B.PROJ_EINVAL
        assert rows(fn, k=33) == B.PROJ_EUNSUPPORTED
        assert rows(fn, m=2 ** 31) == B.PROJ_EUNSUPPORTED
        assert rows(fn, a=17) == B.PROJ_EALIGN
        assert rows(fn, slot=18) == B.PROJ_EALIGN
    grad = lambda ys=16, dys=16, dw=16: lib.proj_moe_combine_backward(16, 8, ys, 8, 16, None, 4, 8, 2, 0, dys, 8, dw, None)  # noqa: E731
    assert grad(dys=None, dw=None) == B.PROJ_EINVAL
    assert grad(ys=None) == B.PROJ_EINVAL
    assert grad(dw=18) == B.PROJ_EALIGN
    back = lambda mode=0, logits=16, dl=16, lddl=8: lib.proj_moe_route_backward(logits, 8, 4, 8, 2, mode, 16, 16, 16, dl, lddl, None)  # noqa: E731
    assert back(dl=None) == B.PROJ_EINVAL
    assert back(mode=1, logits=None) == B.PROJ_EINVAL
    assert back(mode=3) == B.PROJ_EINVAL
    assert back(lddl=7) == B.PROJ_EINVAL
    assert back(dl=18) == B.PROJ_EALIGN
    with pytest.raises(B.ProjError):
        B.proj_moe_gather(None, 8, None, 1, 8, 2, 0, None, 8)
