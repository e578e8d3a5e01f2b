"""Rows of keys and values to the cache and back, and accepted drafts to their places, against plain definitions.

Codes and scales are defined step by step in fp32, and have to be those bits.  Against 64 bits: a code is off by at most
half a step (e4m3: 2^-4 of its size, or 2^-10 below 2^-6; int8: 1/2), and 4 2^-24 of x for the reciprocal, the product
and the scale's own rounding.  A value read back has one rounding of fp32 and one to its type.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B
from gemv_projection_layers_gb300 import build as libbuild

from kv_plain import DT, Cache, int32, offsets_of, quantise

GUARD = 7.0


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return B.load()


def rows(m, kv, D, dtype, seed, ld_more=0):
    """m rows [m, kv D] with ld_more columns behind each, and what they hold [m, kv, D]."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(m, kv * D + ld_more, generator=gen) * torch.exp(torch.randn(m, 1, generator=gen))
    x = x.to(DT[dtype][0]).cuda()
    return x, x[:, :kv * D].reshape(m, kv, D)


CASES = [
    # fmt, dtype, counts, starts, kv, D, page, layout, columns behind a row
    ("e4m3", "bf16", [1], [0], 1, 128, 64, "head", 0),
    ("e4m3", "fp16", [3, 0, 5, 1], [7, 3, 30, 0], 3, 64, 16, "head", 8),
    ("int8", "bf16", [2, 33, 1], [15, 0, 99], 2, 128, 1, "token", 0),
    ("int8", "fp16", [17, 40], [31, 200], 5, 64, 48, "token", 64),
    ("rows", "bf16", [9, 1, 0, 2], [1, 2, 3, 100], 8, 128, 100, "head", 0),
    ("rows", "fp16", [5], [1000], 1, 64, 7, "token", 16),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dtype,counts,starts,kv,D,page,layout,more", CASES)
def test_write_and_read(fmt, dtype, counts, starts, kv, D, page, layout, more):
    lens = [s + n for s, n in zip(starts, counts)]
    c = Cache(fmt, dtype, lens, kv, D, page, layout)
    want = Cache(fmt, dtype, lens, kv, D, page, layout)
    m = sum(counts) + 3  # the last three are no sequence's
    kr, k = rows(m, kv, D, dtype, 1, more)
    vr, v = rows(m, kv, D, dtype, 2, more)
    off, start = offsets_of(counts), int32(starts)
    B.proj_kv_write(c.c, off, start, m, kr, kr.stride(0), vr, vr.stride(0))
    at = 0
    for b, n in enumerate(counts):
        want.put(b, starts[b], k[at:at + n].cpu(), v[at:at + n].cpu())
        at += n
    got, exp = c.raw(), want.raw()
    for n in got:
        assert torch.equal(got[n], exp[n]), n
    out = [torch.full((m, kv * D + more), GUARD, device="cuda", dtype=DT[dtype][0]) for _ in range(2)]
    B.proj_kv_read(c.c, off, start, m, out[0], kv * D + more, out[1], kv * D + more)
    u = DT[dtype][2]
    at = 0
    for b, n in enumerate(counts):
        for name, o, x in (("k", out[0], k), ("v", out[1], v)):
            o = o[at:at + n, :kv * D].reshape(n, kv, D).cpu().double()
            ref = c.get(name, b, starts[b], n)
            if fmt == "rows":
                assert torch.equal(o, ref)
                continue
            assert bool(((o - ref).abs() <= (u + 2.0 ** -24) * ref.abs() + 2.0 ** -25).all())
            x = x[at:at + n].cpu().double()
            s = x.abs().amax(-1, keepdim=True) / (448.0 if fmt == "e4m3" else 127.0)
            half = torch.maximum(x.abs() * 2.0 ** -4, s * 2.0 ** -10) if fmt == "e4m3" else s / 2
            assert bool(((ref - x).abs() <= half * (1 + 2.0 ** -20) + 4 * 2.0 ** -24 * x.abs()).all())
        at += n
    for o in out:  # rows of no sequence, and what stands behind a row
        assert bool((o[at:] == GUARD).all()) and bool((o[:, kv * D:] == GUARD).all())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_write_of_extremes(fmt, dtype):
    """Zeros, the smallest and largest numbers, values on borders, NaN and infinities."""
    D, T = 64, DT[dtype][0]
    x = torch.zeros(8, D)
    x[1, 3] = 2.0 ** -133 if dtype == "bf16" else 2.0 ** -24
    x[2] = float(torch.finfo(T).max) * torch.linspace(-1, 1, D)
    x[3] = torch.arange(D) * 14.0 - 448.0  # steps and halves of steps of both formats
    x[4], x[4, 7] = 1.0, math.nan
    x[5], x[5, 9] = 2.0, math.inf
    x[6], x[6, 60] = -3.0, -math.inf
    x[7] = -1e-30 * torch.arange(D) if dtype == "bf16" else -2.0 ** -20 * torch.arange(D)
    x = x.to(T)
    c, want = Cache(fmt, dtype, [8], 1, D, 16), Cache(fmt, dtype, [8], 1, D, 16)
    d = x.cuda()
    B.proj_kv_write(c.c, offsets_of([8]), int32([0]), 8, d, D, d, D)
    want.put(0, 0, x[:, None], x[:, None])
    for n, t in c.raw().items():
        if n in ("k", "v"):
            assert torch.equal(t, want.raw()[n]), n
    for n in ("k_scale", "v_scale"):
        assert torch.equal(c.t[n].nan_to_num(nan=-1.0), want.t[n].nan_to_num(nan=-1.0))
    out = torch.zeros(8, D, device="cuda", dtype=T)
    B.proj_kv_read(c.c, offsets_of([8]), int32([0]), 8, out, D, None, 0)
    assert out[4:7].isnan().all() and out[:4].isfinite().all() and out[7].isfinite().all()
    assert bool((out[0] == 0).all())


@pytest.mark.gpu
def test_places_without_a_page():
    """Positions beyond the table, before 0, or of pages that do not exist: not written, read as zeros."""
    c = Cache("e4m3", "bf16", [40, 40], 2, 64, 16)
    c.d_table[0, 1] = c.pages       # positions 16 .. 31
    c.d_table[1, 0] = -5            # positions 0 .. 15
    before = c.raw()
    kr, _ = rows(8, 2, 64, "bf16", 3)
    last = c.width * 16
    for off, start in (([0, 4, 8], [18, 5]), ([0, 4, 8], [last, -4]), ([0, 4, 8], [2 ** 31 - 3, -2 ** 31])):
        B.proj_kv_write(c.c, int32(off), int32(start), 8, kr, 128, kr, 128)
        assert all(torch.equal(t, before[n]) for n, t in c.raw().items())
        out = torch.full((8, 128), GUARD, device="cuda", dtype=torch.bfloat16)
        B.proj_kv_read(c.c, int32(off), int32(start), 8, out, 128, None, 0)
        assert bool((out == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("off", [[-5, 4, 400], [3, 2, 9], [8, 8, 8], [0, 0, 8], [2, 4, 6]])
def test_offsets_out_of_range(off):
    """Offsets beyond 0 .. m or decreasing: rows of no sequence are left, and nothing beside the sequences' pages is written."""
    c = Cache("int8", "fp16", [64, 64], 1, 64, 16, spare=8)
    kr, _ = rows(8, 1, 64, "fp16", 4)
    B.proj_kv_write(c.c, int32(off), int32([0, 0]), 8, kr, 64, kr, 64)
    mine = set(c.table[c.table >= 0].tolist())
    for p in range(c.pages):
        if p not in mine:
            assert c.t["k_scale"][p].isnan().all()
    out = torch.full((8, 64), GUARD, device="cuda", dtype=torch.float16)
    B.proj_kv_read(c.c, int32(off), int32([0, 0]), 8, out, 64, out.clone(), 64)
    for r in range(8):
        owned = any(max(off[b], 0) <= r < off[b + 1] for b in range(2))
        if off == sorted(off):
            assert bool((out[r] == GUARD).all()) == (not owned)


@pytest.mark.gpu
def test_many_sequences():
    """More sequences than a step of the search sees, some without rows."""
    n = 1500
    counts = [(7 * b) % 3 for b in range(n)]
    starts = [b % 5 for b in range(n)]
    c = Cache("int8", "bf16", [s + k for s, k in zip(starts, counts)], 1, 64, 4)
    m = sum(counts)
    kr, k = rows(m, 1, 64, "bf16", 5)
    B.proj_kv_write(c.c, offsets_of(counts), int32(starts), m, kr, 64, kr, 64)
    code, scale = quantise(k, "int8")
    at = 0
    host, host_scale = c.t["k"].cpu(), c.t["k_scale"].cpu()
    for b in range(n):
        page, spot = c.spots(b, starts[b], counts[b])
        assert torch.equal(host[page, :, spot], code[at:at + counts[b]])
        assert torch.equal(host_scale[page, :, spot], scale[at:at + counts[b]])
        at += counts[b]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dtype,kv,D,page,layout", [("e4m3", "bf16", 1, 128, 64, "head"), ("int8", "fp16", 3, 64, 5, "token"),
                                                        ("rows", "fp16", 8, 128, 16, "head")])
def test_move(fmt, dtype, kv, D, page, layout):
    paths = [[0, 1, 2, -1], [1, 3, 8, 30, 31], [], [5], [2, 2, 3], [0, 2, 1, 4], list(range(0, 40, 2)), [-1, 3]]
    kept = [3, 5, 0, 1, 1, 2, 20, 0]
    starts = [0, 6, 3, 14, 2, 9, 31, 4]
    depth = 21
    lens = [s + 40 for s in starts]
    c, want = Cache(fmt, dtype, lens, kv, D, page, layout), Cache(fmt, dtype, lens, kv, D, page, layout)
    for b, n in enumerate(lens):
        x = torch.randn(n, kv, D, generator=c.gen).to(DT[dtype][0])
        c.put(b, 0, x, x * 2)
        want.put(b, 0, x, x * 2)
    raw = want.t
    for b, p in enumerate(paths):
        old = {n: t.clone() for n, t in raw.items()}
        for i, f in enumerate(p[:kept[b]]):
            (fp, fs), (tp, ts) = want.spots(b, starts[b] + f, 1), want.spots(b, starts[b] + i, 1)
            for n, t in raw.items():
                t[tp[0], :, ts[0]] = old[n][fp[0], :, fs[0]]
    table = torch.full((len(paths), depth + 2), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        table[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    table[:, depth:] = 3  # behind a path's depth: not looked at
    after = torch.zeros(len(paths), dtype=torch.int32, device="cuda")
    B.proj_kv_move(c.c, int32(starts), table.cuda(), depth + 2, depth, after)
    assert after.tolist() == [s + k for s, k in zip(starts, kept)]
    got, exp = c.raw(), want.raw()
    for n in got:
        assert torch.equal(got[n], exp[n]), n


@pytest.mark.gpu
def test_move_without_pages():
    """Entries whose source or target has no page stay; the others move."""
    c = Cache("e4m3", "bf16", [64], 1, 64, 16)
    x = torch.randn(64, 1, 64)
    c.put(0, 0, x, x)
    c.d_table[0, 1] = -1
    before = c.raw()
    after = torch.zeros(1, dtype=torch.int32, device="cuda")
    # sources 17 (no page), 33, 2^30 (beyond the table); targets 15, 16 (no page), 17 (no page)
    B.proj_kv_move(c.c, int32([15]), int32([[2, 18, 2 ** 30]]), 3, 3, after)
    assert after.item() == 18
    assert all(torch.equal(t, before[n]) for n, t in c.raw().items())
    B.proj_kv_move(c.c, int32([14]), int32([[2 ** 31 - 1]]), 1, 1, after)
    assert after.item() == 15
    assert all(torch.equal(t, before[n]) for n, t in c.raw().items())


def _fields(**change):
    """A valid cache's fields with made-up addresses: for calls that are refused, or have nothing to do."""
    f = dict(format=B.PROJ_KV_E4M3, dtype=B.PROJ_BF16, pages=4, page=16, heads=2, D=64, k=1 << 20, v=1 << 21, k_scale=1 << 22, v_scale=1 << 23,
             page_stride=2048, head_stride=1024, token_stride=64, table=1 << 24, ldt=3, width=3, sequences=2)
    return B.kv_cache(**{**f, **change})


REFUSED = [
    (dict(format=3), B.PROJ_EINVAL), (dict(dtype=B.PROJ_FP32), B.PROJ_EINVAL), (dict(pages=0), B.PROJ_EINVAL), (dict(page=0), B.PROJ_EINVAL),
    (dict(heads=0), B.PROJ_EINVAL), (dict(width=0, ldt=0), B.PROJ_EINVAL), (dict(sequences=-1), B.PROJ_EINVAL), (dict(ldt=2), B.PROJ_EINVAL),
    (dict(k=None), B.PROJ_EINVAL), (dict(v=None), B.PROJ_EINVAL), (dict(table=None), B.PROJ_EINVAL), (dict(k_scale=None), B.PROJ_EINVAL),
    (dict(format=B.PROJ_KV_ROWS), B.PROJ_EINVAL), (dict(token_stride=63), B.PROJ_EINVAL), (dict(D=80, token_stride=80), B.PROJ_EUNSUPPORTED),
    (dict(heads=1025), B.PROJ_EUNSUPPORTED), (dict(page=65537), B.PROJ_EUNSUPPORTED), (dict(pages=1 << 31), B.PROJ_EUNSUPPORTED),
    (dict(sequences=65537), B.PROJ_EUNSUPPORTED), (dict(width=1 << 26, ldt=1 << 26), B.PROJ_EUNSUPPORTED), (dict(k=(1 << 20) + 8), B.PROJ_EALIGN),
    (dict(token_stride=72), B.PROJ_EALIGN), (dict(k_scale=(1 << 22) + 2), B.PROJ_EALIGN), (dict(table=(1 << 24) + 1), B.PROJ_EALIGN),
]


@pytest.mark.parametrize("change,status", REFUSED)
def test_caches_refused(lib, change, status):
    import ctypes
    c = ctypes.byref(_fields(**change))
    assert lib.proj_kv_write(c, 16, 16, 1, 16, 128, 16, 128, None) == status
    assert lib.proj_kv_read(c, 16, 16, 1, 16, 128, 16, 128, None) == status
    assert lib.proj_kv_move(c, 16, 16, 1, 1, None, None) == status
    assert lib.proj_attn_workspace(c, 1, 2) == -1 and B.proj_last_status() == status
    assert B.last_cuda_error()


def test_calls_refused(lib):
    import ctypes
    c = ctypes.byref(_fields())
    for call in (lib.proj_kv_write, lib.proj_kv_read):
        assert call(None, 16, 16, 1, 16, 128, 16, 128, None) == B.PROJ_EINVAL
        assert call(c, 16, 16, -1, 16, 128, 16, 128, None) == B.PROJ_EINVAL
        assert call(c, None, 16, 1, 16, 128, 16, 128, None) == B.PROJ_EINVAL
        assert call(c, 16, None, 1, 16, 128, 16, 128, None) == B.PROJ_EINVAL
        assert call(c, 16, 16, 1, None, 128, None, 128, None) == B.PROJ_EINVAL
        assert call(c, 16, 16, 1, 16, 127, 16, 128, None) == B.PROJ_EINVAL
        assert call(c, 16, 16, 1, 16, 128, 16, 120, None) == B.PROJ_EINVAL
        assert call(c, 16, 16, 1 << 30, 16, 128, 16, 128, None) == B.PROJ_EUNSUPPORTED
        assert call(c, 16, 16, 1, 16, 1 << 31, 16, 128, None) == B.PROJ_EUNSUPPORTED
        assert call(c, 16, 16, 1, 8, 128, 16, 128, None) == B.PROJ_EALIGN
        assert call(c, 16, 16, 1, 16, 132, 16, 128, None) == B.PROJ_EALIGN
        assert call(c, 18, 16, 1, 16, 128, 16, 128, None) == B.PROJ_EALIGN
        assert call(c, None, None, 0, None, 128, None, 128, None) == B.PROJ_OK
    assert lib.proj_kv_write(c, 16, 16, 1, 16, 128, None, 128, None) == B.PROJ_EINVAL
    assert lib.proj_kv_move(c, None, 16, 4, 4, None, None) == B.PROJ_EINVAL
    assert lib.proj_kv_move(c, 16, None, 4, 4, None, None) == B.PROJ_EINVAL
    assert lib.proj_kv_move(c, 16, 16, 3, 4, None, None) == B.PROJ_EINVAL
    assert lib.proj_kv_move(c, 16, 32, 4, -1, None, None) == B.PROJ_EINVAL
    assert lib.proj_kv_move(c, 16, 32, 4, 4, 16, None) == B.PROJ_EINVAL
    assert lib.proj_kv_move(c, 16, 34, 4, 4, None, None) == B.PROJ_EALIGN
    assert lib.proj_kv_move(c, 16, 32, 1 << 31, 4, None, None) == B.PROJ_EUNSUPPORTED
    assert lib.proj_kv_move(c, 16, None, 0, 0, None, None) == B.PROJ_OK
    none = ctypes.byref(_fields(sequences=0, table=None))
    assert lib.proj_kv_write(none, None, None, 4, 16, 128, 16, 128, None) == B.PROJ_OK
    assert lib.proj_kv_move(none, None, None, 4, 4, None, None) == B.PROJ_OK
