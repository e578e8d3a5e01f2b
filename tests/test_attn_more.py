"""More of the attention over the cache: rows around the kernels' tiles, references that move, long caches, calls with
offsets and starts that are out of range.  Bounds as in test_attn.py."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B
from gemv_projection_layers_gb300 import build as libbuild

from kv_plain import DT, Cache, int32, offsets_of
from test_attn import GUARD, Call, tree


@pytest.fixture(scope="module", autouse=True)
def lib():
    libbuild.build()
    return B.load()


@pytest.mark.gpu
@pytest.mark.parametrize("T,G", [(2, 8), (17, 1), (4, 8), (16, 4), (13, 5), (16, 8), (43, 3), (32, 8), (257, 1), (3, 11)])
@pytest.mark.parametrize("fmt,dtype,D", [("rows", "bf16", 128), ("e4m3", "fp16", 64), ("int8", "bf16", 128)])
def test_rows_around_a_tile(T, G, fmt, dtype, D):
    """Items of 16, 17, 32, 64, 65, 128, 129, 256, 257 and 33 rows."""
    c = Call(fmt, dtype, [T, T], [130, 63], 2, G, D, 32, [tree, tree], B.PROJ_GATE_SIGMOID, seed=T * 31 + G)
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 4, 12])
@pytest.mark.parametrize("fmt,dtype", [("rows", "fp16"), ("int8", "bf16")])
@pytest.mark.parametrize("up", [True, False])
def test_references_that_move(T, fmt, dtype, up):
    """Scores that rise (or fall) along the keys by hundreds, and values whose scales do, so that every reference moves often."""
    c = Call(fmt, dtype, [T], [700], 1, 8, 64, 16, [tree], seed=17, scale=1.0)
    n = 700 + T
    rise = torch.linspace(0, 1, n) if up else torch.linspace(1, 0, n)
    gen = torch.Generator().manual_seed(3)
    k = torch.randn(n, 1, 64, generator=gen) * 0.05
    k[:, :, 0] = 300.0 * rise[:, None]
    v = torch.randn(n, 1, 64, generator=gen) * torch.exp2(12.0 * rise)[:, None, None]
    c.cache.put(0, 0, k.to(DT[dtype][0]), v.to(DT[dtype][0]))
    c.q[:, 0::64] = 1.0  # each head's first dimension
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("T,G", [(1, 4), (9, 4)])
def test_many_sequences_of_either_kernel(T, G):
    n = 150
    counts = [(b * 5) % (T + 1) for b in range(n)] if T > 1 else [b % 2 for b in range(n)]
    counts[0] = T
    c = Call("e4m3", "bf16", [T - k % 2 if k else 0 for k in counts], [(b * 11) % 90 for b in range(n)], 1, G, 64, 16, None, seed=18)
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 6])
def test_a_cache_beyond_32_bits(T):
    """Pages whose bytes lie beyond 2^32: write, read, move, attend."""
    kv, D, page, G = 4, 128, 64, 8
    pages = (5 << 30) // (kv * page * D)
    k, v = (torch.zeros(pages, kv, page, D, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, kv, page), math.nan, device="cuda") for _ in range(2))
    c = Call("int8", "bf16", [T], [100], kv, G, D, page, None, seed=19)
    width = 4 + Cache.more // page
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, :3] = int32([pages - 1, pages - 2, pages // 2 + 3])
    far = B.kv_cache(format=B.PROJ_KV_INT8, dtype=B.PROJ_BF16, pages=pages, page=page, heads=kv, D=D, k=k, v=v, k_scale=ks, v_scale=vs,
                     page_stride=kv * page * D, head_stride=page * D, token_stride=D, table=table, ldt=width, width=width, sequences=1)
    n = 100 + T
    rows_k = torch.randn(n, kv * D, device="cuda").bfloat16()
    rows_v = torch.randn(n, kv * D, device="cuda").bfloat16()
    B.proj_kv_write(far, int32([0, n]), int32([0]), n, rows_k, kv * D, rows_v, kv * D)
    c.cache.put(0, 0, rows_k.view(n, kv, D).cpu(), rows_v.view(n, kv, D).cpu())
    back = torch.zeros_like(rows_k)
    B.proj_kv_read(far, int32([0, n]), int32([0]), n, back, kv * D, None, 0)
    ref = c.cache.get("k", 0, 0, n).reshape(n, -1)
    assert bool(((back.cpu().double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -24) * ref.abs() + 2.0 ** -30).all())
    args = c.args()
    args.cache = ctypes.addressof(far)
    B.proj_attn(args)
    c.check()
    if T > 1:
        B.proj_kv_move(far, int32([100]), int32([[1, 4]]), 2, 2)
        for i, f in enumerate((1, 4)):
            at = [(table[0, p // page].item(), p % page) for p in (100 + i, 100 + f)]
            assert torch.equal(k[at[0][0], :, at[0][1]].cpu(), c.cache.t["k"][c.cache.spots(0, 100 + f, 1)[0].item(), :, (100 + f) % page].cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("off", [[-3, 4, 400], [5, 2, 7], [8, 8, 8], [0, 0, 8], [3, 5, 7]])
def test_offsets_out_of_range(T, off):
    """Offsets beyond 0 .. m, or decreasing: rows of no sequence are left as they are."""
    c = Call("rows", "bf16", [8 * T, 0], [40, 40], 1, 4, 64, 16, None, seed=20)
    o = [x * T for x in off]
    c.run(offsets=int32(o))
    torch.cuda.synchronize()
    if off == sorted(off):
        for r in range(8 * T):
            owned = any(max(o[b], 0) <= r < o[b + 1] for b in range(2))
            assert bool((c.out[r] == GUARD).all()) == (not owned) and bool((c.lse[r] == GUARD).all()) == (not owned)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 9])
def test_starts_out_of_range(T):
    """A negative start counts as 0; drafts behind the table's end have no place and are not seen."""
    c = Call("e4m3", "bf16", [T, T], [0, 30], 1, 4, 64, 16, None, seed=21)
    c.start.copy_(int32([-7, 30]))
    c.run()
    c.check()
    last = c.cache.width * 16
    for s in (last - 1, last, 2 ** 31 - 1):
        c = Call("e4m3", "bf16", [T], [48], 1, 4, 64, 16, None, seed=22)
        c.cache.d_table[0, 3:] = c.cache.d_table[0, 0]  # the table's last place is a page too
        last = c.cache.width * 16
        c.start.copy_(int32([min(s, 2 ** 31 - 1)]))
        c.run()
        k, v = (torch.cat([c.cache.get(i, 0, 0, 48)] + [c.cache.get(i, 0, 0, 16)] * (c.cache.width - 3)).numpy() for i in ("k", "v"))
        q = c.q.reshape(T, 4, 64).cpu().double().numpy()
        for r in range(T):
            n = min(max(s, 0) + r + 1, last)
            p = np.einsum("hd,kd->hk", q[r], k[:n, 0]) * float(np.float32(c.scale))
            p = np.exp(p - p.max(1, keepdims=True))
            ref = (p / p.sum(1, keepdims=True)) @ v[:n, 0]
            got = c.out[r].reshape(4, 64).cpu().double().numpy()
            assert np.abs(got - ref).max() <= 2.0 ** -6 * np.abs(ref).max() + 2.0 ** -8 * np.abs(v).max()


@pytest.mark.gpu
def test_no_sequences_and_no_rows():
    c = Call("rows", "fp16", [0, 0], [5, 9], 1, 4, 64, 16, None, behind=4, seed=23)
    c.run()
    assert bool((c.out == GUARD).all()) and bool((c.lse == GUARD).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 8])
def test_one_page_for_many_sequences(T):
    """Sequences that share the pages of a common beginning."""
    c = Call("int8", "fp16", [T, T, T], [64, 80, 64], 1, 4, 64, 16, None, seed=24)
    shared = c.cache.table[0, :4].clone()
    for b in (1, 2):
        c.cache.table[b, :4] = shared
    c.cache.d_table.copy_(c.cache.table)
    c.run()
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("T,G,D", [(1, 8, 128), (2, 8, 128), (1, 3, 64), (4, 4, 64)])
@pytest.mark.parametrize("dtype,r", [("bf16", 2.0 ** -16), ("fp16", 2.0 ** -22)])
def test_few_rows_of_a_16_bit_cache(T, G, D, dtype, r):
    """Streamed, a probability is the sum of two numbers: off by half a step of what half a step of the first one left."""
    for counts, starts in (([T, T], [500, 40]), ([T] * 250, [(7 * b) % 60 for b in range(250)])):
        c = Call("rows", dtype, counts, starts, 1, G, D, 16, None, seed=25)
        assert "stream" in B.proj_attn_describe(c.cache.c, c.m, c.heads)
        c.r = r
        c.run()
        c.check()


def test_scale_out_of_range_refused():
    """A scale whose product with log2(e) leaves fp32: the exponents are computed in base 2."""
    cache = B.kv_cache(format=B.PROJ_KV_ROWS, dtype=B.PROJ_BF16, pages=1, page=16, heads=1, D=64, k=4096, v=8192,
                       page_stride=1024, head_stride=1024, token_stride=64, table=4096, ldt=1, width=1, sequences=1)
    args = B.attn_args(cache, m=1, heads=1, q=4096, ldq=64, offsets=4096, start=4096, scale=3e38, out=8192, ldo=64,
                       workspace=4096, workspace_bytes=1 << 30)
    assert B.load().proj_attn(ctypes.byref(args), None) == B.PROJ_EINVAL
    assert "scale" in B.last_cuda_error()
