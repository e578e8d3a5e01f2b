"""Attention over caches whose tables have room for a million positions: there the kernel for many rows is taken from 33 rows on,
and most of a table is no page.  The cases and bounds are those of test_attn.py and test_attn_more.py, whose small tables go to
the streaming kernel."""
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B

import test_attn as A
import test_attn_more as M
from kv_plain import Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def wide(monkeypatch):
    A.libbuild.build()
    monkeypatch.setattr(Cache, "more", 1 << 20)


def test_which_kernel():
    """33 rows of a sequence and a head: tcgen05 with such a table, streamed with a small one."""
    for fmt in ("rows", "int8"):
        c = A.Call(fmt, "bf16", [33], [10], 1, 1, 64, 16)
        assert "tcgen05" in B.proj_attn_describe(c.cache.c, c.m, c.heads)
    Cache.more = 0
    c = A.Call("rows", "bf16", [33], [10], 1, 1, 64, 16)
    assert "stream" in B.proj_attn_describe(c.cache.c, c.m, c.heads)


MANY = [i for i, c in enumerate(A.CASES) if -(-sum(c[2]) // len(c[2])) * c[5] > 32]


@pytest.mark.parametrize("case", MANY)
def test_attention(case):
    A.test_attention(case)


@pytest.mark.parametrize("T", [5, 6, 7, 8, 9, 16, 17, 31, 33])
@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("rows", "bf16"), ("int8", "fp16")])
def test_numbers_of_drafts(T, fmt, dtype):
    A.test_numbers_of_drafts(T, fmt, dtype)


@pytest.mark.parametrize("T", [8, 64])
def test_split_over_all_ctas(T):
    A.test_split_over_all_ctas(T)


@pytest.mark.parametrize("spread,scale", [(4.0, 0.125), (0.0, 20.0), (1.0, -0.3), (1.0, 0.0)])
def test_scores_and_scales_that_differ(spread, scale):
    A.test_scores_and_scales_that_differ(spread, scale, 12)


@pytest.mark.parametrize("fmt,dtype,T,G", [("rows", "fp16", 40, 4), ("e4m3", "bf16", 70, 2), ("rows", "bf16", 12, 12), ("int8", "bf16", 90, 2),
                                           ("rows", "bf16", 5, 8), ("e4m3", "fp16", 9, 7)])
def test_no_finite_number_in_unseen_drafts(fmt, dtype, T, G):
    A.test_no_finite_number_in_unseen_drafts(fmt, dtype, T, G)


def test_no_finite_number_in_codes():
    A.test_no_finite_number_in_codes()


@pytest.mark.parametrize("T", [6, 40])
def test_pages_that_do_not_exist(T):
    A.test_pages_that_do_not_exist(T)


def test_masks_shorter_than_the_drafts():
    A.test_masks_shorter_than_the_drafts()


def test_in_place_and_without_lse():
    A.test_in_place_and_without_lse(24)


def test_same_bits_and_two_streams():
    A.test_same_bits_and_two_streams(12)


@pytest.mark.parametrize("T,G", [(4, 16), (8, 8), (43, 3)])
def test_graphs_of_growing_sequences(T, G):
    """A captured call, replayed while the sequences get shorter: units, items and shares follow."""
    c = A.Call("e4m3", "bf16", [T, T], [700, 300], 1, G, 64, 64, None, seed=31)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.run(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.run(side)
    for _ in range(4):
        c.out.fill_(A.GUARD)
        c.lse.fill_(A.GUARD)
        graph.replay()
        torch.cuda.synchronize()
        c.check()
        c.starts = [max(0, s - 97) for s in c.starts]
        c.start.copy_(A.int32(c.starts))
        torch.cuda.synchronize()
    assert B.proj_attn_device_status() == 0


@pytest.mark.parametrize("T,G", [(17, 4), (16, 4), (13, 5), (16, 8), (43, 3), (32, 8), (257, 1), (3, 11)])
@pytest.mark.parametrize("fmt,dtype,D", [("rows", "bf16", 128), ("e4m3", "fp16", 64), ("int8", "bf16", 128)])
def test_rows_around_a_tile(T, G, fmt, dtype, D):
    M.test_rows_around_a_tile(T, G, fmt, dtype, D)


@pytest.mark.parametrize("T", [5, 12])
@pytest.mark.parametrize("fmt,dtype", [("rows", "fp16"), ("int8", "bf16")])
@pytest.mark.parametrize("up", [True, False])
def test_references_that_move(T, fmt, dtype, up):
    M.test_references_that_move(T, fmt, dtype, up)


def test_many_sequences():
    M.test_many_sequences_of_either_kernel(9, 16)


@pytest.mark.parametrize("T", [6, 40])
def test_a_cache_beyond_32_bits(T):
    M.test_a_cache_beyond_32_bits(T)


@pytest.mark.parametrize("off", [[-3, 4, 400], [5, 2, 7], [8, 8, 8], [0, 0, 8], [3, 5, 7]])
def test_offsets_out_of_range(off):
    M.test_offsets_out_of_range(20, off)


def test_one_page_for_many_sequences():
    M.test_one_page_for_many_sequences(16)
