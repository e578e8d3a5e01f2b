"""A workspace that is aligned to 16 bytes and no more, of exactly the size asked for, between guards."""
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B

import test_attn as A
from kv_plain import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,fmt,dtype,counts,starts,kv,G,D,more", [
    ("CTAs", "e4m3", "bf16", [1], [5000], 1, 8, 128, 0), ("CTAs", "rows", "fp16", [4, 4], [900, 3000], 2, 4, 64, 0),
    ("warps", "int8", "bf16", [2] * 44, [300] * 44, 8, 4, 64, 0), ("warps", "rows", "bf16", [1] * 700, [90] * 700, 1, 8, 128, 0),
    ("tcgen05", "e4m3", "bf16", [8, 3], [2000, 70], 1, 8, 128, 1 << 20), ("tcgen05", "rows", "fp16", [70], [1500], 2, 4, 64, 1 << 20)])
def test_aligned_to_16_bytes(kind, fmt, dtype, counts, starts, kv, G, D, more, monkeypatch):
    A.libbuild.build()
    monkeypatch.setattr(Cache, "more", more)
    c = A.Call(fmt, dtype, counts, starts, kv, G, D, 16, None, B.PROJ_GATE_SIGMOID, seed=71)
    assert kind in B.proj_attn_describe(c.cache.c, c.m, c.heads)
    c.run()
    torch.cuda.synchronize()
    want, want_lse, size = c.out.clone(), c.lse.clone(), c.room.numel()
    for shift in (16, 48):
        whole = torch.full((size + 128,), 255, device="cuda", dtype=torch.uint8)
        assert whole.data_ptr() % 32 == 0
        room = whole[shift:shift + size]
        c.out.fill_(A.GUARD)
        c.lse.fill_(A.GUARD)
        c.run(workspace=room, workspace_bytes=size)
        torch.cuda.synchronize()
        assert torch.equal(c.out, want) and torch.equal(c.lse, want_lse)
        assert bool((whole[:shift] == 255).all()) and bool((whole[shift + size:] == 255).all())
    c.check()
    assert B.proj_attn_device_status() == 0
