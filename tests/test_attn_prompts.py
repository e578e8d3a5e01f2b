"""Attention of prompts: hundreds of rows of a sequence, alone and beside single tokens, chains without a mask.  Bounds as in test_attn.py."""
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B

import test_attn as A
from kv_plain import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,starts", [([1100], [0]), ([777, 1, 1, 0, 37, 1], [5, 0, 900, 64, 63, 129]), ([513, 2], [700, 3000])])
@pytest.mark.parametrize("fmt,dtype,kv,G,D", [("rows", "bf16", 1, 3, 64), ("e4m3", "bf16", 1, 4, 128), ("int8", "fp16", 2, 1, 64),
                                              ("rows", "fp16", 1, 2, 128)])
@pytest.mark.parametrize("more", [0, 1 << 20], ids=["narrow", "wide"])
def test_prompts(counts, starts, fmt, dtype, kv, G, D, more, monkeypatch):
    A.libbuild.build()
    monkeypatch.setattr(Cache, "more", more)
    c = A.Call(fmt, dtype, counts, starts, kv, G, D, 48, None, B.PROJ_GATE_SIGMOID, more=8, behind=2, seed=sum(counts))
    c.run()
    c.check()
    assert B.proj_attn_device_status() == 0
