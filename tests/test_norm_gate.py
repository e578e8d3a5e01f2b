"""The gradient of a sigmoid gate where the gate is nearly shut or nearly open.

The slope is sigmoid(x) sigmoid(-x), a product of two values that are each known to their own last
places, so the bound goes by the slope itself.  (test_norm's goes by slope + g, for gates about 0.)
"""
import pytest

torch = pytest.importorskip("torch")

from test_norm import Cc, Cr, DT, TINY, Case, backward, grads64, near

from gemv_projection_layers_gb300 import binding as B

GATES = [-30.0, -20.0, -17.5, -10.0, -5.0, -1.0, 0.0, 1.0, 5.0, 8.0, 10.0, 12.0, 17.5, 20.0, 30.0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gate", [B.PROJ_GATE_CHANNEL, B.PROJ_GATE_ELEMENT, B.PROJ_GATE_TOKEN])
@pytest.mark.parametrize("m,D", [(15, 64), (31, 333), (7, 1000), (5, 2048), (4, 4096), (3, 8192), (2, 5001), (2, 16384)])
def test_slope(m, D, gate, dtype):
    c = Case(m, D, dtype, gate, B.PROJ_GATE_SIGMOID, D)
    raw = c.gate[:m, :D] if gate == B.PROJ_GATE_ELEMENT else c.gate
    places = torch.arange(raw.numel(), device="cuda") % len(GATES)
    raw.copy_(torch.tensor(GATES, device="cuda")[places].view(raw.shape).to(raw.dtype))
    got, _ = backward(c)
    ref, sizes = grads64(c)
    x = raw.double()
    s = torch.sigmoid(x)
    slope = s * torch.sigmoid(-x)
    ref["gate"] = ref["gate"] / ((1 - s) * s) * slope  # autograd's (1 - s) s cancels in 64 bits too
    for n, name in (("dgate", "gate"), ("dy", "y"), ("dresidual", "residual")):
        g = got[n]
        u = DT[dtype][2] if g.dtype != torch.float32 else 2.0 ** -24
        size = sizes[name] * (slope / (slope + s) if n == "dgate" else 1.0)
        near(g, ref[name], u, TINY[dtype] if g.dtype == torch.float16 else 0.0, size, Cc if g.dim() == 1 else Cr)
