"""The combine with many more pieces than the GPU holds at a time, in each of its three accesses.

Bounds as in test_moe: u |ref| + (k + 2) 2^-24 sum |w y|.
"""
import pytest

torch = pytest.importorskip("torch")

from test_moe import DT, plan, rows

from gemv_projection_layers_gb300 import binding as B


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,k,D,extra", [(4000, 1, 264, 0), (1500, 8, 2056, 0), (1000, 9, 1000, 8), (1500, 8, 4100, 0), (1200, 9, 4102, 0),
                                         (3000, 1, 333, 0), (1500, 8, 2501, 0), (1000, 9, 777, 2), (700, 17, 5001, 0)])
def test_combine_of_many_pieces(m, k, D, extra, dtype):
    """A CTA goes from piece to piece many times, each row's neighbours NaN where they do not count."""
    t, kind, u = DT[dtype]
    slot, w, s64 = plan(m, max(k, 16), k, m + D)
    ld, n = D + extra, m * k
    valid = s64 >= 0
    ys = rows(n, D, dtype, 2, ld)
    named = torch.zeros(n, dtype=torch.bool, device="cuda")
    named[s64[valid]] = True
    ys[:n][~named] = float("nan")
    out = torch.full((m + 1, ld), -7.0, device="cuda", dtype=t)
    B.proj_moe_combine(ys, ld, slot, w, m, D, k, kind, out, ld)
    torch.cuda.synchronize()
    for t0 in range(0, m, 500):  # in parts: the 64-bit rows are large
        part = slice(t0, min(m, t0 + 500))
        y64 = torch.where(valid[part][..., None], ys[:n, :D][s64[part].clamp(min=0)].double(), torch.zeros((), device="cuda", dtype=torch.float64))
        terms = w[part].double()[..., None] * y64
        ref = terms.sum(1)
        tol = u * ref.abs() + (k + 2) * 2.0 ** -24 * terms.abs().sum(1) + (2.0 ** -25 if dtype == "fp16" else 0)
        assert ((out[part, :D].double() - ref).abs() <= tol).all()
    assert (out[m:] == -7.0).all() and (out[:, D:] == -7.0).all()
