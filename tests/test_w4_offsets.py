"""Experts' offsets that decrease, which a caller should not pass: nothing but the rows of x is touched, and
every value is a right one of some expert's.  Bounds as in test_w4."""
import pytest

torch = pytest.importorskip("torch")

from test_w4 import Weights, is_exact, make_x

from gemv_projection_layers_gb300 import binding as B


@pytest.mark.gpu
@pytest.mark.parametrize("m,N,K", [(146, 536, 2050), (146, 130, 200), (600, 536, 520), (20, 300, 4200)])
def test_offsets_that_decrease(m, N, K):
    """Rows claimed by several experts: every value is one of theirs, or what stood there."""
    claims = [0, m, 0, m // 2, 3, m, 1, m - 1, 0]
    E = len(claims) - 1
    with Weights(E, N, K, 64, False, "bf16", m) as w:
        x, ld = make_x(m, K, "bf16", m)
        off = torch.tensor(claims, dtype=torch.int32, device="cuda")
        out = torch.full((m + 2, N), -7.0, device="cuda", dtype=torch.bfloat16)
        B.proj_w4_run_experts(w.h, x, ld, m, off, out, N)
        torch.cuda.synchronize()
        assert (out[m:] == -7.0).all()
        got, fine = out[:m].double(), out[:m] == -7.0
        x64 = x[:m, :K].double()
        for e in range(E):
            rows = slice(claims[e], max(claims[e], claims[e + 1]))
            w64 = w.w64(e)
            ref, S = x64[rows] @ w64.t(), x64[rows].abs() @ w64.abs().t()
            tol = 2.0 ** -8 * ref.abs() + ((K / 16 + 64) * 2.0 ** -23 + (0.0 if is_exact(w.h, m) else 2.0 ** -8)) * S
            fine[rows] |= (got[rows] - ref).abs() <= tol
        assert fine.all()
