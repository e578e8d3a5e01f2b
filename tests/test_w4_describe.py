"""What proj_w4_describe says of a stack of one matrix, which proj_w4_run and proj_w4_run_experts both take."""
import pytest

torch = pytest.importorskip("torch")

from test_w4 import Weights

from gemv_projection_layers_gb300 import binding as B


@pytest.mark.gpu
@pytest.mark.parametrize("m,N,K,run,experts", [
    (300, 8192, 512, "256-token tiles", "128-token tiles"),  # tiles of rows from anywhere are kept to 128
    (4, 512, 512, "16 rows", "32 rows"),  # experts' streamed blocks go in pairs
    (50, 512, 512, "64-token tiles", None),
])
def test_both_calls_are_described(m, N, K, run, experts):
    with Weights(1, N, K, 64, False, "bf16", 1) as w:
        text = B.proj_w4_describe(w.h, m)
        first, _, second = text.partition("; with offsets: ")
        assert run in first
        assert second == "" if experts is None else experts in second
        assert ("exact" in first) == (m <= 16) and (not second or ("exact" in second) == ("exact" in first))
    with Weights(2, N, K, 64, False, "bf16", 1) as w:
        assert "offsets" not in B.proj_w4_describe(w.h, m)
