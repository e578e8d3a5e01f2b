"""4-bit products with so many tiles that a CTA works on several."""
import pytest

torch = pytest.importorskip("torch")

from test_w4 import Weights, assert_close, is_exact, make_x, offsets_of

from gemv_projection_layers_gb300 import binding as B


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,group,zeros", [("bf16", 128, False), ("fp16", 32, True)])
@pytest.mark.parametrize("m,N,K", [(1100, 8192, 200), (2048, 8192, 513), (3001, 4100, 130), (700, 20000, 64)])
def test_several_256_token_tiles_a_cta(m, N, K, dtype, group, zeros):
    """The one accumulator goes from tile to tile, and the rings go on through them; the last tiles are part-filled."""
    with Weights(1, N, K, group, zeros, dtype, m) as w:
        text = B.proj_w4_describe(w.h, m)
        assert "256-token tiles" in text and -(-m // 256) * -(-N // 128) > 2 * 152
        x, ld = make_x(m, K, dtype, m, extra=m % 2)
        out = torch.full((m + 1, N), -7.0, device="cuda", dtype=x.dtype)
        B.proj_w4_run(w.h, x, ld, m, out, N)
        torch.cuda.synchronize()
        assert (out[m:] == -7.0).all()
        assert_close(out[:m], x[:m, :K].double(), w.w64(0), dtype, is_exact(w.h, m), K)


@pytest.mark.gpu
@pytest.mark.parametrize("m,N,K", [(1100, 8192, 200), (2000, 4100, 513)])
def test_several_128_token_tiles_a_cta_in_a_stack_of_one(m, N, K):
    with Weights(1, N, K, 64, True, "bf16", m) as w:
        x, ld = make_x(m, K, "bf16", m)
        out = torch.full((m + 1, N), -7.0, device="cuda", dtype=x.dtype)
        B.proj_w4_run_experts(w.h, x, ld, m, offsets_of([m - 10], 3), out, N)
        torch.cuda.synchronize()
        assert (out[:3] == -7.0).all() and (out[m - 7:] == -7.0).all()
        assert_close(out[3:m - 7], x[3:m - 7, :K].double(), w.w64(0), "bf16", is_exact(w.h, m), K)
