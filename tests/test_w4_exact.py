"""4-bit products whose weights are not rounded: by the caller's choice, and by themselves where
s (q - z) leaves the range of the 16-bit type.  The bound is test_w4's for exact products."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from test_w4 import DT, assert_close, make_x, offsets_of

from gemv_projection_layers_gb300 import binding as B
from gemv_projection_layers_gb300 import build as libbuild


class Stack:
    """A stack of matrices with the given scales [E, N, groups]."""

    def __init__(self, s, K, group, zeros, dtype, seed, flags=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.E, self.N, _ = s.shape
        self.K, self.group, self.s = K, group, s.to(DT[dtype][0])
        self.q = torch.randint(0, 16, (self.E, self.N, K + K % 2), device="cuda", generator=gen, dtype=torch.uint8)
        codes = (self.q[..., 0::2] | (self.q[..., 1::2] << 4)).contiguous()
        self.z = torch.randint(0, 16, s.shape, device="cuda", generator=gen, dtype=torch.uint8) if zeros else None
        args = (codes, self.s, self.z, self.E, self.N, K, group, DT[dtype][1])
        self.h = B.proj_w4_prepare_ex(*args, flags) if flags else B.proj_w4_prepare(*args)

    def w64(self, e):
        rep = lambda a: a.double().repeat_interleave(self.group, dim=-1)[..., :self.K]  # noqa: E731
        z = 8.0 if self.z is None else rep(self.z[e])
        return (self.q[e, :, :self.K].double() - z) * rep(self.s[e])

    def __enter__(self):
        return self

    def __exit__(self, *a):
        torch.cuda.synchronize()
        assert B.proj_w4_device_status(self.h) == 0
        B.proj_w4_destroy(self.h)


def check(w, x, ld, m, dtype):
    """proj_w4_run, or with E > 1 run_experts with m rows spread over the matrices."""
    out = torch.full((m + 1, w.N), -7.0, device="cuda", dtype=x.dtype)
    if w.E == 1:
        B.proj_w4_run(w.h, x, ld, m, out, w.N)
        o = [0, m]
    else:
        o = [m * e // w.E for e in range(w.E + 1)]
        B.proj_w4_run_experts(w.h, x, ld, m, offsets_of([o[e + 1] - o[e] for e in range(w.E)]), out, w.N)
    torch.cuda.synchronize()
    assert (out[m:] == -7.0).all()
    for e in range(w.E):
        if o[e] < o[e + 1]:
            rows = slice(o[e], o[e + 1])
            assert_close(out[rows], x[rows, :w.K].double(), w.w64(e), dtype, True, w.K)


@pytest.mark.gpu
@pytest.mark.parametrize("E", [1, 3])
@pytest.mark.parametrize("dtype,scale,small,zeros,group", [("fp16", 30000.0, 2.0 ** -10, False, 64), ("fp16", 60000.0, 2.0 ** -11, True, 32),
                                                           ("bf16", 2.0 ** 126, 2.0 ** -118, False, 128), ("bf16", 2.0 ** 127, 2.0 ** -119, True, 64)])
def test_scales_whose_weights_leave_the_range(dtype, scale, small, zeros, group, E):
    """s is in the type's range, s (q - z) is not, the sums are: the same finite values at any number of rows."""
    N, K = 70, 200
    gen = torch.Generator("cuda").manual_seed(E)
    s = scale * (torch.rand(E, N, -(-K // group), device="cuda", generator=gen).double() - 0.5).float()
    s[0, 0, 0] = scale
    with Stack(s, K, group, zeros, dtype, 3) as w:
        for m in (4, 17, 65, 300):
            x, ld = make_x(m, K, dtype, m)
            check(w, x * small, ld, m, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,most", [("fp16", 65504.0), ("bf16", 2.0 ** 127 * (2 - 2.0 ** -7))])
def test_scales_just_in_range_keep_the_fast_kernel(dtype, most):
    """The largest |q - z| is 8 with z = 8, so most / 8 is the last scale whose weights all fit."""
    N, K, m = 40, 128, 50
    s = torch.full((1, N, 2), most / 8, device="cuda", dtype=torch.float64)
    for factor, fits in ((1.0, True), (1.01, False)):
        with Stack((s * factor), K, 64, False, dtype, 4) as w:
            assert ("rounded" in B.proj_w4_describe(w.h, m)) == fits
    z = torch.full((1, N, 2), 7, device="cuda", dtype=torch.uint8)  # |q - z| up to 8 again; with 15 it is 15
    codes = torch.zeros(1, N, K // 2, device="cuda", dtype=torch.uint8)
    for value, fits in ((7, True), (15, False)):
        h = B.proj_w4_prepare(codes, s.to(DT[dtype][0]), z.fill_(value), 1, N, K, 64, DT[dtype][1])
        try:
            assert ("rounded" in B.proj_w4_describe(h, m)) == fits
        finally:
            B.proj_w4_destroy(h)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,group,zeros", [("bf16", 128, False), ("fp16", 32, True)])
@pytest.mark.parametrize("E,N,K", [(1, 130, 1000), (4, 70, 520), (40, 17, 96)])
def test_exact_at_any_number_of_rows_if_asked_for(E, N, K, dtype, group, zeros):
    gen = torch.Generator("cuda").manual_seed(N)
    s = torch.rand(E, N, -(-K // group), device="cuda", generator=gen) * 0.2 - 0.05
    with Stack(s, K, group, zeros, dtype, 5, flags=B.PROJ_W4_EXACT) as w:
        for m in (1, 16, 17, 64, 257, 1500):
            assert "exact" in B.proj_w4_describe(w.h, m)
            x, ld = make_x(m, K, dtype, m)
            check(w, x, ld, m, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("E", [1, 2])
def test_exact_at_the_most_rows(E):
    """2^20 rows are 65,536 tiles of 16, more than a grid has in y."""
    N, K, m = 16, 64, 2 ** 20
    s = torch.rand(E, N, 1, device="cuda") * 0.2 - 0.05
    with Stack(s, K, 64, False, "bf16", 6, flags=B.PROJ_W4_EXACT) as w:
        x, ld = make_x(m, K, "bf16", 1)
        check(w, x, ld, m, "bf16")


def test_flags_are_checked_before_any_device_call():
    libbuild.build()
    lib = B.load()
    st = ctypes.c_int(0)
    assert lib.proj_w4_prepare_ex(16, 16, None, 1, 16, 64, 32, B.PROJ_BF16, 2, ctypes.byref(st)) is None
    assert st.value == B.PROJ_EINVAL and B.last_cuda_error().startswith("proj_w4_prepare")
    assert lib.proj_w4_prepare_ex(None, 16, None, 1, 16, 64, 32, B.PROJ_BF16, B.PROJ_W4_EXACT, ctypes.byref(st)) is None
    assert st.value == B.PROJ_EINVAL
