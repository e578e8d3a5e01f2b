"""Products with 4-bit weights and group scales against the definition in 64 bits.

Tolerance, element by element, from the arithmetic:
  u |ref|                 the output's rounding (u = 2^-8 bf16, 2^-11 fp16; 2^-25 more for fp16
                          results below its normal range),
  (K / 16 + 64) 2^-23 S   fp32 sums: S = sum of |x w|; a chain of at most K / 16 steps of the
                          matrix unit, whose inner sums and the joins of partial sums add a few
                          dozen roundings; 2^-23 because the unit may truncate,
  u S                     only where the call rounds s (q - z) to the type of x first, which
                          proj_w4_describe tells.
"""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B
from gemv_projection_layers_gb300 import build as libbuild

DT = {"bf16": (torch.bfloat16, B.PROJ_BF16, 2.0 ** -8), "fp16": (torch.float16, B.PROJ_FP16, 2.0 ** -11)}


class Weights:
    def __init__(self, E, N, K, group, zeros, dtype, seed):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.E, self.N, self.K, self.group, self.dtype = E, N, K, group, dtype
        ng = -(-K // group)
        self.q = torch.randint(0, 16, (E, N, K), device="cuda", generator=gen, dtype=torch.uint8)
        pad = torch.randint(0, 16, (E, N, K + K % 2), device="cuda", generator=gen, dtype=torch.uint8)
        pad[..., :K] = self.q  # an odd K leaves a half byte with anything in it
        self.codes = (pad[..., 0::2] | (pad[..., 1::2] << 4)).contiguous()
        self.s = (torch.rand(E, N, ng, device="cuda", generator=gen) * 0.2 - 0.05).to(DT[dtype][0])
        self.z = torch.randint(0, 16, (E, N, ng), device="cuda", generator=gen, dtype=torch.uint8) if zeros else None
        self.h = B.proj_w4_prepare(self.codes, self.s, self.z, E, N, K, group, DT[dtype][1])

    def w64(self, e):
        rep = lambda a: a.double().repeat_interleave(self.group, dim=-1)[..., :self.K]  # noqa: E731
        z = 8.0 if self.z is None else rep(self.z[e])
        return (self.q[e].double() - z) * rep(self.s[e])

    def __enter__(self):
        return self

    def __exit__(self, *a):
        torch.cuda.synchronize()
        assert B.proj_w4_device_status(self.h) == 0
        B.proj_w4_destroy(self.h)


def make_x(m, K, dtype, seed, extra=0):
    """m rows; everything a call must not read is NaN: columns from K on, rows from m on."""
    gen = torch.Generator("cuda").manual_seed(seed + 1000)
    ld = (K + 7) // 8 * 8 + 8 * extra
    buf = torch.full((m + 3, ld), float("nan"), device="cuda", dtype=DT[dtype][0])
    buf[:m, :K] = torch.randn(m, K, device="cuda", generator=gen).to(buf.dtype)
    return buf, ld


def assert_close(out, x64, w64, dtype, exact, K):
    u = DT[dtype][2]
    ref = x64 @ w64.t()
    S = x64.abs() @ w64.abs().t()
    tol = u * ref.abs() + ((K / 16 + 64) * 2.0 ** -23 + (0.0 if exact else u)) * S
    if dtype == "fp16":
        tol = tol + 2.0 ** -25
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), ((err - tol).max().item(), err.max().item())


def is_exact(h, m):
    return "exact" in B.proj_w4_describe(h, m)


SHAPES = [  # N, K, group, zeros
    (1, 1, 32, False), (15, 2, 32, True), (16, 31, 64, True), (17, 33, 32, True), (129, 63, 32, False),
    (33, 65, 64, True), (40, 100, 32, True), (64, 129, 128, False), (200, 640, 192, True), (256, 1000, 1024, True),
    (130, 1024, 128, False), (300, 4096, 128, True), (65, 8103, 32, True), (2305, 512, 64, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("N,K,group,zeros", SHAPES)
def test_one_matrix(N, K, group, zeros, dtype):
    with Weights(1, N, K, group, zeros, dtype, N + K) as w:
        w64 = w.w64(0)
        for m in (1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 130, 257):
            x, ld = make_x(m, K, dtype, m, extra=m % 3)
            ldo = N + m % 4
            room = torch.full((m + 2, ldo), -7.0, device="cuda", dtype=x.dtype)
            B.proj_w4_run(w.h, x, ld, m, room, ldo)
            torch.cuda.synchronize()
            assert_close(room[:m, :N], x[:m, :K].double(), w64, dtype, is_exact(w.h, m), K)
            assert (room[m:] == -7.0).all() and (room[:, N:] == -7.0).all(), "wrote outside out"


@pytest.mark.gpu
@pytest.mark.parametrize("m", [1, 5, 40, 200])
def test_out_at_an_odd_element_and_in_a_side_stream(m):
    N, K = 77, 320
    with Weights(1, N, K, 64, True, "bf16", 5) as w:
        x, ld = make_x(m, K, "bf16", 9)
        room = torch.full((m * N + 2,), -7.0, device="cuda", dtype=torch.bfloat16)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        B.proj_w4_run(w.h, x, ld, m, room.data_ptr() + 2, N, s)
        s.synchronize()
        assert room[0] == -7.0 and room[-1] == -7.0
        assert_close(room[1:-1].view(m, N), x[:m, :K].double(), w.w64(0), "bf16", is_exact(w.h, m), K)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [3, 48, 150])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_one_hot_rows_give_the_weights(dtype, m):
    """x = a unit row: out is one column of s (q - z), rounded once to the type of x."""
    N, K = 100, 500
    with Weights(1, N, K, 32, True, dtype, 3) as w:
        cols = torch.arange(m, device="cuda") * 7 % K
        x = torch.zeros(m, 504, device="cuda", dtype=DT[dtype][0])
        x[torch.arange(m, device="cuda"), cols] = 1.0
        out = torch.empty(m, N, device="cuda", dtype=x.dtype)
        B.proj_w4_run(w.h, x, 504, m, out, N)
        torch.cuda.synchronize()
        # (q - z) s has at most 16 significant bits: the same rounding from 32 and from 64 bits
        assert torch.equal(out, w.w64(0)[:, cols].t().float().to(x.dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("m", [4, 100])
def test_infinities_and_nan_stay_in_their_rows(m):
    N, K = 50, 256
    with Weights(1, N, K, 64, False, "bf16", 8) as w:
        x, ld = make_x(m, K, "bf16", 1)
        clean = x.clone()
        x[1, 3] = float("inf")
        x[2, 200] = float("nan")
        a, b = (torch.empty(m, N, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        B.proj_w4_run(w.h, x, ld, m, a, N)
        B.proj_w4_run(w.h, clean, ld, m, b, N)
        torch.cuda.synchronize()
        rest = [i for i in range(m) if i not in (1, 2)]
        assert torch.equal(a[rest], b[rest])
        assert torch.isnan(a[2]).all()
        assert not torch.isfinite(a[1]).any()


def offsets_of(counts, start=0):
    o = [start]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


EXPERT_CASES = [  # counts, first row, rows behind the last expert's
    ([1], 0, 0), ([0, 0, 5, 0], 0, 0), ([3, 0, 9, 1, 40, 0, 8, 17], 0, 0), ([0, 0, 0], 0, 6), ([2, 2, 2], 3, 4),
    ([200, 0, 1], 0, 0), ([1] * 70, 0, 5), ([33, 130, 7, 64, 65], 0, 0), ([0] * 600 + [3] + [0] * 400 + [2], 0, 0),
    ([300, 290, 310], 0, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,group,zeros,N,K", [("bf16", 32, True, 70, 200), ("fp16", 128, False, 129, 513),
                                                   ("bf16", 64, False, 16, 96)])
@pytest.mark.parametrize("case", range(len(EXPERT_CASES)))
def test_experts(case, dtype, group, zeros, N, K):
    counts, start, behind = EXPERT_CASES[case]
    E, m = len(counts), start + sum(counts) + behind
    with Weights(E, N, K, group, zeros, dtype, case) as w:
        x, ld = make_x(m, K, dtype, case)
        x[:start] = float("nan")  # rows of no expert are not read
        x[start + sum(counts):] = float("nan")
        off = offsets_of(counts, start)
        out = torch.full((m, N), -7.0, device="cuda", dtype=x.dtype)
        B.proj_w4_run_experts(w.h, x, ld, m, off, out, N)
        again = torch.full((m, N), -7.0, device="cuda", dtype=x.dtype)
        B.proj_w4_run_experts(w.h, x, ld, m, off, again, N)
        torch.cuda.synchronize()
        assert torch.equal(out, again)
        assert (out[:start] == -7.0).all() and (out[start + sum(counts):] == -7.0).all()
        o = off.tolist()
        for e in range(E):
            if o[e] < o[e + 1]:
                rows = slice(o[e], o[e + 1])
                assert_close(out[rows], x[rows, :K].double(), w.w64(e), dtype, is_exact(w.h, m), K)


@pytest.mark.gpu
def test_experts_offsets_out_of_range_are_moved_into_it():
    N, K, m = 32, 64, 10
    with Weights(3, N, K, 32, False, "bf16", 2) as w:
        x, ld = make_x(m, K, "bf16", 2)
        out = torch.full((m + 2, N), -7.0, device="cuda", dtype=torch.bfloat16)
        off = torch.tensor([-5, 4, 2 ** 30, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
        B.proj_w4_run_experts(w.h, x, ld, m, off, out, N)
        torch.cuda.synchronize()
        assert_close(out[:4], x[:4, :K].double(), w.w64(0), "bf16", is_exact(w.h, m), K)
        assert_close(out[4:m], x[4:m, :K].double(), w.w64(1), "bf16", is_exact(w.h, m), K)
        assert (out[m:] == -7.0).all()


@pytest.mark.gpu
def test_in_a_graph_after_a_producer_on_the_stream():
    """x comes from a kernel just before; the captured pair replays on fresh inputs."""
    N, K, m = 256, 512, 6
    with Weights(1, N, K, 128, False, "bf16", 4) as w:
        src, _ = make_x(m, K, "bf16", 0)
        x = torch.zeros(m, K, device="cuda", dtype=torch.bfloat16)
        out = torch.zeros(m, N, device="cuda", dtype=torch.bfloat16)
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        B.proj_w4_run(w.h, x, K, m, out, N)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            x.copy_(src[:m, :K])
            B.proj_w4_run(w.h, x, K, m, out, N, s)
        for seed in (1, 2):
            src.copy_(make_x(m, K, "bf16", seed)[0])
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert_close(out, src[:m, :K].double(), w.w64(0), "bf16", is_exact(w.h, m), K)


@pytest.mark.gpu
def test_refusals_of_a_handle():
    with Weights(2, 32, 64, 32, False, "bf16", 1) as w:
        x = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
        o = torch.zeros(4, 32, device="cuda", dtype=torch.bfloat16)
        off = torch.zeros(3, device="cuda", dtype=torch.int32)
        lib = B.load()
        X, O, F = x.data_ptr(), o.data_ptr(), off.data_ptr()
        assert lib.proj_w4_run(w.h, X, 64, 4, O, 32, None) == B.PROJ_EINVAL  # two experts
        run = lambda *a: lib.proj_w4_run_experts(w.h, *a, None)  # noqa: E731
        assert run(X, 56, 4, F, O, 32) == B.PROJ_EINVAL
        assert run(X, 64, 4, F, O, 31) == B.PROJ_EINVAL
        assert run(X, 64, -1, F, O, 32) == B.PROJ_EINVAL
        assert run(None, 64, 4, F, O, 32) == B.PROJ_EINVAL
        assert run(X, 64, 4, None, O, 32) == B.PROJ_EINVAL
        assert run(X, 64, 4, F, None, 32) == B.PROJ_EINVAL
        assert run(X + 2, 64, 4, F, O, 32) == B.PROJ_EALIGN
        assert run(X, 68, 4, F, O, 32) == B.PROJ_EALIGN
        assert run(X, 64, 4, F + 2, O, 32) == B.PROJ_EALIGN
        assert run(X, 64, 4, F, O + 1, 32) == B.PROJ_EALIGN
        assert run(X, 64, 2 ** 20 + 1, F, O, 32) == B.PROJ_EUNSUPPORTED
        assert run(None, 64, 0, None, None, 32) == B.PROJ_OK
        assert B.proj_w4_describe(w.h, 4)


def test_refusals_before_any_device_call():
    libbuild.build()
    lib = B.load()
    st = ctypes.c_int(0)

    def prepare(codes=16, scales=16, E=1, N=16, K=64, group=32, dtype=B.PROJ_BF16):
        assert lib.proj_w4_prepare(codes, scales, None, E, N, K, group, dtype, ctypes.byref(st)) is None
        assert B.proj_last_status() == st.value and B.last_cuda_error().startswith("proj_w4_prepare")
        return st.value

    assert prepare(codes=None) == B.PROJ_EINVAL
    assert prepare(scales=None) == B.PROJ_EINVAL
    assert prepare(E=0) == B.PROJ_EINVAL
    assert prepare(N=0) == B.PROJ_EINVAL
    assert prepare(K=0) == B.PROJ_EINVAL
    for group in (0, -64, 16, 48, 96):
        assert prepare(group=group) == B.PROJ_EINVAL
    assert prepare(dtype=B.PROJ_FP32) == B.PROJ_EINVAL
    assert prepare(E=1025) == B.PROJ_EUNSUPPORTED
    assert prepare(K=2 ** 20 + 1) == B.PROJ_EUNSUPPORTED
    assert prepare(scales=17) == B.PROJ_EALIGN
    assert lib.proj_w4_run(None, 16, 64, 1, 16, 16, None) == B.PROJ_EINVAL
    assert lib.proj_w4_run_experts(None, 16, 64, 1, 16, 16, 16, None) == B.PROJ_EINVAL
    assert lib.proj_w4_describe(None, 1, None, 0) == B.PROJ_EINVAL
    assert lib.proj_w4_device_status(None, None, None) == B.PROJ_EINVAL
    lib.proj_w4_destroy(None)
    with pytest.raises(B.ProjError):
        B.proj_w4_run(0, 16, 64, 1, 16, 16)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,group,zeros,N,K", [("bf16", 128, False, 40, 4200), ("fp16", 32, True, 70, 4096), ("bf16", 64, True, 33, 5001)])
@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 9, 1, 17, 0], [2, 2, 2, 0, 0, 6], [70, 1, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0]])
def test_experts_of_long_rows(counts, dtype, group, zeros, N, K):
    """K long enough that few rows are streamed; some experts have several tiles all the same."""
    E, m = len(counts), sum(counts)
    with Weights(E, N, K, group, zeros, dtype, E) as w:
        x, ld = make_x(m, K, dtype, E)
        off = offsets_of(counts)
        out = torch.full((m + 1, N), -7.0, device="cuda", dtype=x.dtype)
        B.proj_w4_run_experts(w.h, x, ld, m, off, out, N)
        torch.cuda.synchronize()
        assert (out[m:] == -7.0).all()
        o = off.tolist()
        for e in range(E):
            if o[e] < o[e + 1]:
                rows = slice(o[e], o[e + 1])
                assert_close(out[rows], x[rows, :K].double(), w.w64(e), dtype, is_exact(w.h, m), K)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,group,zeros,N,K", [("bf16", 32, True, 520, 513), ("fp16", 128, False, 700, 96)])
@pytest.mark.parametrize("counts", [[1, 0, 2] * 100, [0] * 100 + [1] * 200 + [0, 0, 29]])
def test_many_experts_of_few_rows(counts, dtype, group, zeros, N, K):
    """So many of them that short rows are not streamed either: tiles with one or two rows on the tensor cores."""
    E, m = len(counts), sum(counts)
    with Weights(E, N, K, group, zeros, dtype, E) as w:
        assert not is_exact(w.h, m)
        x, ld = make_x(m, K, dtype, E)
        off = offsets_of(counts)
        out = torch.full((m + 1, N), -7.0, device="cuda", dtype=x.dtype)
        B.proj_w4_run_experts(w.h, x, ld, m, off, out, N)
        torch.cuda.synchronize()
        assert (out[m:] == -7.0).all()
        o = off.tolist()
        for e in range(E):
            if o[e] < o[e + 1]:
                rows = slice(o[e], o[e + 1])
                assert_close(out[rows], x[rows, :K].double(), w.w64(e), dtype, is_exact(w.h, m), K)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,group,zeros,N,K", [("bf16", 128, False, 40, 4200), ("fp16", 32, True, 270, 2050), ("bf16", 64, True, 129, 600)])
@pytest.mark.parametrize("counts", [[7], [0, 30, 0, 65, 1, 128, 0], [0, 0, 100], [40, 0, 0], [200, 1, 130, 0], [0, 900, 3]])
def test_experts_with_few_tiles_of_long_rows(counts, dtype, group, zeros, N, K):
    """K is split over clusters, some of which have no tile."""
    E, m = len(counts), sum(counts)
    with Weights(E, N, K, group, zeros, dtype, E + 1) as w:
        x, ld = make_x(m, K, dtype, E)
        off = offsets_of(counts)
        out, again = (torch.full((m + 1, N), -7.0, device="cuda", dtype=x.dtype) for _ in range(2))
        B.proj_w4_run_experts(w.h, x, ld, m, off, out, N)
        B.proj_w4_run_experts(w.h, x, ld, m, off, again, N)
        torch.cuda.synchronize()
        assert torch.equal(out, again) and (out[m:] == -7.0).all()
        o = off.tolist()
        for e in range(E):
            if o[e] < o[e + 1]:
                rows = slice(o[e], o[e + 1])
                assert_close(out[rows], x[rows, :K].double(), w.w64(e), dtype, is_exact(w.h, m), K)


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[40000] + [1, 0] * 511 + [3], [70000, 0, 1, 75000]])
def test_experts_with_more_token_tiles_than_the_table_holds(counts):
    E, m, N, K = len(counts), sum(counts), 17, 96
    with Weights(E, N, K, 32, False, "bf16", 6) as w:
        x, ld = make_x(m, K, "bf16", 6)
        off = offsets_of(counts)
        out = torch.full((m, N), -7.0, device="cuda", dtype=x.dtype)
        B.proj_w4_run_experts(w.h, x, ld, m, off, out, N)
        torch.cuda.synchronize()
        o = off.tolist()
        for e in [i for i in range(E) if counts[i] > 1] + [1, 3, 101]:
            if e < E and o[e] < o[e + 1]:
                rows = slice(o[e], o[e + 1])
                assert_close(out[rows], x[rows, :K].double(), w.w64(e), "bf16", is_exact(w.h, m), K)


@pytest.mark.gpu
def test_dependent_calls_back_to_back():
    """Each call's x is the call before's out, on one stream, across both kernels: the first loads that do not
    wait for the kernel before are the weights' only."""
    m, N = 40, 512
    with Weights(1, N, N, 64, False, "bf16", 12) as a, Weights(1, N, N, 128, True, "bf16", 13) as b:
        x = (torch.randn(m, N, device="cuda") * 0.1).bfloat16()
        bufs = [torch.zeros(m, N, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
        for rows in (m, 8):  # tensor cores, streamed
            for _ in range(5):
                src = x
                for i, w in enumerate((a, b, a, b)):
                    B.proj_w4_run(w.h, src, N, rows, bufs[i], N)
                    src = bufs[i]
            torch.cuda.synchronize()
            src = x
            for i, w in enumerate((a, b, a, b)):
                assert_close(bufs[i][:rows], src[:rows].double(), w.w64(0), "bf16", is_exact(w.h, rows), N)
                src = bufs[i]
