"""The norms at a block's ends and their gradients against the definition in 64 bits.

Bounds, element by element: u |ref| for the output's own rounding, plus C 2^-23 of the sum of the
sizes of the terms that make it up.  C = 64 for a row's values (chains of at most 16 terms a thread
and a tree of 10 in each of the two sums, their square roots, and under 20 roundings per element),
128 for sums over tokens, whose chains are longer.
"""
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B
from gemv_projection_layers_gb300 import build as libbuild

DT = {"bf16": (torch.bfloat16, B.PROJ_BF16, 2.0 ** -8), "fp16": (torch.float16, B.PROJ_FP16, 2.0 ** -11),
      "fp32": (torch.float32, B.PROJ_FP32, 2.0 ** -24)}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 0.0}
EPS, ALPHA, BETA = 1e-5, 0.7, -1.3
Cr, Cc = 64 * 2.0 ** -23, 128 * 2.0 ** -23


class Case:
    """Inputs with their own strides; what must not be read is NaN."""

    def __init__(self, m, D, dtype, gate, act, seed, extra=0, plain=False, no_y=False, no_w=False, zero_row=True):
        self.m, self.D, self.dtype, self.gate_mode, self.act = m, D, dtype, gate, act
        self.plain, self.no_y, self.ld = plain, no_y, D + extra
        gen = torch.Generator("cuda").manual_seed(seed)
        t = DT[dtype][0]

        def mat(scale=1.0):
            buf = torch.full((m + 1, self.ld), float("nan"), device="cuda", dtype=t)
            buf[:m, :D] = (torch.randn(m, D, device="cuda", generator=gen) * scale).to(t)
            return buf

        vec = lambda: (1 + 0.3 * torch.randn(D, device="cuda", generator=gen)).to(t)  # noqa: E731
        self.y, self.r, self.dout, self.dh = (None if no_y else mat(3.0)), mat(), mat(), mat()
        if m > 2 and not no_y and zero_row:
            self.y[1, :D] = 0  # a row of zeros
        self.gate = [lambda: None, vec, mat, lambda: torch.randn(m, device="cuda", generator=gen).to(t)][gate]()
        self.w_post = None if no_w or plain or no_y else vec()
        self.w_pre = None if no_w else vec()

    def named(self):
        return dict(m=self.m, D=self.D, dtype=DT[self.dtype][1], gate_mode=self.gate_mode, gate_act=self.act, y_plain=int(self.plain),
                    eps=EPS, alpha=ALPHA, beta=BETA, y=self.y, ldy=self.ld, residual=self.r, ldr=self.ld, gate=self.gate,
                    ldg=self.ld, w_post=self.w_post, w_pre=self.w_pre)

    def leaves(self):
        m, D = self.m, self.D
        d = {"residual": self.r[:m, :D].double()}
        if self.y is not None:
            d["y"] = self.y[:m, :D].double()
        for n in ("w_post", "w_pre"):
            if getattr(self, n) is not None:
                d[n] = getattr(self, n).double()
        if self.gate is not None:
            d["gate"] = (self.gate[:m, :D] if self.gate_mode == 2 else self.gate).double()
        return d

    def forward64(self, d):
        """out, normed, the rsqrt factors and the sizes of out's terms."""
        # the scalars are the call's fp32 values
        eps, alpha, beta = (float(torch.tensor(v, dtype=torch.float32)) for v in (EPS, ALPHA, BETA))
        u, size, rp = alpha * d["residual"], (alpha * d["residual"]).abs(), None
        if "y" in d:
            n = d["y"]
            if not self.plain:
                rp = (d["y"].pow(2).mean(1) + eps).rsqrt()
                n = d["y"] * rp[:, None]
                if "w_post" in d:
                    n = n * d["w_post"]
            if self.gate_mode:
                g = torch.sigmoid(d["gate"]) if self.act else d["gate"]
                n = n * (g[:, None] if self.gate_mode == 3 else g)
            u, size = u + beta * n, size + (beta * n).abs()
        ru = (u.pow(2).mean(1) + eps).rsqrt()
        h = u * ru[:, None]
        if "w_pre" in d:
            h = h * d["w_pre"]
        return u, h, rp, ru, size


def near(got, ref, u, tiny, size, C):
    err = (got.double() - ref).abs()
    tol = u * ref.abs() + tiny + C * size
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), (err - tol).max().item()


GRID = [(1, 1, 0), (1, 8, 0), (2, 7, 1), (5, 64, 0), (3, 513, 0), (33, 512, 0), (4, 1000, 8), (17, 2048, 3), (2, 4100, 0), (3, 8192, 0),
        (2, 8200, 8), (2, 16384, 0), (1, 16383, 0), (700, 96, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,D,extra", GRID)
def test_forward(m, D, extra, dtype):
    t, _, u = DT[dtype]
    for gate in range(4):
        c = Case(m, D, dtype, gate, (m + gate) % 2, D + gate, extra, no_w=gate == 3 and m % 2 == 0)
        out, normed = (torch.full((m + 1, c.ld), -7.0, device="cuda", dtype=t) for _ in range(2))
        rp, ru = (torch.full((m + 1,), -7.0, device="cuda") for _ in range(2))
        B.proj_norm(B.norm_args(**c.named(), out=out, ldo=c.ld, normed=normed, ldn=c.ld, rstd_post=rp, rstd_pre=ru))
        torch.cuda.synchronize()
        v, h, rp64, ru64, size = c.forward64(c.leaves())
        wide = ru64[:, None] * size * (c.w_pre.double().abs() if c.w_pre is not None else 1.0)
        # the factor's relative error is that of the sum under the root, whose terms grow with out's
        spread = (size.pow(2).mean(1, keepdim=True) * ru64[:, None].pow(2)).clamp(min=1.0)
        near(out[:m, :D], v, u, TINY[dtype], size, Cr)
        near(normed[:m, :D], h, u, TINY[dtype], wide * spread, Cr)
        near(rp[:m], rp64, 0, 0, rp64, Cr)
        near(ru[:m], ru64, 0, 0, ru64 * spread[:, 0], Cr)
        assert (out[m:] == -7.0).all() and (out[:, D:] == -7.0).all() and (normed[m:] == -7.0).all() and (normed[:, D:] == -7.0).all()
        assert rp[m] == -7.0 and ru[m] == -7.0


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["no block", "plain", "plain gated", "only out", "only normed", "in place"])
@pytest.mark.parametrize("m,D", [(3, 256), (2, 333), (5, 8192)])
def test_forward_forms(m, D, form):
    c = Case(m, D, "bf16", 2 if form == "plain gated" else 0, 1, 11, no_y=form == "no block", plain=form.startswith("plain"))
    v, h, _, ru64, size = c.forward64(c.leaves())
    wide = ru64[:, None] * size * c.w_pre.double().abs()
    spread = (size.pow(2).mean(1, keepdim=True) * ru64[:, None].pow(2)).clamp(min=1.0)
    u = DT["bf16"][2]
    if form == "in place":
        B.proj_norm(B.norm_args(**c.named(), out=c.r, ldo=c.ld, normed=c.y, ldn=c.ld))
        out, normed = c.r, c.y
    else:
        out, normed = (torch.empty(m, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        B.proj_norm(B.norm_args(**c.named(), out=None if form == "only normed" else out, ldo=D,
                                normed=None if form == "only out" else normed, ldn=D))
    torch.cuda.synchronize()
    if form != "only normed":
        near(out[:m, :D], v, u, 0, size, Cr)
    if form != "only out":
        near(normed[:m, :D], h, u, 0, wide * spread, Cr)


def backward(c, want_dout=True, want_dh=True):
    m, D, t = c.m, c.D, DT[c.dtype][0]
    v, h, rp, ru, size = c.forward64(c.leaves())
    new = lambda: torch.full((m + 1, c.ld), -7.0, device="cuda", dtype=t)  # noqa: E731
    col = lambda: torch.full((D + 1,), -7.0, device="cuda")  # noqa: E731
    got = {"dresidual": new()}
    if c.y is not None:
        got["dy"] = new()
    if c.w_post is not None:
        got["dw_post"] = col()
    if c.w_pre is not None and want_dh:
        got["dw_pre"] = col()
    if c.gate is not None:
        got["dgate"] = [None, col, new, lambda: torch.full((m + 1,), -7.0, device="cuda", dtype=t)][c.gate_mode]()
    room = torch.full((max(16, B.proj_norm_workspace(m, D)),), 0xFF, device="cuda", dtype=torch.uint8)
    args = B.norm_grad_args(**c.named(), **got, rstd_post=None if rp is None else rp.float(), rstd_pre=ru.float(),
                            dout=c.dout if want_dout else None, lddo=c.ld, dnormed=c.dh if want_dh else None, lddn=c.ld, lddy=c.ld,
                            lddr=c.ld, lddg=c.ld, workspace=room, workspace_bytes=room.numel())
    B.proj_norm_backward(args)
    first = {n: g.clone() for n, g in got.items()}
    B.proj_norm_backward(args)  # sums in a fixed order: the same bits again
    torch.cuda.synchronize()
    for n in got:
        assert torch.equal(got[n], first[n]), n
        if got[n].dim() == 2:
            assert (got[n][m:] == -7.0).all() and (got[n][:, D:] == -7.0).all()
            got[n] = got[n][:m, :D]
        else:
            assert got[n][-1] == -7.0
            got[n] = got[n][:-1]
    return got, room


def grads64(c, want_dout=True, want_dh=True):
    """Autograd of the definition, and sizes of the terms of each gradient."""
    m, D = c.m, c.D
    alpha, beta = (float(torch.tensor(v, dtype=torch.float32)) for v in (ALPHA, BETA))
    d = {n: v.clone().requires_grad_() for n, v in c.leaves().items()}
    v, h, rp, ru, size = c.forward64(d)
    zero = torch.zeros_like(v)
    dout = c.dout[:m, :D].double() if want_dout else zero
    dh = c.dh[:m, :D].double() if want_dh else zero
    ref = dict(zip(d, torch.autograd.grad([v, h], list(d.values()), [dout, dh], allow_unused=True)))
    with torch.no_grad():
        w_pre = d["w_pre"].abs() if "w_pre" in d else 1.0
        un = size * ru[:, None]  # terms of u ru
        tt = (dh * w_pre).abs() if want_dh else zero
        spread = (size.pow(2).mean(1, keepdim=True) * ru[:, None].pow(2)).clamp(min=1.0)
        du = dout.abs() + ru[:, None] * (tt + un * (tt * un).mean(1, keepdim=True)) * spread
        sizes = {"residual": abs(alpha) * du, "w_pre": (dh.abs() * un * spread).sum(0)}
        if "y" in d:
            g = torch.ones_like(v)
            slope = g
            if c.gate_mode:
                raw = torch.sigmoid(d["gate"]) if c.act else d["gate"]
                sl = raw * (1 - raw) if c.act else torch.ones_like(raw)
                fit = (lambda a: a[:, None].expand_as(v)) if c.gate_mode == 3 else (lambda a: a.expand_as(v))
                g, slope = fit(raw).abs(), fit(sl).abs()
            yn = d["y"].abs() * (rp[:, None] if rp is not None else 1.0)
            w_post = d["w_post"].abs() if "w_post" in d else 1.0
            cc = abs(beta) * g * du
            b = cc * w_post
            sizes["y"] = rp[:, None] * (b + yn * (b * yn).mean(1, keepdim=True)) if rp is not None else cc
            sizes["w_post"] = (cc * yn).sum(0)
            dg = abs(beta) * yn * w_post * du * (slope + (g if c.act else 0))
            sizes["gate"] = {0: None, 1: dg.sum(0), 2: dg, 3: dg.sum(1)}[c.gate_mode]
    return ref, sizes


NAMES = {"dy": "y", "dresidual": "residual", "dw_post": "w_post", "dw_pre": "w_pre", "dgate": "gate"}


def check_backward(c, **want):
    got, _ = backward(c, **want)
    ref, sizes = grads64(c, **want)
    for n, g in got.items():
        u = DT[c.dtype][2] if g.dtype != torch.float32 else 2.0 ** -24
        tiny = TINY[c.dtype] if g.dtype == torch.float16 else 0.0
        r = ref[NAMES[n]]
        near(g, torch.zeros_like(sizes[NAMES[n]]) if r is None else r, u, tiny, sizes[NAMES[n]], Cc if g.dim() == 1 else Cr)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,D,extra", GRID)
def test_backward(m, D, extra, dtype):
    for gate in range(4):
        check_backward(Case(m, D, dtype, gate, (m + gate) % 2, D + gate, extra, no_w=gate == 3 and m % 2 == 0))


# More rows than are on the GPU at a time, so that the rows ahead go around their room: a warp a row, four
# warps, eight and sixteen; rows on and off 16 bytes.
MANY = [(6000, 40, 0), (5000, 301, 0), (5200, 512, 0), (2000, 776, 8), (1300, 1025, 0), (1000, 2050, 6), (500, 6000, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,D,extra", MANY)
def test_forward_many_rows(m, D, extra, dtype):
    test_forward(m, D, extra, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m,D,extra", MANY)
def test_backward_many_rows(m, D, extra, dtype):
    """Sums over tokens: a few rows a thread, at most 4 + 19 + 32 partial sums, and the 64 of a row's values."""
    for gate in (1, 2, 3):
        check_backward(Case(m, D, dtype, gate, gate % 2, D + gate, extra))


@pytest.mark.gpu
@pytest.mark.parametrize("form", ["no block", "plain", "plain gated", "plain token", "no dout", "no dnormed"])
@pytest.mark.parametrize("m,D", [(3, 256), (2, 333), (5, 8192)])
def test_backward_forms(m, D, form):
    gate = {"plain gated": 2, "plain token": 3, "no dout": 1, "no dnormed": 3}.get(form, 0)
    c = Case(m, D, "bf16", gate, 1, 11, no_y=form == "no block", plain=form.startswith("plain"))
    check_backward(c, want_dout=form != "no dout", want_dh=form != "no dnormed")


@pytest.mark.gpu
@pytest.mark.parametrize("gate,act", [(0, 0), (1, 1), (2, 1), (2, 0), (3, 1)])
def test_backward_against_differences(gate, act):
    """Central differences of the forward kernel itself, along a random direction of every input."""
    m, D, h = 6, 200, 2.0 ** -6
    c = Case(m, D, "fp32", gate, act, 21, zero_row=False)  # no step is small at sqrt(eps)
    got, _ = backward(c)
    ref, sizes = grads64(c)
    d = c.leaves()
    gen = torch.Generator("cuda").manual_seed(5)
    way = {n: torch.randn(v.shape, device="cuda", generator=gen).double() for n, v in d.items()}
    c1, c2 = c.dout[:m, :D].double(), c.dh[:m, :D].double()

    def both(sign):
        """The loss from the kernel's outputs and from 64 bits, and the size of its terms."""
        moved = {n: (v + sign * h * way[n]).float() for n, v in d.items()}
        k = Case(m, D, "fp32", gate, act, 21, zero_row=False)
        k.y[:m, :D], k.r[:m, :D], k.w_post[:], k.w_pre[:] = moved["y"], moved["residual"], moved["w_post"], moved["w_pre"]
        if gate == 2:
            k.gate[:m, :D] = moved["gate"]
        elif gate:
            k.gate[:] = moved["gate"]
        out, normed = (torch.empty(m, D, device="cuda") for _ in range(2))
        B.proj_norm(B.norm_args(**k.named(), out=out, ldo=D, normed=normed, ldn=D))
        torch.cuda.synchronize()
        v, hh, _, ru, size = k.forward64(k.leaves())
        spread = (size.pow(2).mean(1, keepdim=True) * ru[:, None].pow(2)).clamp(min=1.0)
        terms = (c1.abs() * size).sum() + (c2.abs() * size * ru[:, None] * k.w_pre.double().abs() * spread).sum()
        return (c1 * out.double()).sum() + (c2 * normed.double()).sum(), (c1 * v).sum() + (c2 * hh).sum(), terms

    up, up64, su = both(1)
    down, down64, sd = both(-1)
    slope = sum((got[n].double() * way[NAMES[n]]).sum() for n in got)
    slope64 = sum((ref[n] * way[n]).sum() for n in ref)
    truncation = abs((up64 - down64) / (2 * h) - slope64)
    rounding = Cr * (su + sd) / (2 * h) + sum((Cc * sizes[n] * way[n].abs()).sum() for n in ref)
    assert abs((up - down) / (2 * h) - slope) <= truncation + rounding
    assert truncation <= 0.05 * sum((ref[n].abs() * way[n].abs()).sum() for n in ref)  # the step is small enough to say something


@pytest.mark.gpu
def test_no_rows():
    D = 64
    cols = [torch.full((D,), -7.0, device="cuda") for _ in range(3)]
    B.proj_norm(B.norm_args(m=0, D=D, ldr=D, out=None, eps=EPS))
    B.proj_norm_backward(B.norm_grad_args(m=0, D=D, ldr=D, eps=EPS, gate_mode=B.PROJ_GATE_CHANNEL, dw_post=cols[0], dw_pre=cols[1],
                                          dgate=cols[2]))
    torch.cuda.synchronize()
    assert all((c == 0).all() for c in cols)


def test_refusals_before_any_device_call():
    libbuild.build()
    lib = B.load()

    def code(fn, make, base, **change):
        try:
            fn(make(**{**base, **change}))
        except B.ProjError as e:
            assert B.last_cuda_error().startswith("proj_norm")
            return e.status
        raise AssertionError(f"not refused: {change}")

    base = dict(m=4, D=8, dtype=0, eps=EPS, y=16, ldy=8, residual=16, ldr=8, w_post=16, w_pre=16, out=16, ldo=8, normed=32, ldn=8)
    f = lambda **c: code(B.proj_norm, B.norm_args, base, **c)  # noqa: E731
    gbase = dict(m=4, D=8, dtype=0, eps=EPS, y=16, ldy=8, residual=16, ldr=8, w_post=16, w_pre=16, rstd_post=16, rstd_pre=16, dout=16,
                 lddo=8, dnormed=16, lddn=8, dy=32, lddy=8, dresidual=32, lddr=8, dw_post=32, dw_pre=32, workspace=64,
                 workspace_bytes=1 << 30)
    g = lambda **c: code(B.proj_norm_backward, B.norm_grad_args, gbase, **c)  # noqa: E731
    for both in (f, g):
        assert both(m=-1) == B.PROJ_EINVAL
        assert both(D=0) == B.PROJ_EINVAL
        assert both(dtype=3) == B.PROJ_EINVAL
        assert both(gate_mode=4) == B.PROJ_EINVAL
        assert both(gate_mode=1) == B.PROJ_EINVAL  # no gate given
        assert both(gate=16) == B.PROJ_EINVAL  # gate without a mode
        assert both(gate_act=2, gate=16, gate_mode=1) == B.PROJ_EINVAL
        assert both(y_plain=2) == B.PROJ_EINVAL
        assert both(y_plain=1) == B.PROJ_EINVAL  # with w_post
        assert both(y=None) == B.PROJ_EINVAL  # with w_post
        assert both(eps=-1.0) == B.PROJ_EINVAL
        assert both(eps=float("nan")) == B.PROJ_EINVAL
        assert both(residual=None) == B.PROJ_EINVAL
        assert both(ldy=7) == B.PROJ_EINVAL
        assert both(ldr=7) == B.PROJ_EINVAL
        assert both(gate_mode=2, gate=16, ldg=7) == B.PROJ_EINVAL
        assert both(m=2 ** 31) == B.PROJ_EUNSUPPORTED
        assert both(y=17) == B.PROJ_EALIGN
        assert both(w_pre=17) == B.PROJ_EALIGN
        assert both(rstd_pre=18) == B.PROJ_EALIGN
    big = dict(D=16385, ldy=16385, ldr=16385)
    assert f(**big, ldo=16385, ldn=16385) == B.PROJ_EUNSUPPORTED
    assert g(**big, lddo=16385, lddn=16385, lddy=16385, lddr=16385) == B.PROJ_EUNSUPPORTED
    assert f(out=None, normed=None) == B.PROJ_EINVAL
    assert f(ldo=7) == B.PROJ_EINVAL
    assert f(ldn=7) == B.PROJ_EINVAL
    assert f(out=17) == B.PROJ_EALIGN
    assert g(dout=None, dnormed=None) == B.PROJ_EINVAL
    assert g(rstd_post=None) == B.PROJ_EINVAL
    assert g(rstd_pre=None) == B.PROJ_EINVAL
    assert g(dgate=16) == B.PROJ_EINVAL
    assert g(lddy=7) == B.PROJ_EINVAL
    assert g(lddr=7) == B.PROJ_EINVAL
    assert g(workspace=None) == B.PROJ_EINVAL
    assert g(workspace_bytes=16) == B.PROJ_EINVAL
    assert g(workspace=8) == B.PROJ_EALIGN
    assert g(dw_post=18) == B.PROJ_EALIGN
    assert g(dy=17) == B.PROJ_EALIGN
    assert lib.proj_norm(None, None) == B.PROJ_EINVAL
    assert lib.proj_norm_backward(None, None) == B.PROJ_EINVAL
    assert lib.proj_norm_workspace(-1, 8) == -1
    assert lib.proj_norm_workspace(1, 16385) == -1
    with pytest.raises(TypeError):
        B.norm_args(nonsense=1)
