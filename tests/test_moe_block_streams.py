"""examples/moe_block.py: every step of the block on one stream, and no more than its buffers hold."""
import contextlib
import importlib.util

import pytest

torch = pytest.importorskip("torch")

from test_moe_block import PATH

from gemv_projection_layers_gb300 import binding as B


def example():
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


class Library:
    """Stands for the binding: notes which call went to which stream."""

    def __init__(self, seen):
        self.seen = seen

    def __getattr__(self, name):
        if name.startswith("PROJ_"):
            return getattr(B, name)
        if name == "norm_args":
            return dict
        return lambda *a: self.seen.append((name, a[-1]))


class Current:
    """torch's current stream, with no device."""

    def __init__(self, monkeypatch, first):
        self.stream = first
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.stream)
        monkeypatch.setattr(torch.cuda, "stream", self.change)

    @contextlib.contextmanager
    def change(self, stream):
        before, self.stream = self.stream, stream
        yield
        self.stream = before


def block_without_device(ex, tokens):
    block = object.__new__(ex.MoeBlock)
    block.k, block.inner, block.tokens = 2, 4, tokens
    rows = tokens * block.k
    for name in ("router", "up", "down"):
        setattr(block, name, 1)
    for name in ("w_in", "w_post", "w_next", "gate", "logits", "weight", "expert", "slot", "order", "offsets", "xs", "ys", "room"):
        setattr(block, name, torch.zeros(1))
    block.h, block.y, block.out, block.next = (torch.zeros(tokens, ex.HIDDEN) for _ in range(4))
    block.mid, block.act = torch.zeros(rows, 8), torch.zeros(rows, 4)
    return block


@pytest.mark.parametrize("given", ["side", None])
def test_every_step_on_one_stream(given, monkeypatch):
    ex, seen = example(), []
    monkeypatch.setattr(ex, "B", Library(seen))
    current = Current(monkeypatch, "current")
    silu = torch.nn.functional.silu
    monkeypatch.setattr(torch.nn.functional, "silu", lambda x: (seen.append(("silu", current.stream)), silu(x))[1])
    block_without_device(ex, 3)(torch.zeros(3, ex.HIDDEN), given)
    assert len(seen) == 9
    assert {stream for _, stream in seen} == {given or "current"}, seen
    assert current.stream == "current"


@pytest.mark.parametrize("rows,width", [(4, 0), (3, -8), (3, 8)])
def test_a_residual_that_does_not_fit_is_refused(rows, width, monkeypatch):
    """Before any step: the calls would run past the block's buffers or the residual's."""
    ex, seen = example(), []
    monkeypatch.setattr(ex, "B", Library(seen))
    Current(monkeypatch, "current")
    block = block_without_device(ex, 3)
    with pytest.raises(ValueError):
        block(torch.zeros(rows, ex.HIDDEN + width))
    with pytest.raises(ValueError):
        block(torch.zeros(3, 2 * ex.HIDDEN)[:, ::2])
    assert not seen


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["given", "current"])
def test_a_side_stream_gives_the_same(where):
    ex = example()
    m = 300
    block = ex.MoeBlock(m, inner=128, k=4, group=64, seed=1)
    try:
        residual = torch.randn(m, ex.HIDDEN, device="cuda").bfloat16()
        want = [t.clone() for t in block(residual)]
        for _ in range(20):
            block.mid.fill_(float("nan"))
            block.act.fill_(float("nan"))
            torch.cuda.synchronize()
            side = torch.cuda.Stream()
            if where == "given":
                got = block(residual, side)
            else:
                with torch.cuda.stream(side):
                    got = block(residual)
            side.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    finally:
        block.close()
