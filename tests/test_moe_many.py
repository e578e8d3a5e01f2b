"""The expert sort of so many tokens that every block's counts are not summed by every block."""
import pytest

torch = pytest.importorskip("torch")

from gemv_projection_layers_gb300 import binding as B


def sort_args(m, E, k, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    ids = torch.randint(-1, E, (m, k), device="cuda", generator=gen, dtype=torch.int32)
    new = lambda *s: torch.full(s, -99, device="cuda", dtype=torch.int32)  # noqa: E731
    room = torch.empty(max(16, B.proj_moe_workspace(m, E, k)), dtype=torch.uint8, device="cuda")
    return ids, (new(E + 1), new(m * k), new(m, k)), room


@pytest.mark.gpu
@pytest.mark.parametrize("m,E,k", [(2 ** 20, 1024, 8), (300000, 1024, 32), (2 ** 20 + 77, 256, 8), (400001, 700, 5)])
def test_sort_of_many_tokens(m, E, k):
    ids, (offsets, order, slot), room = sort_args(m, E, k, m)
    room.fill_(0xFF)
    B.proj_moe_sort(ids, m, E, k, offsets, order, slot, room, room.numel())
    torch.cuda.synchronize()
    flat = torch.where(ids < 0, E, ids).reshape(-1).long()
    ranked = torch.sort(flat, stable=True).indices
    ends = torch.cumsum(torch.bincount(flat, minlength=E + 1), 0)[:E]
    assert offsets[0] == 0 and torch.equal(offsets[1:].long(), ends)
    kept = int(ends[-1])
    assert torch.equal(order[:kept].long(), ranked[:kept]) and (order[kept:] == -1).all()
    want = torch.full_like(flat, -1)
    want[ranked[:kept]] = torch.arange(kept, device="cuda")
    assert torch.equal(slot.reshape(-1).long(), want)


@pytest.mark.gpu
def test_time_of_the_sort_grows_with_the_tokens():
    """Four times the tokens take four times as long, give or take; with the square of them it would be sixteen."""
    def best(m, E=1024, k=8):
        ids, out, room = sort_args(m, E, k, 1)
        times = []
        for _ in range(8):
            start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            B.proj_moe_sort(ids, m, E, k, *out, room, room.numel())
            stop.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(stop))
        return min(times[2:])

    assert best(2 ** 20) <= 8 * best(2 ** 18)
