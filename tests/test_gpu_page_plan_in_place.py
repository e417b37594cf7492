"""qmm_page_plan with seq_lens in past_lens' place: what separate arrays give, with one
block of tokens and with many."""
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from paged_util import i32, pages  # noqa: E402


def plan(past, new, page, free, width, table, in_place):
    b, t = len(past), sum(new)
    lens = i32(past)
    got = {"table": table.clone(), "starts": i32([9] * (b + 1)), "seq": lens if in_place else i32([9] * b),
           "positions": i32([9] * t), "slots": i32([9] * t), "next": i32([9])}
    qmm.qmm_page_plan(lens, i32(new), b, free, free.numel(), None, page, got["table"], width, t, got["starts"],
                      got["seq"], got["positions"], got["slots"], got["next"])
    return got


@pytest.mark.parametrize("requests,most_past,most_new", [
    (5, 300, 20), (300, 90, 1), (700, 4000, 1), (64, 500, 600), (1500, 60, 40), (3, 0, 90000)])
def test_lengths_in_place(requests, most_past, most_new):
    rng = random.Random(requests)
    page = 16
    past = [rng.randint(0, most_past) for _ in range(requests)]
    new = [rng.randint(0, most_new) for _ in range(requests)]
    held, need = [pages(p, page) for p in past], [pages(p + n, page) - pages(p, page) for p, n in zip(past, new)]
    width = max(a + b for a, b in zip(held, need)) + 1
    ids = rng.sample(range(10 ** 6), sum(held) + sum(need))
    table = [[-7] * width for _ in past]
    for row, n in zip(table, held):
        for j in range(n):
            row[j] = ids.pop()
    table, free = i32(table), i32(ids + [1])
    apart = plan(past, new, page, free, width, table, False)
    assert apart["seq"].tolist() == [p + n for p, n in zip(past, new)]
    assert apart["positions"].tolist() == [p + i for p, n in zip(past, new) for i in range(n)]
    for _ in range(10):
        got = plan(past, new, page, free, width, table, True)
        for k in apart:
            assert torch.equal(got[k], apart[k]), k
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def test_a_captured_step_moves_on_by_itself():
    """The lengths and the free list's count pass through one graph, replayed for 40 steps."""
    b, page, steps = 600, 8, 40
    width = pages(b % 7 + 7 + steps, page) + 2
    past = [x % 7 for x in range(b)]
    lens, new, table = i32(past), i32([1] * b), torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(b, device="cuda")
    free, count, moved = torch.arange(b, b * width, dtype=torch.int32, device="cuda"), i32([0]), i32([0])
    starts, positions, slots = i32([0] * (b + 1)), i32([0] * b), i32([0] * b)
    # A request of length 0 holds no page; its first entry is taken at the first step.
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        qmm.qmm_page_plan(lens, new, b, free, free.numel(), count, page, table, width, b, starts, lens, positions,
                          slots, moved)
        count.copy_(moved)
    for step in range(steps):
        graph.replay()
        want = torch.tensor([p + step for p in past], device="cuda", dtype=torch.int32)
        assert torch.equal(positions, want) and torch.equal(lens, want + 1)
        rows = torch.arange(b, device="cuda")
        assert torch.equal(slots, table[rows, (want // page).long()] * page + want % page)
    held = [pages(n, page) for n in lens.tolist()]
    ids = [i for row, n in zip(table.tolist(), held) for i in row[:n]]
    assert len(set(ids)) == len(ids) and int(count) == sum(held) - sum(p > 0 for p in past)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
