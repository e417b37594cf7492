"""qmm_page_plan against a host loop over requests and tokens: exact."""
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from paged_util import i32, pages  # noqa: E402

@pytest.fixture(autouse=True)
def clear_what_earlier_calls_left():
    """The device error word holds what any earlier call reported until it is read."""
    qmm.qmm_get_device_error()


def plan(past, new, page, free, first=None, width=None, extra=0, room=None, seed=0):
    """The call on a table whose held entries are distinct ids, and the loop's result."""
    rng = random.Random(seed)
    width = width or max([pages(max(p, 0) + max(n, 0), page) for p, n in zip(past, new)] + [1]) + 2
    ids = rng.sample(range(1000, 1000 + 4 * len(past) * width + 1), len(past) * width)
    table = [[ids[b * width + j] if j < pages(max(p, 0), page) else -7 for j in range(width)]
             for b, p in enumerate(past)]
    room = sum(max(n, 0) for n in new) + extra if room is None else room
    t = {"table": i32(table).reshape(len(past), width), "starts": i32([99] * (len(past) + 1)),
         "seq": i32([99] * len(past)), "positions": i32([99] * room), "slots": i32([99] * room),
         "next_out": i32([99])}
    args = (i32(past), i32(new), i32(free), i32([first]) if first is not None else None)
    qmm.qmm_page_plan(args[0], args[1], len(past), args[2], len(free), args[3], page, t["table"], width,
                      room, t["starts"], t["seq"], t["positions"], t["slots"], t["next_out"])
    got = {k: v.cpu().tolist() for k, v in t.items()}
    want = {"starts": [0], "seq": [], "positions": [], "slots": []}
    at, bad = max(first or 0, 0), (first or 0) < 0
    for b, (p, n) in enumerate(zip(past, new)):
        bad |= p < 0 or n < 0
        p, n = max(p, 0), max(n, 0)
        if p + n > width * page:
            bad = True
            p = min(p, width * page)
            n = width * page - p
        for j in range(pages(p, page), pages(p + n, page)):
            table[b][j] = free[at] if at < len(free) else -1
            at += 1
        for i in range(n):
            pos = p + i
            pid = table[b][pos // page]
            bad |= pid < 0
            want["positions"].append(pos)
            want["slots"].append(pid * page + pos % page if pid >= 0 else -1)
        want["starts"].append(want["starts"][-1] + n)
        want["seq"].append(p + n)
    bad |= want["starts"][-1] > room
    want["starts"] = [min(s, room) for s in want["starts"]]
    want["positions"] = (want["positions"] + [0] * room)[:room]
    want["slots"] = (want["slots"] + [-1] * room)[:room]
    want["table"], want["next_out"] = table, [max(max(first or 0, 0), min(at, len(free)))]
    for k in want:
        assert got[k] == want[k], k
    return qmm.QMM_ERR_INDEX if bad else qmm.QMM_OK


@pytest.mark.parametrize("page", [1, 7, 16, 24, 256])
@pytest.mark.parametrize("requests,most_past,most_new", [
    (1, 0, 1), (1, 5000, 1), (3, 100, 700), (511, 300, 1), (512, 300, 2), (513, 300, 3), (1500, 60, 9)])
def test_plans(page, requests, most_past, most_new):
    rng = random.Random(requests + page)
    past = [rng.randint(0, most_past) for _ in range(requests)]
    new = [rng.randint(0, most_new) for _ in range(requests)]
    free = list(range(10 ** 5, 10 ** 5 + 3 + sum(pages(a + b, page) for a, b in zip(past, new))))
    rng.shuffle(free)
    assert plan(past, new, page, free, rng.choice([None, 0, 2]), extra=rng.choice([0, 5])) == qmm.QMM_OK
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def test_whole_pages_and_their_ends():
    for past, new in [(16, 16), (15, 1), (15, 2), (0, 0), (32, 0), (31, 33), (0, 16), (0, 17)]:
        assert plan([past, 3], [new, 1], 16, list(range(50, 60))) == qmm.QMM_OK


def test_no_requests():
    assert plan([], [], 16, [1], extra=3) == qmm.QMM_OK


@pytest.mark.parametrize("past,new,free,kw", [
    ([0, 10], [40, 30], [5, 6, 7], {}),                    # the free list runs out
    ([0, 10], [4, 30], [], {}),
    ([4, -3], [2, 5], [5, 6, 7], {}),                      # a negative length
    ([4, 3], [-2, 5], [5, 6, 7], {}),
    ([4, 3], [2, 5], [5, 6, 7], {"first": -4}),
    ([30, 3], [40, 5], [5, 6, 7, 8, 9], {"width": 3}),     # a request outgrows its row
    ([100, 3], [1, 5], [5, 6, 7, 8, 9], {"width": 3}),
    ([4, 3], [20, 50], list(range(9)), {"room": 33}),      # tokens outgrow their room
    ([4, 3], [20, 50], list(range(9)), {"room": 10}),
])
def test_what_does_not_fit_is_cut_and_reported(past, new, free, kw):
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    assert plan(past, new, 16, free, **kw) == qmm.QMM_ERR_INDEX
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def test_slots_past_31_bits_are_refused():
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    t = [i32([0] * n) for n in (2, 1, 2, 2, 1)]
    qmm.qmm_page_plan(i32([0]), i32([2]), 1, i32([2 ** 30]), 1, None, 4, i32([[0, 0]]), 2, 2, t[0], t[1],
                      t[2], t[3], t[4])
    assert t[3].tolist() == [-1, -1]
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
