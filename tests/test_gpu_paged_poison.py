"""qmm_paged_attention over keys and values that are not finite where rows see them:
what comes out, and that it costs what a clean call costs."""
import math
import statistics

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from paged_util import TYPES, Pool, attend, queries  # noqa: E402


@pytest.fixture(autouse=True)
def clear_what_earlier_calls_left():
    """The device error word holds what any earlier call reported until it is read."""
    qmm.qmm_get_device_error()


def setup(lens, group, dim, dtype):
    pool = Pool([a + b for a, b in lens], 16, 2, dim, dtype, seed=3)
    news = [b for _, b in lens]
    return pool, queries(pool, sum(news), 2 * group, 4), news


def micros(call):
    times = []
    for _ in range(4):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        call()
        end.record()
        end.synchronize()
        times.append(1000 * start.elapsed_time(end))
    return statistics.median(times[1:])


# Few rows: one long cache in many pieces; whole items.  Many rows: pieces, whole items.
SHAPES = {"long": [(60000, 1)], "many": [(900, 1)] * 200, "chunk": [(20000, 64)], "prompts": [(0, 700)] * 12}


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64), ("f32", 64), ("bf16", 256)])
@pytest.mark.parametrize("shape", sorted(SHAPES))
@pytest.mark.parametrize("what", ["q", "k"])
def test_a_row_whose_scores_are_not_finite_costs_what_others_cost(dtype, dim, shape, what):
    """A row that sees a NaN score is NaN, and nothing is done for it again: one warp that
    walked all of the row's keys took 130 ms over the long cache, 2.6 ms over the many.
    The bound, three times the clean call's time, is far from either."""
    lens = SHAPES[shape]
    pool, q, news = setup(lens, 4, dim, dtype)
    call = lambda: attend(pool, q, news, 8, dim ** -0.5)  # noqa: E731
    clean, clean_lse = call()
    before = micros(call)
    if what == "q":
        q[-1, 0, 0] = math.nan  # head 0 of the last token
    else:
        page, row = pool.place(len(lens) - 1, 5)
        pool.k[page, 0, row, dim - 1] = math.nan  # key 5 of the last request's first key head
    out, lse = call()
    after = micros(call)
    gone = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    if what == "q":
        gone[-1, 0] = True
    else:
        past, new = lens[-1]
        gone[sum(news) - new + max(0, 5 - past):, :4] = True
    assert out[gone].isnan().all() and lse[gone].isnan().all()
    assert torch.equal(out[~gone], clean[~gone]) and torch.equal(lse[~gone], clean_lse[~gone])
    assert after <= 3 * before + 50, "%.0f us against %.0f" % (after, before)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 64), ("f32", 64), ("bf16", 256)])
@pytest.mark.parametrize("shape", sorted(SHAPES))
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_a_value_that_is_not_finite_where_rows_see_it_costs_little(dtype, dim, shape, value):
    """V of key 5 of the last request's first head is not finite in one column, every
    score is: the rows that see it are not finite there, of themselves, and only the few
    that do not see it beside those that do are done again.  With all of them it took 130
    ms over the long cache, 24 ms for the prompts (0.45 now).  The bound is ten times the clean call's time, for prompts whose
    rows each look over their item's other keys."""
    lens = SHAPES[shape]
    pool, q, news = setup(lens, 4, dim, dtype)
    scale = 0.3 * dim ** -0.5
    call = lambda: attend(pool, q, news, 8, scale)  # noqa: E731
    clean, clean_lse = call()
    before = micros(call)
    page, row = pool.place(len(lens) - 1, 5)
    pool.v[page, 0, row, dim // 2] = value
    out, lse = call()
    after = micros(call)
    hit = torch.zeros_like(out, dtype=torch.bool)
    past, new = lens[-1]
    hit[sum(news) - new + max(0, 5 - past):, :4, dim // 2] = True
    assert (out[hit].isnan() if math.isnan(value) else out[hit] == value).all()
    assert torch.equal(lse, clean_lse)
    bound = (3 * TYPES[dtype][2] + (past + new) * 2.0 ** -23 + 2.0 ** -13) * max(
        float(v[v.isfinite()].abs().max()) for v in pool.values)
    assert (out[~hit].double() - clean[~hit].double()).abs().max() <= bound
    assert after <= 10 * before + 50, "%.0f us against %.0f" % (after, before)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f32", 64), ("bf16", 24)])
@pytest.mark.parametrize("lens", [[(2000, 1), (30, 2)], [(1900, 200)], [(0, 300), (0, 40)], [(100, 1)]])
@pytest.mark.parametrize("column", [0, -1])
def test_an_infinite_value_is_seen_in_its_column_alone(dtype, dim, lens, column):
    """V of key 20 of the first request is infinite in one column: infinite there for the
    rows that see it, as the weights are positive; all else as before."""
    pool, q, news = setup(lens, 4, dim, dtype)
    scale = 0.3 * dim ** -0.5
    clean, clean_lse = attend(pool, q, news, 8, scale)
    page, row = pool.place(0, 20)
    pool.v[page, 1, row, column] = math.inf
    out, lse = attend(pool, q, news, 8, scale)
    hit = torch.zeros_like(out, dtype=torch.bool)
    past, new = lens[0]
    hit[max(0, 20 - past):new, 4:, column] = True
    assert (out[hit] == math.inf).all()
    assert out[~hit].isfinite().all() and torch.equal(lse, clean_lse)
    # Rows done again round their output once more and no weight, and add in another
    # order: 3 roundings to the type, n of sums, and the scores' (2^-13 is far above).
    bound = (3 * TYPES[dtype][2] + sum(lens[0]) * 2.0 ** -23 + 2.0 ** -13) * max(
        float(v[v.isfinite()].abs().max()) for v in pool.values)
    assert (out[~hit].double() - clean[~hit].double()).abs().max() <= bound
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
