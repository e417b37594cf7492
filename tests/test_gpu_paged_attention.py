"""qmm_paged_attention against the definition in 64 bits: types, head layouts,
lengths from none to thousands, pages that end inside key tiles, masks that
leave rows empty, non-finite keys and values where no row looks."""
import math
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from paged_util import Pool, attend, check, i32, queries, workspace  # noqa: E402

@pytest.fixture(autouse=True)
def clear_what_earlier_calls_left():
    """The device error word holds what any earlier call reported until it is read."""
    qmm.qmm_get_device_error()


# (past, new) of each request.
DECODE = [(0, 1), (1, 1), (37, 1), (300, 1), (64, 1)]
DRAFTS = [(0, 3), (129, 5), (700, 2), (15, 1), (50, 0)]
MIXED = [(0, 70), (33, 1), (500, 17), (0, 1), (128, 128), (3, 0)]
PROMPTS = [(0, 200), (0, 1), (0, 129), (0, 64)]
LONG = [(1900, 300), (0, 700)]
SHAPES = {"decode": DECODE, "drafts": DRAFTS, "mixed": MIXED, "prompts": PROMPTS, "long": LONG}


def setup(lens, page, kv, group, dim, dtype, layout="hnd", seed=3):
    pool = Pool([a + b for a, b in lens], page, kv, dim, dtype, layout, seed)
    news = [b for _, b in lens]
    return pool, queries(pool, sum(news), kv * group, seed + 1), news, kv * group, dim ** -0.5


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", sorted(SHAPES))
@pytest.mark.parametrize("kv,group,dim,page,layout", [
    (2, 4, 128, 16, "hnd"),
    (3, 1, 64, 16, "nhd"),
    (1, 7, 80, 24, "hnd"),
    (2, 3, 128, 7, "nhd"),
    (1, 40, 64, 32, "hnd"),
    (2, 2, 96, 200, "hnd"),
    (1, 5, 8, 64, "nhd"),
    (1, 2, 256, 16, "hnd"),
])
def test_shapes(dtype, shape, kv, group, dim, page, layout):
    check(*setup(SHAPES[shape], page, kv, group, dim, dtype, layout), what="%s %s" % (dtype, shape))
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", ["decode", "drafts", "mixed", "long"])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 100), (False, 0), (False, 64), (True, 4000)])
def test_masks(dtype, shape, causal, window):
    check(*setup(SHAPES[shape], 16, 2, 4, 64 if window == 100 else 128, dtype), causal=causal,
          window=window, what="%s %s %s" % (shape, causal, window))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 3, 8, 64, 128, 129, 256])
def test_pages(dtype, page):
    check(*setup([(0, 1), (130, 1), (300, 1)], page, 2, 4, 128, dtype), what="decode")
    check(*setup([(0, 40), (257, 130), (100, 33)], page, 2, 4, 128, dtype), what="chunk")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("keys", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257])
def test_key_counts_around_tiles(dtype, keys):
    check(*setup([(keys - 1, 1)], 16, 1, 8, 128, dtype), what="decode")
    check(*setup([(0, keys)], 16, 1, 8, 128, dtype), what="prompt")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("requests,past,new", [
    (32, 100, 3), (33, 100, 3), (33, 40, 90), (129, 60, 2), (700, 30, 2), (1400, 9, 2), (40, 20, 300)])
def test_many_requests(dtype, requests, past, new):
    """More requests than a warp's lanes or a block's threads plan at once; some idle, some long."""
    rng = random.Random(requests + past + new)
    lens = [(rng.randint(0, past), rng.choice([0, 1, 1, rng.randint(0, new)])) for _ in range(requests)]
    lens[requests // 2] = (past, new)
    lens[-1] = (past // 2, new)
    check(*setup(lens, 16, 1, 4, 64, dtype), what="%d requests" % requests)


@pytest.mark.parametrize("kv,group", [(1, 17), (2, 33), (1, 128), (1, 130), (1, 200)])
@pytest.mark.parametrize("lens", [[(30, 1), (5, 1)], [(90, 40), (0, 3)]])
def test_wide_groups(kv, group, lens):
    """Groups of more heads than an item has rows are walked in slices."""
    for dtype in ("bf16", "f32"):
        check(*setup(lens, 16, kv, group, 64, dtype), what="group %d" % group)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("news,lens", [([5, 1, 40], [2, 0, 7]), ([200, 3], [150, 0]), ([1, 1], [0, 9])])
def test_rows_that_see_nothing(dtype, news, lens):
    """More new tokens than keys: the first rows come before every key."""
    pool = Pool(lens, 16, 2, 128, dtype)
    q = queries(pool, sum(news), 8)
    check(pool, q, news, 8, 0.1)
    out, lse = attend(pool, q, news, 8, 0.1)
    empty = news[0] - lens[0]
    assert empty > 0 and (out[:empty] == 0).all() and (lse[:empty] == -math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens", [[(100, 1), (5, 1)], [(40, 60)], [(200, 300), (0, 150)]])
@pytest.mark.parametrize("poison", [math.inf, math.nan])
def test_keys_that_a_row_does_not_see_have_no_part_in_it(dtype, lens, poison):
    """Non-finite K and V at the last token of each request: only its own row sees them."""
    pool, q, news, heads, scale = setup(lens, 16, 2, 4, 128, dtype)
    for b, (past, new) in enumerate(lens):
        page, row = pool.place(b, past + new - 1)
        pool.k[page, :, row] = poison
        pool.v[page, :, row] = poison
    out, lse = attend(pool, q, news, heads, scale)
    clean = setup(lens, 16, 2, 4, 128, dtype)[0]
    ref, ref_lse = attend(clean, q, news, heads, scale)
    last = torch.zeros(sum(news), dtype=torch.bool)
    at = 0
    for n in news:
        at += n
        last[at - 1] = True
    assert out[last.cuda()].isnan().any()
    rest = (~last).cuda()
    assert out[rest].isfinite().all() and lse[rest].isfinite().all()
    if rest.any():
        check(clean, q, news, heads, scale, got=(torch.where(rest[:, None, None], out, ref),
                                                 torch.where(rest[:, None], lse, ref_lse)))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_scores_far_from_zero(dtype):
    """Scores in the hundreds, of both signs: the running maximum moves a lot."""
    for lens in ([(600, 1)], [(300, 200)]):
        pool = Pool([a + b for a, b in lens], 16, 2, 128, dtype, scale=4.0)
        q = queries(pool, sum(b for _, b in lens), 8, scale=6.0)
        check(pool, q, [b for _, b in lens], 8, 128 ** -0.5)
        check(pool, q, [b for _, b in lens], 8, -(128 ** -0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(1000, 1)] * 3, [(300, 200), (40, 90)]])
def test_strides_streams_and_no_lse(dtype, lens):
    pool, q, news, heads, scale = setup(lens, 16, 2, 4, 64, dtype)
    t = sum(news)
    wide = torch.full((t, heads * 64 + 72), math.nan, dtype=pool.dt, device="cuda")
    wide[:, 16:16 + heads * 64] = q.reshape(t, -1)
    out = torch.full((t, heads * 64 + 24), 5.0, dtype=pool.dt, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        attend(pool, wide[:, 16:], news, heads, scale, q_stride=wide.stride(0), out=out,
               out_stride=out.stride(0), lse=False)
    side.synchronize()
    assert (out[:, heads * 64:] == 5.0).all()
    check(pool, q, news, heads, scale, got=(out[:, :heads * 64].reshape(t, heads, 64), None))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(4000, 1)], [(2000, 1), (10, 1), (900, 3)], [(3000, 100), (50, 400)]])
def test_repeats_bit_for_bit_and_under_a_graph(dtype, lens):
    pool, q, news, heads, scale = setup(lens, 16, 2, 4, 128, dtype)
    first, first_lse = attend(pool, q, news, heads, scale)
    check(pool, q, news, heads, scale, got=(first, first_lse))
    for _ in range(3):
        again, lse = attend(pool, q, news, heads, scale)
        assert torch.equal(again, first) and torch.equal(lse, first_lse)
    # What the hint says changes speed, not results beyond rounding.
    check(pool, q, news, heads, scale, max_new=1)
    check(pool, q, news, heads, scale, max_new=5000)
    cache, ws, out = pool.cache(), workspace(), torch.empty_like(first)
    starts, seq = [0], i32([a + b for a, b in lens])
    for n in news:
        starts.append(starts[-1] + n)
    starts = i32(starts)
    args = (q, heads * 128, sum(news), heads, cache, pool.table, pool.width, starts, seq, len(news),
            max(news), scale, True, 0, out, heads * 128, None, ws, ws.numel() * 4)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        qmm.qmm_paged_attention(*args)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(100, 1), (40, 1)], [(100, 90), (40, 33)]])
def test_pages_outside_the_pool_read_as_zero_and_are_reported(dtype, lens):
    pool, q, news, heads, scale = setup(lens, 16, 2, 4, 128, dtype)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    for bad in (-1, pool.num, 2 ** 31 - 1):
        pool.table[0, 2] = bad
        pool.keys[0][:, 32:48] = 0.0
        pool.values[0][:, 32:48] = 0.0
        check(pool, q, news, heads, scale, what="page %d" % bad)
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    """A pool whose last pages start past 2^31 elements (only they are written)."""
    page, dim = 16, 128
    heads = 2
    stride = page * dim * heads
    num = 2 ** 31 // stride + 40
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    lens = [(70, 1), (30, 40)]
    small = Pool([a + b for a, b in lens], page, heads, dim, dtype)
    news = [b for _, b in lens]
    q = queries(small, sum(news), 8)
    big_k = torch.empty(num, heads, page, dim, dtype=dt, device="cuda")
    big_v = torch.empty(num, heads, page, dim, dtype=dt, device="cuda")
    big_k[-small.num:], big_v[-small.num:] = small.k, small.v
    small.k, small.v = big_k, big_v
    small.table = small.table + (num - small.num)
    small.num = num
    check(small, q, news, 8, 0.1)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def test_nothing_to_do():
    pool = Pool([5], 16, 2, 128, "bf16")
    c, ws = pool.cache(), workspace()
    L = qmm.lib()
    assert L.qmm_paged_attention(None, 1024, 0, 8, c, None, 1, None, None, 0, 0, 1.0, 1, 0, None, 1024,
                                 None, None, 0, 0) == qmm.QMM_OK
    # All requests idle, and room past the last token: the rows there stay.
    out = torch.full((4, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    q = queries(pool, 4, 8)
    qmm.qmm_paged_attention(q, 1024, 4, 8, c, pool.table, pool.width, i32([0, 0]), i32([5]), 1, 4, 1.0,
                            True, 0, out, 1024, None, ws, ws.numel() * 4)
    assert (out == 7.0).all()
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("lens", [[(3000, 1), (700, 2)], [(2000, 300)]])
def test_waits_that_run_out_are_reported_and_the_next_call_is_right(lens):
    """One poll a wait: whether a wait runs out depends on timing (a poll may be
    suspended until the copy lands); either way the kernel drains its copies and
    returns, and the next call is right."""
    pool, q, news, heads, scale = setup(lens, 16, 2, 4, 128, "bf16")
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    before = qmm.qmm_set_wait_limit(1)
    try:
        attend(pool, q, news, heads, scale)
        torch.cuda.synchronize()
    finally:
        qmm.qmm_set_wait_limit(before)
    assert qmm.qmm_get_device_error() in (qmm.QMM_OK, qmm.QMM_ERR_TIMEOUT)
    check(pool, q, news, heads, scale)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
