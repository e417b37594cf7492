"""qmm_moe_route: ids equal to a plain sort's, weights within fp32's roundings."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from moe_util import TYPES, routed  # noqa: E402


def run(logits, top, sigmoid, normalize, scale, guard=64):
    t, e = logits.shape
    ids = torch.full((t * top + guard,), -9, dtype=torch.int32, device="cuda")
    weights = torch.full((t * top + guard,), -9.0, device="cuda")
    kind = {dt: k for dt, k in TYPES.values()}[logits.dtype]
    qmm.qmm_moe_route(logits.cuda(), kind, t, e, top, int(sigmoid), normalize, scale, ids, weights)
    torch.cuda.synchronize()
    assert (ids[t * top:] == -9).all() and (weights[t * top:] == -9.0).all()
    return ids[:t * top].cpu().view(t, top), weights[:t * top].cpu().view(t, top)


def check(logits, top, sigmoid, normalize, scale=1.0):
    ids, weights = run(logits, top, sigmoid, normalize, scale)
    want_ids, want = routed(logits, top, sigmoid, normalize, scale)
    assert torch.equal(ids, want_ids)
    # exp of an argument off by 2^-24 of its size (at most 2^8 here before it underflows),
    # sums of 1024 in fp32, three divisions and products; below 2^-126 in absolute terms
    err = (weights.double() - want).abs()
    assert (err <= want.abs() * (2.0 ** -15) + abs(scale) * 2.0 ** -120).all(), err.max()
    return ids, weights


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("tokens,experts,top", [(1, 1, 1), (3, 8, 2), (9, 31, 31), (17, 33, 5), (64, 64, 6),
                                                (7, 100, 32), (16, 128, 8), (33, 256, 8), (5, 300, 9),
                                                (4, 513, 1), (6, 1024, 32)])
def test_sizes(tokens, experts, top, sigmoid, normalize, kind):
    g = torch.Generator().manual_seed(tokens * experts + top)
    logits = (torch.randn(tokens, experts, generator=g) * 3).to(TYPES[kind][0])
    check(logits, top, sigmoid, normalize, 2.5 if top % 2 else 1.0)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
def test_masks_ties_and_values_that_are_not_finite(sigmoid, normalize):
    inf, nan = math.inf, math.nan
    g = torch.Generator().manual_seed(8)
    x = torch.randn(12, 70, generator=g)
    x[0] = -inf                                 # nothing open
    x[1] = nan
    x[2, 10:] = -inf                            # fewer open than chosen
    x[2, :8] = nan
    x[3] = 1.5                                  # all equal
    x[4, ::2], x[4, 1::2] = 0.0, -0.0           # zeros of both signs
    x[5, [3, 40]] = inf                         # shared by two
    x[6] = torch.finfo(torch.float32).min       # a mask of the type's lowest value
    x[6, 69] = 0.0
    x[7] = torch.linspace(-300, 88, 70)
    x[8, 5] = 3.4e38
    x[9] = -200.0
    x[10, 33] = inf
    x[10, 34] = nan
    ids, weights = check(x, 12, sigmoid, normalize)
    assert (weights[:2] == 0).all() and torch.equal(ids[0], torch.arange(12, dtype=torch.int32))
    assert weights.isfinite().all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
def test_masks_and_ties_of_16_bit_logits(kind, sigmoid, normalize):
    inf, nan = math.inf, math.nan
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(12, 300, generator=g) * 4).round() / 4        # many equal logits
    x[0], x[1] = -inf, nan
    x[2, 6:] = -inf
    x[2, :5] = -nan
    x[3, ::2], x[3, 1::2] = -0.0, 0.0
    x[4, [299, 7]] = inf
    x[5] = torch.finfo(TYPES[kind][0]).min
    x[6] = torch.finfo(TYPES[kind][0]).tiny
    x[6, 200] = -torch.finfo(TYPES[kind][0]).tiny
    x[7] = -torch.linspace(0, 60000, 300)
    ids, weights = check(x.to(TYPES[kind][0]), 9, sigmoid, normalize)
    assert (weights[:2] == 0).all() and torch.equal(ids[3], torch.arange(9, dtype=torch.int32))


def test_many_tokens_and_bf16_ties():
    g = torch.Generator().manual_seed(2)
    logits = torch.randn(5000, 128, generator=g).to(torch.bfloat16)
    check(logits, 8, False, True)


def test_replayed_on_another_stream():
    x = torch.randn(40, 96, device="cuda")
    ids = torch.empty(40, 4, dtype=torch.int32, device="cuda")
    weights = torch.empty(40, 4, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.qmm_moe_route(x, qmm.QMM_F32, 40, 96, 4, qmm.QMM_SCORE_SOFTMAX, True, 1.0, ids, weights)
    s = torch.cuda.Stream()
    x.neg_()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph.replay()
    s.synchronize()
    assert torch.equal(ids.cpu(), routed(x.cpu(), 4, False, True, 1.0)[0])
