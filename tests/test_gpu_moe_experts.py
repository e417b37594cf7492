"""qmm_moe_experts and qmm_moe_layer against 64-bit results, within derived bounds."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from moe_util import TYPES, Layer, random_ids, reference, routed, workspace  # noqa: E402


def run(layer, x, ids, weights, out, guard=64):
    t, top = ids.shape
    dt, kind = TYPES[out]
    y = torch.full((t * layer.hidden + guard,), 77.0, dtype=dt, device="cuda")
    ws, n = workspace(t, top, layer.hidden, layer.inner)
    x_kind = {d: k for d, k in TYPES.values()}[x.dtype]
    qmm.qmm_moe_experts(x, x_kind, t, ids, weights, top, layer.handle, y, kind, ws, n)
    torch.cuda.synchronize()
    assert (y[t * layer.hidden:] == 77.0).all() and (ws[n:] == 0xFF).all()
    return y[:t * layer.hidden].view(t, layer.hidden)


def check(layer, x, ids, weights, out):
    qmm.qmm_get_device_error()  # (other tests may have left theirs)
    y = run(layer, x, ids, weights, out)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    want, far = reference(layer, x, ids, weights, y.dtype)
    ratio = ((y.double() - want).abs() / (far + 1e-30)).max().item()
    assert ratio <= 1.0, ratio
    assert torch.equal(y, run(layer, x, ids, weights, out))  # bit for bit
    return y


def tokens(t, hidden, kind, seed=0):
    g = torch.Generator().manual_seed(seed + t)
    return torch.randn(t, hidden, generator=g).to(TYPES[kind][0]).cuda()


@pytest.mark.parametrize("bits", [1, 2, 3, 4, 5, 6, 8])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_bits_and_groups(bits, group):
    for kind, sb, out in (("bf16", "bf16", "bf16"), ("f32", "f32", "f32"), ("f16", "f16", "f16")):
        layer = Layer(5, 3 * group if group < 128 else 256, 128 + group, bits, group, sb, bits * group)
        ids, weights = random_ids(3, 2, 5, bits)
        check(layer, tokens(3, layer.hidden, kind), ids, weights, out)


@pytest.mark.parametrize("x,sb,out", [("bf16", "f16", "f32"), ("bf16", "f32", "bf16"), ("f16", "bf16", "f32"),
                                      ("f16", "f32", "f16"), ("f32", "bf16", "f32"), ("f32", "f16", "f32")])
def test_mixed_types(x, sb, out):
    layer = Layer(4, 320, 192, 4, 64, sb, 3)
    ids, weights = random_ids(5, 3, 4, 1)
    check(layer, tokens(5, 320, x), ids, weights, out)


@pytest.mark.parametrize("t,top,experts,hidden,inner", [
    (1, 1, 1, 64, 64), (1, 8, 16, 1024, 320), (2, 1, 7, 64, 1024), (8, 2, 4, 512, 128), (9, 3, 3, 256, 448),
    (16, 8, 64, 256, 192), (17, 2, 2, 192, 64), (33, 1, 1, 128, 256), (64, 8, 32, 320, 128), (16, 32, 40, 64, 64),
    (64, 2, 1024, 64, 64), (5, 4, 200, 2048, 64), (3, 2, 5, 64, 4160), (20, 4, 6, 4096, 64),
])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_shapes(t, top, experts, hidden, inner, kind):
    layer = Layer(experts, hidden, inner, 4, 64, "bf16", t)
    ids, weights = random_ids(t, top, experts, top)
    check(layer, tokens(t, hidden, kind), ids, weights, kind)


def test_every_slot_one_expert_and_the_same_expert_twice():
    layer = Layer(6, 256, 128, 4, 64, "bf16", 1)
    for t, top in ((64, 8), (40, 3), (1, 5)):
        ids = torch.full((t, top), 4, dtype=torch.int32, device="cuda")
        weights = torch.rand(t, top, device="cuda") - 0.3
        check(layer, tokens(t, 256, "bf16"), ids, weights, "bf16")


def test_weights_of_zero_leave_their_experts_out():
    """Expert 3's weights are NaN and its slots have weight 0: y has no part of them."""
    layer = Layer(5, 128, 192, 4, 32, "bf16", 2)
    for part in layer.parts:
        part[1][3] = math.nan
    ids = torch.tensor([[0, 3], [3, 3], [2, 1]], dtype=torch.int32, device="cuda")
    weights = torch.tensor([[0.5, 0.0], [0.0, -0.0], [0.25, 2.0]], device="cuda")
    y = run(layer, tokens(3, 128, "bf16"), ids, weights, "f32")
    clean = Layer(5, 128, 192, 4, 32, "bf16", 2)
    want, far = reference(clean, tokens(3, 128, "bf16"), ids, weights, y.dtype)
    assert (y[1] == 0).all() and ((y.double() - want).abs() <= far).all()


def test_values_that_are_not_finite_stay_with_their_token():
    layer = Layer(4, 128, 128, 4, 64, "bf16", 6)
    ids, weights = random_ids(20, 2, 4, 3)
    for kind, out in (("bf16", "bf16"), ("f32", "f32")):
        x = tokens(20, 128, kind)
        want, far = reference(layer, x, ids, weights, x.dtype)
        x[3, 5], x[11, 100] = math.nan, math.inf
        y = run(layer, x, ids, weights, out)
        assert not y[3].isfinite().any() and not y[11].isfinite().any()
        keep = [i for i in range(20) if i not in (3, 11)]
        assert ((y.double() - want).abs() <= far)[keep].all()


def test_ids_outside_are_reported_and_left_out():
    layer = Layer(4, 128, 64, 4, 64, "bf16", 7)
    ids, weights = random_ids(6, 3, 4, 5)
    bad = ids.clone()
    bad[2, 1], bad[4, 0] = 4, -1
    x = tokens(6, 128, "bf16")
    qmm.qmm_get_device_error()
    y = run(layer, x, bad, weights, "bf16")
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    want, far = reference(layer, x, bad, weights, y.dtype)
    assert ((y.double() - want).abs() <= far).all()


def test_large_and_small_values():
    """fp32 x near its limits (three parts of it must hold), fp16 x at 65504, tiny x."""
    layer = Layer(3, 128, 64, 8, 64, "f32", 8)
    ids, weights = random_ids(4, 2, 3, 2)
    for scale in (1e-30, 1e-3, 1e3):
        x = tokens(4, 128, "f32") * scale
        check(layer, x, ids, weights, "f32")
    x = (tokens(4, 128, "f16").float() * 2e4).clamp(-65504, 65504).to(torch.float16)
    check(layer, x, ids, weights * 1e-9, "f32")


@pytest.mark.parametrize("bits", [1, 2, 3, 4, 6, 8])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_with_values_from_two_to_26(bits, kind):
    """Tokens below and above the size at which codes are scaled instead of x, in the same
    expert and alone; and silu(gate) * up that crosses it though x does not."""
    layer = Layer(3, 192, 128, bits, 64, "f32", bits)
    x = tokens(24, 192, kind).float()
    x[3] *= 2.0 ** 26
    x[9] *= 2.0 ** 40
    x[10, 5] = 2.0 ** 26
    x[11, 5] = 2.0 ** 26 * (1 - 2.0 ** -8)
    x[17] *= 3e4
    x[18] *= 2.0 ** -80
    x = x.to(TYPES[kind][0])
    ids = torch.tensor([[t % 3, (t + 1) % 3] for t in range(24)], dtype=torch.int32, device="cuda")
    weights = torch.rand(24, 2, device="cuda") + 0.1
    check(layer, x, ids, weights, "f32")
    for t in (3, 9, 11, 17):
        check(layer, x[t:t + 1].clone(), ids[t:t + 1].clone(), weights[t:t + 1].clone(), "f32")


@pytest.mark.parametrize("counts", [(7, 8, 9), (16, 17, 1), (24, 8, 25)])
def test_passes_over_an_expert(counts):
    """Experts with about a whole number of passes of 8 slots."""
    layer = Layer(3, 256, 192, 4, 64, "bf16", 5)
    ids = torch.tensor([e for e, n in enumerate(counts) for _ in range(n)], dtype=torch.int32, device="cuda")[:, None]
    weights = torch.rand(sum(counts), 1, device="cuda") + 0.1
    check(layer, tokens(sum(counts), 256, "bf16"), ids, weights, "f32")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("sigmoid,normalize", [(False, True), (True, False)])
@pytest.mark.parametrize("t,experts,top", [(1, 8, 2), (16, 40, 6), (7, 300, 4), (64, 16, 8), (2, 1024, 32)])
def test_layer_is_route_and_experts(t, experts, top, sigmoid, normalize, kind):
    """Bit for bit what the two calls give, and near the 64-bit result."""
    layer = Layer(experts, 128, 64, 4, 64, "bf16", t)
    g = torch.Generator().manual_seed(t)
    logits = torch.randn(t, experts, generator=g)
    logits[0, : experts // 2] = -math.inf
    logits = logits.to(TYPES[kind][0]).cuda()
    x = tokens(t, 128, "bf16")
    ids = torch.empty(t, top, dtype=torch.int32, device="cuda")
    weights = torch.empty(t, top, device="cuda")
    qmm.qmm_moe_route(logits, TYPES[kind][1], t, experts, top, int(sigmoid), normalize, 1.5, ids, weights)
    y = torch.empty(t, 128, dtype=torch.bfloat16, device="cuda")
    ws, n = workspace(t, top, 128, 64)
    qmm.qmm_moe_layer(x, qmm.QMM_BF16, t, logits, TYPES[kind][1], top, int(sigmoid), normalize, 1.5,
                      layer.handle, y, qmm.QMM_BF16, ws, n)
    assert torch.equal(y, run(layer, x, ids, weights, "bf16"))
    want_ids, want_weights = routed(logits.cpu(), top, sigmoid, normalize, 1.5)
    want, far = reference(layer, x, want_ids.cuda(), want_weights.cuda(), y.dtype)
    assert ((y.double() - want).abs() <= far + 1e-30).all()


def test_a_row_without_experts_is_zero():
    layer = Layer(4, 64, 64, 4, 64, "bf16", 1)
    logits = torch.full((3, 4), -math.inf, device="cuda")
    logits[1] = 0.5
    y = torch.full((3, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    ws, n = workspace(3, 2, 64, 64)
    qmm.qmm_moe_layer(tokens(3, 64, "bf16"), qmm.QMM_BF16, 3, logits, qmm.QMM_F32, 2, qmm.QMM_SCORE_SOFTMAX,
                      True, 1.0, layer.handle, y, qmm.QMM_BF16, ws, n)
    assert (y[[0, 2]] == 0).all() and (y[1] != 0).any()


def test_captured_replayed_and_two_at_once():
    """Two graphs with a workspace each, on two streams at once, and again with new inputs."""
    layer = Layer(16, 512, 256, 4, 64, "bf16", 4)
    calls = []
    for i in range(2):
        x, logits = tokens(8, 512, "bf16", i), torch.randn(8, 16, device="cuda")
        y = torch.empty_like(x)
        ws, n = workspace(8, 3, 512, 256)
        args = (x, qmm.QMM_BF16, 8, logits, qmm.QMM_F32, 3, qmm.QMM_SCORE_SOFTMAX, True, 1.0, layer.handle, y,
                qmm.QMM_BF16, ws, n)
        qmm.qmm_moe_layer(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qmm.qmm_moe_layer(*args)
        calls.append((x, logits, y, graph, torch.cuda.Stream(), args, ws))
    for x, logits, *_ in calls:
        x.mul_(0.5)
        logits.neg_()
    torch.cuda.synchronize()
    for _ in range(20):
        for c in calls:
            with torch.cuda.stream(c[4]):
                c[3].replay()
    torch.cuda.synchronize()
    for x, logits, y, *_ in calls:
        ids, weights = routed(logits.cpu(), 3, False, True, 1.0)
        want, far = reference(layer, x, ids.cuda(), weights.cuda(), y.dtype)
        assert ((y.double() - want).abs() <= far).all()


def test_a_prompt_takes_the_router_and_the_gathered_products():
    """Many tokens: qmm_moe_route's ids, sorted, drive qmm_gather_qmm for each product; the
    few-token layer gives the same for the first of them."""
    layer = Layer(8, 256, 128, 4, 64, "bf16", 12)
    t, top = 96, 2
    x, logits = tokens(t, 256, "bf16"), torch.randn(t, 8, device="cuda")
    ids = torch.empty(t, top, dtype=torch.int32, device="cuda")
    weights = torch.empty(t, top, device="cuda")
    qmm.qmm_moe_route(logits, qmm.QMM_F32, t, 8, top, qmm.QMM_SCORE_SOFTMAX, True, 1.0, ids, weights)
    order = ids.flatten().sort(stable=True).indices
    rhs = ids.flatten()[order].contiguous()
    rows = x[order // top].contiguous()

    def product(part, rows, n, k):
        out = torch.empty(t * top, n, device="cuda")
        w, s, b = layer.parts[part]
        qmm.qmm_gather_qmm(rows, t * top, 1, w, s, b, 8, n, k, None, rhs, t * top, 1, 64, 4, 1, out, qmm.QMM_F32)
        return out

    gate, up = product(0, rows, 128, 256), product(1, rows, 128, 256)
    h = (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)
    z = product(2, h, 256, 128) * weights.flatten()[order, None]
    y = torch.zeros(t, 256, device="cuda").index_add_(0, order // top, z)
    few = run(layer, x[:64].contiguous(), ids[:64].contiguous(), weights[:64].contiguous(), "f32")
    # gather_qmm rounds weights to bf16 (2^-9 each), h here too: some 2^-8 of the terms' size
    size = y.double().pow(2).mean().sqrt()
    assert ((few - y[:64]).abs().max() <= 16 * 2.0 ** -8 * size)
