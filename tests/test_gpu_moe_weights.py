"""Weights of qmm_moe_route are as near to 64 bits as the formula evaluated in fp32 is."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from moe_util import TYPES, routed  # noqa: E402


def scores(logits, sigmoid):
    if sigmoid:
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("spread", [1, 4, 10])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
def test_rms_of_relative_errors(normalize, sigmoid, spread, kind):
    """Root of the mean square over 32768 weights: at most a quarter above torch's in fp32
    (other orders of sums, a product by the scale of 1)."""
    dt, k = TYPES[kind]
    logits = (torch.randn(4096, 256, generator=torch.Generator().manual_seed(spread)) * spread).to(dt).cuda()
    ids = torch.empty(4096, 8, dtype=torch.int32, device="cuda")
    weights = torch.empty(4096, 8, device="cuda")
    qmm.qmm_moe_route(logits, k, 4096, 256, 8, int(sigmoid), normalize, 1.0, ids, weights)

    def off(w):
        want = scores(logits.double(), sigmoid).gather(1, ids.long())
        if normalize:
            want = want / want.sum(1, keepdim=True)
        return ((w.double() - want) / want).pow(2).mean().sqrt().item()

    plain = scores(logits.float(), sigmoid).gather(1, ids.long())
    if normalize:
        plain = plain / plain.sum(1, keepdim=True)
    assert off(weights) <= 1.25 * off(plain)


def test_logits_of_more_than_two_to_31():
    """8 400 000 tokens over 256 experts: the first rows, those about element 2^31, the last."""
    tokens, experts, top = 8400000, 256, 8
    logits = torch.empty(tokens, experts, dtype=torch.bfloat16, device="cuda")
    logits.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    ids = torch.empty(tokens, top, dtype=torch.int32, device="cuda")
    weights = torch.empty(tokens, top, device="cuda")
    qmm.qmm_moe_route(logits, qmm.QMM_BF16, tokens, experts, top, qmm.QMM_SCORE_SOFTMAX, True, 1.0, ids, weights)
    for first in (0, 2 ** 31 // experts - 32, tokens - 64):
        rows = slice(first, first + 64)
        want_ids, want = routed(logits[rows].cpu(), top, False, True, 1.0)
        assert torch.equal(ids[rows].cpu(), want_ids)
        assert ((weights[rows].cpu().double() - want).abs() <= 2.0 ** -18 * want).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("first", [30.0, -0.5, -10.0, -60.0, -64.5, -100.0, -3000.0])
def test_normalized_sigmoids_keep_their_ratios(first, kind):
    """Logits 0 to 80 below the largest: every weight to a few roundings (2^-24 of the
    difference, 16 more), and what lies below 2^-126."""
    dt, k = TYPES[kind]
    logits = (first - torch.linspace(0, 80, 32))[None].to(dt)
    ids = torch.empty(1, 32, dtype=torch.int32, device="cuda")
    weights = torch.empty(1, 32, device="cuda")
    qmm.qmm_moe_route(logits.cuda(), k, 1, 32, 32, qmm.QMM_SCORE_SIGMOID, True, 1.0, ids, weights)
    want_ids, want = routed(logits, 32, True, True, 1.0)
    assert torch.equal(ids.cpu(), want_ids)
    far = want * (100 + 16) * 2.0 ** -24 + 2.0 ** -126
    assert ((weights.cpu().double() - want).abs() <= far).all()
