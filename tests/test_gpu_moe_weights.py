"""Weights of qmm_moe_route are as near to 64 bits as the formula evaluated in fp32 is."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from moe_util import TYPES  # noqa: E402


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
