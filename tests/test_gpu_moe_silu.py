"""The activation of qmm_moe_experts where its parts leave fp32's normal numbers."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from moe_util import TYPES  # noqa: E402
from test_gpu_moe_exact import Codes, one_expert, pick  # noqa: E402


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gates_far_below_zero(kind):
    """gate = x, up = 2^100: silu(gate) * up is an ordinary number although exp(gate) is
    subnormal, or 1 + exp(-gate) is near fp32's end.  Off by exp's own roundings (its result is
    a multiple of 2^-149, off by 2 units of its last place), the product's and the sum's."""
    hidden = inner = 128
    at = torch.arange(inner) % 127 + 1
    up = pick(inner, hidden, torch.zeros(inner, dtype=torch.long))
    layer = Codes(pick(inner, hidden, at), up, pick(hidden, inner, torch.arange(hidden) % inner), 4, 64, (1.0, 2.0 ** 100, 1.0))
    x = -torch.linspace(60, 104, 8 * hidden).reshape(8, hidden)
    x[:, 0] = 1.0
    x = x.to(TYPES[kind][0]).cuda()
    y = one_expert(layer, x).double()
    gate = x.double()[:, at[torch.arange(hidden) % inner]]
    e = torch.exp(gate)
    want = gate * e / (1 + e) * 2.0 ** 100
    far = want.abs() * 2.0 ** -20 + gate.abs() * 2.0 ** (2 - 149 + 100)
    assert ((y - want).abs() <= far).all()


def test_ordinary_gates():
    """Within a few roundings of fp32 (2^-24 each: exp two of its last place, the sum, the
    quotient two, two products, the parts' and the sums' none)."""
    hidden = inner = 128
    at = torch.arange(inner) % 127 + 1
    layer = Codes(pick(inner, hidden, at), pick(inner, hidden, torch.zeros(inner, dtype=torch.long)),
                  pick(hidden, inner, torch.arange(hidden) % inner), 4, 64)
    x = torch.linspace(-60, 60, 8 * hidden).reshape(8, hidden)
    x[:, 0] = 1.0
    y = one_expert(layer, x.cuda()).cpu().double()
    gate = x.double()[:, at[torch.arange(hidden) % inner]]
    want = gate * torch.sigmoid(gate)
    assert ((y - want).abs() <= want.abs() * 16 * 2.0 ** -24).all()
