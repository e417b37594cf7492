"""qmm_moe_experts where every product and sum is a whole number that fp32 holds (or the same
times a power of two), so that the result is known bit for bit."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from moe_util import TYPES, Layer, random_ids, reference, workspace  # noqa: E402


def pack(codes, bits):
    """int32 words of [.., columns] codes, little-endian bit by bit."""
    bit = codes[..., None] >> torch.arange(bits) & 1
    words = bit.reshape(*codes.shape[:-1], -1, 32).long() << torch.arange(32)
    words = words.sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


class Codes(Layer):
    """One expert of given codes, scales 1 (or `scales` for gate, up and down), biases 0."""

    def __init__(self, gate, up, down, bits, group, scales=(1.0, 1.0, 1.0)):
        self.experts, self.hidden, self.inner, self.bits, self.group, self.sb = 1, gate.shape[1], gate.shape[0], bits, group, qmm.QMM_F32
        self.parts = []
        for c, s in zip((gate, up, down), scales):
            full = torch.full((1, c.shape[0], c.shape[1] // group), s, device="cuda")
            self.parts.append((pack(c, bits)[None].cuda(), full, torch.zeros_like(full)))
        self.handle = qmm.Experts(*self.parts, self.sb, 1, self.hidden, self.inner, group, bits)


def run(layer, x, ids, weights, out):
    dt, kind = TYPES[out]
    t, top = ids.shape
    y = torch.empty(t, layer.hidden, dtype=dt, device="cuda")
    ws, n = workspace(t, top, layer.hidden, layer.inner)
    x_kind = {d: k for d, k in TYPES.values()}[x.dtype]
    qmm.qmm_moe_experts(x, x_kind, t, ids, weights, top, layer.handle, y, kind, ws, n)
    return y


def one_expert(layer, x, out="f32"):
    ids = torch.zeros(x.shape[0], 1, dtype=torch.int32, device="cuda")
    return run(layer, x, ids, torch.ones(x.shape[0], 1, device="cuda"), out)


def pick(rows, columns, at, code=1):
    """One code in each row r, in column at[r]."""
    c = torch.zeros(rows, columns, dtype=torch.long)
    c[torch.arange(rows), at] = code
    return c


# Column 0 of x is 1 and up picks it; a gate of 20 or more is its own silu in fp32
# (1 + exp(-20) rounds to 1); down picks: y is then gate, to the last bit.


@pytest.mark.parametrize("bits", [1, 4, 6, 8])
@pytest.mark.parametrize("group", [32, 128])
def test_fp32_keeps_24_bits(bits, group):
    """Gate picks a value of x of 24 significant bits (dropping the last of x's or h's three
    parts would change it)."""
    hidden, inner, t = 256, 384, 5
    g = torch.Generator().manual_seed(bits)
    at = torch.randint(1, hidden, (inner,), generator=g)
    back = torch.randint(0, inner, (hidden,), generator=g)
    layer = Codes(pick(inner, hidden, at), pick(inner, hidden, torch.zeros(inner, dtype=torch.long)),
                  pick(hidden, inner, back), bits, group)
    x = (torch.randint(2 ** 23, 2 ** 24, (t, hidden), generator=g) | 1).float()
    x[:, 0] = 1.0
    y = one_expert(layer, x.cuda())
    assert torch.equal(y.cpu(), x[:, at[back]])


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bits", [2, 4, 5, 8])
def test_sums_of_24_bits(bits, kind):
    """A sum of codes times x with one large term among small ones, below 2^24: nothing of it
    may be lost.  (A code taken as an unnormalised number loses the small ones.)"""
    hidden, inner, t, group = 128, 64, 8, 64
    top = 2 ** bits - 1
    g = torch.Generator().manual_seed(bits)
    codes = torch.randint(0, min(top, 2) + 1, (inner, hidden), generator=g)
    codes[:, 0] = 0
    codes[:, 1 + torch.randint(0, 63, (1,), generator=g)] = top
    large = codes[0].argmax().item()
    x = torch.randint(-3, 4, (t, hidden), generator=g).float() * 2 + 1
    x[:, 0] = 1.0
    # the large term near, and all of them below, 2^23; fp16 ends at 65504
    x[:, large] = min(2 ** 23 // (top + 1), 2 ** 15) if kind == "f16" else 2 ** 23 // (top + 1)
    layer = Codes(codes, pick(inner, hidden, torch.zeros(inner, dtype=torch.long)),
                  pick(hidden, inner, torch.arange(hidden) % inner), bits, group)
    x = x.to(TYPES[kind][0])
    want = x.double() @ codes.double().T
    assert (want >= 20).all() and (want < 2 ** 24).all()
    y = one_expert(layer, x.cuda())
    assert torch.equal(y.cpu().double(), want[:, torch.arange(hidden) % inner])


@pytest.mark.parametrize("part,power,kind", [(p, n, k) for p in "xh" for n in (-80, -40, 60, 100) for k in ("bf16", "f32")] +
                         [("x", -100, "bf16")])  # (below 2^-110 parts of x or h leave bf16)
@pytest.mark.parametrize("bits", [4, 8])
def test_powers_of_two_move_to_the_scales(bits, power, part, kind):
    """x (or silu(gate) * up) times 2^power and the scales times 2^-power: the same bits.  For
    x, gate's and up's scales; for h, up's against down's."""
    base = Layer(4, 256, 192, bits, 64, "f32", bits)
    moved = Layer(4, 256, 192, bits, 64, "f32", bits)
    for i, sign in ((0, -1), (1, -1)) if part == "x" else ((1, 1), (2, -1)):
        for t in moved.parts[i][1:]:
            t.mul_(2.0 ** (sign * power))
    ids, weights = random_ids(6, 2, 4, 1)
    x = torch.randn(6, 256, generator=torch.Generator().manual_seed(2)).to(TYPES[kind][0]).cuda()
    y = run(base, x, ids, weights, "f32")
    z = run(moved, (x.double() * 2.0 ** power).to(x.dtype) if part == "x" else x, ids, weights, "f32")
    assert torch.equal(y, z)
    want, far = reference(base, x, ids, weights, y.dtype)
    assert ((y.double() - want).abs() <= far).all()


@pytest.mark.parametrize("bits", [4, 8])
def test_x_near_the_largest_value(bits):
    """Scales (2^-121 and more, so that they are normal) bring sums of x of 2^118 back, of which
    128 codes of 8 bits times x would not fit."""
    base, moved = Layer(2, 128, 128, bits, 128, "f32", bits), Layer(2, 128, 128, bits, 128, "f32", bits)
    for i in (0, 1):
        for b, m in zip(base.parts[i][1:], moved.parts[i][1:]):
            b.mul_(2.0 ** 10)
            m.mul_(2.0 ** (10 - 118))
    ids = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    weights = torch.ones(2, 1, device="cuda")
    x = (torch.rand(2, 128, generator=torch.Generator().manual_seed(1)) + 1).bfloat16().cuda()
    y, z = run(base, x, ids, weights, "f32"), run(moved, x * 2.0 ** 118, ids, weights, "f32")
    assert y.isfinite().all() and torch.equal(y, z)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_a_token_does_not_depend_on_the_values_of_others(kind):
    layer = Layer(3, 192, 128, 4, 64, "bf16", 4)
    x = torch.randn(16, 192, generator=torch.Generator().manual_seed(3)).to(TYPES[kind][0]).cuda()
    ids = torch.tensor([[t % 3, (t + 1) % 3] for t in range(16)], dtype=torch.int32, device="cuda")
    weights = torch.rand(16, 2, device="cuda") + 0.1
    y = run(layer, x, ids, weights, "f32")
    x[5] *= 2.0 ** 40
    x[11] = float("nan")
    z = run(layer, x, ids, weights, "f32")
    keep = [t for t in range(16) if t not in (5, 11)]
    assert torch.equal(y[keep], z[keep])


@pytest.mark.parametrize("x,sb", [("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16")])
@pytest.mark.parametrize("bits", [2, 4, 8])
def test_outputs_in_fp32_are_near(x, sb, bits):
    """Relative to the norm of y: each of the three products in a row may lose 8 units of 2^-23
    of its norm (a group's few sums, a fused multiply-add a group), its inputs kept whole."""
    layer = Layer(8, 1024, 768, bits, 64, sb, bits)
    ids, weights = random_ids(12, 3, 8, 5)
    v = torch.randn(12, 1024, generator=torch.Generator().manual_seed(5)).to(TYPES[x][0]).cuda()
    y = run(layer, v, ids, weights, "f32").double()
    want, _ = reference(layer, v, ids, weights, torch.float32)
    off = ((y - want).norm() / want.norm()).item()
    print("off by %.2e" % off)
    assert off <= 3 * 8 * 2.0 ** -23
