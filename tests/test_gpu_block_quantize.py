"""qmm_block_quantize against its definition in 64 bits, bit for bit."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from block_util import TYPES, blocks, quantized, values  # noqa: E402


def run(x, block_rows, kind, guard=256):
    rows, cols = x.shape
    codes = torch.full((rows * cols + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-rows // block_rows) * blocks(cols) + guard,), -7.0, device="cuda")
    qmm.qmm_block_quantize(x.cuda(), kind, rows, cols, block_rows, codes, scales)
    torch.cuda.synchronize()
    assert (codes[rows * cols:] == 0xA5).all() and (scales[scales.numel() - guard:] == -7.0).all()
    return codes[:rows * cols].cpu().view(rows, cols), scales[:-guard].cpu().view(-1, blocks(cols))


def check(x, block_rows, kind):
    codes, scales = run(x, block_rows, kind)
    want, want_scales = quantized(x, block_rows)
    assert torch.equal(torch.nan_to_num(scales, 7.5, 8.5), torch.nan_to_num(want_scales, 7.5, 8.5))
    assert torch.equal(scales.isnan(), want_scales.isnan())
    got = values(codes)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(9.0), want.nan_to_num(9.0))
    return codes


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (31, 4096), (128, 128), (129, 400), (257, 1040)])
def test_values(rows, cols, block_rows, kind):
    dt, k = TYPES[kind]
    g = torch.Generator().manual_seed(rows * cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    x[torch.rand(rows, cols, generator=g) < 0.01] *= 40
    check(x.to(dt), block_rows, k)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_borders(kind):
    """Blocks whose largest value is 448 * s: the quotients lie on and next to the borders
    between codes, and among the smallest codes."""
    dt, k = TYPES[kind]
    rows = []
    for s in (1.0, 0.75, 1.9921875, 2.0 ** -60, 3.0 * 2.0 ** 40):
        row = torch.zeros(2048, dtype=torch.float64)
        n = torch.arange(2048, dtype=torch.float64)
        row[:1024] = (n[:1024] + 0.5) * 2.0 ** -10 * s            # up to 1 in half steps of small codes
        row[1024:] = (16 + n[1024:] % 32 + 0.5) * 2.0 ** (n[1024:] // 32 % 9 - 5) * s / 2
        row.clamp_(max=448 * s)
        row[::128] = 448 * s
        rows += [row, -row, row * (1 + 2.0 ** -20)]
    x = torch.stack(rows).clamp(-3e38, 3e38).float().to(dt)
    for block_rows in (1, 128):
        check(x, block_rows, k)


def test_many_quotients_near_a_border():
    """Single-precision values chosen one unit around border * scale."""
    g = torch.Generator().manual_seed(5)
    rows, top = 64, 1.0 + torch.rand(64, 1, generator=g)
    scale = (top.double() / 448).float()
    from block_util import grid
    border = (grid()[1:] + grid()[:-1]) / 2
    t = border[torch.randint(0, 126, (rows, 1024), generator=g)]
    x = (t * scale.double()).float()
    bits = x.view(torch.int32) + torch.randint(-2, 3, (rows, 1024), generator=g, dtype=torch.int32)
    x = torch.minimum(bits.view(torch.float32), top)
    x[:, ::128] = top
    check(x, 1, qmm.QMM_F32)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_zeros_smallest_and_not_finite(block_rows):
    x = torch.randn(256, 512, generator=torch.Generator().manual_seed(1))
    x[3, 5] = float("nan")
    x[140, 140] = float("inf")
    x[200, 300] = -float("inf")
    x[0, 128:256] = 0.0
    x[1, 128:256] = -0.0
    x[2, 256:384] = 2.0 ** -140
    x[5, 256:384] = torch.tensor([2.0 ** -149, 2.0 ** -117] * 64)
    check(x, block_rows, qmm.QMM_F32)
    check(torch.zeros(130, 128), block_rows, qmm.QMM_F32)
    check(torch.full((130, 128), 2.0 ** -149), block_rows, qmm.QMM_F32)
    check(torch.full((130, 128), 3.3e38).to(torch.bfloat16), block_rows, qmm.QMM_BF16)


def test_another_stream_and_replay():
    x = torch.randn(64, 512, device="cuda").to(torch.bfloat16)
    codes, scales = torch.empty(64, 512, dtype=torch.uint8, device="cuda"), torch.empty(64, 4, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        qmm.qmm_block_quantize(x, qmm.QMM_BF16, 64, 512, 1, codes, scales)
    s.synchronize()
    with torch.cuda.graph(graph):
        qmm.qmm_block_quantize(x, qmm.QMM_BF16, 64, 512, 1, codes, scales)
    x.mul_(3)
    graph.replay()
    torch.cuda.synchronize()
    want, want_scales = quantized(x.cpu(), 1)
    assert torch.equal(values(codes.cpu()), want) and torch.equal(scales.cpu(), want_scales)
