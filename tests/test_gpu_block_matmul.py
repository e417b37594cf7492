"""qmm_block_matmul against the product in 64 bits, within bounds of its fp32 sums."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from block_util import TYPES, bound, operands, product  # noqa: E402


def run(a, sa, w, sw, kind, guard=64):
    dt, k = TYPES[kind]
    m, n = a.shape[0], w.shape[0]
    y = torch.full((m * n + guard,), -3.0, dtype=dt, device="cuda")
    qmm.qmm_get_device_error()  # (other tests may have left theirs)
    qmm.qmm_block_matmul(a.cuda(), sa.cuda(), m, w.cuda(), sw.cuda(), n, a.shape[1], y, k)
    torch.cuda.synchronize()
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    assert (y[m * n:] == -3.0).all()
    return y[:m * n].view(m, n)


def check(m, n, k, kind, seed=0):
    a, sa, w, sw = operands(m, n, k, 1000 * m + n + k + seed)
    y = run(a, sa, w, sw, kind)
    want, terms = product(a.cuda(), sa.cuda(), w.cuda(), sw.cuda())
    far = (y.double() - want).abs() / bound((want, terms), k, y.dtype)
    assert far.max() <= 1.0, (m, n, k, kind, far.max().item(), far.argmax().item())
    assert torch.equal(y, run(a, sa, w, sw, kind))  # bit for bit


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 16), (1, 4096, 4096), (2, 130, 144), (7, 257, 1024), (8, 64, 128), (9, 1000, 528), (16, 512, 2048),
    (17, 384, 2064), (33, 127, 112), (64, 1024, 256), (65, 1021, 1040), (100, 640, 384), (128, 256, 512),
    (129, 129, 129 * 16), (200, 1024, 1024), (256, 512, 128), (257, 513, 272), (300, 96, 16),
])
def test_sizes(m, n, k, kind):
    check(m, n, k, kind)


@pytest.mark.parametrize("m,n,k", [(1, 16384, 64), (3, 14336, 4096), (16, 128, 16384), (40, 11008, 4096),
                                   (512, 4096, 4096), (1000, 2051, 4112), (4096, 768, 16), (2048, 14336, 256)])
def test_larger(m, n, k):
    check(m, n, k, "bf16")
    check(m, n, k, "f32", 1)


@pytest.mark.parametrize("m", [1, 5, 16, 48, 130, 300])
def test_exact_where_sums_are(m):
    """Small whole numbers and scales of powers of two: every sum is exact, so is y."""
    g = torch.Generator().manual_seed(m)
    k, n = 1056, 270
    code = lambda r: torch.randint(-8, 9, (r, k), generator=g).float().to(torch.float8_e4m3fn).view(torch.uint8)
    a, w = code(m), code(n)
    sa = torch.exp2(torch.randint(-2, 3, (m, 9), generator=g).float())
    sw = torch.exp2(torch.randint(-2, 3, (3, 9), generator=g).float())
    want, _ = product(a, sa, w, sw)
    assert torch.equal(run(a, sa, w, sw, "f32").double().cpu(), want)


@pytest.mark.parametrize("m", [1, 20, 140])
def test_every_code(m):
    """One code a row of W against one-hot rows: y is the code's value, NaN codes among them."""
    w = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 272)
    a = torch.zeros(m, 272, dtype=torch.uint8)
    one = torch.ones(1).to(torch.float8_e4m3fn).view(torch.uint8)
    for i in range(m):
        a[i, (i * 37) % 272] = one
    y = run(a, torch.ones(m, 3), w, torch.ones(2, 3), "f32").cpu()
    want = w[:, 0].view(torch.float8_e4m3fn).float().expand(m, 256)
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("m", [3, 200])
def test_not_finite_stays_in_its_row(m):
    a, sa, w, sw = operands(m, 200, 256, 9)
    want, terms = product(a, sa, w, sw)
    a2, sa2 = a.clone(), sa.clone()
    a2[1, 7] = 0x7F
    sa2[2, 1] = float("inf")
    y = run(a2, sa2, w, sw, "f32").double().cpu()
    assert y[1].isnan().all() and not y[2].isfinite().any()
    keep = [i for i in range(m) if i not in (1, 2)]
    assert ((y - want).abs() <= bound((want, terms), 256, torch.float32))[keep].all()


def test_large_and_small_values_keep_their_scales():
    """Blocks whose scales are 2^60 and 2^-60: y is the large block's product."""
    a, sa, w, sw = operands(20, 140, 256, 3)
    sa[:, 0] *= 2.0 ** 60
    sw[:, 1] *= 2.0 ** -60
    y = run(a, sa, w, sw, "f32").double().cpu()
    want, terms = product(a, sa, w, sw)
    assert ((y - want).abs() <= bound((want, terms), 256, torch.float32)).all()


def test_replayed_with_new_values():
    for m in (4, 150):
        a, sa, w, sw = [t.cuda() for t in operands(m, 256, 512, m)]
        y = torch.empty(m, 256, dtype=torch.bfloat16, device="cuda")
        args = (a, sa, m, w, sw, 256, 512, y, qmm.QMM_BF16)
        qmm.qmm_block_matmul(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qmm.qmm_block_matmul(*args)
        sa.mul_(0.5)
        a.copy_(a.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        want, terms = product(a, sa, w, sw)
        assert ((y.double() - want).abs() <= bound((want, terms), 512, y.dtype)).all()


def test_quantize_then_multiply():
    """Both operators as a projection uses them: the product of the quantized values, and
    within e4m3's rounding (half a step, 2^-4 of a value, on each side) of the unquantized."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(37, 656, generator=g).to(torch.bfloat16).cuda()
    v = torch.randn(300, 656, generator=g).to(torch.bfloat16).cuda()
    a, sa = torch.empty(37, 656, dtype=torch.uint8, device="cuda"), torch.empty(37, 6, device="cuda")
    w, sw = torch.empty(300, 656, dtype=torch.uint8, device="cuda"), torch.empty(3, 6, device="cuda")
    y = torch.empty(37, 300, dtype=torch.bfloat16, device="cuda")
    qmm.qmm_block_quantize(x, qmm.QMM_BF16, 37, 656, 1, a, sa)
    qmm.qmm_block_quantize(v, qmm.QMM_BF16, 300, 656, 128, w, sw)
    qmm.qmm_block_matmul(a, sa, 37, w, sw, 300, 656, y, qmm.QMM_BF16)
    want, terms = product(a, sa, w, sw)
    assert ((y.double() - want).abs() <= bound((want, terms), 656, y.dtype)).all()
    full, size = x.double() @ v.double().T, x.double().abs() @ v.double().abs().T
    # the smallest codes are 2^-9 apart: half of that, of each scale, beside half a step
    low = (sa.max() * 2.0 ** -10) * v.double().abs().sum(1) + (sw.max() * 2.0 ** -10) * x.double().abs().sum(1)[:, None]
    assert ((y.double() - full).abs() <= size * (2.0 ** -3 + 2.0 ** -8 + 2.0 ** -8) + 2 * low).all()


@pytest.mark.parametrize("m,n,k", [(4, 1024, 4096), (100, 640, 4096), (1024, 12800, 1024)])
def test_a_wait_that_runs_out_is_reported(m, n, k):
    """One poll a wait and operands that come from memory: loads and products in flight
    retire, the status is reported, and the next call is right."""
    a, sa, w, sw = [t.cuda() for t in operands(m, n, k, 8)]
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    qmm.qmm_get_device_error()
    seen = []
    before = qmm.qmm_set_wait_limit(1)
    try:
        for _ in range(10):
            flush.zero_()
            qmm.qmm_block_matmul(a, sa, m, w, sw, n, k, y, qmm.QMM_BF16)
            seen.append(qmm.qmm_get_device_error())
    finally:
        qmm.qmm_set_wait_limit(before)
    assert set(seen) <= {qmm.QMM_OK, qmm.QMM_ERR_TIMEOUT} and qmm.QMM_ERR_TIMEOUT in seen
    check(m, n, k, "bf16")


@pytest.mark.parametrize("m,n,k,kind", [(3000, 4104, 256, "bf16"), (3000, 4100, 384, "f32"), (3001, 4099, 128, "f16"),
                                        (129, 16640, 272, "f32"), (1300, 8200, 144, "bf16")])
def test_tiles_at_the_edges_of_y(m, n, k, kind):
    """Rows of y that TMA can address and rows that it cannot, last tiles of a few rows and
    columns, steps that are and are not a multiple of four."""
    check(m, n, k, kind)
