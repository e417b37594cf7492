"""Block-scaled codes and products of more than 2^31 elements."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from block_util import TYPES, bound, product, quantized  # noqa: E402


def random_codes(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    c.random_(0, 256, generator=g)
    return torch.where(c & 0x7F == 0x7F, torch.zeros_like(c), c)  # no NaN


def random_scales(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.rand(rows, cols, generator=g, device="cuda") / 1000 + 1e-4


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_codes_of_more_than_two_to_31(block_rows, kind):
    """600000 x 4096 elements: the first rows, those about element 2^31, the last ones."""
    rows, cols = 600000, 4096
    g = torch.Generator(device="cuda").manual_seed(block_rows)
    x = torch.empty(rows, cols, dtype=TYPES[kind][0], device="cuda").normal_(generator=g)
    codes = torch.full((rows * cols + 64,), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.empty(-(-rows // block_rows), cols // 128, device="cuda")
    qmm.qmm_block_quantize(x, TYPES[kind][1], rows, cols, block_rows, codes, scales)
    assert (codes[rows * cols:] == 0x55).all()
    got = codes[:rows * cols].view(rows, cols)
    for first in (0, 2 ** 31 // cols // 128 * 128 - 128, rows // 128 * 128 - 128):
        last = min(first + 256, rows)
        want, s = quantized(x[first:last].cpu(), block_rows)
        assert torch.equal(scales[first // block_rows:-(-last // block_rows)].cpu(), s)
        assert torch.equal(got[first:last].cpu().view(torch.float8_e4m3fn).double(), want)


@pytest.mark.parametrize("m,n,k,kind", [
    (70001, 31000, 128, "bf16"),  # y of 2.17e9 elements, tiles by TMA
    (70000, 31001, 128, "f16"),   # rows of y that TMA cannot address
    (3, 1100000, 2048, "f32"),    # W of 2.25e9 codes, few rows
    (600, 1100000, 2048, "bf16"),  # and many
    (1100000, 130, 2048, "bf16"),  # A of 2.25e9 codes
])
def test_products_of_more_than_two_to_31(m, n, k, kind):
    a, w = random_codes(m, k, 1), random_codes(n, k, 2)
    sa, sw = random_scales(m, k // 128, 3), random_scales(-(-n // 128), k // 128, 4)
    dt, out = TYPES[kind]
    y = torch.full((m * n + 64,), -3.0, dtype=dt, device="cuda")
    qmm.qmm_get_device_error()
    qmm.qmm_block_matmul(a, sa, m, w, sw, n, k, y, out)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    assert (y[m * n:] == -3.0).all()
    y = y[:m * n].view(m, n)
    # rows and columns (by blocks of 128 of W) at both ends and about element 2^31 of A, W and y
    tops = sorted({0, max(m - 64, 0), min(2 ** 31 // k, max(m - 64, 0)), min(2 ** 31 // n, max(m - 64, 0))})
    lefts = sorted({0, (n - 1) // 128 * 128, min(2 ** 31 // k, n - 1) // 128 * 128})
    for i in tops:
        for j in lefts:
            rows, cols = slice(i, min(i + 64, m)), slice(j, min(j + 128, n))
            want, terms = product(a[rows], sa[rows], w[cols], sw[j // 128:j // 128 + 1])
            far = bound((want, terms), k, dt)
            assert ((y[rows, cols].double() - want).abs() <= far).all(), (i, j)
