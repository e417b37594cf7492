"""qmm_block_matmul at sizes about the borders between its kernels and their splits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from block_util import bound, operands, product  # noqa: E402
from test_gpu_block_matmul import check, run  # noqa: E402


@pytest.mark.parametrize("n,k", [(1000, 4096), (4096, 4112), (14336, 2048), (520, 1040), (4100, 512), (256, 256)])
@pytest.mark.parametrize("m", [1, 4, 5, 9, 16, 17, 32, 33, 64, 65, 97, 128, 129, 144, 200, 384, 513])
def test_rows(m, n, k):
    check(m, n, k, "bf16")


@pytest.mark.parametrize("m,n,k", [(1, 40000, 4096), (16, 40000, 4096), (17, 40000, 4096), (16, 19456, 4096),
                                   (16, 19457, 4096), (32, 9729, 4096), (33, 9728, 4096), (64, 4865, 4096)])
def test_wide(m, n, k):
    check(m, n, k, "f32")


@pytest.mark.parametrize("m", [3, 200])
def test_scales_whose_product_leaves_fp32(m):
    """Scales of a block are multiplied first: 2^-160 is 0, the block has no part in y; 2^128 is
    infinite, and so is y where the block's sum is not 0."""
    a, sa, w, sw = operands(m, 300, 384, m)
    sa[:, 1], sw[:, 1] = 2.0 ** -80, 2.0 ** -80
    y = run(a, sa, w, sw, "f32").double().cpu()
    sa[:, 1] = 0
    want, terms = product(a, sa, w, sw)
    assert ((y - want).abs() <= bound((want, terms), 384, torch.float32)).all()
    sa[:, 1], sw[:, 1] = 2.0 ** 64, 2.0 ** 64
    y = run(a, sa, w, sw, "f32")
    assert not y.isfinite().any()
