"""qmm_block_matmul at sizes about the borders between its kernels and their splits."""
import pytest

pytestmark = pytest.mark.gpu

pytest.importorskip("torch")
from test_gpu_block_matmul import check  # noqa: E402


@pytest.mark.parametrize("n,k", [(1000, 4096), (4096, 4112), (14336, 2048), (520, 1040), (4100, 512), (256, 256)])
@pytest.mark.parametrize("m", [1, 4, 5, 9, 16, 17, 32, 33, 64, 65, 97, 128, 129, 144, 200, 384, 513])
def test_rows(m, n, k):
    check(m, n, k, "bf16")


@pytest.mark.parametrize("m,n,k", [(1, 40000, 4096), (16, 40000, 4096), (17, 40000, 4096), (16, 19456, 4096),
                                   (16, 19457, 4096), (32, 9729, 4096), (33, 9728, 4096), (64, 4865, 4096)])
def test_wide(m, n, k):
    check(m, n, k, "f32")
