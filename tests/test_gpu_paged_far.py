"""qmm_paged_attention at the far end of what lengths can count: 2^31 - 1 keys of one
request, its pages the same few over and over, a window over the last of them."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from paged_util import TYPES, Pool, attend, check, queries  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("new", [1, 3, 90])
@pytest.mark.parametrize("page,dim,window", [(4096, 64, 1), (4096, 128, 100), (4104, 64, 300), (4099, 64, 1000)])
def test_the_last_keys_that_a_length_can_count(dtype, new, page, dim, window):
    """What a request of the last two pages' keys alone gives, page for page."""
    n = 2 ** 31 - 1
    width = -(-n // page)
    first = (width - 2) * page  # the first key of the last two pages
    near = Pool([n - first], page, 1, dim, dtype, spare=1)
    q = queries(near, new, 4)
    want, want_lse = attend(near, q, [new], 4, 0.1, window=window)
    check(near, q, [new], 4, 0.1, got=(want, want_lse), window=window)
    last = near.table[0, :2].clone()
    near.table = torch.full((1, width), near.table_host[0][2], dtype=torch.int32, device="cuda")
    near.table[0, -2:] = last
    near.width = width
    out, lse = attend(near, q, [new], 4, 0.1, window=window, seq=[n])
    # The same keys in other tiles: weights and sums round otherwise.
    u = TYPES[dtype][2]
    bound = (3 * u + window * 2.0 ** -23 + 2.0 ** -13) * float(near.values[0].abs().max())
    assert (out.double() - want.double()).abs().max() <= bound
    assert (lse - want_lse).abs().max() <= window * 2.0 ** -23 + 2.0 ** -13
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
