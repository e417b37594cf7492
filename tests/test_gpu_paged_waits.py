"""The prompt kernel's bounded waits, made to run out: every role stops, copies and
products in flight retire, tensor memory is freed, the status is reported, and the next
call is right.  (The other attention kernels have no waits that could run out.)"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from paged_util import Pool, attend, check, queries  # noqa: E402


@pytest.mark.parametrize("dtype,dim,page", [("bf16", 128, 16), ("f16", 64, 24), ("bf16", 128, 7)])
@pytest.mark.parametrize("lens", [[(2000, 300)], [(0, 700), (100, 40), (900, 64)]])
def test_a_wait_that_runs_out_is_reported(dtype, dim, page, lens):
    """One poll a wait, and nothing in L2: a poll may stay suspended for a while, but not
    for as long as the queries, table entries and keys take to come from memory.  Seen
    in 50 of 50 calls; one of ten is asked for."""
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    pool = Pool([a + b for a, b in lens], page, 2, dim, dtype)
    news = [b for _, b in lens]
    q = queries(pool, sum(news), 8)
    qmm.qmm_get_device_error()
    seen = []
    before = qmm.qmm_set_wait_limit(1)
    try:
        for _ in range(10):
            flush.zero_()
            attend(pool, q, news, 8, 0.1)
            seen.append(qmm.qmm_get_device_error())
    finally:
        qmm.qmm_set_wait_limit(before)
    assert set(seen) <= {qmm.QMM_OK, qmm.QMM_ERR_TIMEOUT} and qmm.QMM_ERR_TIMEOUT in seen
    check(pool, q, news, 8, 0.1)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
