"""qmm_paged_attention with a workspace anywhere that its contract allows: any address
that is a multiple of 16, a slice of a larger buffer for instance."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
import paged_util  # noqa: E402
from paged_host import workspace_bases  # noqa: E402
from paged_util import Pool, attend, check, queries  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(3000, 1)], [(2000, 300)], [(900, 100), (2500, 1), (40, 2)]])
def test_slices_of_a_larger_buffer(dtype, lens, tmp_path, monkeypatch):
    """Items are cut in all of these, so their pieces pass through the workspace."""
    size = qmm.QMM_ATTENTION_WORKSPACE_BYTES
    arena = torch.full((size // 4 + 64,), math.nan, device="cuda")
    slices = [arena[x // 4:(x + size) // 4] for x in (0, 16, 32, 48, 112)]
    # Nothing is launched unless the base that the host computes can take the kernels' stores.
    for base, _ in workspace_bases(tmp_path, [s.data_ptr() for s in slices], size):
        assert base % 32 == 0
    pool = Pool([a + b for a, b in lens], 16, 2, 128, dtype)
    news = [b for _, b in lens]
    q = queries(pool, sum(news), 8)
    first, first_lse = attend(pool, q, news, 8, 0.1)
    check(pool, q, news, 8, 0.1, got=(first, first_lse))
    for s in slices:
        monkeypatch.setattr(paged_util, "workspace", lambda s=s: s)
        out, lse = attend(pool, q, news, 8, 0.1)
        assert torch.equal(out, first) and torch.equal(lse, first_lse)
    # Neither before nor behind the last slice is anything written.
    arena.fill_(math.nan)
    attend(pool, q, news, 8, 0.1)
    at = 112 // 4
    assert arena[:at].isnan().all() and arena[at + size // 4:].isnan().all()
