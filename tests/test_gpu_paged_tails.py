"""qmm_paged_attention in fp16 where one key's weight stands far above a long tail: each
of the others is near or below what fp16 holds beside 1, together they count."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from paged_util import Pool, attend, check, queries  # noqa: E402


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("requests,new,group", [(40, 1, 4), (40, 3, 2), (10, 40, 2), (10, 300, 1)])
@pytest.mark.parametrize("peak", ["first", "last"])
@pytest.mark.parametrize("depth", [20.6, 23.3, 25.7, 27.0])
def test_a_flat_tail_far_below_one_peak(dim, requests, new, group, peak, depth):
    """The peak's value is 0 and the tail's are 1 to 2, so the output is the tail's alone.
    Requests enough (of the same pages) that few blocks share one's keys: a key is
    rounded beside the keys that its block and warp have seen.

    Bounds: scores are one exact product (q and k differ from 0 in one column) times the
    scale, two roundings, off by 2^-22 of the largest in log2 (27 at most), so a weight
    by 2^-17; sums of n terms by n 2^-23 (n = 20000: 0.24 %); a weight by its rounding,
    u = 2^-11 of it, or, too small for all of its bits, by 2^-32 of the largest at most
    (of the two kernels'); the output by u.  A tail rounded beside 1 would be off by up
    to 2^-25 a key, 4 % to all of it here."""
    n, page, kv = 20000, 64, 8
    pool = Pool([n], page, kv, dim, "f16")
    pool.table = pool.table.repeat(requests, 1)
    k, v = torch.zeros(n, dim), 1.0 + torch.rand(n, dim, generator=torch.Generator().manual_seed(5))
    scale = 0.125
    k[:, 3] = -depth * math.log(2.0) / scale / 8.0
    top = 0 if peak == "first" else n - new  # a key that every row sees
    k[top], v[top] = 0.0, 0.0
    k, v = k.half(), v.half()
    rows = torch.arange(n)
    pages = torch.tensor(pool.table_host[0])[rows // page].cuda()
    pool.k[pages, :, (rows % page).cuda()] = k.cuda()[:, None]
    pool.v[pages, :, (rows % page).cuda()] = v.cuda()[:, None]
    q = torch.zeros(requests * new, kv * group, dim, dtype=torch.float16, device="cuda")
    q[:, :, 3] = 8.0
    out, lse = attend(pool, q, [new] * requests, kv * group, scale, seq=[n] * requests)
    # Row i of a request sees keys 0 .. n - new + i.
    w = torch.exp(k[:, 3].double() * 8.0 * scale)
    mass, whole = torch.cumsum(w, 0)[n - new:], torch.cumsum(w[:, None] * v.double(), 0)[n - new:]
    want = (whole / mass[:, None])[None, :, None]
    u = 2.0 ** -11
    rel = 2.0 ** -17 + n * 2.0 ** -23 + max(u, 2.0 ** (depth - 32)) + u
    got = out.double().cpu().reshape(requests, new, kv * group, dim)
    worst = ((got - want).abs() / want).max()
    assert worst <= rel, "off by %.4g, bound %.4g" % (float(worst), rel)
    z = (lse.double().cpu().reshape(requests, new, -1) - mass.log()[None, :, None]).abs().max()
    assert z <= 2.0 ** -17 + n * 2.0 ** -23
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("lens", [[(3000, 1), (50, 2)], [(500, 300), (0, 90)]])
def test_values_at_the_ends_of_the_range(lens):
    """Weights raised above 1 times values near fp16's largest stay finite."""
    pool = Pool([a + b for a, b in lens], 16, 2, 128, "f16")
    news = [b for _, b in lens]
    pool.v.mul_(2.0 ** 13)
    pool.values = [x * 2.0 ** 13 for x in pool.values]
    assert max(float(x.abs().max()) for x in pool.values) > 30000
    check(pool, queries(pool, sum(news), 8), news, 8, 128 ** -0.5)
