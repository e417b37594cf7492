"""qmm_paged_attention with scores so large that fp32 counts them in ones and fours."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from paged_util import TYPES, Pool, attend  # noqa: E402


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("size", range(18, 27))
@pytest.mark.parametrize("lens", [[(900, 1), (70, 2)], [(300, 300), (0, 130)]])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_one_key_takes_all(dtype, size, lens, sign):
    """Scores are one exact product a key, up to 2^size, and the largest that a row sees is
    2^(size - 7) above the others: 2^11 and more, so all weights but its own are 0 and the
    output is its value.  Bounds: the weight beside its reference, a rounded score, is any
    number: 16-bit types round it and the output once each, 2 u; 2^-22 for the sums.
    The statistic is the largest score, three roundings of 2^-24."""
    pool = Pool([a + b for a, b in lens], 16, 1, 64, dtype, seed=size)
    news = [b for _, b in lens]
    g = torch.Generator().manual_seed(size)
    q = torch.zeros(sum(news), 4, 64, dtype=pool.dt, device="cuda")
    q[:, :, 5] = sign * 2.0 ** (size // 2)
    want, stat = [], []
    for b, (past, new) in enumerate(lens):
        n = past + new
        k = torch.randint(64, 96, (n,), generator=g).double()
        k[0] = 96
        k[torch.randperm(n, generator=g)[:24].sort().values] = torch.arange(97, 121).double()  # the maximum climbs
        keys = sign * k * 2.0 ** (size - size // 2 - 7)
        for p in range(-(-n // 16)):
            page, rows = pool.table_host[b][p], min(16, n - 16 * p)
            pool.k[page, 0, :rows] = 0
            pool.k[page, 0, :rows, 5] = keys[16 * p:16 * p + rows].to(pool.dt).cuda()
        for i in range(new):
            top = int(k[:past + i + 1].argmax())
            want.append(pool.values[b][0, top])
            stat.append(float(k[top]) * 2.0 ** (size - 7))
    out, lse = attend(pool, q, news, 4, 1.0)
    want = torch.stack(want)[:, None]
    bound = (2 * TYPES[dtype][2] + 2.0 ** -22) * want.abs()
    assert ((out.cpu().double() - want).abs() <= bound).all()
    stat = torch.tensor(stat, dtype=torch.float64)[:, None]
    assert ((lse.cpu().double() - stat).abs() <= 2.0 ** -21 * stat).all()
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens", [(500, 1), (40, 200)])
@pytest.mark.parametrize("value", [2.0 ** 9, -(2.0 ** 9)])
def test_all_scores_the_same(dtype, lens, value):
    """All 2^24 or -2^24: each key weighs alike, and the weight's rounding is one for all
    of them.  Bounds: u for it, u for the output, n 2^-23 for sums of n."""
    pool = Pool([sum(lens)], 16, 1, 64, dtype)
    pool.k.fill_(value)
    q = torch.full((lens[1], 4, 64), 2.0 ** 9, dtype=pool.dt, device="cuda")
    out, _ = attend(pool, q, [lens[1]], 4, 1.0)
    v = pool.values[0][0]
    count = torch.arange(lens[0] + 1, sum(lens) + 1)[:, None]
    want = (torch.cumsum(v, 0)[lens[0]:] / count)[:, None]
    bound = 2 * TYPES[dtype][2] * want.abs() + (sum(lens) * 2.0 ** -23 + 2.0 ** -20) * v.abs().max()
    assert ((out.cpu().double() - want).abs() <= bound).all()
