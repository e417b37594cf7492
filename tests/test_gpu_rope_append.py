"""qmm_rope_append against complex products in 64 bits."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from paged_util import TYPES, i32  # noqa: E402

@pytest.fixture(autouse=True)
def clear_what_earlier_calls_left():
    """The device error word holds what any earlier call reported until it is read."""
    qmm.qmm_get_device_error()


def run(t, hq, hk, d, r, sections, dtype, page=16, layout="hnd", interleaved=False, in_place=False,
        positions=None, slots=None, rows=500, seed=0, pad=0):
    dt, kind, u = TYPES[dtype]
    g = torch.Generator().manual_seed(seed)
    num = -(-t // page) + 3
    shape = (num, hk, page, d) if layout == "hnd" else (num, page, hk, d)
    pools = [torch.full(shape, 9.0, dtype=dt, device="cuda") for _ in range(2)]
    if layout == "nhd":
        pools = [p.transpose(1, 2) for p in pools]
    qkv = torch.randn(t, (hq + 2 * hk) * d + pad, generator=g).to(dt).cuda()
    q, k, v = (qkv[:, a * d:b * d] for a, b in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
    x = qkv.cpu().double()[:, :(hq + 2 * hk) * d].reshape(t, hq + 2 * hk, d)
    if positions is None:
        positions = torch.randint(0, rows, (len(sections), t), generator=g).tolist()
    if slots is None:
        slots = torch.randperm(num * page, generator=g)[:t].tolist()
    angle = torch.rand(rows, r // 2, generator=g) * 6.3
    table = torch.cat([angle.cos(), angle.sin()], 1)
    out = q if in_place else torch.full((t, hq * d + 8), 9.0, dtype=dt, device="cuda")
    s = pools[0].stride()
    cache = qmm.PagedCache(pools[0], pools[1], kind, num, page, hk, d, s[0], s[1], s[2])
    qmm.qmm_rope_append(q, qkv.stride(0), k, qkv.stride(0), v, qkv.stride(0), t, hq, i32(positions), sections,
                        table.cuda(), rows, r, interleaved, i32(slots), out, out.stride(0), cache)
    # The definition, pair by pair.
    axis = sum(([a] * n for a, n in enumerate(sections)), [])
    turned, tol = x.clone(), torch.zeros_like(x)
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        pos = torch.tensor(positions[axis[i]])
        ok = (pos >= 0) & (pos < rows)
        row = table.double()[pos.clamp(0, rows - 1)]
        c = torch.where(ok, row[:, i], 0.0)[:, None]
        s_ = torch.where(ok, row[:, r // 2 + i], 0.0)[:, None]
        h = slice(0, hq + hk)
        turned[:, h, a] = x[:, h, a] * c - x[:, h, b] * s_
        turned[:, h, b] = x[:, h, b] * c + x[:, h, a] * s_
        # two products and a sum in fp32 (each 2^-24 of the terms), one rounding to the type
        size = (x[:, h, a].abs() + x[:, h, b].abs()) * 2.0 ** -22
        tol[:, h, a] = tol[:, h, b] = size
    tol = tol + turned.abs() * u + (2.0 ** -25 if dtype == "f16" else 0.0)
    got = out.cpu().double()[:, :hq * d].reshape(t, hq, d)
    assert ((got - turned[:, :hq]).abs() <= tol[:, :hq]).all(), "q"
    if not in_place:
        assert (out[:, hq * d:] == 9.0).all()
    want = [torch.full((num, hk, page, d), 9.0, dtype=torch.float64) for _ in range(2)]
    room = torch.zeros(num, hk, page, d, dtype=torch.float64)
    for i, slot in enumerate(slots):
        if 0 <= slot < num * page:
            want[0][slot // page, :, slot % page] = turned[i, hq:hq + hk]
            want[1][slot // page, :, slot % page] = x[i, hq + hk:]
            room[slot // page, :, slot % page] = tol[i, hq:hq + hk]
    assert ((pools[0].cpu().double() - want[0]).abs() <= room).all(), "k"
    assert torch.equal(pools[1].cpu().double(), want[1]), "v"


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,hq,hk,d,r,sections", [
    (1, 32, 8, 128, 128, [64]),
    (17, 8, 8, 64, 64, [32]),
    (5, 7, 1, 80, 32, [16]),
    (33, 3, 3, 96, 96, [20, 14, 14]),
    (130, 4, 2, 128, 128, [16, 24, 24]),
    (9, 6, 2, 256, 64, [1, 30, 0, 1]),
    (4, 5, 5, 16, 16, [3, 5]),
    (3, 1, 1, 24, 16, [8]),
    (700, 2, 1, 128, 128, [63, 1]),
])
def test_rotates_and_appends(dtype, interleaved, t, hq, hk, d, r, sections):
    run(t, hq, hk, d, r, sections, dtype, interleaved=interleaved)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


@pytest.mark.parametrize("page,layout,pad", [(1, "hnd", 0), (7, "nhd", 8), (200, "hnd", 24), (16, "nhd", 0)])
def test_layouts(page, layout, pad):
    for dtype in ("bf16", "f32"):
        run(50, 8, 2, 64, 64, [32], dtype, page=page, layout=layout, pad=pad)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(interleaved):
    for dtype in ("bf16", "f16", "f32"):
        run(40, 8, 2, 128, 64, [16, 16], dtype, in_place=True, interleaved=interleaved)


def test_tokens_without_a_slot_are_not_kept():
    run(6, 4, 2, 64, 64, [32], "bf16", slots=[3, -1, 0, -1, 20, 9])
    assert qmm.qmm_get_device_error() == qmm.QMM_OK


def test_slots_and_positions_outside_are_reported():
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    run(4, 4, 2, 64, 64, [32], "bf16", slots=[3, 10 ** 6, 0, 2 ** 31 - 1])
    assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX
    for dtype in ("bf16", "f32"):
        run(4, 4, 2, 64, 64, [16, 16], dtype, positions=[[1, 500, 3, -1], [0, 1, 2 ** 31 - 1, 3]])
        assert qmm.qmm_get_device_error() == qmm.QMM_ERR_INDEX


def test_no_tokens():
    c = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    cache = qmm.PagedCache(c, c, qmm.QMM_BF16, 1, 16, 1, 64, 1024, 1024, 64)
    qmm.qmm_rope_append(None, 64, None, 64, None, 64, 0, 1, None, [32], None, 5, 64, 0, None, None, 64, cache)
    assert not math.isnan(float(c.sum()))
