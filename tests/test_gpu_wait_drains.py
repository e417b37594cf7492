"""A kernel whose wait runs out leaves only when its own copies have landed, whichever of its
roles stopped.  Sizes at which every load fits its ring, so that the loading role has no wait
that could run out, behind a flushed L2, each followed at once (nothing waits in between) by a
call that uses the shared memory again and must be right."""
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm, synth  # noqa: E402
import moe_util  # noqa: E402
from block_util import bound, operands, product  # noqa: E402
from gpu_util import assert_within_tolerance, dev, empty_out, weight  # noqa: E402
from paged_util import Pool, attend, check, queries  # noqa: E402

TRIES = 10


@pytest.fixture(scope="module")
def flush():
    return torch.empty(1 << 28, dtype=torch.uint8, device="cuda")


def stopped_then_right(flush, call, right):
    """Runs call() with one poll a wait, then right() with the default; the statuses seen."""
    qmm.qmm_get_device_error()
    seen = []
    for _ in range(TRIES):
        flush.zero_()
        before = qmm.qmm_set_wait_limit(1)
        try:
            call()
        finally:
            qmm.qmm_set_wait_limit(before)
        right()
        seen.append(qmm.qmm_get_device_error())
    assert set(seen) <= {qmm.QMM_OK, qmm.QMM_ERR_TIMEOUT}
    return seen


@pytest.mark.parametrize("m,n,k", [(4, 1024, 4096),      # few rows: 4 steps a block, 5 stages
                                   (100, 640, 2048),     # 7 tiles of them: 2 steps a block
                                   (1024, 12800, 256)])  # tiles of many rows: 2 steps a tile, 4 stages
def test_block_product(flush, m, n, k):
    a, sa, w, sw = [t.cuda() for t in operands(m, n, k, 8)]
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    again = torch.empty_like(y)

    def call(out):
        qmm.qmm_block_matmul(a, sa, m, w, sw, n, k, out, qmm.QMM_BF16)

    seen = stopped_then_right(flush, lambda: call(y), lambda: call(again))
    assert qmm.QMM_ERR_TIMEOUT in seen
    want, terms = product(a, sa, w, sw)
    assert ((again.double() - want).abs() <= bound((want, terms), k, y.dtype)).all()


@pytest.mark.parametrize("bits", [4, 6])
@pytest.mark.parametrize("m,n,k,sure", [(256, 14336, 128, False),   # two steps: x and W fit their rings
                                        (256, 14336, 256, True),    # four: W does
                                        (1024, 14336, 128, True)])  # three tiles a block, two steps each
def test_quantized_product(flush, m, n, k, bits, sure):
    """(One poll may stay suspended until a first load has come; where more than that is waited
    for, waits ran out in every call.)"""
    w = synth.quant_weight(820 + m, n, k, bits, 64)
    x = synth.x_bf16(821 + m, m, k)
    px, parts = dev(x), weight(w)
    y, again = (empty_out((m, n), qmm.QMM_BF16) for _ in range(2))

    def call(out):
        qmm.qmm_quantized_matmul(px, m, *parts, n, k, 1, 64, bits, out, qmm.QMM_BF16)

    seen = stopped_then_right(flush, lambda: call(y), lambda: call(again))
    assert not sure or qmm.QMM_ERR_TIMEOUT in seen
    ref, absy = oracle.qmm(x, m, w.packed, w.scales, w.biases, n, k, True, 64, bits)
    assert_within_tolerance(again, ref, absy, "after a wait that ran out")


@pytest.mark.parametrize("dtype,dim,page", [("bf16", 128, 16), ("f16", 64, 24), ("bf16", 128, 7)])
def test_prompt_of_one_tile(flush, dtype, dim, page):
    """Keys of one tile: queries, K and V fit the ring (pages of 7 are copied by the lanes)."""
    pool = Pool([100], page, 2, dim, dtype)
    q = queries(pool, 100, 8)
    got = []
    seen = stopped_then_right(flush, lambda: attend(pool, q, [100], 8, 0.1),
                              lambda: got.append(attend(pool, q, [100], 8, 0.1)))
    assert qmm.QMM_ERR_TIMEOUT in seen
    for g in got:
        check(pool, q, [100], 8, 0.1, got=g)


class FarLayer(moe_util.Layer):
    """Experts made on the GPU, whole memory's random words."""

    def __init__(self, experts, hidden, inner, bits, group):
        self.experts, self.hidden, self.inner, self.bits, self.group = experts, hidden, inner, bits, group
        g = torch.Generator(device="cuda").manual_seed(bits)

        def part(rows, cols):
            words = torch.empty(experts, rows, cols * bits // 32, dtype=torch.int32, device="cuda")
            for e in range(experts):
                words[e].random_(-2 ** 31, 2 ** 31 - 1, generator=g)
            s = torch.empty(experts, rows, cols // group, dtype=torch.bfloat16, device="cuda").uniform_(0.002, 0.02, generator=g)
            return words, s.mul_(8 / 2 ** (bits - 1)), s * -2 ** (bits - 1)

        self.parts = [part(inner, hidden), part(inner, hidden), part(hidden, inner)]
        self.handle = qmm.Experts(*self.parts, qmm.QMM_BF16, experts, hidden, inner, group, bits)


@pytest.mark.parametrize("experts,hidden,inner,bits,group", [
    (1024, 2048, 4096, 8, 64),  # experts spread over 8.6 GB each of gate, up and down
    (1024, 992, 2080, 6, 32),   # rows of gate and up that the lanes copy
])
def test_expert_layer(flush, experts, hidden, inner, bits, group):
    """Weights far apart in memory: a chunk takes longer than a poll may stay suspended.  (Waits
    of the first case ran out in every call measured; in the second, and with weights of less than a
    few GB, none was seen to.  It depends on memory alone, so the status may be either.)"""
    t, top = 64, 8
    layer = FarLayer(experts, hidden, inner, bits, group)
    ids, weights = moe_util.random_ids(t, top, experts, 3)
    x = torch.randn(t, hidden, generator=torch.Generator().manual_seed(t)).bfloat16().cuda()
    y, again = (torch.empty(t, hidden, device="cuda") for _ in range(2))
    ws, n = moe_util.workspace(t, top, hidden, inner)

    def call(to):
        qmm.qmm_moe_experts(x, qmm.QMM_BF16, t, ids, weights, top, layer.handle, to, qmm.QMM_F32, ws, n)

    print(stopped_then_right(flush, lambda: call(y), lambda: call(again)))
    few = [0, 31, 63]
    want, far = moe_util.reference(layer, x[few], ids[few], weights[few], again.dtype)
    assert ((again[few].double() - want).abs() <= far).all()
