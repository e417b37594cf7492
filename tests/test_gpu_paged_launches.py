"""How many kernels a qmm_paged_attention call launches: the few-rows kernel and the
many-rows kernel, each with its join, only where a request can be of its kind."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from mlx_grouped_affine_gb300 import qmm  # noqa: E402
from paged_util import Pool, check, i32, queries, workspace  # noqa: E402


def launches(pool, q, news, heads, scale):
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    out, ws = torch.empty_like(q), workspace()
    args = (q, heads * pool.dim, sum(news), heads, pool.cache(), pool.table, pool.width, i32(starts),
            i32([k.shape[1] for k in pool.keys]), len(news), max(news), scale, True, 0, out, heads * pool.dim, None,
            ws, ws.numel() * 4)
    qmm.qmm_paged_attention(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        qmm.qmm_paged_attention(*args)
    count = ctypes.c_size_t()
    nodes = ctypes.CDLL("libcuda.so.1").cuGraphGetNodes
    nodes.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)]
    assert nodes(graph.raw_cuda_graph(), None, ctypes.byref(count)) == 0
    return count.value


@pytest.mark.parametrize("group,lens,want", [
    (4, [(300, 1), (5, 2)], 2),              # few rows each
    (4, [(300, 90), (0, 40)], 2),            # many rows each
    (4, [(300, 90), (50, 1)], 4),            # both
    (4, [(300, 90), (50, 0)], 4),            # the host cannot know that the other is idle
    (33, [(300, 90), (50, 0)], 2),           # a group wider than 32 rows: never few
    (40, [(100, 64), (9, 1), (3, 0)], 2),
])
def test_launches(group, lens, want):
    pool = Pool([a + b for a, b in lens], 16, 1, 64, "bf16")
    news = [b for _, b in lens]
    q = queries(pool, sum(news), group)
    check(pool, q, news, group, 0.125)
    assert launches(pool, q, news, group, 0.125) == want
