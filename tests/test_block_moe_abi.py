"""Host-side tests of the block-scaled and mixture-of-experts calls (no GPU): invalid
arguments are refused before anything is launched (pointers are never dereferenced)."""
import ctypes

import pytest

from mlx_grouped_affine_gb300 import qmm

A = 1 << 30
STEP = 1 << 28
BAD, UNSUPPORTED, OK = qmm.QMM_ERR_INVALID_ARG, qmm.QMM_ERR_UNSUPPORTED, qmm.QMM_OK


def at(i):
    """Addresses far apart."""
    return A + i * STEP


def quantize(**kw):
    a = dict(x=at(0), dt=qmm.QMM_BF16, rows=4, cols=256, br=1, codes=at(1), scales=at(2))
    a.update(kw)
    return qmm.lib().qmm_block_quantize(a["x"], a["dt"], a["rows"], a["cols"], a["br"], a["codes"],
                                        a["scales"], 0)


def matmul(**kw):
    a = dict(a=at(0), sa=at(1), M=4, w=at(2), sw=at(3), N=64, K=256, y=at(4), dt=qmm.QMM_BF16)
    a.update(kw)
    return qmm.lib().qmm_block_matmul(a["a"], a["sa"], a["M"], a["w"], a["sw"], a["N"], a["K"], a["y"],
                                      a["dt"], 0)


def route(**kw):
    a = dict(l=at(0), dt=qmm.QMM_F32, T=4, E=16, k=2, sc=0, norm=1, scale=1.0, ids=at(1), w=at(2))
    a.update(kw)
    return qmm.lib().qmm_moe_route(a["l"], a["dt"], a["T"], a["E"], a["k"], a["sc"], a["norm"], a["scale"],
                                   a["ids"], a["w"], 0)


def handle(**kw):
    a = dict(gate=(at(10), at(11), at(12)), up=(at(13), at(14), at(15)), down=(at(16), at(17), at(18)),
             sb_dtype=qmm.QMM_BF16, experts=16, hidden=256, inner=128, group_size=64, bits=4)
    a.update(kw)
    return qmm.Experts(**a)


def experts(e=None, **kw):
    a = dict(x=at(0), dt=qmm.QMM_BF16, T=4, ids=at(1), w=at(2), k=2, y=at(3), yd=qmm.QMM_BF16, ws=at(4),
             n=1 << 20)
    a.update(kw)
    return qmm.lib().qmm_moe_experts(a["x"], a["dt"], a["T"], a["ids"], a["w"], a["k"],
                                     handle() if e is None else e, a["y"], a["yd"], a["ws"], a["n"], 0)


def layer(e=None, **kw):
    a = dict(x=at(0), dt=qmm.QMM_BF16, T=4, l=at(1), ld=qmm.QMM_F32, k=2, sc=0, norm=1, scale=1.0, y=at(3),
             yd=qmm.QMM_BF16, ws=at(4), n=1 << 20)
    a.update(kw)
    return qmm.lib().qmm_moe_layer(a["x"], a["dt"], a["T"], a["l"], a["ld"], a["k"], a["sc"], a["norm"],
                                   a["scale"], handle() if e is None else e, a["y"], a["yd"], a["ws"],
                                   a["n"], 0)


def refused(status, op, word, want=BAD):
    assert status == want
    assert op + ":" in qmm.qmm_last_error() and word in qmm.qmm_last_error(), qmm.qmm_last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(rows=-1), "rows"), (dict(cols=-16), "cols"), (dict(cols=24), "multiple of 16"),
    (dict(rows=2 ** 31), "rows"), (dict(br=0), "block_rows"), (dict(br=64), "block_rows"), (dict(x=0), "x must"),
    (dict(codes=at(1) + 8), "codes"), (dict(scales=0), "scales"), (dict(codes=at(0) + 1024), "codes lies over x"),
    (dict(scales=at(0)), "scales lies over x"), (dict(scales=at(1) + 16), "overlap"),
])
def test_block_quantize_refuses(kw, word):
    refused(quantize(**kw), "qmm_block_quantize", word)


@pytest.mark.parametrize("kw,word", [
    (dict(M=-1), "M (-1)"), (dict(N=-1), "N (-1)"), (dict(K=0), "K"), (dict(K=100), "multiple of 16"),
    (dict(N=2 ** 31), "N"), (dict(a=0), "a must"), (dict(sa=at(1) + 4), "a_scales"), (dict(w=at(2) + 8), "w must"),
    (dict(sw=0), "w_scales"), (dict(y=0), "y must"), (dict(y=at(2) + 16), "y lies over w"),
    (dict(y=at(1)), "y lies over a_scales"),
])
def test_block_matmul_refuses(kw, word):
    refused(matmul(**kw), "qmm_block_matmul", word)


ROUTING = [(dict(k=0), "top_k"), (dict(k=17), "top_k"), (dict(sc=2), "scoring"), (dict(norm=2), "normalize"),
           (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"), (dict(l=0), "logits"),
           (dict(l=at(1) + 2), "logits")]


@pytest.mark.parametrize("kw,word", ROUTING + [
    (dict(T=-1), "tokens"), (dict(E=0), "experts"), (dict(E=1025), "experts"), (dict(E=64, k=33), "top_k"),
    (dict(ids=0), "ids"), (dict(w=at(2) + 4), "weights"), (dict(ids=at(0)), "ids lies over logits"),
    (dict(w=at(1) + 16), "overlap"),
])
def test_moe_route_refuses(kw, word):
    refused(route(**kw), "qmm_moe_route", word)


COMMON = [(dict(T=-1), "tokens"), (dict(T=65), "tokens"), (dict(T=64, k=9), "at most"), (dict(x=0), "x must"),
          (dict(y=at(3) + 8), "y must"), (dict(ws=0), "workspace"), (dict(ws=at(4) + 4), "workspace"),
          (dict(n=100), "workspace needs"), (dict(n=-1), "workspace"), (dict(y=at(0)), "y lies over x"),
          (dict(ws=at(0) + 16), "workspace lies over x"), (dict(ws=at(3) + 16), "overlap"),
          (dict(y=at(16) + 64), "y lies over down"), (dict(ws=at(12)), "workspace lies over gate_biases")]


@pytest.mark.parametrize("kw,word", COMMON + [(dict(k=0), "top_k"), (dict(k=33), "top_k"), (dict(ids=0), "ids"),
                                              (dict(w=at(2) + 2), "weights"), (dict(y=at(1)), "y lies over ids")])
def test_moe_experts_refuses(kw, word):
    refused(experts(**kw), "qmm_moe_experts", word)


@pytest.mark.parametrize("kw,word", COMMON + ROUTING + [(dict(y=at(1)), "y lies over logits")])
def test_moe_layer_refuses(kw, word):
    refused(layer(**kw), "qmm_moe_layer", word)


@pytest.mark.parametrize("kw,word", [
    (dict(experts=0), "experts"), (dict(experts=1025), "experts"), (dict(hidden=0), "hidden"),
    (dict(hidden=96), "hidden"), (dict(inner=100), "inner"), (dict(inner=-64), "inner"), (dict(group_size=16), "group"),
    (dict(bits=7), "bits"), (dict(bits=0), "bits"), (dict(gate=(0, at(11), at(12))), "gate must"),
    (dict(up=(at(13), at(14) + 2, at(15))), "up_scales"), (dict(down=(at(16), at(17), 0)), "down_biases"),
])
def test_experts_that_are_refused(kw, word):
    refused(experts(handle(**kw)), "qmm_moe_experts", word)
    refused(layer(handle(**kw)), "qmm_moe_layer", word)


def test_unknown_types():
    assert quantize(dt=3) == UNSUPPORTED and matmul(dt=-1) == UNSUPPORTED and route(dt=9) == UNSUPPORTED
    assert experts(dt=4) == UNSUPPORTED and layer(ld=4) == UNSUPPORTED
    assert experts(handle(sb_dtype=5)) == UNSUPPORTED
    refused(experts(yd=qmm.QMM_F16), "qmm_moe_experts", "output dtype", UNSUPPORTED)
    null = ctypes.POINTER(qmm.Experts)()
    assert qmm.lib().qmm_moe_experts(A, 1, 1, A, A, 1, null, A, 1, A, 1 << 20, 0) == BAD
    assert qmm.lib().qmm_moe_layer(A, 1, 1, A, 0, 1, 0, 1, 1.0, null, A, 1, A, 1 << 20, 0) == BAD


def test_empty_outputs_are_no_ops():
    assert quantize(rows=0, x=0, codes=0, scales=0) == OK and quantize(cols=0) == OK
    assert matmul(M=0, y=0) == OK and matmul(N=0) == OK
    assert route(T=0, l=0) == OK
    assert experts(T=0, x=0, ids=0) == OK and layer(T=0, l=0) == OK


def test_workspace_sizes():
    n = qmm.qmm_moe_workspace_bytes
    assert 0 < n(1, 1, 64, 64) <= n(64, 8, 64, 64) <= n(64, 8, 4096, 14336) < 1 << 27
    assert n(65, 1, 64, 64) == n(64, 9, 64, 64) == n(1, 0, 64, 64) == n(1, 33, 64, 64) == n(-1, 1, 64, 64) == -1
    assert n(1, 1, -1, 64) == n(1, 1, 64, 2 ** 31) == -1
