"""Host-side tests of the paged-attention calls (no GPU): every invalid argument
is refused before anything is launched (the pointers are never dereferenced)."""
import ctypes

import pytest

from mlx_grouped_affine_gb300 import qmm

A = 1 << 20
BAD, UNSUPPORTED, OK = qmm.QMM_ERR_INVALID_ARG, qmm.QMM_ERR_UNSUPPORTED, qmm.QMM_OK


def cache(**kw):
    c = dict(k=A, v=A, dtype=qmm.QMM_BF16, num_pages=10, page_size=16, heads=2, head_dim=64,
             page_stride=2048, head_stride=1024, token_stride=64)
    c.update(kw)
    return qmm.PagedCache(**c)


def plan(**kw):
    a = dict(past=A, new=A, B=2, free=A, F=5, nxt=None, page=16, table=A, stride=8, T=4, starts=A, seq=A,
             pos=A, slots=A, out=A)
    a.update(kw)
    return qmm.lib().qmm_page_plan(a["past"], a["new"], a["B"], a["free"], a["F"], a["nxt"], a["page"],
                                   a["table"], a["stride"], a["T"], a["starts"], a["seq"], a["pos"],
                                   a["slots"], a["out"], 0)


def rope(c=None, **kw):
    a = dict(q=A, qs=256, k=A, ks=128, v=A, vs=128, T=0, heads=4, pos=A, sec=[32], table=A, rows=9, r=64,
             inter=0, slots=A, out=A, os=256)
    a.update(kw)
    sec = None if a["sec"] is None else (ctypes.c_int32 * max(1, len(a["sec"])))(*a["sec"])
    axes = a.get("axes", 1 if a["sec"] is None else len(a["sec"]))
    return qmm.lib().qmm_rope_append(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["T"], a["heads"],
                                     a["pos"], axes, sec, a["table"], a["rows"], a["r"], a["inter"],
                                     a["slots"], a["out"], a["os"], cache() if c is None else c, 0)


def attend(c=None, **kw):
    a = dict(q=A, qs=256, T=3, heads=4, table=A, stride=8, starts=A, seq=A, B=0, most=1, scale=1.0,
             causal=1, window=0, out=A, os=256, lse=A, ws=A, bytes=qmm.QMM_ATTENTION_WORKSPACE_BYTES)
    a.update(kw)
    return qmm.lib().qmm_paged_attention(a["q"], a["qs"], a["T"], a["heads"], cache() if c is None else c,
                                         a["table"], a["stride"], a["starts"], a["seq"], a["B"], a["most"],
                                         a["scale"], a["causal"], a["window"], a["out"], a["os"], a["lse"],
                                         a["ws"], a["bytes"], 0)


def refused(status, *words):
    assert status == BAD
    for w in words:
        assert w in qmm.qmm_last_error(), (w, qmm.qmm_last_error())


@pytest.mark.parametrize("kw,word", [
    (dict(B=-1), "requests"), (dict(F=-1), "free_count"), (dict(T=2 ** 31), "tokens"),
    (dict(page=0), "page_size"), (dict(page=65537), "page_size"), (dict(stride=0), "table_stride"),
    (dict(starts=0), "starts"), (dict(out=A + 4), "next_free_out"), (dict(past=0), "past_lens"),
    (dict(new=A + 8), "new_lens"), (dict(table=0), "block_table"), (dict(seq=0), "seq_lens"),
    (dict(free=0), "free_pages"), (dict(pos=0), "positions"), (dict(slots=A + 2), "slots"),
    (dict(nxt=A), "next_free"), (dict(nxt=A + 4), "next_free"),
])
def test_page_plan_refuses(kw, word):
    refused(plan(**kw), "qmm_page_plan:", word)


@pytest.mark.parametrize("kw,word", [
    (dict(head_dim=0), "head_dim"), (dict(head_dim=60), "head_dim"), (dict(head_dim=264), "head_dim"),
    (dict(page_size=0), "page_size"), (dict(num_pages=0), "num_pages"), (dict(num_pages=2 ** 27), "num_pages"),
    (dict(heads=0), "heads"), (dict(heads=3), "heads"), (dict(page_stride=2044), "strides"),
    (dict(head_stride=32), "strides"), (dict(token_stride=2 ** 40), "strides"), (dict(token_stride=-64), "strides"),
    (dict(k=0), "k and v"), (dict(v=A + 2), "k and v"),
])
def test_caches_that_are_refused(kw, word):
    refused(rope(cache(**kw)), "qmm_rope_append:", word)
    refused(attend(cache(**kw)), "qmm_paged_attention:", word)


def test_null_cache_and_unknown_dtype():
    L = qmm.lib()
    refused(L.qmm_rope_append(A, 256, A, 128, A, 128, 1, 4, A, 1, (ctypes.c_int32 * 1)(32), A, 9, 64, 0, A, A,
                              256, None, 0), "null cache")
    assert rope(cache(dtype=3)) == UNSUPPORTED and attend(cache(dtype=-1)) == UNSUPPORTED


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), "tokens"), (dict(rows=0), "max_positions"), (dict(r=0), "rotary_dim"),
    (dict(r=24, sec=[12]), "rotary_dim"), (dict(r=80, sec=[40]), "rotary_dim"), (dict(inter=2), "interleaved"),
    (dict(sec=[]), "axes"), (dict(sec=[8] * 5), "axes"), (dict(sec=None, axes=1), "axes"),
    (dict(sec=[31]), "sections"), (dict(sec=[40, -8]), "negative"), (dict(heads=3), "heads"),
    (dict(qs=248), "stride of q "), (dict(ks=132), "stride of k"), (dict(vs=64), "stride of v"),
    (dict(os=0), "stride of q_out"), (dict(T=1, q=0), "q must"), (dict(T=1, k=A + 2), "k must"),
    (dict(T=1, v=0), "v must"), (dict(T=1, out=0), "q_out must"), (dict(os=512), "same stride"),
    (dict(T=1, pos=0), "positions"), (dict(T=1, slots=A + 4), "slots"), (dict(T=1, table=0), "cos_sin"),
])
def test_rope_append_refuses(kw, word):
    refused(rope(**kw), "qmm_rope_append:", word)


@pytest.mark.parametrize("kw,word", [
    (dict(T=-1), "tokens"), (dict(B=-1), "requests"), (dict(most=-1), "max_new"), (dict(window=-1), "window"),
    (dict(window=2 ** 31), "window"), (dict(stride=0), "table_stride"), (dict(causal=2), "causal"),
    (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"), (dict(heads=5), "heads"),
    (dict(qs=128), "stride of q"), (dict(os=260), "stride of out"), (dict(q=0), "q must"),
    (dict(out=A + 8), "out must"), (dict(B=2, table=0), "block_table"), (dict(B=2, starts=A + 4), "starts"),
    (dict(B=2, seq=0), "seq_lens"), (dict(B=2, lse=A + 4), "lse"), (dict(B=2, ws=0), "workspace"),
    (dict(B=2, bytes=qmm.QMM_ATTENTION_WORKSPACE_BYTES - 1), "workspace"),
])
def test_paged_attention_refuses(kw, word):
    refused(attend(**kw), "qmm_paged_attention:", word)


def test_empty_calls_are_no_ops():
    assert rope(T=0, q=0, k=0, v=0, out=0, pos=0, slots=0, table=0, os=256) == OK
    assert attend(T=0, B=2, q=0, out=0, table=0, starts=0, seq=0, ws=0) == OK
    assert attend(B=0, table=0, starts=0, seq=0, ws=0, bytes=0) == OK


def test_the_binding_raises():
    with pytest.raises(qmm.QmmError) as e:
        qmm.qmm_paged_attention(A, 256, 3, 4, cache(page_size=0), A, 8, A, A, 2, 1, 1.0, True, 0, A, 256, None,
                                A, 64 << 20, stream=0)
    assert e.value.status == BAD
