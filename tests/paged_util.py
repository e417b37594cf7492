"""The paged-attention tests' inputs and their plain 64-bit results: block tables
by a host loop, rotations by complex products, attention row by row of the
definition.  Shares nothing with the library."""
import math

import torch

from mlx_grouped_affine_gb300 import qmm

# torch type, library type, unit roundoff (2^-p of a p-bit significand: half an
# ulp at the bottom of a binade)
TYPES = {"bf16": (torch.bfloat16, qmm.QMM_BF16, 2.0 ** -8), "f16": (torch.float16, qmm.QMM_F16, 2.0 ** -11),
         "f32": (torch.float32, qmm.QMM_F32, 2.0 ** -24)}


def pages(n, page):
    return -(-n // page)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Pool:
    """K and V pools whose rows that no request holds are NaN, and the requests'
    table (entries past a request's pages point at a page of NaN)."""

    def __init__(self, lens, page, heads, dim, dtype, layout="hnd", seed=0, spare=2, scale=1.0):
        dt, self.kind, _ = TYPES[dtype]
        g = torch.Generator().manual_seed(seed)
        held = [pages(n, page) for n in lens]
        self.num = sum(held) + spare
        order = torch.randperm(self.num, generator=g).tolist()
        self.width = max(held + [1]) + 1
        self.table_host = [[order[-1]] * self.width for _ in lens]
        shape = (self.num, heads, page, dim)
        k = torch.full(shape, math.nan)
        v = torch.full(shape, math.nan)
        self.keys, self.values = [], []
        at = 0
        for b, n in enumerate(lens):
            kb = (scale * torch.randn(heads, n, dim, generator=g)).to(dt)
            vb = torch.randn(heads, n, dim, generator=g).to(dt)
            self.keys.append(kb.double())
            self.values.append(vb.double())
            for p in range(held[b]):
                page_id = order[at]
                at += 1
                self.table_host[b][p] = page_id
                rows = min(page, n - p * page)
                k[page_id, :, :rows] = kb[:, p * page:p * page + rows].float()
                v[page_id, :, :rows] = vb[:, p * page:p * page + rows].float()
        if layout == "nhd":
            self.k, self.v = (x.transpose(1, 2).contiguous().to(dt).cuda().transpose(1, 2) for x in (k, v))
        else:
            self.k, self.v = (x.to(dt).cuda() for x in (k, v))
        self.table = i32(self.table_host)
        self.page, self.heads, self.dim, self.dt, self.dtype = page, heads, dim, dt, dtype

    def cache(self):
        s = self.k.stride()
        return qmm.PagedCache(self.k, self.v, self.kind, self.num, self.page, self.heads, self.dim,
                              s[0], s[1], s[2])

    def place(self, request, key):
        """(page, row) of a request's key."""
        return self.table_host[request][key // self.page], key % self.page


_workspace = {}


def workspace():
    if "w" not in _workspace:
        # Whatever it holds: NaN in every word.
        _workspace["w"] = torch.full((qmm.QMM_ATTENTION_WORKSPACE_BYTES // 4,), math.nan, device="cuda")
    return _workspace["w"]


def attend(pool, q, news, q_heads, scale, causal=True, window=0, seq=None, max_new=None, lse=True,
           q_stride=None, out=None, out_stride=None, stream=None, requests=None, lens=None):
    """The library's call; returns (out [T, Hq, D], lse [T, Hq] or None)."""
    d = pool.dim
    t = sum(news)
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    seq = [k.shape[1] for k in pool.keys] if seq is None else seq
    if out is None:
        out = torch.full((t, q_heads, d), 7.0, dtype=pool.dt, device="cuda")
    z = torch.full((t, q_heads), 7.0, device="cuda") if lse else None
    starts_d, seq_d, ws = i32(starts), i32(seq), workspace()
    qmm.qmm_paged_attention(q, q_heads * d if q_stride is None else q_stride, t, q_heads, pool.cache(),
                            pool.table, pool.width, starts_d, seq_d, len(news),
                            max(news) if max_new is None else max_new, scale, causal, window, out,
                            q_heads * d if out_stride is None else out_stride, z, ws, ws.numel() * 4,
                            stream=stream)
    return out, z


def expect(pool, q, news, q_heads, scale, causal=True, window=0, seq=None):
    """64-bit out, lse and the bounds of their errors.

    Bounds, from the arithmetic that the header states.  With A the largest
    scale * sum |q||k| of a row's keys and n of them: scores are off by at most
    ds = 2 (D + 8) 2^-24 A (fp32 sums of exact products, truncated or
    rounded) plus the scaling's two roundings, 2^-22 |s|; a weight by 2 ds + 2^-20
    relatively; sums of n fp32 terms by n 2^-23.  16-bit types round each
    weight (u) and the output (u); an fp16 weight below 2^-14 of the largest is
    off by up to 2^-24 of it instead.  All of it multiplies sum w |v|.
    """
    d, group = pool.dim, q_heads // pool.heads
    u = TYPES[pool.dtype][2]
    outs, lses, out_tol, lse_tol = [], [], [], []
    at = 0
    for b, new in enumerate(news):
        n_keys = pool.keys[b].shape[1] if seq is None else seq[b]
        qb = q[at:at + new].cpu().double().reshape(new, pool.heads, group, d)
        at += new
        k, v = pool.keys[b][:, :n_keys], pool.values[b][:, :n_keys]
        s = torch.einsum("ihgd,hjd->ihgj", qb, k) * scale
        mag = torch.einsum("ihgd,hjd->ihgj", qb.abs(), k.abs()) * abs(scale)
        pos = torch.arange(new)[:, None] + (n_keys - new)
        key = torch.arange(n_keys)[None]
        see = torch.ones(new, n_keys, dtype=torch.bool)
        if causal:
            see &= key <= pos
        if window:
            see &= key > pos - window
        see = see[:, None, None]
        s = torch.where(see, s, torch.tensor(-math.inf, dtype=torch.float64))
        if n_keys == 0:
            outs.append(torch.zeros(new, pool.heads, group, d, dtype=torch.float64))
            lses.append(torch.full((new, pool.heads, group), -math.inf, dtype=torch.float64))
            out_tol.append(torch.zeros_like(outs[-1]))
            lse_tol.append(torch.zeros_like(lses[-1]))
            continue
        z = torch.logsumexp(s, -1)
        w = torch.where(see, torch.exp(s - torch.where(z.isfinite(), z, 0.0)[..., None]), 0.0)
        v0 = v.nan_to_num(0.0, 0.0, 0.0)
        outs.append(torch.einsum("ihgj,hjd->ihgd", w, v0))
        spread = torch.einsum("ihgj,hjd->ihgd", w, v0.abs())
        a = torch.where(see, mag, 0.0).amax(-1)
        ds = 2 * (d + 8) * 2.0 ** -24 * a + 2.0 ** -22 * a
        count = see.sum(-1).double().expand_as(z)
        rel = 2 * ds + 2.0 ** -20 + count * 2.0 ** -23 + (u if pool.dtype != "f32" else 0.0)
        tol = rel[..., None] * spread + u * outs[-1].abs()
        if pool.dtype == "f16":
            top = w.amax(-1)
            tol = tol + (count * top)[..., None] * 2.0 ** -24 * v0.abs().amax((0, 1, 2)) + 2.0 ** -25
        out_tol.append(tol)
        lses.append(z)
        lse_tol.append(ds + 2.0 ** -20 + count * 2.0 ** -23 + z.nan_to_num(0, 0, 0).abs() * 2.0 ** -22)
    t = sum(news)
    shape = (t, q_heads, d)
    return (torch.cat(outs).reshape(shape), torch.cat(lses).reshape(t, q_heads),
            torch.cat(out_tol).reshape(shape), torch.cat(lse_tol).reshape(t, q_heads))


def check(pool, q, news, q_heads, scale, got=None, what="", **how):
    shape = {k: v for k, v in how.items() if k in ("causal", "window", "seq")}
    out, lse = attend(pool, q, news, q_heads, scale, **how) if got is None else got
    ref, ref_lse, tol, lse_tol = expect(pool, q, news, q_heads, scale, **shape)
    out = out.cpu().double()
    off = (out - ref).abs() - tol
    assert not out.isnan().any(), "%s: NaN in %s" % (what, out.isnan().nonzero()[0].tolist())
    assert (off <= 0).all(), "%s: %d of %d outside, worst %.3g past its bound at %s" % (
        what, int((off > 0).sum()), off.numel(), float(off.max()),
        (off == off.max()).nonzero()[0].tolist())
    if lse is not None:
        z = lse.cpu().double()
        none = ref_lse == -math.inf
        assert (z[none] == -math.inf).all(), what
        assert ((z - ref_lse).abs()[~none] <= lse_tol[~none]).all(), "%s: lse off by %.3g" % (
            what, float((z - ref_lse).abs()[~none].max()))


def queries(pool, t, q_heads, seed=1, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(t, q_heads, pool.dim, generator=g)).to(pool.dt).cuda()
