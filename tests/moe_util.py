"""Plain 64-bit forms of the mixture-of-experts calls, and their inputs."""
import math

import torch

from mlx_grouped_affine_gb300 import qmm

TYPES = {"f32": (torch.float32, qmm.QMM_F32), "bf16": (torch.bfloat16, qmm.QMM_BF16),
         "f16": (torch.float16, qmm.QMM_F16)}


def packed(count, rows, cols, bits, group, dtype, g):
    words = torch.randint(-2 ** 31, 2 ** 31, (count, rows, cols * bits // 32), generator=g, dtype=torch.int64)
    s = (torch.rand(count, rows, cols // group, generator=g) * 0.018 + 0.002) * 8 / 2 ** (bits - 1)
    b = -s * 2 ** (bits - 1) + torch.randn(s.shape, generator=g) * 1e-3
    return words.to(torch.int32).cuda(), s.to(dtype).cuda(), b.to(dtype).cuda()


class Layer:
    """Random experts on the GPU."""

    def __init__(self, experts, hidden, inner, bits, group, sb="bf16", seed=0):
        g = torch.Generator().manual_seed(seed)
        dt, self.sb = TYPES[sb]
        self.experts, self.hidden, self.inner, self.bits, self.group = experts, hidden, inner, bits, group
        self.parts = [packed(experts, inner, hidden, bits, group, dt, g),
                      packed(experts, inner, hidden, bits, group, dt, g),
                      packed(experts, hidden, inner, bits, group, dt, g)]
        self.handle = qmm.Experts(*self.parts, self.sb, experts, hidden, inner, group, bits)

    def dense(self, part, e):
        """(weight, |scale * code| + |bias|) of expert e in 64 bits, codes bit by bit."""
        words, scales, biases = (t[e] for t in self.parts[part])
        bit = (words[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        stream = bit.reshape(words.shape[0], -1, self.bits).double()
        codes = stream @ (2.0 ** torch.arange(self.bits, device="cuda", dtype=torch.float64))
        s = scales.double().repeat_interleave(self.group, 1)
        b = biases.double().repeat_interleave(self.group, 1)
        return codes * s + b, (codes * s).abs() + b.abs()


def workspace(tokens, top, hidden, inner, fill=0xFF):
    """Exactly the bytes asked for, holding NaN patterns, between guards."""
    n = qmm.qmm_moe_workspace_bytes(tokens, top, hidden, inner)
    return torch.full((n + 512,), fill, dtype=torch.uint8, device="cuda"), n


def reference(layer, x, ids, weights, out_dtype):
    """(y, bound) in 64 bits.  The bound follows the sums: n additions of fp32, cut or
    rounded, cost n * 2^-23 of the sum of magnitudes; a few roundings more (scales, biases,
    planes of x) 8; silu's slope is below 1.1 and its own error 2^-20; silu * up keeps 15
    bits (23 in fp32)."""
    d = x.double()
    y, far = torch.zeros_like(d), torch.zeros_like(d)
    eps = 2.0 ** -23
    keep = 2.0 ** -22 if x.dtype == torch.float32 else 2.0 ** -15
    for e in sorted(set(ids.flatten().tolist())):
        if not 0 <= e < layer.experts:
            continue
        share = torch.where(ids == e, weights, torch.zeros_like(weights)).double()
        mass, share = share.abs().sum(1, keepdim=True), share.sum(1, keepdim=True)
        at = (mass[:, 0] > 0).nonzero()[:, 0]
        if at.numel() == 0:
            continue
        r = d[at]
        (wg, ag), (wu, au), (wd, ad) = (layer.dense(i, e) for i in range(3))
        g, u = r @ wg.T, r @ wu.T
        dg, du = (r.abs() @ ag.T) * (layer.hidden + 8) * eps, (r.abs() @ au.T) * (layer.hidden + 8) * eps
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + h.abs() * (keep + 2.0 ** -20)
        z = h @ wd.T
        dz = dh @ ad.T + (h.abs() + dh) @ ad.T * (layer.inner + 8) * eps
        y[at] += share[at] * z
        far[at] += mass[at] * (dz + z.abs() * 2.0 ** -18)  # weights and the sum over experts
    return y, far + y.abs() * torch.finfo(out_dtype).eps / 2


def routed(logits, top, sigmoid, normalize, scale):
    """(ids, weights in 64 bits) of CPU logits, by sorting."""
    l = logits.double()
    l = torch.where(l.isnan(), -math.inf, l)
    ids = torch.tensor([sorted(range(l.shape[1]), key=lambda e: (-row[e], e))[:top] for row in l.tolist()],
                       dtype=torch.int32).reshape(l.shape[0], top)
    if sigmoid:
        score = torch.sigmoid(l)
    else:
        m = l.amax(1, keepdim=True)
        score = torch.where(l == m, 1.0, torch.exp(l - m)).double()
        score = torch.where(l == -math.inf, 0.0, score)
        total = score.sum(1, keepdim=True)
        score = torch.where(total > 0, score / total, 0.0)
    w = score.gather(1, ids.long())
    if normalize:
        if sigmoid:
            # sigmoids below 2^-1074 vanish even in 64 bits, their ratios do not: exponentials of
            # log sigmoid(l) = -log(1 + exp(-l)) relative to the largest
            chosen = l.gather(1, ids.long())
            log = torch.nn.functional.logsigmoid(chosen)
            w = torch.where(chosen == -math.inf, 0.0, torch.exp(log - log[:, :1]))
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return ids, w * scale


def random_ids(tokens, top, experts, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(experts, generator=g)[:top] for _ in range(tokens)]).to(torch.int32)
    weights = torch.rand(tokens, top, generator=g) + 0.05
    return ids.cuda(), weights.cuda()
