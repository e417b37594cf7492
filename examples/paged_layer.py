"""One decoder layer's attention block over a paged cache, on quantized weights.

Requests of different lengths share a pool of cache pages.  Each step takes any
number of new tokens of each request (a prompt, a chunk of one, single tokens) and
runs, without a copy to the host in between:

  qmm_page_plan           block table, slots and positions from the lengths
  qmm_quantized_matmul    one fused q/k/v projection
  qmm_rope_append         rotary positions; k and v into the cache
  qmm_paged_attention     the step's tokens over their requests' pages
  qmm_quantized_matmul    the output projection

Run as a program it takes the same tokens in one step and in several, and prints
how far the outputs are apart.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mlx_grouped_affine_gb300 import qmm  # noqa: E402


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class QuantizedLinear:
    """y = x . dequant(W)^T for a bf16 W [out, in], stored in 4-bit codes."""

    def __init__(self, w, bits=4, group=64):
        self.n, self.k = w.shape
        self.bits, self.group = bits, group
        self.codes = torch.empty(self.n, self.k * bits // 32, dtype=torch.int32, device="cuda")
        self.scales = torch.empty(self.n, self.k // group, dtype=torch.bfloat16, device="cuda")
        self.biases = torch.empty_like(self.scales)
        qmm.qmm_quantize(w, self.n, self.k, group, bits, self.codes, self.scales, self.biases)

    def __call__(self, x):
        y = torch.empty(x.shape[0], self.n, dtype=torch.bfloat16, device="cuda")
        qmm.qmm_quantized_matmul(x, x.shape[0], self.codes, self.scales, self.biases, self.n, self.k, 1,
                                 self.group, self.bits, y, qmm.QMM_BF16)
        return y


class PagedLayer:
    """The weights of one layer, its cache pool, and the requests' tables and lengths."""

    def __init__(self, hidden=1024, q_heads=16, kv_heads=4, head_dim=64, page=16, pages=256, requests=4,
                 max_tokens=2048, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.page = q_heads, kv_heads, head_dim, page

        def weight(n, k):
            return QuantizedLinear((torch.randn(n, k, generator=g, device="cuda") * k ** -0.5).bfloat16())

        self.qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.out = weight(hidden, q_heads * head_dim)
        pool = (pages, kv_heads, page, head_dim)
        self.k_cache = torch.zeros(pool, dtype=torch.bfloat16, device="cuda")
        self.v_cache = torch.zeros(pool, dtype=torch.bfloat16, device="cuda")
        s = self.k_cache.stride()
        self.cache = qmm.PagedCache(self.k_cache, self.v_cache, qmm.QMM_BF16, pages, page, kv_heads, head_dim,
                                    s[0], s[1], s[2])
        self.table = torch.full((requests, -(-max_tokens // page)), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.next_free = [i32([0]), i32([0])]  # the count moves from one to the other
        self.past = i32([0] * requests)
        angle = torch.arange(max_tokens, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(head_dim // 2, device="cuda", dtype=torch.float64) * 2 / head_dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        self.workspace = torch.empty(qmm.QMM_ATTENTION_WORKSPACE_BYTES, dtype=torch.uint8, device="cuda")

    def step(self, x, new_lens):
        """x [sum(new_lens), hidden]: the new tokens of each request, one request after another."""
        t, b = x.shape[0], len(new_lens)
        hq, hk, d = self.q_heads, self.kv_heads, self.head_dim
        starts, seq, positions, slots = i32([0] * (b + 1)), i32([0] * b), i32([0] * t), i32([0] * t)
        qmm.qmm_page_plan(self.past, i32(new_lens), b, self.free, self.free.numel(), self.next_free[0], self.page,
                          self.table, self.table.stride(0), t, starts, seq, positions, slots, self.next_free[1])
        self.next_free.reverse()
        qkv = self.qkv(x)
        q, k, v = qkv.split([hq * d, hk * d, hk * d], 1)
        turned = torch.empty(t, hq * d, dtype=torch.bfloat16, device="cuda")
        qmm.qmm_rope_append(q, q.stride(0), k, k.stride(0), v, v.stride(0), t, hq, positions, [d // 2], self.cos_sin,
                            self.cos_sin.shape[0], d, False, slots, turned, hq * d, self.cache)
        mixed = torch.empty_like(turned)
        qmm.qmm_paged_attention(turned, hq * d, t, hq, self.cache, self.table, self.table.stride(0), starts, seq, b,
                                max(new_lens), d ** -0.5, True, 0, mixed, hq * d, None, self.workspace,
                                self.workspace.numel())
        self.past = seq
        return self.out(mixed)


def run(lengths=(300, 7, 129, 64), steps=((200, 0, 129, 1), (99, 5, 0, 62), (1, 1, 0, 1), (0, 1, 0, 0))):
    """The same tokens in one step and in `steps`; returns the largest difference over the outputs' rms."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    x = [torch.randn(n, 1024, generator=g, device="cuda").bfloat16() for n in lengths]
    whole = PagedLayer(requests=len(lengths)).step(torch.cat(x), list(lengths)).float().split(list(lengths))
    layer, done, got = PagedLayer(requests=len(lengths)), [0] * len(lengths), [[] for _ in lengths]
    for news in steps:
        y = layer.step(torch.cat([x[b][done[b]:done[b] + n] for b, n in enumerate(news)]), list(news)).float()
        for b, part in enumerate(y.split(list(news))):
            got[b].append(part)
            done[b] += news[b]
    assert done == list(lengths)
    assert qmm.qmm_get_device_error() == qmm.QMM_OK
    rms = torch.cat(whole).square().mean().sqrt()
    return float(max((torch.cat(a) - w).abs().max() for a, w in zip(got, whole)) / rms)


if __name__ == "__main__":
    print("one step against several: largest difference %.4f of the outputs' rms" % run())
