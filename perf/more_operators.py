"""Cases of the operators for block-scaled 8-bit floats and mixture-of-experts layers:
what a decoder layer with routed experts multiplies besides its attention.

  quantize  values to e4m3 codes with one fp32 scale for each block of 128 columns
  matmul    product of such activations (a scale per row and 128 columns) and weights
            (a scale per 128 x 128 block)
  route     the top experts of each token and their weights, from router logits
  experts   gated feed-forward of given experts for a few tokens, affine 1-8 bit weights
  layer     the same from router logits: routing and experts in one call
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
BITS = [1, 2, 3, 4, 4, 4, 5, 6, 8, 8]
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


def listed():
    return [
        # A decode step's activations before a product, 16 requests: latency counts.
        quantize("quantize decode", 16, 4096, "bf16", 1),
        # A whole projection's weight from a checkpoint in single precision.
        quantize("quantize weight f32", 11008, 4096, "f32", 128),
        # The smallest product: one token through a square projection.
        matmul("matmul decode", 1, 4096, 4096, "bf16"),
        # Drafted tokens of a few requests, sizes that fill no tile, columns that end inside a block.
        matmul("matmul odd f32", 77, 1021, 4208, "f32"),
        # A prompt through the widest projection of a feed-forward block: the largest product.
        matmul("matmul prompt", 2048, 14336, 4096, "bf16"),
        # A decode step's routing.
        route("route decode", 16, 128, 8, "f32", "softmax", True),
        # A prompt's routing over many experts, some of them closed to some tokens.
        route("route prompt bf16", 8192, 256, 8, "bf16", "sigmoid", True, masked=0.2),
        # One token of one request through many small experts.
        layer("layer one token", 1, 128, 8, 2048, 768, 4, 64, "bf16"),
        # A decode step of a batch: most experts are asked for, each by few tokens.
        layer("layer batch", 16, 64, 8, 2048, 1024, 4, 64, "bf16"),
        # Single precision, 8 bits, wide groups, more tokens than experts.
        layer("layer f32", 48, 32, 4, 1024, 512, 8, 128, "f32", "sigmoid", False),
        # Few wide experts of an 8B-class block, two for each token: the most bytes.
        experts("experts wide", 16, 8, 2, 4096, 14336, 4, 64, "bf16"),
        # Half precision, codes that straddle words, narrow groups, sizes that fill no tile.
        experts("experts odd f16", 5, 16, 3, 992, 416, 6, 32, "f16"),
    ]


def quantize(name, rows, cols, dtype, block_rows):
    return dict(name=name, op="quantize", rows=rows, cols=cols, dtype=dtype, block_rows=block_rows)


def matmul(name, m, n, k, dtype):
    return dict(name=name, op="matmul", m=m, n=n, k=k, dtype=dtype)


def route(name, tokens, count, top, dtype, scoring, normalize, masked=0.0, scale=1.0):
    return dict(name=name, op="route", tokens=tokens, experts=count, top=top, dtype=dtype,
                scoring=scoring, normalize=normalize, masked=masked, scale=scale)


def experts(name, tokens, count, top, hidden, inner, bits, group, dtype):
    return dict(name=name, op="experts", tokens=tokens, experts=count, top=top, hidden=hidden,
                inner=inner, bits=bits, group=group, dtype=dtype)


def layer(name, tokens, count, top, hidden, inner, bits, group, dtype, scoring="softmax",
          normalize=True, scale=1.0):
    return dict(name=name, op="layer", tokens=tokens, experts=count, top=top, hidden=hidden,
                inner=inner, bits=bits, group=group, dtype=dtype, scoring=scoring,
                normalize=normalize, scale=scale)


def log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "route", "experts", "layer", "layer"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize":
        cols = 16 * log_int(rng, 1, 1024)
        c = quantize("", log_int(rng, 1, min(20000, 40000000 // cols)), cols, dtype, rng.choice([1, 1, 128]))
    elif op == "matmul":
        n, k = log_int(rng, 1, 16384), 16 * log_int(rng, 1, 1024)
        m = rng.choice([log_int(rng, 1, 16), log_int(rng, 1, 256), log_int(rng, 1, 8192)])
        c = matmul("", max(1, min(m, 120000000000 // (n * k))), n, k, dtype)
    elif op == "route":
        count = log_int(rng, 1, 1024)
        c = route("", log_int(rng, 1, 16384), count, log_int(rng, 1, min(count, 32)), dtype,
                  rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6, rng.choice([0.0, 0.0, 0.3, 0.9]),
                  rng.choice([1.0, 2.5]))
    else:
        group = rng.choice([32, 64, 64, 64, 128])
        hidden = group * log_int(rng, 1, 4096 // group)
        inner = group * log_int(rng, 1, 14336 // group)
        bits = rng.choice(BITS)
        each = 3 * hidden * inner * max(0.5, bits / 8 + 2 * BYTES[dtype] / group)
        count = log_int(rng, 1, max(1, min(256, int(700000000 // each))))
        tokens = log_int(rng, 1, 64)
        top = log_int(rng, 1, min(count, 16, 512 // tokens))
        if op == "experts":
            c = experts("", tokens, count, top, hidden, inner, bits, group, dtype)
        else:
            c = layer("", tokens, count, top, hidden, inner, bits, group, dtype,
                      rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6, rng.choice([1.0, 2.5]))
    del c["name"]
    return c


def blocks(n):
    return -(-n // 128)


def work(case):
    op = case["op"]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        scales = (r if case["block_rows"] == 1 else blocks(r)) * blocks(c)
        return {"bytes": r * c * (BYTES[case["dtype"]] + 1) + 4 * scales, "flops": 2 * r * c}
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k + 4 * (m + blocks(n)) * blocks(k) + m * n * BYTES[case["dtype"]],
                "flops": 2 * m * n * k}
    t, e, top = case["tokens"], case["experts"], case["top"]
    if op == "route":
        return {"bytes": t * e * BYTES[case["dtype"]] + 8 * t * top, "flops": 3 * t * e}
    # The experts that t tokens ask for, on average, each read once.
    used = min(t * top, e * (1 - (1 - top / e) ** t))
    weights = 3 * case["hidden"] * case["inner"]
    b = BYTES[case["dtype"]]
    each = weights * case["bits"] / 8 + 2 * b * weights / case["group"]
    routing = 8 * t * top if op == "experts" else 4 * t * e
    return {"bytes": int(used * each + 2 * t * case["hidden"] * b + routing),
            "flops": 2 * t * top * weights}


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def packed(rows, cols, bits, group, count, g, dtype):
    """`count` weights [rows, cols]: uniform codes, scales in [0.002, 0.02], biases that
    centre them, as (words, scales, biases)."""
    words = torch.randint(-2 ** 31, 2 ** 31, (count, rows, cols * bits // 32), generator=g, device="cuda",
                          dtype=torch.int32)
    shape = (count, rows, cols // group)
    s = (torch.rand(shape, generator=g, device="cuda") * 0.018 + 0.002) * 8 / 2 ** (bits - 1)
    b = -s * 2 ** (bits - 1) + torch.randn(shape, generator=g, device="cuda") * 1e-3
    return words, s.to(dtype), b.to(dtype)


def prepare(case, seed):
    g, op, s = generator(seed), case["op"], dict(case)
    dt = DTYPES[case["dtype"]]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        # Rows of different size and a few values far above the rest, as activations have them.
        x = normal((r, c), g, torch.float32) * torch.exp(normal((r, 1), g, torch.float32))
        far = torch.rand((r, c), generator=g, device="cuda") < 0.001
        s["x"] = torch.where(far, x * 30, x).to(dt)
        s["codes"] = torch.empty((r, c), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((r if case["block_rows"] == 1 else blocks(r), blocks(c)), device="cuda")
        return s
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = (normal((m, k), g, torch.float32) * 120).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["w"] = (normal((n, k), g, torch.float32) * 120).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["a_scales"] = torch.exp(normal((m, blocks(k)), g, torch.float32) * 0.5) / 120
        s["w_scales"] = torch.exp(normal((blocks(n), blocks(k)), g, torch.float32) * 0.5) / 2400
        s["y"] = torch.empty((m, n), dtype=dt, device="cuda")
        return s
    t, e, top = case["tokens"], case["experts"], case["top"]
    if op == "route":
        logits = normal((t, e), g, torch.float32) * 2
        closed = torch.rand((t, e), generator=g, device="cuda") < case["masked"]
        s["logits"] = logits.masked_fill(closed, -math.inf).to(dt)
        s["ids"] = torch.empty((t, top), dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty((t, top), device="cuda")
        return s
    h, i, bits, group = case["hidden"], case["inner"], case["bits"], case["group"]
    s["gate"] = packed(i, h, bits, group, e, g, dt)
    s["up"] = packed(i, h, bits, group, e, g, dt)
    s["down"] = packed(h, i, bits, group, e, g, dt)
    s["x"] = normal((t, h), g, dt)
    s["y"] = torch.empty((t, h), dtype=dt, device="cuda")
    logits = normal((t, e), g, torch.float32)
    if op == "layer":
        s["logits"] = logits
    else:
        best = torch.topk(logits, top)
        s["ids"] = best.indices.to(torch.int32)
        s["weights"] = torch.softmax(best.values, -1)
    if own:
        from mlx_grouped_affine_gb300 import qmm
        s["handle"] = qmm.Experts(s["gate"], s["up"], s["down"], kind(dt), e, h, i, group, bits)
        size = qmm.qmm_moe_workspace_bytes(t, top, h, i)
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


def kind(dtype):
    from mlx_grouped_affine_gb300 import qmm
    return {torch.bfloat16: qmm.QMM_BF16, torch.float16: qmm.QMM_F16, torch.float32: qmm.QMM_F32}[dtype]


def run(s):
    return {"quantize": run_quantize, "matmul": run_matmul, "route": run_route, "experts": run_experts,
            "layer": run_experts}[s["op"]](s)


def run_quantize(s):
    x, r, c = s["x"], s["rows"], s["cols"]
    if own:
        from mlx_grouped_affine_gb300 import qmm
        qmm.qmm_block_quantize(x, kind(x.dtype), r, c, s["block_rows"], s["codes"], s["scales"])
        return {"codes": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    rb = s["block_rows"]
    rows, cols = -(-r // rb), blocks(c)
    p = torch.zeros((rows * rb, cols * 128), device=x.device)
    p[:r, :c] = x.float()
    p = p.view(rows, rb, cols, 128)
    top = p.abs().amax((1, 3))
    scales = (top / torch.full_like(top, E4M3_MAX)).clamp(min=SCALE_MIN)  # a tensor: a true division
    # The nearest code of the quotient itself: 64 bits keep every quotient off the borders
    # between codes that it is not on.
    q = p.double() / scales[:, None, :, None].double()
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    q = (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    q = torch.copysign(q, p.double()).view(rows * rb, cols * 128)[:r, :c]
    return {"codes": q.float().to(torch.float8_e4m3fn), "scales": scales}


def widened(codes, scales, rows):
    """e4m3 codes times their blocks' scales, fp32; `rows` rows share a scale."""
    v = codes.view(torch.float8_e4m3fn).float()
    s = scales.repeat_interleave(rows, 0)[: v.shape[0]].repeat_interleave(128, 1)[:, : v.shape[1]]
    return v * s


def run_matmul(s):
    if own:
        from mlx_grouped_affine_gb300 import qmm
        qmm.qmm_block_matmul(s["a"], s["a_scales"], s["m"], s["w"], s["w_scales"], s["n"], s["k"], s["y"],
                             kind(s["y"].dtype))
        return s["y"]
    return (widened(s["a"], s["a_scales"], 1) @ widened(s["w"], s["w_scales"], 128).T).to(s["y"].dtype)


def routed(logits, top, scoring, normalize, scale):
    """The `top` experts of each row and their weights: largest logits first, the lowest
    index of equal ones; -infinity (and NaN) has weight 0."""
    l = logits.float()
    l = torch.where(torch.isnan(l), -math.inf, l)
    ids = torch.sort(l, dim=-1, descending=True, stable=True).indices[:, :top]
    if scoring == "softmax":
        m = l.amax(-1, keepdim=True)
        score = torch.where(l == m, 1.0, torch.exp(l - m))
        score = torch.where(l == -math.inf, 0.0, score)
        total = score.sum(-1, keepdim=True)
        score = torch.where(total > 0, score / total, 0.0)
    else:
        score = 1 / (1 + torch.exp(-l))
    weights = score.gather(1, ids)
    if normalize:
        total = weights.sum(-1, keepdim=True)
        weights = torch.where(total > 0, weights / total, 0.0)
    return ids.to(torch.int32), weights * scale


def run_route(s):
    if own:
        from mlx_grouped_affine_gb300 import qmm
        scoring = qmm.QMM_SCORE_SOFTMAX if s["scoring"] == "softmax" else qmm.QMM_SCORE_SIGMOID
        qmm.qmm_moe_route(s["logits"], kind(s["logits"].dtype), s["tokens"], s["experts"], s["top"], scoring,
                          s["normalize"], s["scale"], s["ids"], s["weights"])
        return {"ids": s["ids"], "weights": s["weights"]}
    ids, weights = routed(s["logits"], s["top"], s["scoring"], s["normalize"], s["scale"])
    return {"ids": ids, "weights": weights}


def dense(weight, e, cols, bits, group):
    """Expert e's weight in fp32: scale * code + bias."""
    words, scales, biases = weight
    bit = torch.arange(cols, device=words.device) * bits
    at, shift = bit // 32, bit % 32
    w = words[e].long() & 0xFFFFFFFF
    w = w | (torch.cat([w[:, 1:], w[:, :1]], 1) << 32)
    codes = (w[:, at] >> shift) & (2 ** bits - 1)
    s, b = scales[e].float(), biases[e].float()
    return codes.float() * s.repeat_interleave(group, 1) + b.repeat_interleave(group, 1)


def run_experts(s):
    if own:
        from mlx_grouped_affine_gb300 import qmm
        dt = kind(s["x"].dtype)
        if s["op"] == "layer":
            scoring = qmm.QMM_SCORE_SOFTMAX if s["scoring"] == "softmax" else qmm.QMM_SCORE_SIGMOID
            qmm.qmm_moe_layer(s["x"], dt, s["tokens"], s["logits"], qmm.QMM_F32, s["top"], scoring,
                              s["normalize"], s["scale"], s["handle"], s["y"], dt, s["workspace"],
                              s["workspace"].numel())
        else:
            qmm.qmm_moe_experts(s["x"], dt, s["tokens"], s["ids"], s["weights"], s["top"], s["handle"],
                                s["y"], dt, s["workspace"], s["workspace"].numel())
        return s["y"]
    if s["op"] == "layer":
        ids, weights = routed(s["logits"], s["top"], s["scoring"], s["normalize"], s["scale"])
    else:
        ids, weights = s["ids"], s["weights"]
    x, bits, group = s["x"].float(), s["bits"], s["group"]
    y = torch.zeros_like(x)
    for e in range(s["experts"]):
        share = torch.where(ids == e, weights, 0.0).sum(1, keepdim=True)
        g = x @ dense(s["gate"], e, s["hidden"], bits, group).T
        u = x @ dense(s["up"], e, s["hidden"], bits, group).T
        z = (g / (1 + torch.exp(-g)) * u) @ dense(s["down"], e, s["inner"], bits, group).T
        y += share * z
    return y.to(s["x"].dtype)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        return exact_quantize(s)
    if op == "matmul":
        return exact_matmul(s)
    if op == "route":
        if case["tokens"] * case["experts"] > 4000000:
            return None
        return {"ids": None, "weights": exact_weights(s)[1]}
    if op == "layer":
        chosen, weights = exact_weights(s)
    else:
        chosen, weights = s["ids"].tolist(), s["weights"].double()
    tokens = {}
    for t, row in enumerate(chosen):
        for j, e in enumerate(row):
            tokens.setdefault(e, []).append((t, j))
    x = s["x"].double()
    y = torch.zeros_like(x)
    for e, where in tokens.items():
        at = torch.tensor([t for t, _ in where], device=x.device)
        share = torch.stack([weights[t, j] for t, j in where])
        rows = x[at]
        g = product64(rows, s["gate"], e, case)
        h = g * torch.sigmoid(g) * product64(rows, s["up"], e, case)
        y.index_add_(0, at, product64(h, s["down"], e, case) * share[:, None])
    return y


def product64(x, weight, e, case):
    """x . w^T for expert e in 64 bits, some rows at a time, codes put together bit by bit."""
    words, scales, biases = (part[e] for part in weight)
    n, k, bits, group = words.shape[0], x.shape[1], case["bits"], case["group"]
    got = []
    place = torch.arange(32, device=words.device, dtype=torch.int32)
    value = 2.0 ** torch.arange(bits, device=words.device, dtype=torch.float64)
    step = max(1, 4000000 // k)
    for r in range(0, n, step):
        stream = ((words[r:r + step, :, None] >> place) & 1).reshape(-1, k, bits)
        codes = (stream.double() @ value).reshape(-1, k // group, group)
        w = codes * scales[r:r + step, :, None].double() + biases[r:r + step, :, None].double()
        got.append(x @ w.reshape(-1, k).T)
    return torch.cat(got, 1)


def exact_weights(s):
    """Chosen experts (nested lists) and weights (64 bits) of each token."""
    l = s["logits"].double().cpu()
    top = s["top"]
    chosen = [sorted(range(len(row)), key=lambda e: (-row[e], e))[:top] for row in l.tolist()]
    ids = torch.tensor(chosen)
    if s["scoring"] == "softmax":
        score = torch.exp(l - torch.logsumexp(l, -1, keepdim=True)).nan_to_num(0.0)
    else:
        score = torch.sigmoid(l)
    w = torch.gather(score, 1, ids)
    if s["normalize"]:
        w = (w / w.sum(-1, keepdim=True)).nan_to_num(0.0)
    return chosen, (w * s["scale"]).cuda()


def exact_matmul(s):
    m, n, k = s["m"], s["n"], s["k"]
    a = s["a"].view(torch.float8_e4m3fn).to(torch.float64)
    w = s["w"].view(torch.float8_e4m3fn).to(torch.float64)
    y = torch.zeros((m, n), dtype=torch.float64, device=a.device)
    rows = torch.arange(n, device=a.device) // 128
    for b in range(blocks(k)):
        cut = slice(128 * b, min(k, 128 * b + 128))
        y += (a[:, cut] @ w[:, cut].T) * s["a_scales"][:, b, None].double() * s["w_scales"][rows, b].double()
    return y


def exact_quantize(s):
    x, r, c, rb = s["x"].double(), s["rows"], s["cols"], s["block_rows"]
    # All 256 codes' values in order, and the borders between neighbours.
    grid = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    border = (grid[1:] + grid[:-1]) / 2
    codes, scales = torch.empty_like(x), []
    for j in range(0, c, 128):
        part = x[:, j:j + 128]
        top = part.abs().amax(1)
        if rb > 1:
            top = torch.stack([p.max() for p in top.split(rb)])
        scale = (top / torch.full_like(top, E4M3_MAX)).float().clamp(min=SCALE_MIN)
        scales.append(scale)
        q = part / scale.double().repeat_interleave(rb)[:r, None]
        at = torch.searchsorted(border, q.abs())
        # On a border the even code: the one below where its index is even.
        on = (at < border.numel()) & (border[at.clamp(max=border.numel() - 1)] == q.abs())
        at = torch.where(on & (at % 2 == 1), at + 1, at)
        codes[:, j:j + 128] = torch.copysign(grid[at], q)
    return {"codes": codes, "scales": torch.stack(scales, 1).double()}


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(4)]:
        print(case, work(case))
