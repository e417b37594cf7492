"""Cases of the paged-attention operators: what one decoder layer does between its
q/k/v projections and its output projection when requests share a paged cache.

  plan       block table, slot map and positions of a step, from request lengths
  append     rotary positions (one or several axes) on q and k, K and V into the cache
  attention  a chunk of new tokens of each request over its pages, grouped heads

Request lengths come from the case alone (`lens` seeds them), values and page
orders from the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # A decode step's bookkeeping: one new token for each of 256 running requests.
        plan("plan decode step", 256, (1, 1), (1, 8191), 16),
        # Admission of prompts beside running requests: 1000 requests, some idle, chunks up to 512.
        plan("plan mixed step", 1000, (0, 512), (0, 4000), 32),
        # One decode step of a small batch: 16 tokens, latency counts.
        append("append decode", 16, 32, 8, 128, 128, 1, "bf16", 16, "hnd"),
        # A prompt chunk with image and video tokens: three position axes.
        append("append video chunk", 8192, 32, 8, 128, 128, 3, "bf16", 16, "hnd"),
        # Odd sizes, half of each head rotated, token-major pages.
        append("append partial f16", 1021, 12, 4, 80, 32, 2, "f16", 24, "nhd"),
        # The smallest attention call: one request, one token, a short cache.
        attention("decode single", 1, (1, 1), (1000, 1000), 32, 8, 128, "bf16", 16, "hnd"),
        # A decode step of a batch whose requests are of very different lengths.
        attention("decode batch ragged", 64, (1, 1), (100, 8000), 32, 8, 128, "bf16", 16, "hnd"),
        # A few requests deep into a long context: the cache is the work.
        attention("decode long f16", 3, (1, 1), (60000, 131000), 16, 2, 64, "f16", 64, "nhd"),
        # Drafted tokens checked together, a sliding window, plain multi-head layout.
        attention("verify window", 16, (1, 7), (500, 6000), 16, 16, 128, "bf16", 32, "hnd", window=2048),
        # A chunk of a long prompt over what is already cached.
        attention("chunk over cache", 1, (500, 512), (32000, 32000), 32, 8, 128, "bf16", 16, "hnd"),
        # Whole prompts of different lengths packed together: the largest call.
        attention("prompts packed", 3, (2000, 8192), (0, 0), 32, 8, 128, "bf16", 16, "hnd"),
        # Single precision, where every product and sum is.
        attention("mixed f32", 5, (1, 130), (0, 2000), 8, 2, 64, "f32", 16, "hnd"),
    ]


def plan(name, requests, new, past, page, lens=1):
    return dict(name=name, op="plan", requests=requests, min_new=new[0], max_new=new[1],
                min_past=past[0], max_past=past[1], page=page, lens=lens)


def append(name, tokens, q_heads, kv_heads, head_dim, rotary, axes, dtype, page, layout,
           interleaved=False):
    return dict(name=name, op="append", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads,
                head_dim=head_dim, rotary=rotary, axes=axes, dtype=dtype, page=page, layout=layout,
                interleaved=interleaved)


def attention(name, requests, new, past, q_heads, kv_heads, head_dim, dtype, page, layout,
              window=0, causal=True, lens=1):
    return dict(name=name, op="attention", requests=requests, min_new=new[0], max_new=new[1],
                min_past=past[0], max_past=past[1], q_heads=q_heads, kv_heads=kv_heads,
                head_dim=head_dim, dtype=dtype, page=page, layout=layout, window=window,
                causal=causal, lens=lens)


def log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "attention", "attention"])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128, 200])
    lens = rng.randrange(1 << 20)
    if op == "plan":
        requests = log_int(rng, 1, 2000)
        most = log_int(rng, 1, max(1, min(2048, 256000 // requests)))
        c = plan("", requests, (rng.choice([0, 1]), most), (0, log_int(rng, 1, 8192)), page, lens)
    elif op == "append":
        group = rng.choice([1, 2, 3, 4, 7, 8])
        kv = rng.choice([1, 2, 4, 8]) if group < 7 else rng.choice([1, 2, 4])
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        c = append("", log_int(rng, 1, 8192 if dim < 256 else 4096), kv * group, kv, dim,
                   rng.choice([dim, dim, 32]) if dim % 16 == 0 else 32, rng.choice([1, 1, 2, 3]),
                   rng.choice(["bf16", "f16", "f32"]) if dim < 256 else "bf16", page,
                   rng.choice(["hnd", "nhd"]), rng.random() < 0.3)
    else:
        kind = rng.choice(["decode", "verify", "chunk", "prompts", "f32"])
        group = rng.choice([1, 2, 3, 4, 5, 8])
        kv = rng.choice([1, 2, 4, 8]) if group < 5 else rng.choice([1, 2, 4])
        dim = rng.choice([64, 80, 96, 128, 128])
        dtype = rng.choice(["bf16", "bf16", "f16"])
        layout = rng.choice(["hnd", "hnd", "nhd"])
        window = rng.choice([0, 0, 0, log_int(rng, 1, 4096)])
        causal = rng.random() < 0.9
        if kind == "decode":
            requests = log_int(rng, 1, 128)
            new, past = (1, 1), (0, log_int(rng, 1, min(100000, 500000 // requests)))
        elif kind == "verify":
            requests = log_int(rng, 1, 48)
            new, past = (0, log_int(rng, 2, 16)), (0, log_int(rng, 1, min(16000, 250000 // requests)))
        elif kind == "chunk":
            requests = log_int(rng, 1, 4)
            new, past = (1, log_int(rng, 17, 1024 // requests)), (0, log_int(rng, 1, 24000 // requests))
        elif kind == "prompts":
            requests = log_int(rng, 1, 4)
            new, past = (1, log_int(rng, 2, 6000 // requests)), (0, 0)
        else:
            requests, dtype = log_int(rng, 1, 8), "f32"
            new, past = (1, log_int(rng, 1, 128)), (0, log_int(rng, 1, 3000))
        c = attention("", requests, new, past, kv * group, kv, dim, dtype, page, layout, window,
                      causal, lens)
    del c["name"]
    return c


def lengths(case):
    """(past, new) of each request: the first is the longest, the rest spread below it."""
    rng = random.Random(case["lens"])
    got = []
    for b in range(case["requests"]):
        lo, hi = case["min_new"], case["max_new"]
        new = hi if b == 0 else rng.randint(lo, hi)
        lo, hi = case["min_past"], case["max_past"]
        got.append((hi if b == 0 else rng.randint(lo, hi), new))
    return got


def pages(tokens, page):
    return -(-tokens // page)


def sections(case):
    """Frequency pairs of each axis: near-equal runs, the first the longest."""
    half, axes = case["rotary"] // 2, case["axes"]
    small = half // axes
    return [half - small * (axes - 1)] + [small] * (axes - 1)


def visible(case):
    """Per request: keys of each row summed over its rows, and keys that some row sees."""
    got = []
    for past, new in lengths(case):
        n, w = past + new, case["window"]
        total, first = 0, n
        for i in range(new):
            p = past + i
            hi = p + 1 if case["causal"] else n
            lo = max(0, p - w + 1) if w else 0
            total += max(0, hi - lo)
            first = min(first, lo)
        got.append((total, n - first if new else 0))
    return got


def work(case):
    if case["op"] == "plan":
        b, t, fresh, p = case["requests"], 0, 0, case["page"]
        for past, new in lengths(case):
            t += new
            fresh += pages(past + new, p) - pages(past, p)
        return {"bytes": 4 * (2 * b + 2 * fresh + 2 * b + 3 + 2 * t), "flops": 0}
    d, hq, hk, e = case["head_dim"], case["q_heads"], case["kv_heads"], BYTES[case["dtype"]]
    if case["op"] == "append":
        t, r = case["tokens"], case["rotary"]
        return {"bytes": t * (2 * (hq + 2 * hk) * d * e + 4 * (case["axes"] + 1) + 4 * r),
                "flops": 3 * t * (hq + hk) * r}
    t = sum(new for _, new in lengths(case))
    seen = visible(case)
    keys = sum(k for _, k in seen)
    return {"bytes": 2 * keys * hk * d * e + 4 * keys // case["page"] + t * hq * (2 * d * e + 4),
            "flops": 4 * d * hq * sum(n for n, _ in seen)}


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def cache_of(case, num_pages, g):
    """K and V pools [pages, heads, page, dim], in memory head-major or token-major."""
    h, p, d = case["kv_heads"], case["page"], case["head_dim"]
    shape = (num_pages, h, p, d) if case["layout"] == "hnd" else (num_pages, p, h, d)
    got = []
    for _ in range(2):
        c = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(DTYPES[case["dtype"]])
        got.append(c if case["layout"] == "hnd" else c.transpose(1, 2))
    return got


def prepare(case, seed):
    g = generator(seed)
    i32 = dict(dtype=torch.int32, device="cuda")
    s = dict(case)
    if case["op"] == "plan":
        lens, p = lengths(case), case["page"]
        b, t = len(lens), sum(new for _, new in lens)
        held = [pages(past, p) for past, _ in lens]
        need = sum(pages(past + new, p) for past, new in lens) - sum(held)
        width = max(pages(past + new, p) for past, new in lens) + 3
        ids = torch.randperm(sum(held) + need + 7, generator=g, device="cuda").to(torch.int32)
        table = torch.full((b, width), -1, **i32)
        held = torch.tensor(held, device="cuda")
        table[torch.arange(width, device="cuda")[None] < held[:, None]] = ids[: int(held.sum())]
        s.update(past=torch.tensor([x for x, _ in lens], **i32), new=torch.tensor([x for _, x in lens], **i32),
                 free=ids[int(held.sum()):].clone(), next_in=torch.full((1,), 2, **i32), table=table, tokens=t,
                 starts=torch.empty(b + 1, **i32), seq=torch.empty(b, **i32), positions=torch.empty(t, **i32),
                 slots=torch.empty(t, **i32), next_out=torch.empty(1, **i32))
        return s
    dt, hq, hk, d = DTYPES[case["dtype"]], case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        t, p, r = case["tokens"], case["page"], case["rotary"]
        num = pages(t, p) + 5
        s["k_cache"], s["v_cache"] = cache_of(case, num, g)
        # One fused projection's output: q, k and v are column ranges of it.
        s["qkv"] = torch.randn(t, (hq + 2 * hk) * d, generator=g, device="cuda").to(dt)
        order = torch.randperm(num, generator=g, device="cuda")
        at = torch.arange(t, device="cuda")
        s["slots"] = (order[at // p] * p + at % p).to(torch.int32)
        # Text counts up on every axis; the middle half is a picture of 24 columns.
        start = int(torch.randint(0, 1000, (1,), generator=g, device="cuda"))
        pos = torch.stack([start + at] * case["axes"])
        if case["axes"] > 1:
            lo, hi = t // 4, 3 * t // 4
            cell = torch.arange(hi - lo, device="cuda")
            pos[0, lo:hi] = start + lo + cell // 576
            pos[-1, lo:hi] = start + lo + cell % 24
            pos[1:-1, lo:hi] = start + lo + cell // 24 % 24
        s["positions"] = pos.to(torch.int32).contiguous()
        rows = start + t + 1
        inv = 10000.0 ** (-torch.arange(r // 2, device="cuda", dtype=torch.float64) * 2 / r)
        angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        s["q_out"] = torch.empty(t, hq, d, dtype=dt, device="cuda")
        return s
    lens, p = lengths(case), case["page"]
    t = sum(new for _, new in lens)
    held = [pages(past + new, p) for past, new in lens]
    width, num = max(held) + 2, sum(held) + 3
    s["k_cache"], s["v_cache"] = cache_of(case, num, g)
    # Half of the heads look widely, half at a few keys.
    sharp = torch.where(torch.arange(hq, device="cuda") % 2 == 0, 1.0, 3.0)
    s["q"] = (torch.randn(t, hq, d, generator=g, device="cuda") * sharp[:, None]).to(dt)
    table = torch.full((len(lens), width), -1, **i32)
    counts = torch.tensor(held, device="cuda")
    ids = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    table[torch.arange(width, device="cuda")[None] < counts[:, None]] = ids[: sum(held)]
    starts = [0]
    for _, new in lens:
        starts.append(starts[-1] + new)
    s.update(table=table, starts=torch.tensor(starts, **i32), seq=torch.tensor([a + b for a, b in lens], **i32),
             tokens=t, most=max(new for _, new in lens), out=torch.empty(t, hq, d, dtype=dt, device="cuda"),
             lse=torch.empty(t, hq, dtype=torch.float32, device="cuda"),
             workspace=torch.empty(64 << 20, dtype=torch.uint8, device="cuda"))
    return s


def run(s):
    if s["op"] == "plan":
        return run_plan(s)
    return run_append(s) if s["op"] == "append" else run_attention(s)


def run_plan(s):
    if own:
        from mlx_grouped_affine_gb300 import qmm
        qmm.qmm_page_plan(s["past"], s["new"], s["requests"], s["free"], s["free"].numel(), s["next_in"],
                          s["page"], s["table"], s["table"].stride(0), s["tokens"], s["starts"], s["seq"],
                          s["positions"], s["slots"], s["next_out"])
        return {k: s[k] for k in ("table", "starts", "seq", "positions", "slots", "next_out")}
    past, new, p = s["past"].long(), s["new"].long(), s["page"]
    seq = past + new
    held, total = (past + p - 1) // p, (seq + p - 1) // p
    need = total - held
    offset = torch.cumsum(need, 0) - need
    column = torch.arange(s["table"].shape[1], device=past.device)
    fresh = (column >= held[:, None]) & (column < total[:, None])
    source = s["next_in"].long() + offset[:, None] + column - held[:, None]
    table = torch.where(fresh, s["free"][source.clamp(0, s["free"].numel() - 1)], s["table"])
    ends = torch.cumsum(new, 0)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    token = torch.arange(s["tokens"], device=past.device)
    request = torch.searchsorted(ends, token, right=True)
    pos = past[request] + token - starts[request]
    slots = table[request, pos // p].long() * p + pos % p
    i32 = torch.int32
    return {"table": table, "starts": starts.to(i32), "seq": seq.to(i32), "positions": pos.to(i32),
            "slots": slots.to(i32), "next_out": (s["next_in"] + need.sum()).to(i32)}


def run_append(s):
    t, hq, hk, d, r = s["tokens"], s["q_heads"], s["kv_heads"], s["head_dim"], s["rotary"]
    q, k, v = s["qkv"].split([hq * d, hk * d, hk * d], 1)
    if own:
        from mlx_grouped_affine_gb300 import qmm
        kind = {torch.bfloat16: qmm.QMM_BF16, torch.float16: qmm.QMM_F16, torch.float32: qmm.QMM_F32}[q.dtype]
        c = s["k_cache"]
        cache = qmm.PagedCache(c, s["v_cache"], kind, c.shape[0], s["page"], hk, d, c.stride(0), c.stride(1),
                               c.stride(2))
        qmm.qmm_rope_append(q, q.stride(0), k, k.stride(0), v, v.stride(0), t, hq, s["positions"],
                            sections(s), s["cos_sin"], s["cos_sin"].shape[0], r, s["interleaved"],
                            s["slots"], s["q_out"], hq * d, cache)
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    axis = torch.repeat_interleave(torch.arange(s["axes"], device=q.device),
                                   torch.tensor(sections(s), device=q.device))
    at = s["positions"].long()[axis].T
    pair = torch.arange(r // 2, device=q.device)
    cos, sin = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, pair + r // 2][:, None]

    def turned(x):
        x = x.reshape(t, -1, d).float()
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if s["interleaved"] else (x[..., : r // 2], x[..., r // 2: r])
        y = (a * cos - b * sin, b * cos + a * sin)
        y = torch.stack(y, -1).flatten(-2) if s["interleaved"] else torch.cat(y, -1)
        return torch.cat([y, x[..., r:]], -1).to(q.dtype)

    page, row = s["slots"].long() // s["page"], s["slots"].long() % s["page"]
    s["k_cache"][page, :, row] = turned(k)
    s["v_cache"][page, :, row] = v.reshape(t, hk, d)
    return {"q": turned(q), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run_attention(s):
    q, hq, hk, d = s["q"], s["q_heads"], s["kv_heads"], s["head_dim"]
    if own:
        from mlx_grouped_affine_gb300 import qmm
        kind = {torch.bfloat16: qmm.QMM_BF16, torch.float16: qmm.QMM_F16, torch.float32: qmm.QMM_F32}[q.dtype]
        c = s["k_cache"]
        cache = qmm.PagedCache(c, s["v_cache"], kind, c.shape[0], s["page"], hk, d, c.stride(0), c.stride(1),
                               c.stride(2))
        qmm.qmm_paged_attention(q, hq * d, s["tokens"], hq, cache, s["table"], s["table"].stride(0),
                                s["starts"], s["seq"], s["requests"], s["most"], d ** -0.5, s["causal"],
                                s["window"], s["out"], hq * d, s["lse"], s["workspace"],
                                s["workspace"].numel())
        return {"out": s["out"], "lse": s["lse"]}
    b, most, t, p = s["requests"], s["most"], s["tokens"], s["page"]
    starts, seq = s["starts"].long(), s["seq"].long()
    new = starts[1:] - starts[:-1]
    width = s["table"].shape[1] - 2
    # Requests side by side, each padded to the longest: [b, kv heads, group, new, keys].
    key = torch.arange(width * p, device=q.device)
    page = s["table"].long()[:, :width].clamp(min=0)
    k = s["k_cache"][page].transpose(1, 2).reshape(b, hk, 1, width * p, d).float()
    v = s["v_cache"][page].transpose(1, 2).reshape(b, hk, 1, width * p, d).float()
    token = torch.arange(most, device=q.device)
    row = (starts[:-1, None] + token).clamp(max=max(t - 1, 0))
    qs = q[row].reshape(b, most, hk, hq // hk, d).permute(0, 2, 3, 1, 4).float()
    at = (seq - new)[:, None] + token
    see = key < seq[:, None, None]
    if s["causal"]:
        see = see & (key <= at[..., None])
    if s["window"]:
        see = see & (key > at[..., None] - s["window"])
    score = (qs * d ** -0.5) @ k.transpose(-1, -2)
    score.masked_fill_(~see[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    out = (score @ v) / total.clamp(min=1e-37)
    lse = (top + total.log()).squeeze(-1)
    request = torch.searchsorted(starts[1:], torch.arange(t, device=q.device), right=True)
    inside = torch.arange(t, device=q.device) - starts[request]
    out = out.permute(0, 3, 1, 2, 4)[request, inside].reshape(t, hq, d).to(q.dtype)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2)[request, inside].reshape(t, hq)}


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    hq, hk, d, p = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] == "append":
        t, r = case["tokens"], case["rotary"]
        x = s["qkv"].double().reshape(t, hq + 2 * hk, d)
        head = x[:, : hq + hk, :r]
        head = head.reshape(t, hq + hk, r // 2, 2) if case["interleaved"] else head.reshape(t, hq + hk, 2, r // 2).mT
        turn = torch.empty(t, r // 2, dtype=torch.complex128, device="cuda")
        first = 0
        for axis, n in enumerate(sections(case)):
            rows = s["cos_sin"].double()[s["positions"][axis].long()]
            turn[:, first:first + n] = torch.complex(rows[:, first:first + n], rows[:, r // 2 + first:r // 2 + first + n])
            first += n
        z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn[:, None])
        x[:, : hq + hk, :r] = (z if case["interleaved"] else z.mT).reshape(t, hq + hk, r)
        pools = [s["k_cache"].double(), s["v_cache"].double()]
        slot = s["slots"].long()
        for pool, part in zip(pools, (x[:, hq:hq + hk], x[:, hq + hk:])):
            pool[slot // p, :, slot % p] = part
        return {"q": x[:, :hq], "k_cache": pools[0], "v_cache": pools[1]}
    t, w = s["tokens"], case["window"]
    out = torch.zeros(t, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((t, hq), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b, (past, new) in enumerate(lengths(case)):
        n = past + new
        if new == 0:
            continue
        ids = s["table"][b, : pages(n, p)].long()
        for h in range(hk):
            k = s["k_cache"][ids, h].double().reshape(-1, d)[:n]
            v = s["v_cache"][ids, h].double().reshape(-1, d)[:n]
            for j in range(h * (hq // hk), (h + 1) * (hq // hk)):
                for lo in range(0, new, 2048):
                    hi = min(new, lo + 2048)
                    a = s["q"][first + lo:first + hi, j].double() @ k.T / math.sqrt(d)
                    at = past + torch.arange(lo, hi, device="cuda")[:, None]
                    j2 = torch.arange(n, device="cuda")[None]
                    keep = (j2 <= at) | (not case["causal"])
                    if w:
                        keep = keep & (j2 > at - w)
                    a[~keep] = -math.inf
                    z = torch.logsumexp(a, -1)
                    lse[first + lo:first + hi, j] = z
                    out[first + lo:first + hi, j] = torch.exp(a - z[:, None]).nan_to_num(0.0) @ v
        first += new
    return {"out": out, "lse": lse}
