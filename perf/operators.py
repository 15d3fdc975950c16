"""Cases of the framework's single-token and paged-serving operators, and what each computes.

Four operators:

  gemv       y = act(x W^T) for a few rows x (bf16 or fp32) and NVFP4 weights W, without
             quantizing x: the timestep and modulation layers of a denoise step, and the linear
             layers of a single new token.
  plan       block tables and slot maps of a paged cache from request lengths.
  append     new K and V tokens into a paged 8-bit cache (E4M3 codes, one power-of-two scale
             for each page and head).
  attention  softmax(scale q k^T) v over that cache: single tokens, ragged chunks, causal or not.

`run` computes a case in plain torch operations, or with the framework's entry points where `own`
is set; `exact` computes it from the definition in 64 bits.
"""
import math
import random

import torch

own = False

# E2M1 values by code, and the bounds of an 8-bit page scale's exponent
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
E_MIN, E_MAX = -60, 60


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the modulation layer of one denoise timestep: one row, a small square weight
        dict(name="gemv 1x1024x1024", op="gemv", rows=1, n=1024, k=1024, x="bf16", y="bf16",
             act="none"),
        # the FFN up-projection with its GELU for one token
        dict(name="gemv 1x14336x4096 gelu", op="gemv", rows=1, n=14336, k=4096, x="bf16",
             y="bf16", act="gelu"),
        # a down-projection for an odd handful of tokens, fp32 in and out, ragged N
        dict(name="gemv 7x5000x14336 fp32", op="gemv", rows=7, n=5000, k=14336, x="fp32",
             y="fp32", act="none"),
        # one request gets one token: the smallest scheduling step
        dict(name="plan 1 request", op="plan", batch=1, cached_max=1000, new_min=1, new_max=1,
             page=16, spare=4, lens=1),
        # a mixed batch: decode and chunked prefill, long slot map
        dict(name="plan 512 requests", op="plan", batch=512, cached_max=20000, new_min=0,
             new_max=257, page=32, spare=64, lens=2),
        # one new token for each request of a decode batch
        dict(name="append 33 tokens", op="append", batch=33, cached_max=2000, new_min=1,
             new_max=1, heads=8, head_dim=128, page=16, spare=8, lens=3),
        # ragged prefill of many requests, K and V out of a fused projection
        dict(name="append ragged prefill", op="append", batch=24, cached_max=500, new_min=1,
             new_max=1500, heads=8, head_dim=128, page=64, spare=32, lens=5),
        # one request, one token, a short cache: latency
        dict(name="attention 1x777", op="attention", batch=1, q_heads=24, kv_heads=24,
             head_dim=128, page=16, q_min=1, q_max=1, kv_min=777, kv_max=777, causal=True, lens=6),
        # a decode batch with shared heads and ragged lengths
        dict(name="attention decode 64", op="attention", batch=64, q_heads=32, kv_heads=8,
             head_dim=128, page=32, q_min=1, q_max=1, kv_min=1, kv_max=8000, causal=True, lens=7),
        # a few very long caches
        dict(name="attention decode long", op="attention", batch=2, q_heads=40, kv_heads=8,
             head_dim=128, page=64, q_min=1, q_max=1, kv_min=100000, kv_max=131072, causal=True,
             lens=8),
        # chunks of prompts on top of what is cached, causal, shared heads, ragged
        dict(name="attention causal chunks", op="attention", batch=6, q_heads=32, kv_heads=8,
             head_dim=64, page=64, q_min=100, q_max=2048, kv_min=1000, kv_max=4096, causal=True,
             lens=10),
        # a chunk of three latent frames over sinks and window, frame pages, no mask inside
        dict(name="attention 2640x10560", op="attention", batch=1, q_heads=24, kv_heads=24,
             head_dim=128, page=880, q_min=2640, q_max=2640, kv_min=10560, kv_max=10560,
             causal=False, lens=9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gemv", "plan", "append", "attention", "attention"))
    lens = rng.randrange(1 << 20)
    if op == "gemv":
        # any N, K a multiple of 32, one row to sixteen
        return dict(op=op, rows=_log_int(rng, 1, 16), n=_log_int(rng, 64, 14336),
                    k=32 * _log_int(rng, 4, 400), x=rng.choice(("bf16", "bf16", "fp32")),
                    y=rng.choice(("bf16", "fp32")), act=rng.choice(("none", "gelu")))
    page = rng.choice((16, 16, 32, 48, 64, 128, 880))
    if op == "plan":
        return dict(op=op, batch=_log_int(rng, 1, 512), cached_max=_log_int(rng, 1, 20000),
                    new_min=rng.choice((0, 1)), new_max=_log_int(rng, 1, 250), page=page,
                    spare=rng.randrange(0, 64), lens=lens)
    if op == "append":
        batch = _log_int(rng, 1, 48)
        return dict(op=op, batch=batch, cached_max=_log_int(rng, 1, 2000), new_min=1,
                    new_max=_log_int(rng, 1, max(1, 12000 // batch)),
                    heads=rng.choice((1, 2, 4, 8, 24)), head_dim=rng.choice((64, 128)), page=page,
                    spare=rng.randrange(0, 16), lens=lens)
    kv_heads, group = rng.choice(((1, 8), (2, 5), (4, 4), (8, 1), (8, 4), (8, 8), (24, 1)))
    batch = _log_int(rng, 1, 64)
    kv_max = _log_int(rng, 1, max(1, 250000 // batch))
    q_max = 1
    if rng.random() < 0.5:  # chunks of new tokens over the cache
        batch = _log_int(rng, 1, 8)
        kv_max = _log_int(rng, 2, 12000 // batch)
        q_max = _log_int(rng, 2, max(2, min(kv_max, 2000 * 24 // (kv_heads * group))))
    return dict(op=op, batch=batch, q_heads=kv_heads * group, kv_heads=kv_heads,
                head_dim=rng.choice((64, 128, 128)), page=page, q_min=1, q_max=q_max,
                kv_min=max(1, kv_max // 3), kv_max=kv_max, causal=rng.random() < 0.75, lens=lens)


def _spread(case, count, lo, hi):
    """`count` lengths of [lo, hi], the largest among them; they go by the case alone."""
    r = random.Random(case["lens"] * 7919 + count * 31 + lo + hi)
    v = [r.randint(lo, hi) for _ in range(count)]
    v[r.randrange(count)] = hi
    return v


def _request_lens(case):
    cached = _spread(case, case["batch"], 0, case["cached_max"])
    new = _spread(case, case["batch"], case["new_min"], case["new_max"])
    return cached, new


def _attention_lens(case):
    kv = _spread(case, case["batch"], case["kv_min"], case["kv_max"])
    nq = _spread(case, case["batch"], case["q_min"], case["q_max"])
    return [min(a, b) for a, b in zip(nq, kv)], kv


def _pages(tokens, page):
    return -(-tokens // page)


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "gemv":
        m, n, k = case["rows"], case["n"], case["k"]
        size = {"bf16": 2, "fp32": 4}
        return {"bytes": n * k * 9 / 16 + m * k * size[case["x"]] + m * n * size[case["y"]] + 4,
                "flops": 2.0 * m * n * k}
    if op == "attention":
        nq, kv = _attention_lens(case)
        d, hq, hkv = case["head_dim"], case["q_heads"], case["kv_heads"]
        pages = sum(_pages(t, case["page"]) for t in kv)
        seen = sum(a * t - (a * (a - 1) // 2 if case["causal"] else 0) for a, t in zip(nq, kv))
        return {"bytes": 2.0 * sum(kv) * hkv * d + 8 * pages * hkv + 4 * pages +
                sum(nq) * hq * (4 * d + 4) + 8 * len(kv), "flops": 4.0 * seen * hq * d}
    cached, new = _request_lens(case)
    page = case["page"]
    if op == "plan":
        fresh = sum(_pages(c + t, page) - _pages(c, page) for c, t in zip(cached, new))
        return {"bytes": 4.0 * (4 * len(new) + sum(new) + 2 * fresh + 3), "flops": 0.0}
    h, d = case["heads"], case["head_dim"]
    runs = sum(_pages(c + t, page) - c // page for c, t in zip(cached, new))
    return {"bytes": 6.0 * sum(new) * h * d + 4 * sum(new) + 16 * runs * h, "flops": 0.0}


# ---------------------------------------------------------------- inputs
def _tables(case, kv, extra, rng):
    """A block table for requests of `kv` tokens over pages in a random order, and the rest."""
    page, batch = case["page"], len(kv)
    held = [_pages(t, page) for t in kv]
    room = max(1, max(_pages(t + e, page) for t, e in zip(kv, extra)))
    fresh = sum(_pages(t + e, page) - h for t, e, h in zip(kv, extra, held))
    n_pages = sum(held) + fresh + case.get("spare", 2)
    order = list(range(n_pages))
    rng.shuffle(order)
    table = [[-1] * room for _ in range(batch)]
    at = 0
    for b in range(batch):
        table[b][:held[b]] = order[at:at + held[b]]
        at += held[b]
    return (torch.tensor(table, dtype=torch.int32, device="cuda"),
            torch.tensor(order[at:], dtype=torch.int32, device="cuda"), n_pages)


def _cache(g, n_pages, heads, page, dim):
    """Codes and page scales as normal K and V leave them: the largest code of a page near the
    format's largest, exponents that differ by page and head."""
    def plane():
        codes = torch.empty(n_pages, heads, page, dim, dtype=torch.float8_e4m3fn, device="cuda")
        for i in range(0, n_pages, 1024):
            part = codes[i:i + 1024]
            part.copy_((torch.randn(part.shape, generator=g, device="cuda") * 80).clamp(-448, 448))
        exps = torch.randint(-8, -5, (n_pages, heads), generator=g, device="cuda")
        return codes, _pow2(exps)
    k, ks = plane()
    v, vs = plane()
    return dict(k_codes=k, v_codes=v, k_scale=ks, v_scale=vs)


def _pow2(e):
    """2^e as fp32, from its exponent field: -126 <= e <= 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "gemv":
        n, k = case["n"], case["k"]
        w = torch.randn(n, k // 16, 16, generator=g, device="cuda") * 0.02
        s_t = w.abs().max() / 2688
        sb = (w.abs().amax(2) / (6 * s_t)).to(torch.float8_e4m3fn)
        y = w / (sb.float() * s_t).clamp_min(1e-30).unsqueeze(2)
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
        code = torch.bucketize(y.abs(), edges).to(torch.uint8) | ((y < 0).to(torch.uint8) << 3)
        code = code.reshape(n, k // 2, 2)
        s["codes"] = (code[:, :, 0] | (code[:, :, 1] << 4)).contiguous()
        # tensor-core layout of the block scales: tiles of 128 rows x 4 blocks
        rp, cp = -(-n // 128) * 128, -(-(k // 16) // 4) * 4
        pad = torch.zeros(rp, cp, dtype=torch.uint8, device="cuda")
        pad[:n, :k // 16] = sb.view(torch.uint8)
        s["sf"] = pad.view(rp // 128, 4, 32, cp // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)
        s["s_t"] = s_t.reshape(1)
        x = torch.randn(case["rows"], k, generator=g, device="cuda")
        x[:, torch.randperm(k, generator=g, device="cuda")[:8]] *= 30  # outlier channels
        s["x"] = x.to(torch.bfloat16) if case["x"] == "bf16" else x
        return s
    if op == "attention":
        nq, kv = _attention_lens(case)
        s["table"], _, n_pages = _tables(case, kv, [0] * len(kv), rng)
        s.update(_cache(g, n_pages, case["kv_heads"], case["page"], case["head_dim"]))
        s["q"] = torch.randn(sum(nq), case["q_heads"], case["head_dim"], generator=g,
                             device="cuda").to(torch.bfloat16)
        starts = [0]
        for t in nq:
            starts.append(starts[-1] + t)
        s["cu_q"], s["seq_lens"] = _int32(starts), _int32(kv)
        s["max_q"], s["max_kv"] = max(nq), max(kv)
        return s
    cached, new = _request_lens(case)
    s["table"], s["free"], s["n_pages"] = _tables(case, cached, new, rng)
    s["cached"], s["new"], s["tokens"] = _int32(cached), _int32(new), sum(new)
    s["head"] = _int32([0])
    if op == "plan":
        return s
    # append: slots as a plan gives them, K and V the last two thirds of a fused projection
    s.update(_cache(g, s["n_pages"], case["heads"], case["page"], case["head_dim"]))
    s["slots"] = _plan_plain(s)[2]
    h, d = case["heads"], case["head_dim"]
    qkv = torch.randn(s["tokens"], 3, h, d, generator=g, device="cuda")
    qkv *= torch.rand(h, 1, generator=g, device="cuda") * 3.5 + 0.5  # a deviation for each head
    qkv = qkv.to(torch.bfloat16)
    s["k"], s["v"] = qkv[:, 1], qkv[:, 2]
    return s


# ---------------------------------------------------------------- plain forms
def _gelu(y):
    return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))


def _gemv_plain(s):
    case = s["case"]
    n, k = case["n"], case["k"]
    rp, cp = -(-n // 128) * 128, -(-(k // 16) // 4) * 4
    sb = s["sf"].view(rp // 128, cp // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rp, cp)
    sb = sb[:n, :k // 16].contiguous().view(torch.float8_e4m3fn).float()
    table = torch.tensor(E2M1, device="cuda")
    code = torch.stack((s["codes"] & 15, s["codes"] >> 4), 2).int()
    w = table[code.reshape(n, k // 16, 16)] * sb.unsqueeze(2)
    y = (s["x"].float() @ w.reshape(n, k).t()) * s["s_t"]
    if case["act"] == "gelu":
        # a bf16 layer hands its activation the rounded value
        y = _gelu(y.to(torch.bfloat16).float() if case["y"] == "bf16" else y)
    return y.to(torch.bfloat16) if case["y"] == "bf16" else y


def _plan_plain(s):
    page, tokens = s["case"]["page"], s["tokens"]
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    seq = cached + new
    held = (cached + page - 1) // page
    total = (seq + page - 1) // page
    need = total - held
    first = torch.cumsum(need, 0) - need + s["head"].long()
    cu = torch.cat((torch.zeros_like(new[:1]), torch.cumsum(new, 0)))
    # pages held.. total of every request come from the free list
    col = torch.arange(table.shape[1], device="cuda")
    fresh = (col >= held[:, None]) & (col < total[:, None])
    at = (first[:, None] + col - held[:, None]).clamp(0, max(0, s["free"].numel() - 1))
    source = s["free"] if s["free"].numel() else s["free"].new_zeros(1)
    table = torch.where(fresh, source[at], table)
    token = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(cu, token, right=True) - 1
    pos = cached[b] + token - cu[b]
    slots = table[b, pos // page].long() * page + pos % page
    return (seq.int(), cu.int(), slots.int(), table, (s["head"] + need.sum()).int())


def _append_plane(x, codes, scale, slots):
    n_pages, heads, page, dim = codes.shape
    x = x.float()
    where, off = slots.long() // page, slots.long() % page
    amax = torch.zeros(n_pages, heads, device="cuda")
    amax.scatter_reduce_(0, where[:, None].expand(-1, heads), x.abs().amax(2), "amax")
    first = torch.full((n_pages,), page, device="cuda", dtype=torch.int64)
    first.scatter_reduce_(0, where, off, "amin")       # first new slot of each page
    mant, exp = torch.frexp(amax)                      # amax = mant 2^exp, 0.5 <= mant < 1
    e = torch.where(mant <= 0.875, exp - 9, exp - 8)   # smallest e with amax <= 448 2^e
    e = torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    fit = _pow2(e)
    fresh = torch.where((first > 0)[:, None], torch.maximum(scale, fit), fit)
    now = torch.where((first < page)[:, None], fresh, scale)
    # tokens that a grown scale finds in its page are coded again
    old = torch.arange(page, device="cuda")[None, :] < first[:, None]
    again = (old & (first < page)[:, None])[:, None, :] & (now != scale)[:, :, None]
    value = codes.float()
    value = torch.where(again[..., None], value * (scale / now)[..., None, None], value)
    out = value.to(torch.float8_e4m3fn)
    coded = (x / now[where][..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    out.view(torch.uint8)[where, :, off] = coded.view(torch.uint8)
    return out, now


def _attention_plain(s):
    case = s["case"]
    d, hkv, page = case["head_dim"], case["kv_heads"], case["page"]
    group = case["q_heads"] // hkv
    batch, wide = s["table"].shape
    ids = s["table"].long().clamp_min(0)
    tokens = wide * page

    def plane(codes, scale):  # [batch, heads, tokens, dim]
        x = codes[ids].float() * scale[ids][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(batch, hkv, tokens, d)

    k, v = plane(s["k_codes"], s["k_scale"]), plane(s["v_codes"], s["v_scale"])
    nq, kv = s["cu_q"].long().diff(), s["seq_lens"].long()
    most = s["max_q"]
    row = torch.arange(most, device="cuda")
    live = row < nq[:, None]
    at = (s["cu_q"].long()[:-1, None] + row).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][at].float().reshape(batch, most, hkv, group, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(batch, hkv, group * most, d) * d ** -0.5, k.transpose(2, 3))
    x = x.reshape(batch, hkv, group, most, tokens)
    key = torch.arange(tokens, device="cuda")
    last = kv[:, None] - nq[:, None] + row if case["causal"] else (kv - 1)[:, None].expand(-1, most)
    seen = (key <= last[..., None]) & (key < kv[:, None, None])
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(4, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(4, keepdim=True)
    o = torch.matmul(p.reshape(batch, hkv, group * most, tokens), v)
    o = o.reshape(batch, hkv, group, most, d) / total.clamp_min(1e-30)
    lse = (top + torch.log(total)).squeeze(4)
    # [batch, kv heads, group, rows] -> the tokens of each request in turn
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, most, hkv * group, d)
    lse = lse.permute(0, 3, 1, 2).reshape(batch, most, hkv * group)
    return o[live].to(torch.bfloat16), lse[live]


def _run_own(s):
    import nvfp4_w4a4_quantized_08_b200 as nv
    case = s["case"]
    op = case["op"]
    if op == "gemv":
        w = nv.NVFP4Tensor(s["codes"], s["sf"], s["s_t"], case["n"], case["k"], nv.SF_MMA128x4)
        return nv.gemv(s["x"], w, torch.bfloat16 if case["y"] == "bf16" else torch.float32,
                       act=nv.ACT_GELU_TANH if case["act"] == "gelu" else nv.ACT_NONE)
    if op == "plan":
        p = nv.plan_pages(s["cached"], s["new"], s["table"], s["free"], s["head"],
                          page_tokens=case["page"], n_pages=s["n_pages"], max_new=s["tokens"])
        return p.seq_lens, p.cu_new, p.slot_map, s["table"], p.free_head
    cache = nv.KVCache8(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    if op == "append":
        cache.append(s["k"], s["v"], s["slots"])
        return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]
    return cache.attention(s["q"], s["cu_q"], s["seq_lens"], s["table"], max_q=s["max_q"],
                           max_kv=s["max_kv"], causal=case["causal"], return_lse=True)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "gemv":
        return _gemv_plain(state)
    if op == "plan":
        return _plan_plain(state)
    if op == "append":
        k, ks = _append_plane(state["k"], state["k_codes"], state["k_scale"], state["slots"])
        v, vs = _append_plane(state["v"], state["v_codes"], state["v_scale"], state["slots"])
        return k, v, ks, vs
    return _attention_plain(state)


# ---------------------------------------------------------------- definitions in 64 bits
def _exact_gemv(s):
    case = s["case"]
    n, k = case["n"], case["k"]
    r = torch.arange(n, device="cuda")[:, None]
    c = torch.arange(k // 16, device="cuda")[None, :]
    tiles = -(-(k // 16) // 4)
    at = ((r // 128) * tiles + c // 4) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + c % 4
    byte = s["sf"][at].int()
    e, m = byte >> 3, (byte & 7).double()
    scale = torch.where(byte >= 8, (1 + m / 8) * _pow2(e - 7).double(), m / 8 * 2.0 ** -6)
    w = torch.empty(n, k, dtype=torch.float64, device="cuda")
    for half in (0, 1):
        c4 = (s["codes"].int() >> (4 * half)) & 15
        e2, m1 = (c4 >> 1) & 3, (c4 & 1).double()
        mag = torch.where(e2 == 0, 0.5 * m1, (1 + 0.5 * m1) * _pow2(e2 - 1).double())
        w[:, half::2] = torch.where(c4 >= 8, -mag, mag)
    w.view(n, k // 16, 16).mul_(scale.unsqueeze(2))
    y = torch.einsum("mk,nk->mn", s["x"].double(), w) * s["s_t"].double()
    if case["act"] == "gelu":
        y = y / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y


def _exact_plan(s):
    page = s["case"]["page"]
    cached, new = s["cached"].tolist(), s["new"].tolist()
    table, free, head = s["table"].tolist(), s["free"].tolist(), s["head"].item()
    starts, slots = [0], []
    for b, (c, t) in enumerate(zip(cached, new)):
        for pos in range(c, c + t):
            if pos % page == 0:
                table[b][pos // page] = free[head]
                head += 1
            slots.append(table[b][pos // page] * page + pos % page)
        starts.append(starts[-1] + t)
    return (_int32([c + t for c, t in zip(cached, new)]), _int32(starts), _int32(slots),
            _int32(table), _int32([head]))


def _e4m3(x):
    """Nearest E4M3 value, ties to even, the largest finite one beyond it; in 64 bits."""
    a = x.abs()
    e = torch.frexp(a.clamp_min(2.0 ** -6))[1] - 1
    step = _pow2(e - 3).double()
    return torch.copysign((torch.round(a / step) * step).clamp_max(448.0), x)


def _exact_append(s):
    def plane(x, codes, scale):
        x, value, scale = x.double(), codes.double(), scale.double()
        page = codes.shape[2]
        slots = s["slots"].cpu()
        pages = slots // page
        for p in pages.unique().tolist():
            t = (pages == p).nonzero().flatten()
            off = (slots[t] % page).tolist()
            mine = x[t.cuda()]                               # [new tokens, heads, dim]
            amax = mine.abs().amax((0, 2))
            e = torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448)).clamp(E_MIN, E_MAX).int()
            # the logarithm may be off by an ulp
            e += (amax > 448 * _pow2(e).double()).int()
            e -= (amax <= 448 * _pow2(e - 1).double()).int()
            sn = _pow2(e.clamp(E_MIN, E_MAX)).double()
            if min(off) > 0:
                sn = torch.maximum(sn, scale[p])
                n = min(off)
                value[p, :, :n] = _e4m3(value[p, :, :n] * (scale[p] / sn)[:, None, None])
            scale[p] = sn
            value[p, :, off] = _e4m3(mine / sn[:, None]).transpose(0, 1)
        return value, scale
    k, ks = plane(s["k"], s["k_codes"], s["k_scale"])
    v, vs = plane(s["v"], s["v_codes"], s["v_scale"])
    return k, v, ks, vs


def _exact_attention(s):
    case = s["case"]
    d, hkv = case["head_dim"], case["kv_heads"]
    group = case["q_heads"] // hkv
    starts, kv = s["cu_q"].tolist(), s["seq_lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, t in enumerate(kv):
        lo, hi = starts[b], starts[b + 1]
        ids = s["table"][b, :_pages(t, case["page"])].long()
        for h in range(hkv):
            k = (s["k_codes"][ids, h].double() * s["k_scale"][ids, h].double()[:, None, None])
            v = (s["v_codes"][ids, h].double() * s["v_scale"][ids, h].double()[:, None, None])
            k, v = k.reshape(-1, d)[:t], v.reshape(-1, d)[:t]
            for g in range(h * group, (h + 1) * group):
                x = s["q"][lo:hi, g].double() @ k.t() / math.sqrt(d)
                if case["causal"]:
                    last = torch.arange(t - (hi - lo), t, device="cuda")
                    x[torch.arange(t, device="cuda")[None] > last[:, None]] = -math.inf
                lse[lo:hi, g] = torch.logsumexp(x, 1)
                out[lo:hi, g] = torch.softmax(x, 1) @ v
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"gemv": _exact_gemv, "plan": _exact_plan, "append": _exact_append,
            "attention": _exact_attention}[case["op"]](s)
