"""Plain 64-bit forms of the paged 8-bit cache, for its tests: numpy and torch on the CPU,
written from the definitions in include/nvfp4.h."""
from __future__ import annotations

import math

import torch

MIN_EXP, MAX_EXP = -60, 60


def e4m3(x: torch.Tensor) -> torch.Tensor:
    """Nearest E4M3 value (ties to even, saturating at 448) of a float64 tensor."""
    a = x.abs()
    e = torch.frexp(a.clamp_min(2.0 ** -6))[1] - 1
    step = torch.ldexp(torch.ones_like(a), e - 3)
    return torch.copysign((torch.round(a / step) * step).clamp_max(448.0), x)


def plan(cached, new, table, free, head, page):
    """Lists in, lists out: the plan by one walk over the tokens."""
    table = [row[:] for row in table]
    cu, slots = [0], []
    for b, (c, t) in enumerate(zip(cached, new)):
        for pos in range(c, c + t):
            if pos % page == 0:
                table[b][pos // page] = free[head]
                head += 1
            slots.append(table[b][pos // page] * page + pos % page)
        cu.append(cu[-1] + t)
    return [c + t for c, t in zip(cached, new)], cu, slots, table, head


def append(x, value, scale, slots, page):
    """One plane.  x [tokens, heads, dim], value [pages, heads, page, dim] (code values) and
    scale [pages, heads], all float64; slots a list.  Updates value and scale in place."""
    by_page = {}
    for t, s in enumerate(slots):
        if s >= 0:
            by_page.setdefault(s // page, []).append((t, s % page))
    for p, places in by_page.items():
        toks = [t for t, _ in places]
        first = min(o for _, o in places)
        for h in range(x.shape[1]):
            mine = x[toks, h]
            finite = mine[torch.isfinite(mine)]
            amax = float(finite.abs().max()) if finite.numel() else 0.0
            e = MIN_EXP
            while e < MAX_EXP and amax > 448 * 2.0 ** e:
                e += 1
            s = 2.0 ** e
            if first > 0:
                was = float(scale[p, h])
                s = max(s, was)
                if s > was:
                    value[p, h, :first] = e4m3(value[p, h, :first] * (was / s))
            scale[p, h] = s
            for t, o in places:
                row = torch.nan_to_num(x[t, h] / s, nan=0.0, posinf=448.0, neginf=-448.0)
                value[p, h, o] = e4m3(row)


def attention(q, k_value, v_value, k_scale, v_scale, table, nq, kv, page, causal, scale):
    """float64 (out, lse, E, A) of packed queries q [tokens, q_heads, dim]: E = sum p |v| per
    output element, plus what 16-bit weights may lose in a row, A the largest
    scale sum |q k| of a row."""
    tokens, hq, d = q.shape
    hkv = k_value.shape[1]
    group = hq // hkv
    out = torch.zeros(tokens, hq, d, dtype=torch.float64)
    lse = torch.full((tokens, hq), -math.inf, dtype=torch.float64)
    E = torch.zeros_like(out)
    A = torch.zeros_like(lse)
    at = 0
    for b, (n, t) in enumerate(zip(nq, kv)):
        ids = table[b][: -(-t // page)]
        for h in range(hkv):
            if t == 0 or n == 0:
                continue
            k = torch.cat([k_value[p, h] * k_scale[p, h] for p in ids])[:t]
            v = torch.cat([v_value[p, h] * v_scale[p, h] for p in ids])[:t]
            sv = torch.cat([v_scale[p, h].expand(page) for p in ids])[:t]
            for g in range(h * group, (h + 1) * group):
                x = q[at:at + n, g] @ k.t() * scale
                A[at:at + n, g] = (q[at:at + n, g].abs() @ k.abs().t() * scale).amax(1)
                if causal:
                    last = torch.arange(t - n, t)
                    x = x.masked_fill(torch.arange(t)[None] > last[:, None], -math.inf)
                live = torch.isfinite(x).any(1)
                l = torch.logsumexp(x, 1)
                p = torch.where(live[:, None], torch.exp(x - l[:, None].nan_to_num()), 0.0)
                lse[at:at + n, g] = l
                out[at:at + n, g] = p @ v
                E[at:at + n, g] = p @ v.abs() + \
                    t * 2.0 ** -32 * 448 * (p * sv).amax(1, keepdim=True) * 2.0 ** 7
        at += n
    return out, lse, E, A


def assert_attention_close(out, lse, ref):
    """|o - ref| <= 2^-7 (E + A' E) + 2^-8 |ref|: a probability enters the product with V as bf16
    or fp16 (relative half steps of 2^-8 and 2^-11; fp16 weights lose up to 2^-32 of the row's
    largest weight each, counted in E times 2^7), scores are fp32 sums of exact products (error
    2^-20 A, twice in a quotient: A' = 2^-12 A with the factor in front), sums of up to 2^17
    fp32 terms in chains of at most 2^12 add 2^-11 E; together below 2^-7 E (1 + 2^-12 A).
    The output is rounded to bf16 (2^-8).  lse: 2^-19 A for the scores, 2^-18 for the sum and
    the logarithm, relative to max(1, |lse|)."""
    o_ref, l_ref, E, A = ref
    o = out.double().cpu()
    tol = 2.0 ** -7 * E * (1 + 2.0 ** -12 * A[..., None]) + 2.0 ** -8 * o_ref.abs()
    bad = ~((o - o_ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                           o[bad][:4].tolist(), o_ref[bad][:4].tolist())
    if lse is not None:
        l = lse.double().cpu()
        empty = torch.isinf(l_ref)
        assert torch.equal(torch.isinf(l) & (l < 0), empty)
        err = (l - l_ref)[~empty].abs()
        bound = (2.0 ** -19 * A + 2.0 ** -18 * l_ref.abs().clamp_min(1.0))[~empty]
        assert bool((err <= bound).all()), float((err / bound).max())
