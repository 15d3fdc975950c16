"""GPU parity of the paged 8-bit cache: page plans (exact), the quantizing write (exact codes and
scales) and the attention (tests/_kv8.py's bounds), alone and together."""
import contextlib
import math
import random
import time

import pytest
import torch

import nvfp4_w4a4_quantized_08_b200 as nv
from nvfp4_w4a4_quantized_08_b200 import _native as N

import _kv8 as ref

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def clean_status():
    nv.device_status()
    yield
    assert nv.device_status() == N.OK


# ---------------------------------------------------------------- plans
def _tables(cached, new, page, spare, seed):
    r = random.Random(seed)
    held = [-(-c // page) for c in cached]
    room = max([1] + [-(-(c + t) // page) for c, t in zip(cached, new)])
    total = sum(-(-(c + t) // page) for c, t in zip(cached, new)) + spare
    order = list(range(total))
    r.shuffle(order)
    table, at = [[-1] * room for _ in cached], 0
    for b, n in enumerate(held):
        table[b][:n] = order[at:at + n]
        at += n
    return table, order[at:], total


@pytest.mark.parametrize("batch,cached_max,new_max,page", [
    (1, 0, 1, 16), (1, 31, 1, 16), (3, 40, 5, 16), (33, 2000, 1, 32), (65, 300, 400, 64),
    (513, 100, 70, 48), (1025, 64, 3, 16), (8192, 20, 2, 16), (2, 5000, 3000, 880)])
def test_plan(batch, cached_max, new_max, page):
    r = random.Random(batch * 31 + page)
    cached = [r.randint(0, cached_max) for _ in range(batch)]
    new = [r.randint(0, new_max) for _ in range(batch)]
    table, free, n_pages = _tables(cached, new, page, 3, 1)
    head, free = 2, [9999, 9999] + free
    want = ref.plan(cached, new, table, free, head, page)
    room = sum(new) + 7
    dev_table = torch.full((batch, len(table[0]) + 3), -5, dtype=torch.int32, device="cuda")
    dev_table[:, :len(table[0])] = i32(table)
    got = nv.plan_pages(i32(cached), i32(new), dev_table[:, :len(table[0])], i32(free),
                        i32([head]), page_tokens=page, n_pages=n_pages, max_new=room)
    assert got.seq_lens.tolist() == want[0]
    assert got.cu_new.tolist() == want[1]
    assert got.slot_map.tolist() == want[2] + [-1] * 7
    assert dev_table[:, :len(table[0])].tolist() == want[3]
    assert bool((dev_table[:, len(table[0]):] == -5).all())
    assert got.free_head.tolist() == [want[4]]


def test_plan_without_requests_or_tokens():
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    p = nv.plan_pages(none, none, none.view(0, 4), i32([1]), i32([0]), page_tokens=16, n_pages=4,
                      max_new=3)
    assert p.cu_new.tolist() == [0] and p.slot_map.tolist() == [-1] * 3
    assert p.free_head.tolist() == [0] and p.seq_lens.numel() == 0
    p = nv.plan_pages(i32([5, 0]), i32([0, 0]), i32([[1], [0]]), none, i32([0]), page_tokens=16,
                      n_pages=4, max_new=0)
    assert p.seq_lens.tolist() == [5, 0] and p.cu_new.tolist() == [0, 0, 0]
    assert p.slot_map.numel() == 0 and p.free_head.tolist() == [0]


@pytest.mark.parametrize("case,status", [
    ("pages", N.ERR_CAPACITY), ("table", N.ERR_CAPACITY), ("slots", N.ERR_CAPACITY),
    ("negative", N.ERR_INVALID_ARG), ("head", N.ERR_INVALID_ARG), ("huge", N.ERR_CAPACITY)])
def test_plan_is_all_or_nothing(case, status):
    cached, new, max_new, head = [20, 3], [30, 20], 50, 0
    free = [5, 6, 7]
    if case == "pages":
        free = [5, 6]
    if case == "table":
        new = [10, 70]
        max_new = 80
    if case == "slots":
        max_new = 49
    if case == "negative":
        new = [30, -1]
    if case == "head":
        head = 4
    if case == "huge":
        cached, new = [2 ** 31 - 1, 0], [2 ** 31 - 1, 1]
    table = i32([[1, 2, -1, -1], [3, -1, -1, -1]])
    before = table.clone()
    p = nv.plan_pages(i32(cached), i32(new), table, i32(free), i32([head]), page_tokens=16,
                      n_pages=16, max_new=max_new)
    assert nv.device_status() == status
    assert torch.equal(table, before) and p.seq_lens.tolist() == cached
    assert p.cu_new.tolist() == [0, 0, 0] and p.free_head.tolist() == [head]
    assert bool((p.slot_map == -1).all())


def test_plan_with_a_page_outside_the_pool():
    """Page ids outside the cache give no slots and are recorded."""
    p = nv.plan_pages(i32([4, 16]), i32([2, 1]), i32([[99, 0], [1, -1]]), i32([-3]), i32([0]),
                      page_tokens=16, n_pages=8, max_new=3)
    assert p.slot_map.tolist() == [-1, -1, -1]
    assert nv.device_status() == N.ERR_INVALID_ARG


# ---------------------------------------------------------------- append
def _random_cache(n_pages, page, heads, dim, seed, spread=2):
    g = torch.Generator().manual_seed(seed)
    c = nv.KVCache8.empty(n_pages, page, heads, dim)
    for codes, scale in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
        x = (torch.randn(codes.shape, generator=g) * 80).clamp(-448, 448)
        codes.copy_(x.to(torch.float8_e4m3fn))
        e = torch.randint(-7 - spread, -7 + spread + 1, scale.shape, generator=g)
        scale.copy_(torch.ldexp(torch.ones(scale.shape, dtype=torch.float64), e).float())
    return c


def _planes64(c):
    return [t.cpu().double() for t in (c.k_codes, c.v_codes, c.k_scale, c.v_scale)]


def _check_append(c, k, v, slots, before):
    kv, vv, ks, vs = before
    ref.append(k.cpu().double(), kv, ks, slots, c.page_tokens)
    ref.append(v.cpu().double(), vv, vs, slots, c.page_tokens)
    for got, want in zip(_planes64(c), (kv, vv, ks, vs)):
        assert torch.equal(got, want), (got != want).nonzero()[:4].tolist()


@pytest.mark.parametrize("heads,dim,page,counts", [
    (1, 64, 16, [1]), (8, 128, 16, [1, 1, 1, 1, 1]), (3, 128, 32, [40, 1, 17, 0, 64]),
    (2, 64, 64, [130, 3]), (5, 128, 48, [100, 47, 1]), (1, 128, 880, [900, 5]),
    (2, 64, 1024, [1500]), (2, 128, 4096, [4096, 1])])
def test_append(heads, dim, page, counts):
    r = random.Random(page + dim)
    cached = [r.randint(0, 2 * page) for _ in counts]
    table, free, n_pages = _tables(cached, counts, page, 2, 3)
    _, _, slots, _, _ = ref.plan(cached, counts, table, free, 0, page)
    c = _random_cache(n_pages, page, heads, dim, 4)
    before = _planes64(c)
    g = torch.Generator().manual_seed(5)
    qkv = torch.randn(sum(counts), 3, heads, dim, generator=g)
    qkv *= torch.exp2(torch.randint(-6, 7, (sum(counts), 1, 1, 1), generator=g).float())
    qkv = qkv.to(torch.bfloat16).cuda()
    k, v = qkv[:, 1], qkv[:, 2]
    c.append(k, v, i32(slots + [-1, -1]))
    _check_append(c, k, v, slots, before)


def test_append_many_single_tokens():
    """More single tokens than CTAs: several runs a CTA."""
    heads, dim, page, batch = 24, 64, 16, 3000
    c = _random_cache(batch, page, heads, dim, 1)
    slots = [p * page + (7 * p) % page for p in range(batch)]
    before = _planes64(c)
    x = torch.randn(batch, heads, dim, generator=torch.Generator().manual_seed(2)) * 3
    x = x.to(torch.bfloat16).cuda()
    c.append(x, -x, i32(slots))
    # the oracle for a part of them: a page is one run here, and goes by itself
    keep = list(range(0, batch, 97))
    sub = [t[keep] for t in before]
    ref.append(x.cpu().double()[keep], sub[0], sub[2], [i * page + slots[p] % page
                                                        for i, p in enumerate(keep)], page)
    now = _planes64(c)
    assert torch.equal(now[0][keep], sub[0]) and torch.equal(now[2][keep], sub[2])


def test_append_edges():
    """Zeros, the scale's ends, saturation, ties, skipped tokens, -0."""
    c = nv.KVCache8.empty(6, 16, 1, 64)
    x = torch.zeros(6, 1, 64)
    x[1] = 2.0 ** -120
    x[2] = 2.0 ** 100
    x[3, 0, :4] = torch.tensor([448.0, 449.0, 17.0, -0.0])
    x[4, 0, :4] = torch.tensor([1.75 * 2 ** 20, 1.0625 * 2 ** 4, -1.1875 * 2 ** 4, 2.0 ** 3])
    x[5] = 1.0
    x = x.to(torch.bfloat16).cuda()
    slots = [0, 16, 32, 48, 64, -1]
    before = _planes64(c)
    c.append(x, x, i32(slots))
    _check_append(c, x, x, slots, before)
    assert float(c.k_scale[0, 0]) == 2.0 ** -60 and float(c.k_scale[2, 0]) == 2.0 ** 60
    assert float(c.k_scale[5, 0]) == 0.0


def test_append_grows_a_page_token_by_token():
    c = nv.KVCache8.empty(1, 16, 2, 128)
    g = torch.Generator().manual_seed(0)
    for t in range(16):
        x = (torch.randn(1, 2, 128, generator=g) * 2.0 ** (t - 8)).to(torch.bfloat16).cuda()
        before = _planes64(c)
        c.append(x, x * 0.5, i32([t]))
        _check_append(c, x, x * 0.5, [t], before)


def test_append_non_finite_and_bad_slots():
    c = _random_cache(3, 16, 2, 64, 9)
    x = torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(1))
    x[0, 0, 3], x[0, 1, 5], x[1, 0, 0] = float("inf"), float("nan"), -float("inf")
    x = x.to(torch.bfloat16).cuda()
    before = _planes64(c)
    slots = [4, 5, 16]
    c.append(x, x, i32(slots))
    assert nv.device_status() == N.ERR_DOMAIN
    _check_append(c, x, x, slots, before)
    y = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    before = _planes64(c)
    c.append(y, y, i32([48, -2, 2 ** 31 - 1, 33]))   # 48 slots: only the last is one
    assert nv.device_status() == N.ERR_INVALID_ARG
    _check_append(c, y, y, [-1, -1, -1, 33], before)
    c.append(y[:0], y[:0], i32([]))


# ---------------------------------------------------------------- attention
def _attention_case(c, nq, kv, hq, causal, seed, page_seed=0, poison=True, **kw):
    r = random.Random(page_seed)
    page = c.page_tokens
    held = [-(-t // page) for t in kv]
    order = list(range(c.n_pages))
    r.shuffle(order)
    table, at = [], 0
    wide = max([1] + held) + 1
    for n in held:
        table.append(order[at:at + n] + [10 ** 6] * (wide - n))   # never to be read
        at += n
    assert at <= c.n_pages
    if poison:  # what no request holds: NaN codes and scales
        for codes, scale in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
            raw = codes.view(torch.uint8)
            free = torch.tensor(order[at:], dtype=torch.long, device="cuda")
            raw[free] = 0x7F
            scale[free] = float("nan")
            for b, t in enumerate(kv):
                if t % page:
                    raw[table[b][t // page], :, t % page:] = 0xFF
    g = torch.Generator().manual_seed(seed)
    tokens = sum(nq)
    q = torch.randn(tokens + 3, hq, c.head_dim, generator=g).to(torch.bfloat16).cuda()
    cu = [0]
    for n in nq:
        cu.append(cu[-1] + n)
    out = torch.full_like(q, 5.0)
    scale = kw.pop("scale", None)
    o, lse = c.attention(q, i32(cu), i32(kv), i32(table), causal=causal, out=out, scale=scale,
                         return_lse=True, **kw)
    assert o is out and bool((out[tokens:] == 5).all())
    planes = _planes64(c)
    want = ref.attention(q[:tokens].cpu().double(), planes[0], planes[1], planes[2], planes[3],
                         table, nq, kv, page, causal, scale or c.head_dim ** -0.5)
    ref.assert_attention_close(o[:tokens], lse[:tokens], want)
    return q, i32(cu), i32(kv), i32(table), o, lse


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hkv,group", [(1, 1), (2, 3), (3, 8), (1, 16), (2, 20)])
@pytest.mark.parametrize("page", [16, 48])
def test_single_tokens(dim, hkv, group, page):
    kv = [1, 15, 16, 17, 0, 100, 333]
    c = _random_cache(40, page, hkv, dim, 7)
    _attention_case(c, [1] * len(kv), kv, hkv * group, True, 3)


@pytest.mark.parametrize("kv", [[5000], [1, 9000], [4096, 4097, 63]])
@pytest.mark.parametrize("group", [1, 4, 12])
def test_split_ranges(kv, group):
    """Long caches of few requests: ranges on several CTAs, joined."""
    c = _random_cache(sum(-(-t // 64) for t in kv) + 2, 64, 2, 128, 8)
    args = dict(max_kv=max(kv))
    q, cu, lens, table, o, lse = _attention_case(c, [1] * len(kv), kv, 2 * group, True, 4, **args)
    # the hint may be wrong in either direction
    for hint in (1, 700, 10 ** 6, None):
        o2, l2 = c.attention(q, cu, lens, table, max_kv=hint, return_lse=True)
        n = len(kv)
        assert float((o2[:n].float() - o[:n].float()).abs().max()) <= \
            2.0 ** -6 * float(o[:n].float().abs().max())
        assert float((l2[:n] - lse[:n]).abs().max()) <= 1e-4


CHUNKS = [
    ([3, 2, 1], [3, 50, 200]), ([1, 128, 17, 0], [40, 128, 300, 70]), ([129], [129]),
    ([257, 1, 64], [400, 513, 64]), ([300], [1000])]


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,kv", CHUNKS)
@pytest.mark.parametrize("hkv,group,page", [(2, 1, 16), (1, 3, 48), (2, 4, 64), (1, 8, 128)])
def test_chunks(dim, causal, nq, kv, hkv, group, page):
    c = _random_cache(sum(-(-t // page) for t in kv) + 2, page, hkv, dim, 11)
    _attention_case(c, nq, kv, hkv * group, causal, 5, max_q=max(nq))


@pytest.mark.parametrize("hq,n", [(4, 40), (4, 2)])
def test_rows_that_see_nothing(hq, n):
    """More queries than cached tokens: the first rows are zero, their log-sum-exp -inf."""
    for kv in (0, 1, 17):
        c = _random_cache(6, 16, 2, 128, 12)   # a new one: what is free is made NaN
        nq = n + kv
        *_, o, lse = _attention_case(c, [nq, 1], [kv, 3], hq, True, 6, max_q=nq)
        assert not o[:nq - kv].any() and bool((lse[:nq - kv] == -float("inf")).all())


@pytest.mark.parametrize("nq", [1, 30])
def test_page_scales_far_apart(nq):
    """V scales 2^40 apart, the large ones under negligible probabilities and the other way
    round: the weights go by their product."""
    c = _random_cache(12, 16, 1, 128, 13, spread=0)
    for p in range(12):
        c.v_scale[p] = 2.0 ** (20 if p % 3 else -20)
        c.k_scale[p] = 2.0 ** (-4 if p % 2 else -9)
    _attention_case(c, [nq], [180], 4, True, 7, poison=False, max_q=nq)
    c.v_scale[:] = 2.0 ** 60
    _attention_case(c, [nq], [180], 4, True, 8, poison=False, max_q=nq)
    c.v_scale[:] = 2.0 ** -60
    _attention_case(c, [nq], [180], 4, True, 9, poison=False, max_q=nq)


@pytest.mark.parametrize("nq", [1, 20])
@pytest.mark.parametrize("mult", [0.0, 1e-30, 30.0, 1e3])
def test_sharp_and_flat_scores(nq, mult):
    c = _random_cache(30, 16, 2, 64, 14)
    g = torch.Generator().manual_seed(1)
    q = (torch.randn(nq, 4, 64, generator=g) * mult).to(torch.bfloat16).cuda()
    kv = 470
    table = list(range(30))
    o, lse = c.attention(q, i32([0, nq]), i32([kv]), i32([table]), max_q=nq, return_lse=True)
    p = _planes64(c)
    want = ref.attention(q.cpu().double(), *p, [table], [nq], [kv], 16, True, 0.125)
    ref.assert_attention_close(o, lse, want)


@pytest.mark.parametrize("nq", [1, 50])
def test_offsets_past_32_bits(nq):
    """A pool above 2^32 bytes for each of K and V, the request in its last pages."""
    page, heads, dim = 4096, 16, 128
    n_pages = (1 << 32) // (page * heads * dim) + 3
    c = nv.KVCache8.empty(n_pages, page, heads, dim)
    small = _random_cache(2, page, heads, dim, 15)
    for name in ("k_codes", "v_codes", "k_scale", "v_scale"):
        src, dst = getattr(small, name), getattr(c, name)
        if src.dtype != torch.float32:
            src, dst = src.view(torch.uint8), dst.view(torch.uint8)
        dst[-2:] = src
    q = torch.randn(nq, heads, dim, generator=torch.Generator().manual_seed(2))
    q = q.to(torch.bfloat16).cuda()
    x = torch.randn(10, heads, dim, generator=torch.Generator().manual_seed(3))
    x = x.to(torch.bfloat16).cuda()
    kv = page + 100
    for cache, ids in ((c, [n_pages - 1, n_pages - 2]), (small, [1, 0])):
        cache.append(x, x, i32([ids[1] * page + 90 + i for i in range(10)]))
    got = c.attention(q, i32([0, nq]), i32([kv]), i32([[n_pages - 1, n_pages - 2]]), max_q=nq)
    want = small.attention(q, i32([0, nq]), i32([kv]), i32([[1, 0]]), max_q=nq)
    assert torch.equal(got, want)


@pytest.mark.parametrize("nq", [1, 40])
def test_bad_lengths_and_pages_are_cut_and_recorded(nq):
    c = _random_cache(4, 16, 1, 128, 16)
    q = torch.randn(2 * nq, 4, 128, generator=torch.Generator().manual_seed(2))
    q = q.to(torch.bfloat16).cuda()
    table = i32([[0, 1], [2, 3]])
    good = c.attention(q, i32([0, nq, 2 * nq]), i32([32, 20]), table, max_q=nq)
    for cu, lens, tab in [
            ([0, nq, 2 * nq], [33, 20], table),          # longer than the table
            ([0, nq, 2 * nq], [32, -5], table),          # negative
            ([0, nq, 2 * nq + 1], [32, 20], table),      # past the queries
            ([-1, nq, 2 * nq], [32, 20], table),
            ([0, nq, nq - 1], [32, 20], table),          # descending
            ([0, nq, 2 * nq], [32, 20], i32([[0, 4], [-1, 3]])),
            ([0, nq, 2 * nq], [32, 20], i32([[0, 2 ** 31 - 1], [-2 ** 31, 3]]))]:
        c.attention(q, i32(cu), i32(lens), tab, max_q=nq)
        assert nv.device_status() == N.ERR_INVALID_ARG
    # a request with more queries than the bound: the rest of the batch still holds
    again = c.attention(q, i32([0, nq, 2 * nq]), i32([32, 20]), table, max_q=nq)
    assert torch.equal(again, good)


@pytest.mark.parametrize("nq", [1, 40])
def test_tokens_of_bad_pages_are_left_out(nq):
    c = _random_cache(4, 16, 2, 64, 17)
    q = torch.randn(nq, 4, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    o = c.attention(q, i32([0, nq]), i32([48]), i32([[1, 77, 3]]), causal=False, max_q=nq)
    assert nv.device_status() == N.ERR_INVALID_ARG
    want = c.attention(q, i32([0, nq]), i32([32]), i32([[1, 3]]), causal=False, max_q=nq)
    assert float((o.float() - want.float()).abs().max()) <= 2.0 ** -6 * float(want.float().abs().max())
    o, lse = c.attention(q, i32([0, nq]), i32([16]), i32([[-1]]), causal=False, max_q=nq,
                         return_lse=True)
    assert nv.device_status() == N.ERR_INVALID_ARG
    assert not o.any() and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("nq", [1, 40])
def test_nan_queries_stay_in_their_rows(nq):
    c = _random_cache(4, 16, 1, 128, 18)
    q = torch.randn(nq, 4, 128, generator=torch.Generator().manual_seed(2))
    q = q.to(torch.bfloat16).cuda()
    args = (i32([0, nq]), i32([60]), i32([[0, 1, 2, 3]]))
    good = c.attention(q, *args, max_q=nq)
    q[0, 1, 5] = float("nan")
    got = c.attention(q, *args, max_q=nq)
    assert bool(got[0, 1].isnan().all())
    got[0, 1] = good[0, 1]
    assert torch.equal(got, good)


@pytest.mark.parametrize("nq", [1, 37])
def test_strided_queries_and_outputs(nq):
    c = _random_cache(10, 16, 2, 128, 19)
    hq, d = 4, 128
    qkv = torch.randn(nq, (hq + 4) * d, generator=torch.Generator().manual_seed(2))
    qkv = qkv.to(torch.bfloat16).cuda()
    q = qkv[:, :hq * d].view(nq, hq, d)
    args = (i32([0, nq]), i32([150]), i32([list(range(10))]))
    want = c.attention(q.contiguous(), *args, max_q=nq)
    wide = torch.full((nq, hq * d + 64), 3.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :hq * d].view(nq, hq, d)
    c.attention(q, *args, max_q=nq, out=out)
    assert torch.equal(out, want) and bool((wide[:, hq * d:] == 3).all())


def test_no_queries():
    c = _random_cache(2, 16, 1, 64, 20)
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert c.attention(q, i32([0, 0]), i32([5]), i32([[0]])).shape == (0, 2, 64)


# ---------------------------------------------------------------- together
def _serve(cache, steps, hq, seed, run):
    """Requests that grow: plan, write, attend, step after step.  Yields each step's
    outputs with what the plain forms say of the same device state."""
    g = torch.Generator().manual_seed(seed)
    page, dim, hkv = cache.page_tokens, cache.head_dim, cache.kv_heads
    batch = len(steps[0])
    table = torch.full((batch, 12), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(cache.n_pages, generator=g).int().cuda()
    head, cached = i32([0]), i32([0] * batch)
    for new in steps:
        tokens = sum(new)
        qkv = torch.randn(tokens + 5, hq + 2 * hkv, dim, generator=g).to(torch.bfloat16).cuda()
        p = nv.plan_pages(cached, i32(new), table, free, head, page_tokens=page,
                          n_pages=cache.n_pages, max_new=tokens + 5)
        cache.append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], p.slot_map)
        o, lse = cache.attention(qkv[:, :hq], p.cu_new, p.seq_lens, table, max_q=max(max(new), 1),
                                 return_lse=True)
        planes = _planes64(cache)
        kv = p.seq_lens.tolist()
        want = ref.attention(qkv[:tokens, :hq].cpu().double(), *planes, table.tolist(), new, kv,
                             page, True, dim ** -0.5)
        ref.assert_attention_close(o[:tokens], lse[:tokens], want)
        cached, head = p.seq_lens, p.free_head
    return table, cached


@pytest.mark.parametrize("page,dim,hkv,hq", [(16, 128, 2, 8), (32, 64, 1, 4)])
def test_serving_steps(page, dim, hkv, hq):
    """Prompts of different lengths, then single tokens, a request that joins late and one
    that pauses; the cache against what was written, and the attention against the cache."""
    cache = nv.KVCache8.empty(40, page, hkv, dim)
    steps = [[30, 1, 0, 77], [1, 1, 50, 1], [1, 0, 1, 1], [1, 3, 1, 20], [1, 1, 1, 1]]
    _serve(cache, steps, hq, 1, None)


def test_two_graphs_and_an_eager_call():
    """Decode steps captured into two graphs on one cache and stream, replayed in turn with
    new inputs, an eager call between: the same bits as eager calls."""
    cache = _random_cache(64, 16, 2, 128, 21)
    table = torch.randperm(64, generator=torch.Generator().manual_seed(1)).int().cuda().view(2, 32)
    lens, cu = i32([500, 300]), i32([0, 1, 2])
    qs = [torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(s)).to(torch.bfloat16)
          .cuda() for s in range(4)]
    want = [cache.attention(q, cu, lens, table, max_q=1).clone() for q in qs]
    bufs = [qs[0].clone(), qs[1].clone()]
    graphs, outs = [], []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(cache.attention(b, cu, lens, table, max_q=1))
        graphs.append(g)
    side = torch.cuda.Stream()
    for round_ in range(3):
        a, b = qs[round_ % 4], qs[(round_ + 1) % 4]
        bufs[0].copy_(a)
        bufs[1].copy_(b)
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):   # at the same time, on another stream
            graphs[1].replay()
        eager = cache.attention(qs[3], cu, lens, table, max_q=1)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[round_ % 4])
        assert torch.equal(outs[1], want[(round_ + 1) % 4])
        assert torch.equal(eager, want[3])


@pytest.mark.parametrize("nq", [1, 100])
def test_the_same_bits_every_time(nq):
    cache = _random_cache(200, 16, 2, 128, 22)
    q = torch.randn(nq, 8, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    args = (i32([0, nq]), i32([3000]), torch.arange(200, dtype=torch.int32, device="cuda")[None])
    first = cache.attention(q, *args, max_q=nq)
    for _ in range(5):
        assert torch.equal(cache.attention(q, *args, max_q=nq), first)


@pytest.mark.parametrize("nq", [1, 40])
def test_a_long_run_of_bad_pages_first(nq):
    """Tiles without a single page before the real ones, whose weights are far from 1."""
    c = _random_cache(8, 16, 1, 128, 23)
    c.v_scale[:] = 2.0 ** -25
    q = torch.randn(nq, 4, 128, generator=torch.Generator().manual_seed(2))
    q = q.to(torch.bfloat16).cuda()
    o, lse = c.attention(q, i32([0, nq]), i32([20 * 16]), i32([[-1] * 12 + list(range(8))]),
                         causal=False, max_q=nq, return_lse=True)
    assert nv.device_status() == N.ERR_INVALID_ARG
    want = ref.attention(q.cpu().double(), *_planes64(c), [list(range(8))], [nq], [128], 16, False,
                         128 ** -0.5)
    ref.assert_attention_close(o, lse, want)


@pytest.mark.parametrize("nq", [1, 130])
@pytest.mark.parametrize("step", [0.5, 3.0, 40.0])
def test_scores_that_rise_all_along(nq, step):
    """Every tile has larger scores than the ones before: the reference is raised again and
    again, by little and by much."""
    c = _random_cache(64, 16, 1, 64, 24, spread=0)
    c.k_codes.view(torch.uint8)[:] = 0x38                      # 1.0
    for p in range(64):
        c.k_scale[p] = 2.0 ** -6
        c.k_codes.view(torch.uint8)[p, :, :, : p] = 0x40       # 2.0 in the first p dims
    g = torch.Generator().manual_seed(3)
    q = (torch.rand(nq, 2, 64, generator=g) * step * 8).to(torch.bfloat16).cuda()
    o, lse = c.attention(q, i32([0, nq]), i32([1024]), i32([list(range(64))]), causal=False,
                         max_q=nq, return_lse=True)
    want = ref.attention(q.cpu().double(), *_planes64(c), [list(range(64))], [nq], [1024], 16,
                         False, 0.125)
    ref.assert_attention_close(o, lse, want)


@pytest.mark.parametrize("heads,dim,page", [(3, 128, 880), (1, 64, 304), (2, 128, 112), (9, 64, 16)])
def test_append_runs_of_all_lengths(heads, dim, page):
    """Single tokens between runs that a warp, a CTA and several CTAs hold, skipped tokens
    among them, more tokens than a tile."""
    r = random.Random(heads * page)
    counts = [r.choice((1, 1, 1, 2, 17, 33, 64, 65, 129, 300, 1000)) for _ in range(40)]
    cached = [r.randint(0, 2 * page) for _ in counts]
    table, free, n_pages = _tables(cached, counts, page, 2, 3)
    _, _, slots, _, _ = ref.plan(cached, counts, table, free, 0, page)
    at = 0
    for n in counts:   # a padded batch: some requests' last tokens are not stored
        if n > 1 and r.random() < 0.3:
            slots[at + n - 1] = -1
        at += n
    c = _random_cache(n_pages, page, heads, dim, 4)
    before = _planes64(c)
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(sum(counts), heads, dim, generator=g).mul_(torch.exp2(
        torch.randint(-6, 7, (sum(counts), 1, 1), generator=g).float())) for _ in range(2))
    k, v = k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda()
    c.append(k, v, i32(slots))
    _check_append(c, k, v, slots, before)


def test_two_streams_at_once():
    """Two requests' steps at the same time, on a stream each, with clusters, ranges and the
    workspace of each stream: the same bits as one after the other."""
    torch.manual_seed(0)
    caches = [_random_cache(80, 16, 4, 128, s) for s in (1, 2)]
    w = nv.quantize((torch.randn(512, 1024) * 0.1).to(torch.bfloat16).cuda())
    table = torch.arange(80).int().cuda().view(1, 80)
    lens, cu = i32([1270]), i32([0, 1])
    qs = [torch.randn(1, 8, 128).to(torch.bfloat16).cuda() for _ in range(2)]

    def step(i):
        c = caches[i]
        c.append(qs[i][:, :4], qs[i][:, 4:], i32([79 * 16 + 5]))
        o = c.attention(qs[i], cu, lens, table, max_q=1)
        return o, nv.gemv(o.view(1, 1024), w)
    want = [step(i) for i in range(2)]
    want = [step(i) for i in range(2)]   # (the last page's scale has grown by now)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(i))
    torch.cuda.synchronize()
    for i in range(2):
        for o, y in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(y, want[i][1])
    for s in streams:
        with torch.cuda.stream(s):
            assert nv.device_status() == 0


@pytest.mark.parametrize("n", [2, 40])
def test_output_over_the_queries_is_refused(n):
    c = _random_cache(8, 16, 2, 64, 3)
    q = torch.randn(n, 4, 64, generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    before = q.clone()
    with pytest.raises(nv.NVFP4Error):
        c.attention(q, i32([0, n]), i32([100]), torch.arange(8).int().cuda().view(1, 8), out=q)
    assert torch.equal(q, before)


def test_two_threads():
    """Python threads with a stream each call at the same time: the same bits as alone."""
    import threading
    caches = [_random_cache(64, 16, 2, 64, s) for s in (5, 6)]
    table = torch.arange(64).int().cuda().view(2, 32)
    lens, cu, free, head = i32([400, 37]), i32([0, 1, 2]), i32([63]), i32([0])
    qs = [torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(s)).to(torch.bfloat16)
          .cuda() for s in range(2)]
    want = [c.attention(q, cu, lens, table, return_lse=True) for c, q in zip(caches, qs)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(200):
                p = nv.plan_pages(lens, i32([0, 0]), table, free, head, 16, 64, 0)
                o, l = caches[i].attention(qs[i], cu, p.seq_lens, table, return_lse=True)
                if not (torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])):
                    wrong.append(i)
            if nv.device_status() != 0:
                wrong.append("status")
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# ---------------------------------------------------------------- the ends of the ranges
@pytest.mark.parametrize("max_kv", [1, None])   # one range, or several that are joined
@pytest.mark.parametrize("nq", [1, 33, 200])
@pytest.mark.parametrize("before,e,rise", [(1536, 60, 7), (10240, 55, 17), (1536, 60, 100),
                                           (256, 60, -7), (128, 0, 130)])
def test_v_scales_at_both_ends_of_the_range(before, e, rise, nq, max_kv):
    """V scales 2^-e, then 2^e for one last token whose score is larger (base 2): the normaliser of
    the tokens before has to survive, however far the weights' reference rises."""
    n = before // 16
    c = _random_cache(n + 1, 16, 1, 64, 25, spread=0)
    codes = c.k_codes.view(torch.uint8)
    codes[:] = 0
    codes[n, 0, 0, 0] = 0x38 if rise > 0 else 0xB8             # +-1.0
    c.k_scale[:] = 1.0
    c.v_scale[:n], c.v_scale[n] = 2.0 ** -e, 2.0 ** e
    q = torch.zeros(nq, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    scale = abs(rise) * math.log(2)
    table = list(range(n + 1))
    o, lse = c.attention(q, i32([0, nq]), i32([before + 1]), i32([table]), causal=False, max_q=nq,
                         max_kv=max_kv, scale=scale, return_lse=True)
    want = ref.attention(q.cpu().double(), *_planes64(c), [table], [nq], [before + 1], 16, False,
                         scale)
    ref.assert_attention_close(o, lse, want)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq", [1, 12, 40])
@pytest.mark.parametrize("dim", [64, 128])
def test_pages_never_written(dim, nq, causal):
    """A new cache (scales of 0), as a warm-up before the first tokens meets it: zeros, and the
    log-sum-exp of equal scores."""
    c = nv.KVCache8.empty(8, 16, 2, dim)
    q = torch.randn(2 * nq, 6, dim, generator=torch.Generator().manual_seed(1))
    q = q.to(torch.bfloat16).cuda()
    table, kv = [[0, 1, 2, 3], [4, 5, 6, 7]], [50, 17]
    o, lse = c.attention(q, i32([0, nq, 2 * nq]), i32(kv), i32(table), causal=causal, max_q=nq,
                         return_lse=True)
    want = ref.attention(q.cpu().double(), *_planes64(c), table, [nq, nq], kv, 16, causal,
                         dim ** -0.5)
    ref.assert_attention_close(o, lse, want)
    assert not o.any()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq", [1, 8, 9, 40, 300])
@pytest.mark.parametrize("mult", [0.0, 2.0 ** -130, 1.0])
def test_zero_keys_and_zero_or_tiny_queries(nq, mult, causal):
    """K of zeros gets the smallest scale there is; with q near 0 too, score factors underflow:
    every token weighs the same."""
    c = nv.KVCache8.empty(8, 16, 1, 64)
    g = torch.Generator().manual_seed(2)
    v = torch.randn(67, 1, 64, generator=g).to(torch.bfloat16).cuda()
    c.append(torch.zeros_like(v), v, i32(list(range(50)) + list(range(80, 97))))
    q = (torch.randn(2 * nq, 4, 64, generator=g) * mult).to(torch.bfloat16).cuda()
    table, kv = [[0, 1, 2, 3], [5, 6, 7]], [50, 17]
    o, lse = c.attention(q, i32([0, nq, 2 * nq]), i32(kv), i32([table[0], table[1] + [0]]),
                         causal=causal, max_q=nq, return_lse=True)
    want = ref.attention(q.cpu().double(), *_planes64(c), table, [nq, nq], kv, 16, causal, 0.125)
    ref.assert_attention_close(o, lse, want)


@pytest.mark.parametrize("kv", [40, 3000])
@pytest.mark.parametrize("nq", [1, 40])
def test_v_scales_of_zero_under_low_scores(nq, kv):
    """V pages never written beside K pages that were, all scores far below 0: zeros, no NaN."""
    n = -(-kv // 16)
    c = _random_cache(n, 16, 1, 64, 26, spread=0)
    c.v_scale.zero_()
    c.v_codes.view(torch.uint8)[:] = 0
    c.k_codes.view(torch.uint8)[:] = 0x38
    c.k_scale[:] = 1.0
    q = torch.full((nq, 4, 64), -40.0, dtype=torch.bfloat16, device="cuda")
    table = list(range(n))
    o, lse = c.attention(q, i32([0, nq]), i32([kv]), i32([table]), causal=False, max_q=nq,
                         return_lse=True)
    want = ref.attention(q.cpu().double(), *_planes64(c), [table], [nq], [kv], 16, False, 0.125)
    ref.assert_attention_close(o, lse, want)


@pytest.mark.parametrize("fits", [True, False])
def test_plan_with_the_largest_slot_map(fits):
    """2^31 - 1 slots: the loops over them step past 2^31."""
    p = nv.plan_pages(i32([20, 0]), i32([3, 20 if fits else -1]), i32([[0, 1], [-1, -1]]),
                      i32([5, 4]), i32([0]), page_tokens=16, n_pages=6, max_new=2 ** 31 - 1)
    want = [20, 21, 22, *range(80, 96), *range(64, 68)] if fits else [-1] * 23
    assert p.slot_map[:23].tolist() == want and p.slot_map.numel() == 2 ** 31 - 1
    assert p.cu_new.tolist() == ([0, 3, 23] if fits else [0, 0, 0])
    assert p.seq_lens.tolist() == ([23, 20] if fits else [20, 0])
    assert p.free_head.tolist() == [2 if fits else 0]
    for at in range(23, 2 ** 31 - 1, 1 << 28):
        assert bool((p.slot_map[at:at + (1 << 28)] == -1).all())
    assert nv.device_status() == (N.OK if fits else N.ERR_INVALID_ARG)


@pytest.mark.parametrize("nq", [1, 5, 40])
def test_output_beside_the_queries(nq):
    """Queries and output as parts of one fused buffer: apart, though their spans meet."""
    c = _random_cache(10, 16, 2, 64, 28)
    wide = torch.randn(nq, 12, 64, generator=torch.Generator().manual_seed(2))
    wide = wide.to(torch.bfloat16).cuda()
    before = wide.clone()
    args = (i32([0, nq]), i32([150]), i32([list(range(10))]))
    want = c.attention(before[:, 2:6].contiguous(), *args, max_q=nq)
    for at in (6, 8):
        got = c.attention(wide[:, 2:6], *args, max_q=nq, out=wide[:, at:at + 4])
        assert torch.equal(got, want)
        keep = [h for h in range(12) if not at <= h < at + 4]
        assert torch.equal(wide[:, keep], before[:, keep])
        wide.copy_(before)
    for at in (1, 3, 5):
        with pytest.raises(nv.NVFP4Error):
            c.attention(wide[:, 2:6], *args, max_q=nq, out=wide[:, at:at + 4])
    assert torch.equal(wide, before)


# ---------------------------------------------------------------- captured calls
def _new_stream():
    """A stream that no call has used: captures on it begin without a workspace."""
    for _ in range(32):
        s = torch.cuda.Stream(priority=-1)
        if all(s.cuda_stream != key[1] for key in nv.ops._workspaces):
            return s
    pytest.skip("every stream of the pool has been used")


def test_captured_calls_report_what_goes_wrong():
    """The first calls on a stream are captured, in two graphs: device_status tells what went
    wrong in a replay of either, whatever the other one did."""
    s = _new_stream()
    cached, new, head, table = i32([20]), i32([20]), i32([0]), i32([[0, 1, -1]])
    frees = [i32([]), i32([2])]
    graphs, plans = [], []
    torch.cuda.synchronize()
    for free in frees:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            plans.append(nv.plan_pages(cached, new, table, free, head, page_tokens=16, n_pages=8,
                                       max_new=40))
        graphs.append(g)
    assert nv.device_status() == N.OK
    for _ in range(2):
        graphs[0].replay()
        graphs[1].replay()
        assert nv.device_status() == N.ERR_CAPACITY
        assert nv.device_status() == N.OK
        assert plans[0].seq_lens.tolist() == [20] and plans[1].seq_lens.tolist() == [40]
        graphs[1].replay()
        assert nv.device_status() == N.OK
    new.fill_(-1)
    graphs[1].replay()
    graphs[0].replay()
    assert nv.device_status() == N.ERR_INVALID_ARG
    # the stream's own calls have a workspace apart from its graphs'
    graphs[0].replay()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        nv.plan_pages(i32([1]), i32([1]), table, frees[1], head, 16, 8, 4)
        assert nv.device_status() == N.ERR_INVALID_ARG
        assert nv.device_status() == N.OK


def test_captured_workspaces_belong_to_no_graph():
    """Two graphs of calls that need zeroed words, the first calls of their stream: the second is
    replayed first, and after the other is gone."""
    s = _new_stream()
    x = [torch.randn(300, 512, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda()
         for i in range(2)]
    want = [nv.quantize(t) for t in x]
    got = [nv.ops.empty(300, 512) for _ in x]
    graphs = []
    torch.cuda.synchronize()
    for t, out in zip(x, got):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            nv.quantize(t, out=out)
        graphs.append(g)
    ws = nv.ops._captured_workspaces[(0, s.cuda_stream)]
    assert not ws.any()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= ws.data_ptr() < seg["address"] + seg["total_size"]:
            assert tuple(seg["segment_pool_id"]) == (0, 0)

    def check(i):
        got[i].codes.zero_(), got[i].sf.zero_(), got[i].s_t.zero_()
        graphs[i].replay()
        assert torch.equal(got[i].codes, want[i].codes) and torch.equal(got[i].sf, want[i].sf)
        assert torch.equal(got[i].s_t, want[i].s_t)
    for i in (1, 0, 1):
        check(i)
    graphs[0].reset()
    graphs[0] = None
    torch.cuda.empty_cache()
    check(1)


def test_no_requests_at_all():
    """An idle step: a plan of no requests, and the attention over it."""
    c = _random_cache(4, 16, 1, 64, 27)
    none = i32([])
    p = nv.plan_pages(none, none, none.view(0, 4), i32([1]), i32([0]), page_tokens=16, n_pages=4,
                      max_new=3)
    for tokens in (0, 3):   # (rows of no request are left)
        q = torch.ones(tokens, 2, 64, dtype=torch.bfloat16, device="cuda")
        out = torch.full_like(q, 5.0)
        o, lse = c.attention(q, p.cu_new, p.seq_lens, none.view(0, 4), out=out, return_lse=True)
        assert o is out and bool((out == 5).all()) and lse.shape == (tokens, 2)
        assert c.attention(q, p.cu_new, p.seq_lens, none.view(0, 0)).shape == q.shape


@pytest.mark.parametrize("dim", [64, 128])
def test_waits_that_run_out_report_and_recover(dim):
    """The many-row kernel with a limit of 0 ns: a wait that finds its phase not over yet (the first
    for the codes from memory, say) runs out.  The kernel records it, ends what it has in flight,
    frees tensor memory and returns, soon; the next call with the normal limit is right."""
    c = _random_cache(200, 16, 2, dim, 29)
    q = torch.randn(700, 4, dim, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    q = q.cuda()
    args = (q, i32([0, 400, 700]), i32([1500, 1700]),
            i32([list(range(94)) + [0] * 13, list(range(93, 200))]))
    good = c.attention(*args, max_q=400)
    seen = []
    for _ in range(4):
        try:
            nv.set_wait_limit_ns(0)
            torch.cuda.synchronize()
            began = time.monotonic()
            c.attention(*args, max_q=400)
            seen.append(nv.device_status())
            assert time.monotonic() - began < 1.0   # (a drain that waits for nothing takes 2 s)
        finally:
            nv.set_wait_limit_ns(2_000_000_000)
        assert torch.equal(c.attention(*args, max_q=400), good)
        assert nv.device_status() == N.OK
    assert all(st in (N.OK, N.ERR_TIMEOUT) for st in seen) and N.ERR_TIMEOUT in seen, seen


# ---------------------------------------------------------------- both planes, step by step
@pytest.mark.parametrize("heads,dim", [(24, 64), (8, 128)])
def test_append_many_single_tokens_both_planes(heads, dim):
    """K and V of their own (not one the other's negative) in pages that hold tokens already."""
    page, batch = 16, 3000
    c = _random_cache(batch, page, heads, dim, 30)
    slots = [p * page + (7 * p) % page for p in range(batch)]
    before = _planes64(c)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(batch, heads, dim, generator=g).mul_(torch.exp2(
        torch.randint(-6, 7, (batch, 1, 1), generator=g).float())) for _ in range(2))
    k, v = k.to(torch.bfloat16).cuda(), v.to(torch.bfloat16).cuda()
    c.append(k, v, i32(slots))
    keep = list(range(0, batch, 97))   # a page is one run here, and goes by itself
    sub = [t[keep] for t in before]
    for x, value, scale in ((k, sub[0], sub[2]), (v, sub[1], sub[3])):
        ref.append(x.cpu().double()[keep], value, scale, [i * page + slots[p] % page
                                                          for i, p in enumerate(keep)], page)
    for got, want in zip(_planes64(c), sub):
        assert torch.equal(got[keep], want)


@pytest.mark.parametrize("page,dim,hkv,hq", [(16, 128, 2, 8), (32, 64, 1, 4), (48, 64, 3, 3)])
def test_serving_steps_fill_the_cache(page, dim, hkv, hq):
    """Plans and appends step after step, with an attention between that must change nothing: the
    tables, lengths, codes and scales of K and V are the plain forms' after every step."""
    cache = nv.KVCache8.empty(40, page, hkv, dim)
    steps = [[30, 1, 0, 77], [1, 1, 50, 1], [1, 0, 1, 1], [1, 3, 1, 20], [0, 0, 0, 0], [1, 1, 1, 1]]
    g = torch.Generator().manual_seed(6)
    order = torch.randperm(40, generator=g).tolist()
    free, head, cached = i32(order), i32([0]), i32([0] * 4)
    table = torch.full((4, 12), -1, dtype=torch.int32, device="cuda")
    rows, taken, lens = table.tolist(), 0, [0] * 4
    for new in steps:
        tokens = sum(new)
        qkv = torch.randn(tokens + 5, hq + 2 * hkv, dim, generator=g)
        qkv *= torch.exp2(torch.randint(-6, 7, (tokens + 5, 1, 1), generator=g).float())
        qkv = qkv.to(torch.bfloat16).cuda()
        before = _planes64(cache)
        p = nv.plan_pages(cached, i32(new), table, free, head, page_tokens=page, n_pages=40,
                          max_new=tokens + 5)
        lens, cu, slots, rows, taken = ref.plan(lens, new, rows, order, taken, page)
        k, v = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        cache.append(k, v, p.slot_map)
        cache.attention(qkv[:, :hq], p.cu_new, p.seq_lens, table, max_q=max(max(new), 1))
        assert p.seq_lens.tolist() == lens and p.cu_new.tolist() == cu
        assert p.slot_map.tolist() == slots + [-1] * 5
        assert table.tolist() == rows and p.free_head.tolist() == [taken]
        _check_append(cache, k, v, slots + [-1] * 5, before)
        cached, head = p.seq_lens, p.free_head


@pytest.mark.parametrize("steps,batch,dim,hkv,hq,page,prompt", [
    (60, 1, 128, 2, 8, 16, 37), (60, 3, 64, 2, 6, 16, 100), (40, 16, 128, 4, 16, 32, 300),
    (20, 2, 128, 8, 32, 64, 6000)])
def test_a_chain_of_steps_in_one_graph(steps, batch, dim, hkv, hq, page, prompt):
    """Each step's tokens come from the last step's output through a layer, its lengths and pages
    from the last step's plan, and every call starts while the one before ends: the same bits as
    with a wait after every call."""
    width = -(-(prompt + steps) // page)
    n_pages = batch * (width + 1)

    def run(between, captured):
        g = torch.Generator().manual_seed(5)
        cache = nv.KVCache8.empty(n_pages, page, hkv, dim)
        w = nv.quantize((torch.randn((hq + 2 * hkv) * dim, hq * dim, generator=g) * 0.05)
                        .to(torch.bfloat16).cuda())
        table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        free, one = torch.randperm(n_pages, generator=g).int().cuda(), i32([1] * batch)
        x = torch.randn(batch, hq * dim, generator=g).to(torch.bfloat16).cuda()
        qkv = torch.randn(batch * prompt, hq + 2 * hkv, dim, generator=g).to(torch.bfloat16).cuda()
        p = nv.plan_pages(i32([0] * batch), i32([prompt] * batch), table, free, i32([0]), page,
                          n_pages, batch * prompt)
        cache.append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], p.slot_map)
        outs = [cache.attention(qkv[:, :hq], p.cu_new, p.seq_lens, table, max_q=prompt)]
        graph = torch.cuda.CUDAGraph() if captured else None
        torch.cuda.synchronize()
        with torch.cuda.graph(graph) if captured else contextlib.nullcontext():
            for _ in range(steps):
                qkv = nv.gemv(x, w).view(batch, hq + 2 * hkv, dim)
                between()
                p = nv.plan_pages(p.seq_lens, one, table, free, p.free_head, page, n_pages, batch)
                between()
                cache.append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], p.slot_map)
                between()
                outs.append(cache.attention(qkv[:, :hq], p.cu_new, p.seq_lens, table, max_q=1))
                between()
                x = outs[-1].view(batch, hq * dim)
        if captured:
            graph.replay()
        torch.cuda.synchronize()
        return [*outs, table, cache.k_codes.view(torch.uint8), cache.v_codes.view(torch.uint8),
                cache.k_scale, cache.v_scale], graph
    want, _ = run(torch.cuda.synchronize, False)
    for captured in (False, True):
        got, graph = run(lambda: None, captured)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("batch,most", [(5000, 1), (700, 40)])
def test_many_requests(batch, most):
    """More requests than SMs by far, some without queries, some without tokens."""
    r = random.Random(batch)
    kv = [r.choice((0, 1, 16, 17, r.randint(1, 60))) for _ in range(batch)]
    nq = [r.choice((0, 1, most)) for _ in range(batch)]
    c = _random_cache(sum(-(-t // 16) for t in kv) + 2, 16, 1, 64, 31)
    _attention_case(c, nq, kv, 2, True, 32, max_q=most)
