"""GPU parity: nvfp4_gemv against the 64-bit product with the decoded weights.

Bounds.  S = sum_k |x w|, X = sum_k (largest |x| of the 256 columns around k) |w|:
  representation of x  bf16: 2^-33 X; fp32: 2^-22 S + 2^-43 X
  sums                 16 tensor-core products of 16 columns each (truncating, 2^-23 of the running
                       sum at most) and fp32 additions: (16 2^-23 + 32 2^-24) S = 2^-18.4 S
so |y - ref| <= 2^-18 S + 2^-32 X + 2^-24 |ref|; bf16 output adds half a step, 2^-8 of the value.
GELU (slope at most 1.13): 1.13 times the error of its input (for bf16 output with the input's
own rounding to bf16), 2^-18 |y| for the fp32 evaluation, then the output's rounding."""
import pytest
import torch

import nvfp4_w4a4_quantized_08_b200 as nv

from _util import GELU_SLOPE_MAX, sf_rowmajor

pytestmark = pytest.mark.gpu

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6],
                    dtype=torch.float64)


def _weights(orc, n, k, layout, seed):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(n, k, generator=g) * 0.02).to(torch.bfloat16)
    q = nv.quantize(w.cuda(), sf_layout=layout)
    code = q.codes.cpu().int()
    v = E2M1[torch.stack((code & 15, code >> 4), 2).reshape(n, k).long()]
    sf = torch.from_numpy(sf_rowmajor(orc, q).copy()).view(torch.float8_e4m3fn).double()
    return q, v * sf.repeat_interleave(16, 1) * q.s_t.cpu().double()


def _check(y, x, w, bf16, gelu=False):
    x = x.double().cpu()
    ref = x @ w.t()
    m, k = x.shape
    pad = torch.zeros(m, -(-k // 256) * 256, dtype=torch.float64)
    pad[:, :k] = x.abs()
    near = pad.view(m, -1, 256).amax(2).repeat_interleave(256, 1)[:, :k]
    S, X = x.abs() @ w.abs().t(), near @ w.abs().t()
    tol = 2.0 ** -18 * S + 2.0 ** -32 * X + 2.0 ** -24 * ref.abs()
    if gelu:
        if bf16:
            tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        tol = GELU_SLOPE_MAX * tol + 2.0 ** -18 * ref.abs()
        u = (2 / torch.pi) ** 0.5 * (ref + 0.044715 * ref ** 3)
        ref = 0.5 * ref * (1 + torch.tanh(u))
    if bf16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (y.double().cpu() - ref).abs()
    assert bool((err <= tol).all()), (float((err / tol.clamp_min(1e-300)).max()),
                                      (err > tol).nonzero()[:4].tolist())


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,k", [(130, 1056), (1, 32), (257, 128)])
def test_rows(orc, m, xd, n, k):
    q, w = _weights(orc, n, k, nv.SF_MMA128x4, n + k)
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(m)).to(xd).cuda()
    _check(nv.gemv(x, q), x, w, True)
    _check(nv.gemv(x, q, torch.float32), x, w, False)


@pytest.mark.parametrize("layout", [nv.SF_ROWMAJOR, nv.SF_MMA128x4])
@pytest.mark.parametrize("n,k", [(1000, 14336), (4100, 2080), (64, 8192)])
def test_layouts_and_splits(orc, layout, n, k):
    """Row-major and tensor-core scales; columns split over a cluster and not."""
    q, w = _weights(orc, n, k, layout, 5)
    x = torch.randn(3, k, generator=torch.Generator().manual_seed(1)).cuda()
    _check(nv.gemv(x, q, torch.float32), x, w, False)


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("m", [1, 6])
def test_gelu(orc, bf16, m):
    q, w = _weights(orc, 300, 512, nv.SF_MMA128x4, 9)
    x = (torch.randn(m, 512, generator=torch.Generator().manual_seed(2)) * 4).to(torch.bfloat16)
    y = nv.gemv(x.cuda(), q, torch.bfloat16 if bf16 else torch.float32, act=nv.ACT_GELU_TANH)
    _check(y, x, w, bf16, gelu=True)


@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
def test_wide_range_of_x(orc, xd):
    """Outlier columns, zero rows, tiny and huge rows, subnormal bf16 values."""
    q, w = _weights(orc, 200, 640, nv.SF_MMA128x4, 3)
    x = torch.randn(6, 640, generator=torch.Generator().manual_seed(4))
    x[0, 7] = 3e4
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e30
    x[4, :128] *= 1e-20
    x[5] *= 2.0 ** -130
    x = x.to(xd).cuda()
    y = nv.gemv(x, q, torch.float32)
    keep = torch.tensor([0, 1, 2, 3, 4])
    _check(y[keep.cuda()], x[keep.cuda()], w, False)
    # row 5: sums of 640 products below 2^-126, where fp32 itself has steps of 2^-149
    ref = x[5:].double().cpu() @ w.t()
    assert bool(((y[5:].double().cpu() - ref).abs() <= 640 * 2.0 ** -149 + 2.0 ** -18 *
                 (x[5:].double().cpu().abs() @ w.abs().t())).all())
    assert not y[1].any()


def test_strides_and_out(orc):
    q, w = _weights(orc, 150, 256, nv.SF_MMA128x4, 8)
    wide = torch.randn(5, 400, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    x = wide[:, 64:64 + 256]
    out = torch.full((5, 160), 7.0, dtype=torch.bfloat16, device="cuda")
    assert nv.gemv(x, q, out=out) is out
    _check(out[:, :150], x, w, True)
    assert bool((out[:, 150:] == 7).all())
    one = nv.gemv(wide[2:3, 64:64 + 256], q)
    _check(one, x[2:3], w, True)


def test_matches_itself_graphs_and_streams(orc):
    """Bitwise the same eagerly, on another stream and in a replayed graph with new inputs."""
    q, _ = _weights(orc, 1000, 4096, nv.SF_MMA128x4, 2)
    x = torch.randn(2, 4096, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    x2 = x.flip(1).contiguous()
    want, want2 = nv.gemv(x, q).clone(), nv.gemv(x2, q).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = nv.gemv(x, q)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, want)
    buf = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nv.gemv(buf, q)
    buf.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want2)


def test_near_gemm_and_oracle(orc):
    """The same layer through the quantized GEMM and the unquantized product: the GEMM's own
    oracle of the quantized x bounds how far the two may be apart."""
    q, w = _weights(orc, 256, 512, nv.SF_MMA128x4, 12)
    x = torch.randn(4, 512, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
    qx = nv.quantize(x)
    xq = nv.dequantize(qx)
    # |x - dequantized x| enters the product linearly
    far = (x.double() - xq.double()).abs().cpu() @ w.abs().t()
    y, yq = nv.gemv(x, q, torch.float32), nv.gemm(qx, q, torch.float32)
    S = xq.double().abs().cpu() @ w.abs().t()
    assert bool(((y - yq).double().abs().cpu() <= far + (2e-3 + 2.0 ** -8) * S).all())


@pytest.mark.parametrize("m,xd", [(1, torch.bfloat16), (3, torch.float32), (8, torch.bfloat16),
                                  (16, torch.float32)])
@pytest.mark.parametrize("n,k", [(40, 16384), (1000, 8000), (2100, 4128), (5000, 2080)])
def test_column_splits(m, xd, n, k):
    """Shapes over which the number of CTAs that split the columns runs from 8 to 1, ragged in
    rows and columns: against 64 bits, within the bound of x's representation (2^-22 of each
    256 columns' largest value) and fp32 sums of at most k products in any order."""
    g = torch.Generator().manual_seed(m * n + k)
    w = nv.quantize((torch.randn(n, k, generator=g) * 0.1).to(torch.bfloat16).cuda())
    x = torch.randn(m, k, generator=g).to(xd).cuda()
    got = nv.gemv(x, w, out_dtype=torch.float32)
    wd = nv.dequantize(w).double()                     # rounded to bf16
    err = (got.double() - x.double() @ wd.t()).abs()
    scale = x.double().abs() @ wd.abs().t()
    assert bool((err <= scale * 2.0 ** -8).all())      # half a bf16 step of each weight
    # the splits' sums are one another's up to fp32: rows alone give the same products
    one = torch.cat([nv.gemv(x[i:i + 1], w, out_dtype=torch.float32) for i in range(m)])
    top = x.abs().amax(dim=1, keepdim=True).double()
    tol = scale * 2.0 ** -19 + top * wd.abs().sum(dim=1) * 2.0 ** -21
    assert bool(((got.double() - one.double()).abs() <= tol).all())
    assert torch.equal(got, nv.gemv(x, w, out_dtype=torch.float32))


@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m", [1, 2, 3, 7, 16])
def test_infinities_and_nan(orc, m, xd):
    """An infinite x gives infinities (NaN against a weight of zero, or another infinity's
    opposite), a NaN gives NaN, in its row alone."""
    n, k = 70, 544
    q, w = _weights(orc, n, k, nv.SF_MMA128x4, 13)
    inf = float("inf")
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(m))
    x[0, 5] = inf
    if m > 2:
        x[2, 300], x[2, 301] = -inf, inf
    if m > 3:
        x[3, 40], x[4, 543], x[5, 7] = float("nan"), -inf, inf
        x[5, :256].fill_(inf)
    x = x.to(xd).cuda()
    for dt in (torch.float32, torch.bfloat16):
        got = nv.gemv(x, q, dt).double().cpu()
        want = (x.double().cpu()[:, None] * w[None]).sum(2)
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(got == inf, want == inf) and torch.equal(got == -inf, want == -inf)
        good = x.isfinite().all(1)
        if bool(good.any()):
            _check(got[good.cpu()], x[good], w, dt == torch.bfloat16)


@pytest.mark.parametrize("bf16", [True, False])
def test_gelu_of_negative_values(bf16):
    """The GELU from -8 to 0, where it falls to 1e-14: right relative to itself.  y is exact here
    (one product of short significands); u = sqrt(2 / pi) (y + 0.044715 y^3) takes seven roundings,
    constants included, which reach the result through exp(-2u) as 14 |u| 2^-24; the exponential,
    the sum and the quotient add at most 8 2^-24."""
    code = torch.zeros(7, 16, dtype=torch.uint8)
    code[:, 0] = torch.arange(1, 8)                       # 0.5 .. 6 in the first column
    q = nv.NVFP4Tensor(code.cuda(), torch.full((14,), 0x38, dtype=torch.uint8, device="cuda"),
                       torch.ones(1, device="cuda"), 7, 32, nv.SF_ROWMAJOR)
    x = torch.zeros(16, 32)
    x[:, 0] = -torch.arange(1, 17) / 12.0
    x = x.to(torch.bfloat16).float()
    y = (x[:, :1] * E2M1[1:8].float()).double()
    if bf16:
        y = y.to(torch.bfloat16).double()
    u = (2 / torch.pi) ** 0.5 * (y + 0.044715 * y ** 3)
    want = y / (1 + torch.exp(-2 * u))
    tol = 2.0 ** -24 * (8 + 14 * u.abs()) * want.abs()
    if bf16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    got = nv.gemv(x.cuda(), q, torch.bfloat16 if bf16 else torch.float32, act=nv.ACT_GELU_TANH)
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("m", [1, 4])
def test_output_beside_x(orc, m):
    """x and y as parts of one buffer; over each other they are refused."""
    q, w = _weights(orc, 256, 256, nv.SF_MMA128x4, 14)
    wide = torch.randn(m, 768, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    before = wide.clone()
    for at in (0, 512):
        y = nv.gemv(wide[:, 256:512], q, out=wide[:, at:at + 256])
        _check(y, before[:, 256:512], w, True)
        assert torch.equal(wide[:, 256:512], before[:, 256:512])
    wide.copy_(before)
    for at in (8, 256, 504):
        with pytest.raises(nv.NVFP4Error):
            nv.gemv(wide[:, 256:512], q, out=wide[:, at:at + 256])
    assert torch.equal(wide, before)


@pytest.mark.parametrize("m,xd", [(1, torch.bfloat16), (5, torch.float32)])
def test_offsets_past_32_bits(m, xd):
    """Weights of more than 2^32 bytes of codes: the last rows."""
    n, k = 620000, 14336
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device="cuda")
    sf = torch.randint(0x30, 0x41, (nv.sf_bytes(n, k, nv.SF_ROWMAJOR),), dtype=torch.uint8,
                       device="cuda")
    q = nv.NVFP4Tensor(codes, sf, torch.full((1,), 2.0 ** -9, device="cuda"), n, k, nv.SF_ROWMAJOR)
    assert codes.numel() > 2 ** 32
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(m)).to(xd).cuda()
    y = nv.gemv(x, q, torch.float32)
    for r in (slice(0, 40), slice(n - 200, n)):
        c = codes[r].cpu().int()
        v = E2M1[torch.stack((c & 15, c >> 4), 2).reshape(-1, k).long()]
        s = sf.view(n, k // 16)[r].cpu().view(torch.float8_e4m3fn).double()
        _check(y[:, r], x, v * s.repeat_interleave(16, 1) * 2.0 ** -9, False)
