"""Host-side refusals of the matrix-vector, page-plan and 8-bit cache entry points: every call
has an invalid argument, so it returns before any device work."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import nvfp4_w4a4_quantized_08_b200 as nv
from nvfp4_w4a4_quantized_08_b200 import _native as N
from nvfp4_w4a4_quantized_08_b200 import build as nbuild

FAKE = 0x7F0000001000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    nbuild.build()
    return N.lib()


def _weights(rows=1000, cols=4096, layout=N.SF_MMA128x4):
    return N.Tensor(FAKE, FAKE, FAKE, rows, cols, layout)


def _gemv(L, **kw):
    a = dict(x=FAKE, xd=N.BF16, m=1, ldx=4096, w=_weights(), y=FAKE, yd=N.BF16, ldy=1000,
             act=N.ACT_NONE)
    a.update(kw)
    return L.nvfp4_gemv(a["x"], a["xd"], a["m"], a["ldx"], ctypes.byref(a["w"]), a["y"], a["yd"],
                        a["ldy"], a["act"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), N.ERR_INVALID_ARG), (dict(y=None), N.ERR_INVALID_ARG),
    (dict(xd=2), N.ERR_INVALID_ARG), (dict(yd=-1), N.ERR_INVALID_ARG),
    (dict(act=2), N.ERR_INVALID_ARG), (dict(m=0), N.ERR_INVALID_ARG),
    (dict(m=-1), N.ERR_INVALID_ARG), (dict(ldx=4095), N.ERR_INVALID_ARG),
    (dict(ldy=999), N.ERR_INVALID_ARG), (dict(m=17), N.ERR_UNSUPPORTED_SHAPE),
    (dict(w=_weights(cols=4080)), N.ERR_UNSUPPORTED_SHAPE),
    (dict(w=_weights(layout=7)), N.ERR_INVALID_ARG),
    (dict(w=_weights(rows=0)), N.ERR_INVALID_ARG),
    (dict(x=FAKE + 8), N.ERR_MISALIGNED), (dict(ldx=4100), N.ERR_MISALIGNED),
    (dict(xd=N.FP32, ldx=4098), N.ERR_MISALIGNED), (dict(y=FAKE + 1), N.ERR_MISALIGNED),
    (dict(y=FAKE + 2, yd=N.FP32), N.ERR_MISALIGNED)])
def test_gemv_rejects(L, bad, status):
    assert _gemv(L, **bad) == status


PLAN = dict(cached=FAKE, new=FAKE + 0x1000, batch=4, table=FAKE + 0x2000, stride=8, pages=8,
            free=FAKE + 0x3000, n_free=10, head=FAKE + 0x4000, page=16, n_pages=100,
            seq=FAKE + 0x5000, cu=FAKE + 0x6000, slots=FAKE + 0x7000, max_new=20,
            head_out=FAKE + 0x8000, ws=FAKE + 0x9000, ws_bytes=256)


def _plan(L, **kw):
    a = dict(PLAN, **kw)
    return L.nvfp4_plan_pages(a["cached"], a["new"], a["batch"], a["table"], a["stride"],
                              a["pages"], a["free"], a["n_free"], a["head"], a["page"],
                              a["n_pages"], a["seq"], a["cu"], a["slots"], a["max_new"],
                              a["head_out"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(batch=-1), N.ERR_INVALID_ARG), (dict(pages=9), N.ERR_INVALID_ARG),
    (dict(cached=None), N.ERR_INVALID_ARG), (dict(new=None), N.ERR_INVALID_ARG),
    (dict(table=None), N.ERR_INVALID_ARG), (dict(free=None), N.ERR_INVALID_ARG),
    (dict(head=None), N.ERR_INVALID_ARG), (dict(seq=None), N.ERR_INVALID_ARG),
    (dict(cu=None), N.ERR_INVALID_ARG), (dict(slots=None), N.ERR_INVALID_ARG),
    (dict(head_out=None), N.ERR_INVALID_ARG), (dict(max_new=-1), N.ERR_INVALID_ARG),
    (dict(n_free=-1), N.ERR_INVALID_ARG), (dict(n_pages=0), N.ERR_INVALID_ARG),
    (dict(page=0), N.ERR_INVALID_ARG), (dict(page=24), N.ERR_UNSUPPORTED_SHAPE),
    (dict(page=8192), N.ERR_UNSUPPORTED_SHAPE), (dict(n_pages=1 << 27), N.ERR_UNSUPPORTED_SHAPE),
    (dict(batch=8193), N.ERR_UNSUPPORTED_SHAPE),
    (dict(pages=1 << 27, stride=1 << 27), N.ERR_UNSUPPORTED_SHAPE),
    # outputs that are inputs, or one another, in whole or in part
    (dict(head_out=FAKE + 0x4000), N.ERR_INVALID_ARG), (dict(seq=FAKE), N.ERR_INVALID_ARG),
    (dict(seq=FAKE + 0x1000), N.ERR_INVALID_ARG), (dict(cu=FAKE + 0x5000 + 12), N.ERR_INVALID_ARG),
    (dict(slots=FAKE + 0x2000 + 4 * 31), N.ERR_INVALID_ARG),
    (dict(slots=FAKE + 2), N.ERR_MISALIGNED),
    (dict(ws=None), N.ERR_WORKSPACE), (dict(ws_bytes=16), N.ERR_WORKSPACE),
    (dict(ws=FAKE + 8), N.ERR_MISALIGNED)])
def test_plan_rejects(L, bad, status):
    assert _plan(L, **bad) == status


def _cache8(**kw):
    a = dict(k=FAKE, v=FAKE, ks=FAKE, vs=FAKE, n_pages=100, page=16, heads=8, dim=128)
    a.update(kw)
    return N.Kv8Cache(a["k"], a["v"], a["ks"], a["vs"], a["n_pages"], a["page"], a["heads"],
                      a["dim"])


BAD_CACHES = [
    (dict(k=None), N.ERR_INVALID_ARG), (dict(vs=None), N.ERR_INVALID_ARG),
    (dict(n_pages=0), N.ERR_INVALID_ARG), (dict(heads=0), N.ERR_INVALID_ARG),
    (dict(page=-16), N.ERR_INVALID_ARG), (dict(page=20), N.ERR_UNSUPPORTED_SHAPE),
    (dict(page=4112), N.ERR_UNSUPPORTED_SHAPE), (dict(dim=96), N.ERR_UNSUPPORTED_SHAPE),
    (dict(dim=256), N.ERR_UNSUPPORTED_SHAPE), (dict(heads=65536), N.ERR_UNSUPPORTED_SHAPE),
    (dict(n_pages=1 << 27), N.ERR_UNSUPPORTED_SHAPE), (dict(k=FAKE + 8), N.ERR_MISALIGNED),
    (dict(ks=FAKE + 2), N.ERR_MISALIGNED)]


def _append(L, cache, **kw):
    a = dict(k=FAKE, v=FAKE, stride=1024, tokens=5, slots=FAKE, ws=FAKE, ws_bytes=256)
    a.update(kw)
    return L.nvfp4_kv8_append(ctypes.byref(cache), a["k"], a["v"], a["stride"], a["tokens"],
                              a["slots"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_append_rejects_caches(L, bad, status):
    assert _append(L, _cache8(**bad)) == status


@pytest.mark.parametrize("bad,status", [
    (dict(k=None), N.ERR_INVALID_ARG), (dict(v=None), N.ERR_INVALID_ARG),
    (dict(slots=None), N.ERR_INVALID_ARG), (dict(tokens=-1), N.ERR_INVALID_ARG),
    (dict(tokens=1 << 30), N.ERR_UNSUPPORTED_SHAPE), (dict(stride=1016), N.ERR_INVALID_ARG),
    (dict(stride=1028), N.ERR_MISALIGNED), (dict(k=FAKE + 8), N.ERR_MISALIGNED),
    (dict(slots=FAKE + 1), N.ERR_MISALIGNED), (dict(ws=None), N.ERR_WORKSPACE),
    (dict(ws_bytes=255), N.ERR_WORKSPACE)])
def test_append_rejects(L, bad, status):
    assert _append(L, _cache8(), **bad) == status


def _attention(L, cache, **kw):
    a = dict(cu=FAKE, lens=FAKE, table=FAKE, stride=10, batch=2, pages=10, max_q=3, max_kv=160,
             q=FAKE, qs=4096, tq=6, heads=32, causal=1, scale=0.1, out=FAKE, os=4096, lse=None,
             scratch=FAKE, sb=1 << 40, ws=FAKE, wb=256)
    a.update(kw)
    b = N.Kv8Batch(a["cu"], a["lens"], a["table"], a["stride"], a["batch"], a["pages"],
                   a["max_q"], a["max_kv"])
    return L.nvfp4_kv8_attention(ctypes.byref(cache), ctypes.byref(b), a["q"], a["qs"], a["tq"],
                                 a["heads"], a["causal"], a["scale"], a["out"], a["os"], a["lse"],
                                 a["scratch"], a["sb"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_attention_rejects_caches(L, bad, status):
    assert _attention(L, _cache8(**bad)) == status


@pytest.mark.parametrize("bad,status", [
    (dict(cu=None), N.ERR_INVALID_ARG), (dict(lens=None), N.ERR_INVALID_ARG),
    (dict(table=None), N.ERR_INVALID_ARG), (dict(q=None), N.ERR_INVALID_ARG),
    (dict(out=None), N.ERR_INVALID_ARG), (dict(batch=0), N.ERR_INVALID_ARG),
    (dict(pages=0), N.ERR_INVALID_ARG), (dict(stride=9), N.ERR_INVALID_ARG),
    (dict(max_q=0), N.ERR_INVALID_ARG), (dict(max_kv=0), N.ERR_INVALID_ARG),
    (dict(tq=-1), N.ERR_INVALID_ARG), (dict(heads=0), N.ERR_INVALID_ARG),
    (dict(heads=12), N.ERR_INVALID_ARG), (dict(causal=2), N.ERR_INVALID_ARG),
    (dict(scale=0.0), N.ERR_INVALID_ARG), (dict(scale=float("nan")), N.ERR_INVALID_ARG),
    (dict(scale=float("inf")), N.ERR_INVALID_ARG), (dict(qs=4088), N.ERR_INVALID_ARG),
    (dict(os=4088), N.ERR_INVALID_ARG), (dict(batch=65536), N.ERR_UNSUPPORTED_SHAPE),
    (dict(tq=1 << 27), N.ERR_UNSUPPORTED_SHAPE),
    (dict(pages=1 << 27, stride=1 << 27), N.ERR_UNSUPPORTED_SHAPE),
    (dict(qs=4100), N.ERR_MISALIGNED), (dict(os=4100), N.ERR_MISALIGNED),
    (dict(q=FAKE + 8), N.ERR_MISALIGNED), (dict(out=FAKE + 8), N.ERR_MISALIGNED),
    (dict(lse=FAKE + 2), N.ERR_MISALIGNED), (dict(scratch=FAKE + 8), N.ERR_MISALIGNED),
    (dict(ws=None), N.ERR_WORKSPACE), (dict(wb=16), N.ERR_WORKSPACE)])
def test_attention_rejects(L, bad, status):
    assert _attention(L, _cache8(), **bad) == status


def test_status_string(L):
    assert N.status_string(N.ERR_CAPACITY) == "page pool, block table or slot map too small"


def _cpu_cache():
    return nv.KVCache8.empty(4, 16, 2, 64, device="cpu")


def test_binding_refuses_before_the_library():
    c = _cpu_cache()
    good = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16),
                cu_q=torch.zeros(3, dtype=torch.int32), seq_lens=torch.zeros(2, dtype=torch.int32),
                block_table=torch.zeros(2, 2, dtype=torch.int32))
    for name, t in [
            ("q", torch.zeros(3, 4, 64)), ("q", torch.zeros(3, 256, dtype=torch.bfloat16)),
            ("q", torch.zeros(3, 4, 128, dtype=torch.bfloat16)[..., ::2]),
            ("q", torch.zeros(4, 3, 64, dtype=torch.bfloat16).transpose(0, 1)),
            ("cu_q", torch.zeros(2, dtype=torch.int32)), ("cu_q", torch.zeros(3)),
            ("cu_q", torch.zeros(6, dtype=torch.int32)[::2]),
            ("seq_lens", torch.zeros(2, dtype=torch.int64)),
            ("block_table", torch.zeros(3, 2, dtype=torch.int32)),
            ("block_table", torch.zeros(2, 2, dtype=torch.int32).t().contiguous().t())]:
        with pytest.raises(ValueError):
            c.attention(**{**good, name: t})
    with pytest.raises(ValueError):
        c.attention(**good, out=torch.zeros(2, 4, 64, dtype=torch.bfloat16))
    kv = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    for k, v, s in [(kv.float(), kv, slots), (kv, kv[:2], slots), (kv, kv, slots[:2]),
                    (kv, kv, slots.long()), (kv[:, :1], kv[:, :1], slots),
                    (kv, torch.zeros(3, 4, 64, dtype=torch.bfloat16)[:, :2], slots)]:
        with pytest.raises(ValueError):
            c.append(k, v, s)
    for bad in (lambda: nv.KVCache8(c.k_codes.view(torch.uint8), c.v_codes, c.k_scale, c.v_scale),
                lambda: nv.KVCache8(c.k_codes, c.v_codes[:2], c.k_scale, c.v_scale),
                lambda: nv.KVCache8(c.k_codes, c.v_codes, c.k_scale.double(), c.v_scale),
                lambda: nv.KVCache8(c.k_codes, c.v_codes, c.k_scale[:2], c.v_scale),
                lambda: nv.KVCache8(c.k_codes.transpose(1, 2), c.v_codes.transpose(1, 2),
                                    c.k_scale, c.v_scale)):
        with pytest.raises(ValueError):
            bad()
    i = torch.zeros(2, dtype=torch.int32)
    for args in [(i.long(), i, i.view(2, 1), i, i[:1]), (i, i[:1], i.view(2, 1), i, i[:1]),
                 (i, i, i, i, i[:1]), (i, i, i.view(2, 1), i, i),
                 (i, i, torch.zeros(4, 2, dtype=torch.int32), i, i[:1])]:
        with pytest.raises(ValueError):
            nv.plan_pages(*args, page_tokens=16, n_pages=4, max_new=3)
    w = nv.NVFP4Tensor(torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8),
                       torch.zeros(1), 8, 32, nv.SF_MMA128x4)
    x = torch.zeros(2, 32)
    for bad in (dict(x=x[0]), dict(x=x[:, :16]), dict(x=x.t().contiguous().t()),
                dict(x=x, out=torch.zeros(1, 8)), dict(x=x, out=torch.zeros(2, 7))):
        with pytest.raises(ValueError):
            nv.gemv(w=w, **bad)
    for bad in (dict(x=x.half()), dict(x=x, out=torch.zeros(2, 8).half())):
        with pytest.raises(TypeError):
            nv.gemv(w=w, **bad)


def test_compiled_binding_refuses():
    """What only the compiled binding sees: wrong kinds of argument, numbers that do not fit."""
    c = _cpu_cache()
    i = torch.zeros(2, dtype=torch.int32)
    good = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), cu_q=torch.zeros(3).int(),
                seq_lens=i, block_table=i.view(2, 1))
    for bad in (dict(q=None), dict(cu_q=[0, 1, 2]), dict(max_q=1.5), dict(max_kv="1"),
                dict(scale="1"), dict(out=1)):
        with pytest.raises(TypeError):
            c.attention(**{**good, **bad})
    for bad in (dict(max_q=2 ** 31), dict(max_kv=-2 ** 31 - 1)):
        with pytest.raises(ValueError):
            c.attention(**{**good, **bad})
    with pytest.raises(OverflowError):
        c.attention(**good, max_q=2 ** 64)
    with pytest.raises(TypeError):
        c.append(None, None, i)
    for bad, error in ((dict(max_new=2 ** 31), ValueError), (dict(max_new=-1), ValueError),
                       (dict(max_new=None), TypeError)):
        with pytest.raises(error):
            nv.plan_pages(i, i, i.view(2, 1), i, i[:1], **{**dict(page_tokens=16, n_pages=4,
                                                                 max_new=3), **bad})
    with pytest.raises(ValueError, match="CUDA"):
        c.attention(**good)
    # a cache whose buffers were exchanged is looked at again
    c.k_codes = c.k_codes[:2]
    with pytest.raises(ValueError):
        c.append(torch.zeros(2, 2, 64).bfloat16(), torch.zeros(2, 2, 64).bfloat16(), i)


def test_attention_does_not_write_over_its_queries(L):
    assert _attention(L, _cache8(), q=FAKE, out=FAKE) == N.ERR_INVALID_ARG


@pytest.mark.parametrize("page", [16, 64, 4096])
def test_attention_rejects_tables_too_wide_for_its_look_ahead(L, page):
    """The kernels read table entries of up to 64 steps of 64 tokens past a range: their 32-bit token
    numbers must not wrap there (a negative one would pass for a small one)."""
    most = 0x7FFF0000 // page
    assert most * page + 4096 + 128 < 2 ** 31 <= (2 ** 31 // page - 1) * page + 4096 + 128
    for pages in (most + 1, 2 ** 31 // page - 1):
        assert _attention(L, _cache8(page=page), pages=pages, stride=pages, max_kv=2 ** 31 - 1) == \
            N.ERR_UNSUPPORTED_SHAPE


G = 1 << 30   # buffers far apart


def _apart(cols=1024, rows=1024, **kw):
    """gemv arguments without an overlap: 4 rows, N = K."""
    w = N.Tensor(FAKE + 2 * G, FAKE + 3 * G, FAKE + 4 * G, rows, cols, N.SF_MMA128x4)
    return dict(dict(x=FAKE, m=4, ldx=cols, w=w, y=FAKE + G, ldy=rows), **kw)


@pytest.mark.parametrize("y,ldy", [
    (FAKE, 1024),                       # x itself
    (FAKE + 2 * 1024 * 3, 1024),        # its last row
    (FAKE - 2 * 1024, 1024), (FAKE - 2, 1024), (FAKE + 2, 2048),
    (FAKE + 2 * G, 1024), (FAKE + 2 * G + 1024 * 512 - 2, 1024), (FAKE + 2 * G - 6146, 2048),
    (FAKE + 3 * G + 1024 * 64 - 2, 1024), (FAKE + 4 * G, 1024), (FAKE + 4 * G - 8190, 1024)])
def test_gemv_rejects_outputs_over_inputs(L, y, ldy):
    assert _gemv(L, **_apart(y=y, ldy=ldy)) == N.ERR_INVALID_ARG


def test_gemv_rejects_outputs_that_reach_into_the_next_row(L):
    # x and y share rows of 2048: y begins in x's columns, or ends in the next row's
    for at in (1022, 1026):
        assert _gemv(L, **_apart(ldx=2048, ldy=2048, y=FAKE + 2 * at)) == N.ERR_INVALID_ARG
    # one row each, of different strides
    assert _gemv(L, **_apart(m=1, ldx=1024, ldy=4096, y=FAKE + 2046)) == N.ERR_INVALID_ARG


def _apart8(**kw):
    """attention arguments without an overlap: 6 tokens of 32 heads of 128."""
    return dict(dict(q=FAKE, out=FAKE + G, cu=FAKE + 2 * G, lens=FAKE + 3 * G, table=FAKE + 4 * G,
                     lse=FAKE + 5 * G, scratch=FAKE + 6 * G, ws=FAKE + 7 * G), **kw)


@pytest.mark.parametrize("bad", [
    dict(out=FAKE), dict(out=FAKE + 16), dict(out=FAKE + 2 * 4096 * 5),
    dict(qs=8192, os=8192, out=FAKE + 2 * 4088), dict(qs=8192, os=8192, out=FAKE + 2 * 4104),
    dict(qs=8192, os=4096, out=FAKE + 2 * 4096), dict(lse=FAKE),
    dict(lse=FAKE + G + 2 * 4096 * 6 - 4),
    dict(out=FAKE + 2 * G), dict(out=FAKE + 3 * G - 2 * 4096 * 6 + 16), dict(out=FAKE + 4 * G + 64),
    dict(lse=FAKE + 4 * G + 76), dict(out=FAKE + 8 * G),
    dict(out=FAKE + 9 * G + 100 * 8 * 2048 - 16),
    dict(lse=FAKE + 10 * G), dict(lse=FAKE + 11 * G + 100 * 8 * 4 - 4)])
def test_attention_rejects_outputs_over_inputs(L, bad):
    c = _cache8(k=FAKE + 8 * G, v=FAKE + 9 * G, ks=FAKE + 10 * G, vs=FAKE + 11 * G)
    assert _attention(L, c, **_apart8(**bad)) == N.ERR_INVALID_ARG


@pytest.mark.parametrize("layout", [nv.SF_MMA128x4, nv.SF_ROWMAJOR])
def test_gemv_checks_the_weights_buffers(layout):
    """What the kernel would read past, or read wrongly, is refused by the binding."""
    rows, cols = 200, 96
    nb = nv.sf_bytes(rows, cols, layout)

    def weights(**kw):
        return nv.NVFP4Tensor(**{**dict(
            codes=torch.zeros(rows, cols // 2, dtype=torch.uint8),
            sf=torch.zeros(nb, dtype=torch.uint8), s_t=torch.zeros(1), rows=rows, cols=cols,
            sf_layout=layout), **kw})
    x = torch.zeros(1, cols)
    u8 = torch.uint8
    for bad in (dict(codes=torch.zeros(rows - 1, cols // 2, dtype=u8)),
                dict(codes=torch.zeros(rows, cols, dtype=u8)[:, ::2]),
                dict(codes=torch.zeros(cols // 2, rows, dtype=u8).t()),
                dict(codes=torch.zeros(rows, cols // 2, dtype=torch.int8)),
                dict(codes=torch.zeros(rows, cols // 2)),
                dict(sf=torch.zeros(nb - 1, dtype=u8)), dict(sf=torch.zeros(2 * nb, dtype=u8)[::2]),
                dict(sf=torch.zeros(nb, dtype=torch.int8)),
                dict(s_t=torch.zeros(1, dtype=torch.float64)), dict(s_t=torch.zeros(0)),
                dict(s_t=torch.zeros(2)), dict(rows=rows + 1), dict(rows=2 ** 31), dict(rows=-1)):
        with pytest.raises(ValueError, match="of the weights"):
            nv.gemv(x, weights(**bad))
    with pytest.raises(ValueError, match="CUDA"):
        nv.gemv(x, weights())


def test_build_refuses_another_register_count():
    """The many-row attention's register split holds for 128 registers a thread at launch."""
    def log(*regs):
        return "".join(
            f"ptxas info    : Compiling entry function '_ZN5nvfp4{n}{i}' for 'sm_100a'\n"
            f"ptxas info    : Function properties for _ZN5nvfp4{n}{i}\n"
            "    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads\n"
            f"ptxas info    : Used {r} registers, used 1 barriers\n"
            for i, (n, r) in enumerate(regs))
    both = ("12chunk_kernelILi64EE", 128), ("12chunk_kernelILi128EE", 128)
    nbuild.check_registers(log(("11join_kernel", 40), *both, ("11gemv_kernel", 124)))
    for bad in ([("12chunk_kernelILi64EE", 120), both[1]],
                [both[0], ("12chunk_kernelILi128EE", 168)], [("11join_kernel", 128)], []):
        with pytest.raises(RuntimeError, match="128 registers"):
            nbuild.check_registers(log(*bad))


def test_library_is_built_without_the_binding(monkeypatch, tmp_path):
    """No host compiler or no torch headers: the error comes after libnvfp4.so is there."""
    monkeypatch.setattr(nbuild, "LIB", str(tmp_path / "libnvfp4.so"))
    monkeypatch.setattr(nbuild, "BINDING", str(tmp_path / "_binding.so"))

    def run(cmd, **kw):
        if cmd[0] != nbuild.NVCC:
            raise FileNotFoundError(cmd[0])
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, None, "entry function 'chunk_kernel' for "
                                           "'sm_100a'\nptxas info    : Used 128 registers\n")
    monkeypatch.setattr(nbuild.subprocess, "run", run)
    with pytest.raises(FileNotFoundError):
        nbuild.build()
    assert os.listdir(tmp_path) == ["libnvfp4.so"]


def test_binding_is_rebuilt_for_another_torch(L, monkeypatch, tmp_path):
    monkeypatch.setattr(nbuild, "BINDING", str(tmp_path / "_binding.so"))
    compiled = []

    def run(cmd, **kw):
        compiled.append([a for a in cmd if "TORCH_VERSION" in a])
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(nbuild.subprocess, "run", run)
    nbuild.build_binding()
    nbuild.build_binding()
    assert len(compiled) == 1 and torch.__version__ in compiled[0][0]
    monkeypatch.setattr(torch, "__version__", "1.0")
    nbuild.build_binding()
    nbuild.build_binding()
    assert compiled[1:] == [['-DNVFP4_TORCH_VERSION="1.0"']]
    # and one that is there all the same is not called
    monkeypatch.setattr(nv.ops, "_binding", None)
    with pytest.raises(RuntimeError, match="not 1.0"):
        nv.ops._load_binding()


@pytest.mark.parametrize("scale", [3e38, 2.4e38, -1e-9])
def test_attention_rejects_scales_that_overflow_in_base_2(L, scale):
    assert _attention(L, _cache8(k=FAKE + 8 * G, v=FAKE + 9 * G, ks=FAKE + 10 * G,
                                 vs=FAKE + 11 * G), **_apart8(scale=scale)) == N.ERR_INVALID_ARG


def test_binding_before_init_refuses():
    """The module by itself, without the library's entry points."""
    code = ("import torch\n"
            "from nvfp4_w4a4_quantized_08_b200 import _binding as b\n"
            "z = lambda *s: torch.zeros(*s, dtype=torch.uint8)\n"
            "try:\n"
            "    b.gemv(torch.zeros(1, 32), z(8, 16), z(512), torch.zeros(1), 8, 32, 1,\n"
            "           torch.float32, None, 0)\n"
            "except RuntimeError as e:\n"
            "    print(e)\n")
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert run.stdout.strip() == "init has not been called", run.stderr[-500:]
