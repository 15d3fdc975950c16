"""torch-facing wrappers of the libnvfp4 entry points.

Argument marshalling only: each function passes device pointers, sizes and
``torch.cuda.current_stream()`` to the C ABI, which launches the kernels.  No
step of the NVFP4 path runs in Python or torch.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Dict, List, Optional, Sequence, Tuple

import torch

from . import _native as N
from ._native import NVFP4Error  # noqa: F401  (re-export)


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


_workspaces: Dict[Tuple[int, int], torch.Tensor] = {}


def workspace(device=None) -> torch.Tensor:
    """A zero-filled workspace for the current stream of `device` (cached).
    Calls that share it must stay ordered on that stream."""
    idx = None if device is None else torch.device(device).index
    if idx is None:
        idx = torch.cuda.current_device()
    key = (idx, torch._C._cuda_getCurrentRawStream(idx))
    ws = _workspaces.get(key)
    if ws is None:
        ws = torch.zeros(N.lib().nvfp4_workspace_bytes(), dtype=torch.uint8,
                         device=torch.device("cuda", idx))
        _workspaces[key] = ws
    return ws


@dataclass
class NVFP4Tensor:
    """Device buffers of an NVFP4 tensor (see nvfp4_tensor in include/nvfp4.h)."""
    codes: torch.Tensor   # uint8 [rows, cols/2]
    sf: torch.Tensor      # uint8 [nvfp4_sf_bytes]
    s_t: torch.Tensor     # float32 [1]
    rows: int
    cols: int
    sf_layout: int

    def c_struct(self) -> N.Tensor:
        return N.Tensor(self.codes.data_ptr(), self.sf.data_ptr(), self.s_t.data_ptr(),
                        self.rows, self.cols, self.sf_layout)

    @property
    def device(self):
        return self.codes.device


def codes_bytes(rows: int, cols: int) -> int:
    return int(N.lib().nvfp4_codes_bytes(rows, cols))


def sf_bytes(rows: int, cols: int, sf_layout: int) -> int:
    return int(N.lib().nvfp4_sf_bytes(rows, cols, sf_layout))


def empty(rows: int, cols: int, sf_layout: int = N.SF_MMA128x4, device="cuda") -> NVFP4Tensor:
    nb = sf_bytes(rows, cols, sf_layout)
    if nb == 0 and rows * cols > 0:
        raise NVFP4Error(N.ERR_UNSUPPORTED_SHAPE, "empty")
    return NVFP4Tensor(
        codes=torch.empty(rows, cols // 2, dtype=torch.uint8, device=device),
        sf=torch.empty(max(nb, 1), dtype=torch.uint8, device=device),
        s_t=torch.empty(1, dtype=torch.float32, device=device),
        rows=rows, cols=cols, sf_layout=sf_layout)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return N.BF16
    if t.dtype == torch.float32:
        return N.FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def quantize(x: torch.Tensor, sf_layout: int = N.SF_MMA128x4, s_t: Optional[torch.Tensor] = None,
             out: Optional[NVFP4Tensor] = None, ws: Optional[torch.Tensor] = None,
             amax_in: Optional[torch.Tensor] = None) -> NVFP4Tensor:
    """nvfp4_quantize: x is a 2-D bf16/fp32 CUDA tensor with unit column stride.

    s_t:     a one-element fp32 tensor holding the tensor scale to use, or None.
    amax_in: a one-element fp32 tensor holding max|x| as accumulated by the
             producer (``gemm(..., c_amax=)``); the amax pass is skipped and the
             word is reset to 0 when the launch ends.  Exclusive with s_t.
    """
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("quantize expects a 2-D tensor with contiguous rows")
    rows, cols = x.shape
    if out is None:
        out = empty(rows, cols, sf_layout, x.device)
    ws = workspace(x.device) if ws is None else ws
    st = out.c_struct()
    N.check(N.lib().nvfp4_quantize(x.data_ptr(), _dtype_code(x), rows, cols, x.stride(0),
                                   ctypes.byref(st), _ptr(s_t), _ptr(amax_in), ws.data_ptr(),
                                   ws.numel(), _stream()), "nvfp4_quantize")
    return out


def dequantize(t: NVFP4Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """nvfp4_dequantize -> bf16 [rows, cols]"""
    if out is None:
        out = torch.empty(t.rows, t.cols, dtype=torch.bfloat16, device=t.device)
    st = t.c_struct()
    N.check(N.lib().nvfp4_dequantize(ctypes.byref(st), out.data_ptr(), out.stride(0), _stream()),
            "nvfp4_dequantize")
    return out


def gemm(a: NVFP4Tensor, w: NVFP4Tensor, out_dtype: torch.dtype = torch.bfloat16,
         out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
         c_amax: Optional[torch.Tensor] = None, c_amax_cols: int = 0,
         act: int = N.ACT_NONE) -> torch.Tensor:
    """nvfp4_gemm: C = act(A W^T), [a.rows, w.rows] in bf16 or fp32.

    act:    N.ACT_NONE, or N.ACT_GELU_TANH (the FFN's GELU, tanh form, in the
            epilogue before the output rounding).

    c_amax: fp32 tensor that starts at 0 (or at a smaller running max); the
            kernel raises it to max|C| over the values it stores.  With
            c_amax_cols = 0 one element covers all of C; with c_amax_cols > 0
            (a multiple of 256 dividing N) element g covers columns
            [g * c_amax_cols, (g + 1) * c_amax_cols).
    """
    if c_amax is not None:
        need = 1 if c_amax_cols == 0 else max(1, w.rows // c_amax_cols)
        if c_amax.dtype != torch.float32 or c_amax.numel() < need:
            raise ValueError(f"c_amax needs {need} fp32 elements")
    if out is None:
        out = torch.empty(a.rows, w.rows, dtype=out_dtype, device=a.device)
    ws = workspace(a.device) if ws is None else ws
    sa, sw = a.c_struct(), w.c_struct()
    N.check(N.lib().nvfp4_gemm(ctypes.byref(sa), ctypes.byref(sw), out.data_ptr(),
                               _dtype_code(out), out.stride(0), act, _ptr(c_amax), c_amax_cols,
                               ws.data_ptr(), ws.numel(), _stream()), "nvfp4_gemm")
    return out


class KVCache:
    """The NVFP4 KV cache of one layer: n_slots frame slots for K and V."""

    def __init__(self, n_slots: int, tokens_per_frame: int, heads: int, head_dim: int,
                 device="cuda", scale_rule: int = N.SCALE_ONTO_6):
        """scale_rule: N.SCALE_ONTO_6 (the recipe) or N.SCALE_FOUR_OVER_SIX."""
        per = tokens_per_frame * heads * head_dim
        self.scale_rule = scale_rule
        self.n_slots, self.tpf, self.heads, self.head_dim = n_slots, tokens_per_frame, heads, head_dim
        self.k_codes = torch.zeros(n_slots, per // 2, dtype=torch.uint8, device=device)
        self.v_codes = torch.zeros_like(self.k_codes)
        self.k_sf = torch.zeros(n_slots, per // 16, dtype=torch.uint8, device=device)
        self.v_sf = torch.zeros_like(self.k_sf)
        self.k_st = torch.zeros(n_slots, dtype=torch.float32, device=device)
        self.v_st = torch.zeros_like(self.k_st)

    def c_struct(self) -> N.KvCache:
        return N.KvCache(self.k_codes.data_ptr(), self.v_codes.data_ptr(), self.k_sf.data_ptr(),
                         self.v_sf.data_ptr(), self.k_st.data_ptr(), self.v_st.data_ptr(),
                         self.n_slots, self.tpf, self.heads, self.head_dim, self.scale_rule)

    def quant_chunk(self, k: torch.Tensor, v: torch.Tensor, dst_slots: Sequence[int],
                    ws: Optional[torch.Tensor] = None, k_amax_in: Optional[torch.Tensor] = None,
                    v_amax_in: Optional[torch.Tensor] = None) -> None:
        """nvfp4_kv_quant_chunk.  k, v: bf16 views [tokens, heads*head_dim] (or
        [tokens, heads, head_dim]) with unit stride inside a token.
        k_amax_in, v_amax_in: both None (amax pass), or one-element fp32
        tensors holding max|K|, max|V| from the producer; reset to 0."""
        token_stride = k.stride(0)
        if v.stride(0) != token_stride:
            raise ValueError("k and v must share a token stride")
        slots = (ctypes.c_int32 * len(dst_slots))(*dst_slots)
        ws = workspace(k.device) if ws is None else ws
        cs = self.c_struct()
        N.check(N.lib().nvfp4_kv_quant_chunk(ctypes.byref(cs), k.data_ptr(), v.data_ptr(),
                                             token_stride, slots, len(dst_slots), _ptr(k_amax_in),
                                             _ptr(v_amax_in), ws.data_ptr(), ws.numel(),
                                             _stream()), "nvfp4_kv_quant_chunk")

    def dequant_window(self, slot_ids: Sequence[int], k_out: Optional[torch.Tensor] = None,
                       v_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """nvfp4_kv_dequant_window -> bf16 K, V [n*tokens_per_frame, heads, head_dim]"""
        n = len(slot_ids)
        shape = (n * self.tpf, self.heads, self.head_dim)
        if k_out is None:
            k_out = torch.empty(shape, dtype=torch.bfloat16, device=self.k_codes.device)
        if v_out is None:
            v_out = torch.empty(shape, dtype=torch.bfloat16, device=self.k_codes.device)
        ids = (ctypes.c_int32 * n)(*slot_ids)
        cs = self.c_struct()
        N.check(N.lib().nvfp4_kv_dequant_window(ctypes.byref(cs), ids, n, k_out.data_ptr(),
                                                v_out.data_ptr(), _stream()),
                "nvfp4_kv_dequant_window")
        return k_out, v_out

    def window_attention(self, q: torch.Tensor, slot_ids: Sequence[int],
                         scale: Optional[float] = None,
                         out: Optional[torch.Tensor] = None,
                         ws: Optional[torch.Tensor] = None) -> torch.Tensor:
        """nvfp4_window_attention: softmax(scale q k^T) v over the listed slots,
        read straight from the NVFP4 pools.  q: bf16 [tq, >= heads*head_dim]
        (row stride a multiple of 8, e.g. the Q third of a QKV output) ->
        bf16 [tq, heads*head_dim] (or `out`, same layout as q)."""
        width = self.heads * self.head_dim
        if q.dtype != torch.bfloat16 or q.dim() != 2 or q.stride(1) != 1 or q.shape[1] < width:
            raise ValueError(f"q must be a 2-D bf16 tensor of at least {width} unit-stride columns")
        if scale is None:
            scale = self.head_dim ** -0.5
        if out is None:
            out = torch.empty(q.shape[0], width, dtype=torch.bfloat16, device=q.device)
        elif (out.dtype != torch.bfloat16 or out.dim() != 2 or out.stride(1) != 1 or
              out.shape[0] != q.shape[0] or out.shape[1] < width):
            raise ValueError(f"out must be a 2-D bf16 tensor of {q.shape[0]} rows and at least "
                             f"{width} unit-stride columns")
        n = len(slot_ids)
        ids = (ctypes.c_int32 * n)(*slot_ids)
        cs = self.c_struct()
        ws = workspace(q.device) if ws is None else ws
        N.check(N.lib().nvfp4_window_attention(ctypes.byref(cs), ids, n, q.data_ptr(), q.stride(0),
                                               q.shape[0], float(scale), out.data_ptr(),
                                               out.stride(0), ws.data_ptr(), ws.numel(),
                                               _stream()),
                "nvfp4_window_attention")
        return out


def _launch(fn, what: str, device: torch.device, *args) -> None:
    """Calls an entry point on `device`'s current stream, with `device` current."""
    if device.type != "cuda":
        raise ValueError(f"{what} takes CUDA tensors")
    i = device.index
    if i == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    if status:
        raise NVFP4Error(status, what)


def _check_int32(device: torch.device, name: str, t: torch.Tensor, dims: int = 1) -> None:
    if t.dtype is not torch.int32 or t.device != device or t.dim() != dims:
        raise ValueError(f"{name} must be an int32 tensor of {dims} dimension(s) on {device}")
    if dims == 1:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    elif t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")


def _row_stride(t: torch.Tensor) -> int:
    """The row stride of a 2-D tensor; torch gives any number for a single row."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def gemv(x: torch.Tensor, w: NVFP4Tensor, out_dtype: torch.dtype = torch.bfloat16,
         out: Optional[torch.Tensor] = None, act: int = N.ACT_NONE) -> torch.Tensor:
    """nvfp4_gemv: act(x W^T) for 1 to 16 rows x (bf16 or fp32, unit column
    stride) that are not quantized, and NVFP4 weights -> [x.rows, w.rows] in
    bf16 or fp32.  For more rows quantize x and use gemm."""
    if x.dim() != 2 or x.stride(1) != 1 or x.shape[1] != w.cols:
        raise ValueError(f"gemv expects a 2-D tensor of {w.cols} unit-stride columns")
    if x.device != w.device:
        raise ValueError("x and w must be on one device")
    if out is None:
        out = torch.empty((x.shape[0], w.rows), dtype=out_dtype, device=x.device)
    elif (out.dim() != 2 or out.shape[0] != x.shape[0] or out.shape[1] < w.rows or
          out.stride(1) != 1 or out.device != x.device):
        raise ValueError(f"out must have {x.shape[0]} rows of at least {w.rows} unit-stride "
                         f"columns on {x.device}")
    sw = w.c_struct()
    _launch(N.lib().nvfp4_gemv, "nvfp4_gemv", x.device, x.data_ptr(), _dtype_code(x), x.shape[0],
            _row_stride(x), ctypes.byref(sw), out.data_ptr(), _dtype_code(out), _row_stride(out),
            act)
    return out


@dataclass
class PagePlan:
    """What plan_pages gives: int32 device tensors."""
    seq_lens: torch.Tensor   # [batch] tokens of each request, the new ones included
    cu_new: torch.Tensor     # [batch + 1] offsets of the requests' new tokens
    slot_map: torch.Tensor   # [max_new] slot of each new token, -1 past the last
    free_head: torch.Tensor  # [1] first page of the free list that is still free


def plan_pages(cached_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
               free_pages: torch.Tensor, free_head: torch.Tensor, page_tokens: int, n_pages: int,
               max_new: int, ws: Optional[torch.Tensor] = None) -> PagePlan:
    """nvfp4_plan_pages: pages and slots for each request's new tokens, on the
    device.  block_table [batch, max_pages] is updated in place; the rest are
    new tensors (free_head of the result goes into the next call).  Lengths that
    do not fit are reported by device_status, and then change nothing."""
    dev = block_table.device
    _check_int32(dev, "cached_lens", cached_lens)
    _check_int32(dev, "new_lens", new_lens)
    _check_int32(dev, "block_table", block_table, 2)
    _check_int32(dev, "free_pages", free_pages)
    _check_int32(dev, "free_head", free_head)
    batch, max_pages = block_table.shape
    if cached_lens.shape[0] != batch or new_lens.shape[0] != batch or free_head.shape[0] != 1:
        raise ValueError("plan_pages: cached_lens and new_lens must be [batch], block_table "
                         "[batch, max_pages], free_head [1]")
    if max_new < 0:
        raise ValueError("max_new must not be negative")
    # one allocation for the four results, each on a 16-byte boundary
    a, b = (batch + 3) // 4 * 4, (batch + 4) // 4 * 4
    mem = torch.empty(4 + a + b + max_new, dtype=torch.int32, device=dev)
    head, seq, cu, slots = mem[:1], mem[4:4 + batch], mem[4 + a:5 + a + batch], mem[4 + a + b:]
    ws = workspace(dev) if ws is None else ws
    at = mem.data_ptr()
    _launch(N.lib().nvfp4_plan_pages, "nvfp4_plan_pages", dev, cached_lens.data_ptr(),
            new_lens.data_ptr(), batch, block_table.data_ptr(), _row_stride(block_table),
            max_pages, free_pages.data_ptr(), free_pages.shape[0], free_head.data_ptr(),
            page_tokens, n_pages, at + 16, at + 16 + 4 * a, at + 16 + 4 * (a + b), max_new, at,
            ws.data_ptr(), ws.numel())
    return PagePlan(seq, cu, slots, head)


class KVCache8:
    """The paged 8-bit KV cache of one layer: E4M3 codes [n_pages, kv_heads,
    page_tokens, head_dim] and a power-of-two scale [n_pages, kv_heads] for K and
    for V.  A page holds page_tokens consecutive tokens of one request; which
    page is whose is the callers' (plan_pages keeps block tables)."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor):
        """A cache over buffers of the caller's; see empty() for new ones."""
        shape, dev = k_codes.shape, k_codes.device
        if len(shape) != 4 or v_codes.shape != shape:
            raise ValueError("codes must be [n_pages, kv_heads, page_tokens, head_dim]")
        for t in (k_codes, v_codes):
            if t.dtype != torch.float8_e4m3fn or not t.is_contiguous() or t.device != dev:
                raise ValueError("codes must be contiguous float8_e4m3fn tensors on one device")
        for t in (k_scale, v_scale):
            if (t.dtype != torch.float32 or t.shape != shape[:2] or not t.is_contiguous() or
                    t.device != dev):
                raise ValueError(f"scales must be contiguous fp32 tensors {tuple(shape[:2])}")
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        self.n_pages, self.kv_heads, self.page_tokens, self.head_dim = shape

    @classmethod
    def empty(cls, n_pages: int, page_tokens: int, kv_heads: int, head_dim: int,
              device="cuda") -> "KVCache8":
        codes = [torch.zeros(n_pages, kv_heads, page_tokens, head_dim, dtype=torch.uint8,
                             device=device).view(torch.float8_e4m3fn) for _ in range(2)]
        scale = [torch.zeros(n_pages, kv_heads, dtype=torch.float32, device=device)
                 for _ in range(2)]
        return cls(*codes, *scale)

    def c_struct(self) -> N.Kv8Cache:
        return N.Kv8Cache(self.k_codes.data_ptr(), self.v_codes.data_ptr(),
                          self.k_scale.data_ptr(), self.v_scale.data_ptr(), self.n_pages,
                          self.page_tokens, self.kv_heads, self.head_dim)

    def _rows(self, name: str, t: torch.Tensor, heads: int) -> int:
        """The token stride of a bf16 tensor [tokens, heads, head_dim] or [tokens,
        heads * head_dim] whose tokens are contiguous."""
        d = self.head_dim
        if t.dim() == 3:
            n, h, e = t.shape
            stride, sh, se = t.stride()
            ok = h == heads and e == d and se == 1 and (sh == d or heads == 1)
        else:
            n, e = t.shape if t.dim() == 2 else (0, -1)
            stride = t.stride(0) if t.dim() == 2 else 0
            ok = e == heads * d and t.stride(1) == 1
        if not ok or t.dtype is not torch.bfloat16 or t.device != self.k_codes.device:
            raise ValueError(f"{name} must be a bf16 tensor [tokens, {heads}, {d}] on "
                             f"{self.k_codes.device}, contiguous inside a token")
        return stride if n > 1 else heads * d

    def append(self, k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor,
               ws: Optional[torch.Tensor] = None) -> None:
        """nvfp4_kv8_append: writes the tokens of k and v (bf16 [tokens,
        kv_heads, head_dim], views into a fused projection included) to their
        slots (a plan's slot_map; its first entries, if it is longer)."""
        stride = self._rows("k", k, self.kv_heads)
        tokens = k.shape[0]
        if v.shape[0] != tokens or self._rows("v", v, self.kv_heads) != stride:
            raise ValueError("k and v must share their tokens and a token stride")
        _check_int32(k.device, "slot_map", slot_map)
        if slot_map.shape[0] < tokens:
            raise ValueError(f"slot_map must have at least {tokens} entries")
        ws = workspace(k.device) if ws is None else ws
        cs = self.c_struct()
        _launch(N.lib().nvfp4_kv8_append, "nvfp4_kv8_append", k.device, ctypes.byref(cs),
                k.data_ptr(), v.data_ptr(), stride, tokens, slot_map.data_ptr(), ws.data_ptr(),
                ws.numel())

    def attention(self, q: torch.Tensor, cu_q: torch.Tensor, seq_lens: torch.Tensor,
                  block_table: torch.Tensor, max_q: Optional[int] = None,
                  max_kv: Optional[int] = None, causal: bool = True,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  return_lse: bool = False, ws: Optional[torch.Tensor] = None):
        """nvfp4_kv8_attention: softmax(scale q k^T) v of each request's queries
        over its cached tokens.

        q:         bf16 [tokens, q_heads, head_dim], the requests' queries packed;
                   q_heads a multiple of kv_heads.
        cu_q, seq_lens, block_table: int32 [batch + 1], [batch], [batch, pages] (a
                   plan's cu_new and seq_lens).
        max_q:     no request has more queries (default: all of q's tokens).
        max_kv:    about the longest request (default: the table's width); the
                   split of the work goes by it, not the result.
        causal:    the queries are the requests' last tokens and see no later one.
        Returns out [tokens, q_heads, head_dim] in bf16, and with return_lse the
        fp32 log-sum-exp [tokens, q_heads] too.  Rows of no request are left as
        they are in `out`."""
        if q.dim() != 3 or q.shape[2] != self.head_dim:
            raise ValueError(f"q must be [tokens, q_heads, {self.head_dim}]")
        tokens, heads = q.shape[0], q.shape[1]
        stride = self._rows("q", q, heads)
        dev = q.device
        _check_int32(dev, "cu_q", cu_q)
        _check_int32(dev, "seq_lens", seq_lens)
        _check_int32(dev, "block_table", block_table, 2)
        batch, pages = block_table.shape
        if cu_q.shape[0] != batch + 1 or seq_lens.shape[0] != batch:
            raise ValueError("attention: cu_q must be [batch + 1], seq_lens [batch] and "
                             "block_table [batch, pages]")
        if out is None:
            out = torch.empty((tokens, heads, self.head_dim), dtype=torch.bfloat16, device=dev)
            out_stride = heads * self.head_dim
        elif out.shape != q.shape:
            raise ValueError("out must have q's shape")
        else:
            out_stride = self._rows("out", out, heads)
        lse = torch.empty((tokens, heads), dtype=torch.float32, device=dev) if return_lse else None
        cs = self.c_struct()
        cb = N.Kv8Batch(cu_q.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
                        _row_stride(block_table), batch, pages,
                        max(tokens, 1) if max_q is None else max_q,
                        pages * self.page_tokens if max_kv is None else max_kv)
        ws = workspace(dev) if ws is None else ws
        need = int(N.lib().nvfp4_kv8_attention_scratch_bytes(
            ctypes.byref(cs), ctypes.byref(cb), tokens, heads, int(causal)))
        # a tensor of the call's own: calls on other streams and captured graphs share nothing
        scratch = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        _launch(N.lib().nvfp4_kv8_attention, "nvfp4_kv8_attention", dev, ctypes.byref(cs),
                ctypes.byref(cb), q.data_ptr(), stride, tokens, heads, int(causal),
                self.head_dim ** -0.5 if scale is None else float(scale), out.data_ptr(),
                out_stride, _ptr(lse), _ptr(scratch), need, ws.data_ptr(), ws.numel())
        return (out, lse) if return_lse else out


class SinkPlan:
    """nvfp4_sink_plan: host-side slot planning under the two-level attention
    sinks (global sinks kept for good, shot sinks re-bound at cuts, a local
    window).  next() -> (dst_slots for KVCache.quant_chunk, window slot list
    for KVCache.dequant_window / window_attention)."""

    def __init__(self, n_slots: int, global_sinks: int = 3, shot_sinks: int = 3,
                 window: int = 9):
        self.n_slots = n_slots
        self._h = N.lib().nvfp4_sink_plan_create(n_slots, global_sinks, shot_sinks, window)
        if not self._h:
            raise N.NVFP4Error(N.ERR_INVALID_ARG, "nvfp4_sink_plan_create")

    def next(self, n_frames: int, new_shot: bool = False) -> Tuple[List[int], List[int]]:
        dst = (ctypes.c_int32 * max(1, n_frames))()
        win = (ctypes.c_int32 * self.n_slots)()
        n = ctypes.c_int32(0)
        N.check(N.lib().nvfp4_sink_plan_next(self._h, n_frames, int(bool(new_shot)), dst, win,
                                             ctypes.byref(n)), "nvfp4_sink_plan_next")
        return list(dst[:n_frames]), list(win[:n.value])

    def frame_of_slot(self, slot: int) -> int:
        return int(N.lib().nvfp4_sink_plan_frame_of_slot(self._h, slot))

    def close(self) -> None:
        if getattr(self, "_h", None):
            N.lib().nvfp4_sink_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:  # interpreter shutdown: the library may be gone already
            pass


def device_status(ws: Optional[torch.Tensor] = None) -> int:
    """nvfp4_get_device_status: sync the current stream, read and clear the
    workspace status word."""
    ws = workspace() if ws is None else ws
    return int(N.lib().nvfp4_get_device_status(ws.data_ptr(), _stream()))


def set_wait_limit_ns(ns: int) -> None:
    N.lib().nvfp4_set_wait_limit_ns(int(ns))
