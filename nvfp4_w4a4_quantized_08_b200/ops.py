"""torch-facing wrappers of the libnvfp4 entry points.

Argument marshalling only: each function passes device pointers, sizes and
``torch.cuda.current_stream()`` to the C ABI, which launches the kernels: through
ctypes, or where a kernel takes a few microseconds through csrc/binding.cpp.  No
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
_captured_workspaces: Dict[Tuple[int, int], torch.Tensor] = {}


def workspace(device=None) -> torch.Tensor:
    """A zero-filled workspace for the current stream of `device` (cached).
    Calls that share it must stay ordered on that stream.

    While the stream is being captured: a second one, which the graphs captured
    on it share and which belongs to none of them.  device_status reads it too.
    Graphs of one stream that are replayed at the same time need a `ws` of their
    own, unless only the status word is used (plan_pages, KVCache8)."""
    idx = None if device is None else torch.device(device).index
    current = torch.cuda.current_device() if idx is None else torch._C._cuda_getDevice()
    if idx is None:
        idx = current
    key = (idx, torch._C._cuda_getCurrentRawStream(idx))
    if idx == current:
        captured = torch._C._cuda_isCurrentStreamCapturing()
    else:
        with torch.cuda.device(idx):
            captured = torch._C._cuda_isCurrentStreamCapturing()
    known = _captured_workspaces if captured else _workspaces
    ws = known.get(key)
    if ws is None:
        nbytes = N.lib().nvfp4_workspace_bytes()
        if captured:   # zeros made here would be a node of the graph, made again in each replay
            ws = (_binding or _load_binding()).zeros_outside_capture(nbytes, idx)
        else:
            ws = torch.zeros(nbytes, dtype=torch.uint8, device=torch.device("cuda", idx))
        known[key] = ws
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


_binding = None


def _load_binding():
    """The compiled module behind gemv, plan_pages and KVCache8, whose kernels take
    less time than a ctypes call; it calls the entry points of the same library."""
    global _binding
    N.lib()  # raises if the library has not been built
    try:
        from . import _binding as b
    except ImportError as e:
        raise RuntimeError("the torch binding has not been built for this torch; run python -m "
                           f"nvfp4_w4a4_quantized_08_b200.build ({e})") from e
    # (a binding for another torch may load all the same, and then call what is no longer there)
    built_for = getattr(b, "torch_version", "of no known version")
    if built_for != torch.__version__:
        raise RuntimeError(f"the torch binding has been built for torch {built_for}, not "
                           f"{torch.__version__}; run python -m nvfp4_w4a4_quantized_08_b200.build")
    b.init(N.LIB_PATH, NVFP4Error, workspace)
    _binding = b
    return b


def gemv(x: torch.Tensor, w: NVFP4Tensor, out_dtype: torch.dtype = torch.bfloat16,
         out: Optional[torch.Tensor] = None, act: int = N.ACT_NONE) -> torch.Tensor:
    """nvfp4_gemv: act(x W^T) for 1 to 16 rows x (bf16 or fp32, unit column
    stride) that are not quantized, and NVFP4 weights -> [x.rows, w.rows] in
    bf16 or fp32.  For more rows quantize x and use gemm."""
    return (_binding or _load_binding()).gemv(x, w.codes, w.sf, w.s_t, w.rows, w.cols,
                                              w.sf_layout, out_dtype, out, act)


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
    do not fit are reported by device_status, also where a replayed graph meets
    them, and then change nothing."""
    return PagePlan(*(_binding or _load_binding()).plan_pages(
        cached_lens, new_lens, block_table, free_pages, free_head, page_tokens, n_pages, max_new,
        ws))


class KVCache8:
    """The paged 8-bit KV cache of one layer: E4M3 codes [n_pages, kv_heads,
    page_tokens, head_dim] and a power-of-two scale [n_pages, kv_heads] for K and
    for V.  A page holds page_tokens consecutive tokens of one request; which
    page is whose is the callers' (plan_pages keeps block tables).  Slots, pages
    and lengths outside the buffers, and values that are not finite, are reported
    by device_status, also where a replayed graph meets them."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scale: torch.Tensor,
                 v_scale: torch.Tensor):
        """A cache over buffers of the caller's; see empty() for new ones."""
        self.n_pages, self.kv_heads, self.page_tokens, self.head_dim = (
            _binding or _load_binding()).kv8_shape(k_codes, v_codes, k_scale, v_scale)
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale

    @classmethod
    def empty(cls, n_pages: int, page_tokens: int, kv_heads: int, head_dim: int,
              device="cuda") -> "KVCache8":
        codes = [torch.zeros(n_pages, kv_heads, page_tokens, head_dim, dtype=torch.uint8,
                             device=device).view(torch.float8_e4m3fn) for _ in range(2)]
        scale = [torch.zeros(n_pages, kv_heads, dtype=torch.float32, device=device)
                 for _ in range(2)]
        return cls(*codes, *scale)

    def append(self, k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor,
               ws: Optional[torch.Tensor] = None) -> None:
        """nvfp4_kv8_append: writes the tokens of k and v (bf16 [tokens,
        kv_heads, head_dim], views into a fused projection included) to their
        slots (a plan's slot_map; its first entries, if it is longer)."""
        (_binding or _load_binding()).kv8_append(self.k_codes, self.v_codes, self.k_scale,
                                                 self.v_scale, k, v, slot_map, ws)

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
                   plan's cu_new and seq_lens; a batch of 0 writes nothing).
        max_q:     no request has more queries (default: all of q's tokens).  Worth
                   giving: up to 32 query rows (max_q * q_heads / kv_heads) a
                   request take the kernel for single tokens, more the one for
                   chunks, whose tiles have 256 rows.
        max_kv:    about the longest request (default: the table's width); the
                   split of the work goes by it, not the result.
        causal:    the queries are the requests' last tokens and see no later one.
        Returns out [tokens, q_heads, head_dim] in bf16, and with return_lse the
        fp32 log-sum-exp [tokens, q_heads] too.  Rows of no request are left as
        they are in `out`."""
        return (_binding or _load_binding()).kv8_attention(
            self.k_codes, self.v_codes, self.k_scale, self.v_scale, q, cu_q, seq_lens,
            block_table, max_q, max_kv, causal, scale, out, return_lse, ws)


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
    workspace status word.  Without `ws`: that of the current stream's workspace,
    or where that is OK the first that is not of the workspaces of captured calls
    on the current device, whichever stream their graphs were replayed on (wait
    for the others first)."""
    if ws is not None:
        return int(N.lib().nvfp4_get_device_status(ws.data_ptr(), _stream()))
    status = device_status(workspace())
    for (idx, _), captured in list(_captured_workspaces.items()):
        if status == N.OK and idx == torch.cuda.current_device():
            status = device_status(captured)
    return status


def set_wait_limit_ns(ns: int) -> None:
    N.lib().nvfp4_set_wait_limit_ns(int(ns))
