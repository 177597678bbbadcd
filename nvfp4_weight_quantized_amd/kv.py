"""torch-facing wrappers of the paged NVFP4 key/value cache: argument checks and marshalling only.

One decode or prefill step of an attention layer, on tensors of one GPU:

    plan = kv_plan(kv_lens, new_lens, block_table, free_pages, page_size, num_pages, num_tokens)
    kv_append(cache, k, v, plan.slots)                       # per layer: quantize the new rows
    out = kv_attention(cache, q, plan.query_offsets, plan.seq_lens, block_table)

The plan holds for every layer of the step (all layers share the block table).  Every call only
enqueues kernels on the current stream of its tensors' device and can be captured in a HIP graph.
"""

from __future__ import annotations

import contextlib
import math
from typing import NamedTuple, Optional

import torch

from . import _lib as L
from .ops import _need, _same_device, _shape

_UNIT = 32              # positions per unit of a page
HEAD_DIMS = (64, 128, 256)


_I32, _BF16 = torch.int32, torch.bfloat16
_NOTHING = contextlib.nullcontext()
_I32_END = 2 ** 31


def _public_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# Device index -> hipStream_t, and the current device.  The names that torch's own generated code calls take 0.06 and
# 0.12 us, the public ones 1.14 and 0.23 us (a call has 10 to 20 us of host time); a torch without the former (a CPU
# build) takes the latter.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(index: int):
    """The context in which a launch goes to GPU ``index`` (nothing to do on the current one)."""
    return _NOTHING if _current_device() == index else torch.cuda.device(index)


def _ints(t: torch.Tensor, name: str, ndim: int, dev: Optional[torch.device] = None) -> torch.device:
    """A contiguous int32 GPU tensor (on ``dev``, when given); its device."""
    if not (isinstance(t, torch.Tensor) and t.dtype is _I32 and t.dim() == ndim and t.is_contiguous()):
        _need(t, name, _I32, ndim)
    d = t.device
    if d != dev:
        if dev is not None:
            raise ValueError(f"{name}: on {d}, expected {dev}")
        if d.type != "cuda":
            raise ValueError(f"{name}: must be a GPU tensor")
    return d


class NvFp4KvCache:
    """Pages of keys and values in NVFP4 (layout: include/moe_nvfp4.h), one attention layer's.

    ``pages`` uint8 [num_pages, kv_heads, page_size / 32, 36 * head_dim], contiguous; ``page_size``
    positions per page (a multiple of 32); ``k_gscale`` and ``v_gscale`` the dequant global scales
    (a cached element is e2m1 * e4m3 * gscale).  The content of new pages does not matter: positions
    past a request's length are never used.  All of them are fixed for the life of the object.
    """
    __slots__ = ("_pages", "_struct", "_dev")

    def __init__(self, pages: torch.Tensor, page_size: int, k_gscale: float = 1.0, v_gscale: float = 1.0):
        _need(pages, "pages", torch.uint8, 4)
        p, h, u, b = pages.shape
        if b % 36 or b // 36 not in HEAD_DIMS:
            raise ValueError(f"pages: last dimension {b}, expected 36 * head_dim with head_dim in {HEAD_DIMS}")
        if page_size % _UNIT or page_size != u * _UNIT:
            raise ValueError(f"pages: {u} units of {_UNIT} positions do not make a page of {page_size}")
        if not (0 < page_size <= 65536 and 0 < h <= 1024 and 0 < p * page_size < _I32_END):
            raise ValueError(f"pages: sizes {tuple(pages.shape)} outside the cache's limits")
        for name, d in (("k_gscale", k_gscale), ("v_gscale", v_gscale)):
            if not 2.0 ** -64 <= d <= 2.0 ** 64:      # also refuses NaN
                raise ValueError(f"{name}: a dequant global scale lies in [2^-64, 2^64], got {d!r}")
        self._pages = pages
        self._struct = L.KvCache(p, page_size, h, b // 36, k_gscale, v_gscale, pages.data_ptr())
        self._dev = pages.device

    @classmethod
    def allocate(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int, k_gscale: float = 1.0,
                 v_gscale: float = 1.0, device="cuda") -> "NvFp4KvCache":
        """A cache of ``num_pages`` new pages."""
        if head_dim not in HEAD_DIMS or page_size <= 0 or page_size % _UNIT:
            raise ValueError(f"head_dim in {HEAD_DIMS} and page_size a multiple of {_UNIT} expected")
        return cls(torch.zeros(num_pages, kv_heads, page_size // _UNIT, 36 * head_dim, dtype=torch.uint8,
                               device=device), page_size, k_gscale, v_gscale)

    @property
    def pages(self) -> torch.Tensor:
        return self._pages

    @property
    def page_size(self) -> int:
        return self._struct.page_size

    @property
    def k_gscale(self) -> float:
        return self._struct.k_gscale

    @property
    def v_gscale(self) -> float:
        return self._struct.v_gscale

    @property
    def num_pages(self) -> int:
        return self._struct.num_pages

    @property
    def kv_heads(self) -> int:
        return self._struct.kv_heads

    @property
    def head_dim(self) -> int:
        return self._struct.head_dim


class KvPlan(NamedTuple):
    """One step's index tensors (int32): offsets [R+1], lengths after the step [R], positions and slots
    [num_tokens] (0 and -1 past the last token), and the number of free pages the step takes [1]."""
    query_offsets: torch.Tensor
    seq_lens: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor
    pages_used: torch.Tensor


def kv_plan(kv_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
            page_size: int, num_pages: int, num_tokens: int) -> KvPlan:
    """Plan a step: requests hold ``kv_lens`` positions and add ``new_lens`` tokens (int32 [R]).

    Pages that open are taken from ``free_pages`` (int32) in order and entered into ``block_table``
    (int32 [R, width], in place).  ``num_tokens`` is the row count of the step's tensors; it may exceed
    the sum of ``new_lens`` (a padded batch).  A shortage shows in ``pages_used`` > len(free_pages) and
    in slots of -1, which the append skips.
    """
    dev = _ints(kv_lens, "kv_lens", 1)
    _ints(new_lens, "new_lens", 1, dev)
    _ints(block_table, "block_table", 2, dev)
    _ints(free_pages, "free_pages", 1, dev)
    r = kv_lens.shape[0]
    rows, width = block_table.shape
    if new_lens.shape[0] != r:
        _shape(new_lens, "new_lens", (r,))
    if rows != r:
        raise ValueError(f"block_table: {rows} rows for {r} requests")
    if not 0 <= num_tokens < _I32_END:
        raise ValueError(f"num_tokens {num_tokens}")
    if page_size <= 0 or num_pages <= 0 or page_size * num_pages >= _I32_END:
        raise ValueError(f"{num_pages} pages of {page_size} positions")
    # one allocation for the outputs
    sizes = (r + 1, r, num_tokens, num_tokens, 1)
    buf = torch.empty(2 * r + 2 * num_tokens + 2, dtype=_I32, device=dev)
    at = buf.data_ptr()
    with _on(dev.index):
        st = L.lib().moe_kv_plan(
            kv_lens.data_ptr(), new_lens.data_ptr(), r, page_size, num_pages, free_pages.data_ptr(),
            free_pages.shape[0], block_table.data_ptr(), width, num_tokens, at, at + 4 * (r + 1),
            at + 4 * (2 * r + 1), at + 4 * (2 * r + 1 + num_tokens), at + 4 * (2 * r + 1 + 2 * num_tokens),
            _raw_stream(dev.index))
    if st:
        L.check("moe_kv_plan", st)
    return KvPlan(*buf.split_with_sizes(sizes))


def _rows(t: torch.Tensor, name: str, dim: int, dev: torch.device):
    """Token rows [T, heads, dim] bf16: heads contiguous, any token stride of a multiple of 8 elements.
    (T, heads, token stride)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16:
        raise TypeError(f"{name}: expected a bfloat16 tensor")
    if t.dim() != 3 or t.shape[2] != dim:
        raise ValueError(f"{name}: expected [tokens, heads, {dim}], got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name}: on {t.device}, expected {dev}")
    tokens, heads, _ = t.shape
    s0, s1, s2 = t.stride()
    if tokens:
        if s2 != 1 or (heads > 1 and s1 != dim):
            raise ValueError(f"{name}: heads must be contiguous, got strides {(s0, s1, s2)}")
        if tokens > 1 and (s0 < heads * dim or s0 % 8):
            raise ValueError(f"{name}: token stride {s0}, expected a multiple of 8 of at least {heads * dim}")
        if t.data_ptr() % 16:
            raise ValueError(f"{name}: rows must start at 16-byte boundaries")
    return tokens, heads, s0


def kv_append(cache: NvFp4KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantize rows k, v (bf16 [T, kv_heads, head_dim]) into the cache at ``slots`` (int32 [T]).

    Slots outside the cache (-1: a padded row) are skipped; slots of one call must be distinct.  k and v
    may be slices of a fused projection's output (contiguous heads, any token stride that is a multiple
    of 8).
    """
    c, dev = cache._struct, cache._dev
    kt, kh, ks = _rows(k, "k", c.head_dim, dev)
    vt, vh, vs = _rows(v, "v", c.head_dim, dev)
    _ints(slots, "slots", 1, dev)
    t, h = slots.shape[0], c.kv_heads
    if kt != t or kh != h or vt != t or vh != h:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)}: expected {(t, h, c.head_dim)}")
    with _on(dev.index):
        st = L.lib().moe_nvfp4_kv_append(c, k.data_ptr(), v.data_ptr(), ks, vs, slots.data_ptr(), t,
                                         _raw_stream(dev.index))
    if st:
        L.check("moe_nvfp4_kv_append", st)


def kv_gather(cache: NvFp4KvCache, slots: torch.Tensor):
    """Dequantize the rows at ``slots`` (int32 [n]): (k, v), each bf16 [n, kv_heads, head_dim].

    A slot outside the cache gives a NaN row.
    """
    c, dev = cache._struct, cache._dev
    _ints(slots, "slots", 1, dev)
    n = slots.shape[0]
    k, v = torch.empty(2, n, c.kv_heads, c.head_dim, dtype=_BF16, device=dev).unbind(0)
    with _on(dev.index):
        st = L.lib().moe_nvfp4_kv_gather(c, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), _raw_stream(dev.index))
    if st:
        L.check("moe_nvfp4_kv_gather", st)
    return k, v


def kv_attention_workspace_size(T: int, R: int, heads: int, kv_heads: int, head_dim: int) -> int:
    """Workspace bytes of ``kv_attention`` for T query rows of R requests."""
    return int(L.lib().moe_nvfp4_kv_attention_workspace_size(T, R, heads, kv_heads, head_dim))


def kv_attention(cache: NvFp4KvCache, q: torch.Tensor, query_offsets: torch.Tensor, seq_lens: torch.Tensor,
                 block_table: torch.Tensor, scale: Optional[float] = None, window: int = 0,
                 return_lse: bool = False, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None):
    """Causal attention of query rows q (bf16 [T, heads, head_dim]) over the cache -> bf16 [T, heads, head_dim].

    Rows [query_offsets[r], query_offsets[r+1]) are the last rows of request r, whose cache holds
    ``seq_lens[r]`` positions (these rows' included: append first).  A row sees the positions up to its
    own, with ``window`` > 0 only the last ``window`` of them.  ``scale`` defaults to head_dim^-0.5.
    ``return_lse``: also the natural log-sum-exp of each row's scores, fp32 [T, heads] (-inf for a row
    that sees nothing, whose output is zero).  Rows outside every request (a padded batch) are left as
    they were in a given ``out`` and zeros without it; their ``lse`` is -inf.  q may be a slice of a fused
    projection's output.  Without ``workspace`` the call takes one from torch's allocator where it needs
    one, so calls on several streams do not share it.  ``out`` and ``workspace`` overlap no other argument.
    """
    c, dev = cache._struct, cache._dev
    dim, kv_heads = c.head_dim, c.kv_heads
    t, heads, stride = _rows(q, "q", dim, dev)
    if heads % kv_heads or not 1 <= heads // kv_heads <= 64:
        raise ValueError(f"q: {heads} heads are no multiple (1 to 64) of the cache's {kv_heads}")
    _ints(query_offsets, "query_offsets", 1, dev)
    _ints(seq_lens, "seq_lens", 1, dev)
    _ints(block_table, "block_table", 2, dev)
    r = seq_lens.shape[0]
    rows, width = block_table.shape
    if query_offsets.shape[0] != r + 1:
        _shape(query_offsets, "query_offsets", (r + 1,))
    if rows != r:
        raise ValueError(f"block_table: {rows} rows for {r} requests")
    if scale is None:
        scale = dim ** -0.5
    if not (scale > 0.0 and math.isfinite(scale)):
        raise ValueError(f"scale must be finite and positive, got {scale!r}")
    if not 0 <= window < _I32_END:
        raise ValueError(f"window {window}")
    lib, lse = L.lib(), None
    if out is None:
        attend = lib.moe_nvfp4_kv_attention_fill
        out = torch.empty_like(q) if q.is_contiguous() else torch.empty((t, heads, dim), dtype=_BF16, device=dev)
        if return_lse:
            lse = torch.empty((t, heads), dtype=torch.float32, device=dev)
    else:
        attend = lib.moe_nvfp4_kv_attention
        _need(out, "out", _BF16, 3)
        _shape(out, "out", (t, heads, dim))
        _same_device(cache._pages, ("out", out))
        if return_lse:
            lse = torch.full((t, heads), -math.inf, dtype=torch.float32, device=dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8)
        _same_device(cache._pages, ("workspace", workspace))
    with _on(dev.index):
        while True:
            st = attend(
                c, q.data_ptr(), stride, t, heads, query_offsets.data_ptr(), seq_lens.data_ptr(), r,
                block_table.data_ptr(), width, scale, window, out.data_ptr(), lse.data_ptr() if return_lse else None,
                workspace.data_ptr() if workspace is not None else None,
                workspace.numel() if workspace is not None else 0, _raw_stream(dev.index))
            if st != L.MOE_ERR_WORKSPACE_TOO_SMALL or workspace is not None:
                break
            # short tables need none; nothing has been enqueued
            workspace = torch.empty(lib.moe_nvfp4_kv_attention_workspace_size(t, r, heads, kv_heads, dim),
                                    dtype=torch.uint8, device=dev)
    if st:
        L.check("moe_nvfp4_kv_attention", st)
    return (out, lse) if return_lse else out
