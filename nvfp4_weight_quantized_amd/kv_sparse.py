"""torch-facing wrappers of sparse attention over the paged NVFP4 key/value cache: argument checks and marshalling only.

One step of an attention layer whose rows read a few pages of long contexts, after ``kv_append``:

    kv_index_update(cache, index, plan.query_offsets, plan.seq_lens, block_table, num_tokens)
    chosen = kv_select(index, q, plan.query_offsets, plan.seq_lens, block_table, top_k)
    out = kv_sparse_attention(cache, q, plan.query_offsets, plan.seq_lens, block_table, chosen)

Every call only enqueues kernels on the current stream of its tensors' device and can be captured in a HIP graph.
"""

from __future__ import annotations

import functools
import math
from typing import Optional

import torch

from . import _lib as L
from .kv import _BF16, _I32, _I32_END, _UNIT, HEAD_DIMS, NvFp4KvCache, _ints, _on, _raw_stream, _rows
from .ops import _need, _same_device, _shape

MAX_SELECTED = 1024          # pages chosen for a row
MAX_SELECT_WIDTH = 16384     # columns of a block table that a choice looks at


class NvFp4KvIndex:
    """8-bit means of the keys of a cache's pages, one attention layer's: what ``kv_select`` chooses by.

    ``codes`` int8 [num_pages, kv_heads, head_dim] and ``scales`` float32 [num_pages, kv_heads], contiguous; the mean of
    a page's keys is code * scale * k_gscale.  ``kv_index_update`` fills them; the content for pages that no request
    holds does not matter.  All of them are fixed for the life of the object.
    """
    __slots__ = ("_codes", "_scales", "_struct", "_dev")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, page_size: int):
        _need(codes, "codes", torch.int8, 3)
        _need(scales, "scales", torch.float32, 2)
        p, h, d = codes.shape
        _shape(scales, "scales", (p, h))
        _same_device(codes, ("scales", scales))
        if d not in HEAD_DIMS:
            raise ValueError(f"codes: head_dim {d}, expected one of {HEAD_DIMS}")
        if codes.data_ptr() % 16:
            raise ValueError("codes: must start at a 16-byte boundary")
        if not (0 < page_size <= 65536 and page_size % _UNIT == 0 and 0 < h <= 1024 and 0 < p * page_size < _I32_END):
            raise ValueError(f"codes: {p} pages of {page_size} positions, {h} heads: outside the cache's limits")
        self._codes, self._scales, self._dev = codes, scales, codes.device
        self._struct = L.KvIndex(p, page_size, h, d, codes.data_ptr(), scales.data_ptr())

    @classmethod
    def allocate(cls, cache: NvFp4KvCache) -> "NvFp4KvIndex":
        """An index of zeros for a cache's pages."""
        p, h, d = cache.num_pages, cache.kv_heads, cache.head_dim
        return cls(torch.zeros(p, h, d, dtype=torch.int8, device=cache._dev),
                   torch.zeros(p, h, dtype=torch.float32, device=cache._dev), cache.page_size)

    @property
    def codes(self) -> torch.Tensor:
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        return self._scales

    @property
    def page_size(self) -> int:
        return self._struct.page_size

    @property
    def num_pages(self) -> int:
        return self._struct.num_pages

    @property
    def kv_heads(self) -> int:
        return self._struct.kv_heads

    @property
    def head_dim(self) -> int:
        return self._struct.head_dim


def _step(query_offsets, seq_lens, block_table, dev):
    """Checks a step's index tensors: (requests, table width)."""
    _ints(query_offsets, "query_offsets", 1, dev)
    _ints(seq_lens, "seq_lens", 1, dev)
    _ints(block_table, "block_table", 2, dev)
    r = seq_lens.shape[0]
    rows, width = block_table.shape
    if query_offsets.shape[0] != r + 1:
        _shape(query_offsets, "query_offsets", (r + 1,))
    if rows != r:
        raise ValueError(f"block_table: {rows} rows for {r} requests")
    return r, width


def kv_index_update(cache: NvFp4KvCache, index: NvFp4KvIndex, query_offsets: torch.Tensor, seq_lens: torch.Tensor,
                    block_table: torch.Tensor, num_tokens: int) -> None:
    """Bring the index of every page that holds a row of the step up to what the cache holds now (append first).

    Request r's rows are its last query_offsets[r+1] - query_offsets[r] positions; ``num_tokens`` is the row count of the
    step's tensors.  With offsets that count whole lengths it builds the index of a cache filled earlier.  A physical
    page is touched by one request of a call.
    """
    c, x, dev = cache._struct, index._struct, cache._dev
    if index._dev != dev or (x.num_pages, x.page_size, x.kv_heads, x.head_dim) != (c.num_pages, c.page_size, c.kv_heads,
                                                                                   c.head_dim):
        raise ValueError("index: not of the cache's sizes and device")
    r, width = _step(query_offsets, seq_lens, block_table, dev)
    if not 0 <= num_tokens < _I32_END:
        raise ValueError(f"num_tokens {num_tokens}")
    with _on(dev.index):
        st = L.lib().moe_nvfp4_kv_index_update(c, x, query_offsets.data_ptr(), seq_lens.data_ptr(), r,
                                               block_table.data_ptr(), width, num_tokens, _raw_stream(dev.index))
    if st:
        L.check("moe_nvfp4_kv_index_update", st)


def kv_select(index: NvFp4KvIndex, q: torch.Tensor, query_offsets: torch.Tensor, seq_lens: torch.Tensor,
              block_table: torch.Tensor, top_k: int, first: int = 1, last: int = 1) -> torch.Tensor:
    """The pages that each query row (bf16 [T, heads, head_dim], as for ``kv_attention``) reads -> int32
    [T, kv_heads, top_k]: columns of the block table, ascending, -1 behind them.

    A row chooses among the pages up to its own position: always the ``first`` first and the ``last`` last of them (its
    own among these), and of the others those with the highest products of the kv head's query rows with the pages' means,
    in 8-bit integers (include/moe_nvfp4.h), equal ones the lowest page first.  Rows of no request get -1 only.

    The launch makes room for every column of ``block_table``, however short the requests: for steps of many rows a table of
    1024 columns or fewer is the fast one, and one of 16384 takes several times as long.
    """
    x, dev = index._struct, index._dev
    t, heads, stride = _rows(q, "q", x.head_dim, dev)
    kv_heads = x.kv_heads
    if heads % kv_heads or not 1 <= heads // kv_heads <= 64:
        raise ValueError(f"q: {heads} heads are no multiple (1 to 64) of the index's {kv_heads}")
    r, width = _step(query_offsets, seq_lens, block_table, dev)
    if width > MAX_SELECT_WIDTH:
        raise ValueError(f"block_table: {width} columns, at most {MAX_SELECT_WIDTH} expected")
    if not (first >= 0 and last >= 1 and first + last <= top_k <= MAX_SELECTED):
        raise ValueError(f"top_k {top_k}, first {first}, last {last}: expected first >= 0, last >= 1 and first + last <= "
                         f"top_k <= {MAX_SELECTED}")
    selected = torch.empty(t, kv_heads, top_k, dtype=_I32, device=dev)
    with _on(dev.index):
        st = L.lib().moe_nvfp4_kv_select(x, q.data_ptr(), stride, t, heads, query_offsets.data_ptr(),
                                         seq_lens.data_ptr(), r, block_table.data_ptr(), width, top_k, first, last,
                                         selected.data_ptr(), _raw_stream(dev.index))
    if st:
        L.check("moe_nvfp4_kv_select", st)
    return selected


@functools.lru_cache(maxsize=1024)      # a call's sizes come again every step
def kv_sparse_attention_workspace_size(T: int, R: int, heads: int, kv_heads: int, head_dim: int, page_size: int,
                                       top_k: int) -> int:
    """Workspace bytes of ``kv_sparse_attention`` for T query rows of R requests."""
    return int(L.lib().moe_nvfp4_kv_sparse_attention_workspace_size(T, R, heads, kv_heads, head_dim, page_size, top_k))


def kv_sparse_attention(cache: NvFp4KvCache, q: torch.Tensor, query_offsets: torch.Tensor, seq_lens: torch.Tensor,
                        block_table: torch.Tensor, selected: torch.Tensor, scale: Optional[float] = None,
                        return_lse: bool = False, out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None):
    """``kv_attention`` (without a window) over the pages in ``selected`` only -> bf16 [T, heads, head_dim].

    ``selected`` int32 [T, kv_heads, top_k]: the columns of the block table that each token's rows of a kv head read, in
    ascending order, negative ones behind them (as ``kv_select`` returns them).  A page listed twice counts once; of the
    row's own page the positions up to its own are seen, pages behind it not at all.  A row that sees nothing gets zeros
    and an ``lse`` of -inf.  Everything else is as for ``kv_attention``, ``workspace`` included
    (``kv_sparse_attention_workspace_size`` bytes; none is needed for steps of many rows).
    """
    c, dev = cache._struct, cache._dev
    dim, kv_heads = c.head_dim, c.kv_heads
    t, heads, stride = _rows(q, "q", dim, dev)
    if heads % kv_heads or not 1 <= heads // kv_heads <= 64:
        raise ValueError(f"q: {heads} heads are no multiple (1 to 64) of the cache's {kv_heads}")
    r, width = _step(query_offsets, seq_lens, block_table, dev)
    _ints(selected, "selected", 3, dev)
    st_, sh, top_k = selected.shape
    if st_ != t or sh != kv_heads or not 1 <= top_k <= MAX_SELECTED:
        raise ValueError(f"selected: expected ({t}, {kv_heads}, 1 to {MAX_SELECTED}), got {tuple(selected.shape)}")
    if scale is None:
        scale = dim ** -0.5
    if not (scale > 0.0 and math.isfinite(scale)):
        raise ValueError(f"scale must be finite and positive, got {scale!r}")
    lib, lse = L.lib(), None
    if out is None:
        attend = lib.moe_nvfp4_kv_sparse_attention_fill
        out = torch.empty_like(q) if q.is_contiguous() else torch.empty(t, heads, dim, dtype=_BF16, device=dev)
        if return_lse:
            lse = torch.empty(t, heads, dtype=torch.float32, device=dev)
    else:
        attend = lib.moe_nvfp4_kv_sparse_attention
        _need(out, "out", _BF16, 3)
        _shape(out, "out", (t, heads, dim))
        _same_device(cache._pages, ("out", out))
        if return_lse:
            lse = torch.full((t, heads), -math.inf, dtype=torch.float32, device=dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8)
        _same_device(cache._pages, ("workspace", workspace))
    else:
        need = kv_sparse_attention_workspace_size(t, r, heads, kv_heads, dim, c.page_size, top_k)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    with _on(dev.index):
        st = attend(c, q.data_ptr(), stride, t, heads, query_offsets.data_ptr(), seq_lens.data_ptr(), r,
                    block_table.data_ptr(), width, selected.data_ptr(), top_k, scale, out.data_ptr(),
                    lse.data_ptr() if return_lse else None, workspace.data_ptr() if workspace is not None else None,
                    workspace.numel() if workspace is not None else 0, _raw_stream(dev.index))
    if st:
        L.check("moe_nvfp4_kv_sparse_attention", st)
    return (out, lse) if return_lse else out
