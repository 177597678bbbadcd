"""torch-facing wrappers of rotary positions: argument checks and marshalling only.

    rot = Rotary.from_theta(128, 500000.0)                               # text
    rot = Rotary.from_theta(128, 1000000.0, sections=(16, 24, 24))       # time, height, width
    q = rotary(rot, q, positions)                                        # rows on their own
    q = kv_append_rotary(cache, rot, q, k, v, plan.positions, plan.slots)     # on their way into the cache

Every call only enqueues kernels on the current stream of its tensors' device and can be captured in a HIP graph.
"""

from __future__ import annotations

import math
from typing import Optional, Sequence

import torch

from . import _lib as L
from .kv import NvFp4KvCache, _ints, _on, _raw_stream, _rows
from .ops import _need

_I32, _F64 = torch.int32, torch.float64


class Rotary:
    """Frequencies of rotary positions and what each pair of elements turns by.

    ``inv_freq`` float64 [pairs] on the GPU: pair i of a head turns by position * inv_freq[i], formed in 64 bits
    (magnitudes up to 256).  Pair i is elements (i, pairs + i) of the head, or with ``interleaved`` (2i, 2i + 1);
    elements from 2 * pairs on pass unchanged.  With ``num_axes`` > 1 (time, height, width of images and video) positions
    have a row per axis, and ``axes`` (int32 [pairs] on the GPU) holds each pair's row.  ``scale`` multiplies cosines and
    sines.  All of them are fixed for the life of the object.
    """
    __slots__ = ("_inv_freq", "_axes", "_struct", "_dev")

    def __init__(self, inv_freq: torch.Tensor, head_dim: int, axes: Optional[torch.Tensor] = None, num_axes: int = 1,
                 interleaved: bool = False, scale: float = 1.0):
        _need(inv_freq, "inv_freq", _F64, 1)
        pairs = inv_freq.shape[0]
        if head_dim % 16 or not 16 <= head_dim <= 512:
            raise ValueError(f"head_dim {head_dim}: a multiple of 16 up to 512 expected")
        if pairs % 8 or not 8 <= pairs <= head_dim // 2:
            raise ValueError(f"inv_freq: {pairs} pairs, expected a multiple of 8 up to {head_dim // 2}")
        if not 1 <= num_axes <= 4:
            raise ValueError(f"num_axes {num_axes}: 1 to 4 expected")
        if axes is not None:
            _need(axes, "axes", _I32, 1)
            if axes.shape[0] != pairs:
                raise ValueError(f"axes: {axes.shape[0]} entries for {pairs} pairs")
            if axes.device != inv_freq.device:
                raise ValueError(f"axes: on {axes.device}, expected {inv_freq.device}")
        elif num_axes > 1:
            raise ValueError(f"axes: needed for {num_axes} axes")
        if not math.isfinite(scale):
            raise ValueError(f"scale must be finite, got {scale!r}")
        self._inv_freq, self._axes, self._dev = inv_freq, axes, inv_freq.device
        self._struct = L.RotaryStruct(head_dim, pairs, num_axes, int(bool(interleaved)), scale, inv_freq.data_ptr(),
                                      axes.data_ptr() if axes is not None else None)

    @classmethod
    def from_theta(cls, head_dim: int, theta: float = 10000.0, rotary_dim: Optional[int] = None,
                   sections: Optional[Sequence[int]] = None, spread: bool = False, interleaved: bool = False,
                   scale: float = 1.0, device="cuda") -> "Rotary":
        """inv_freq[i] = theta^(-i / pairs) over the first ``rotary_dim`` elements of a head (default: all).

        ``sections``: pairs of each axis.  They lie one axis after the other, or with ``spread`` in turn (axis 0, 1, 2,
        0, 1, ...) for as long as an axis has pairs left, the first axis taking the rest.
        """
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        if rotary_dim % 2 or not theta > 0.0 or not math.isfinite(theta):
            raise ValueError(f"rotary_dim {rotary_dim} and theta {theta!r}: an even and a positive number expected")
        pairs = rotary_dim // 2
        freq = torch.tensor([theta ** (-i / pairs) for i in range(pairs)], dtype=_F64)
        axes, n = None, 1
        if sections is not None:
            n = len(sections)
            if any(s < 0 for s in sections) or sum(sections) != pairs:
                raise ValueError(f"sections {tuple(sections)}: expected parts of {pairs} pairs")
            order = [a for a, s in enumerate(sections) for _ in range(s)]
            if spread:
                order = [0] * pairs
                for a in range(1, n):
                    at = range(a, n * sections[a], n)
                    if at and at[-1] >= pairs:
                        raise ValueError(f"sections {tuple(sections)}: axis {a} does not fit {pairs} pairs in turn")
                    for i in at:
                        order[i] = a
            axes = torch.tensor(order, dtype=_I32).to(device)
        return cls(freq.to(device), head_dim, axes, n, interleaved, scale)

    @property
    def inv_freq(self) -> torch.Tensor:
        return self._inv_freq

    @property
    def axes(self) -> Optional[torch.Tensor]:
        return self._axes

    @property
    def num_axes(self) -> int:
        return self._struct.axes

    @property
    def head_dim(self) -> int:
        return self._struct.head_dim

    @property
    def pairs(self) -> int:
        return self._struct.pairs


def _positions(rot: Rotary, positions: torch.Tensor, tokens: int) -> int:
    """int32 [tokens] or [num_axes, tokens] on the rotary's device; elements from axis to axis."""
    if not isinstance(positions, torch.Tensor) or positions.dtype is not _I32:
        raise TypeError("positions: expected an int32 tensor")
    if positions.device != rot._dev:
        raise ValueError(f"positions: on {positions.device}, expected {rot._dev}")
    n, shape = rot._struct.axes, positions.shape
    if not (positions.dim() == 1 and n == 1 or positions.dim() == 2 and shape[0] == n) or shape[-1] != tokens:
        raise ValueError(f"positions: expected {(n, tokens) if n > 1 else (tokens,)}, got {tuple(shape)}")
    if tokens > 1 and positions.stride(-1) != 1:
        raise ValueError("positions: the tokens must be contiguous")
    axis = positions.stride(0) if n > 1 else tokens
    if axis < tokens:
        raise ValueError(f"positions: {axis} elements from axis to axis for {tokens} tokens")
    return axis


def _out(out: Optional[torch.Tensor], x: torch.Tensor, name: str, shape, dim: int, dev: torch.device):
    """A new tensor, or a given one that is checked: (tensor, token stride)."""
    tokens, heads = shape
    if out is None:
        return (torch.empty_like(x) if x.is_contiguous() else
                torch.empty(tokens, heads, dim, dtype=torch.bfloat16, device=dev)), heads * dim
    t, h, stride = _rows(out, "out", dim, dev)
    if t != tokens or h != heads:
        raise ValueError(f"out: expected {(tokens, heads, dim)}, got {tuple(out.shape)}")
    if tokens > 1 and out.data_ptr() == x.data_ptr() and stride != x.stride(0):
        raise ValueError(f"out: the rows of {name} with another token stride")
    return out, stride


def rotary(rot: Rotary, x: torch.Tensor, positions: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotate rows x (bf16 [T, heads, head_dim]) by ``positions`` (int32 [T], or [num_axes, T]) -> bf16 rows.

    x and ``out`` may be slices of a fused projection's output (contiguous heads, any token stride that is a multiple of
    8); ``out`` may be x itself, and otherwise overlaps no other argument.
    """
    r, dev = rot._struct, rot._dev
    t, heads, stride = _rows(x, "x", r.head_dim, dev)
    axis = _positions(rot, positions, t)
    out, out_stride = _out(out, x, "x", (t, heads), r.head_dim, dev)
    if t and heads:
        with _on(dev.index):
            st = L.lib().moe_rotary(r, x.data_ptr(), stride, t, heads, positions.data_ptr(), axis, out.data_ptr(),
                                    out_stride, _raw_stream(dev.index))
        if st:
            L.check("moe_rotary", st)
    return out


def kv_append_rotary(cache: NvFp4KvCache, rot: Rotary, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     positions: torch.Tensor, slots: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A step's rows in one launch: q rotated (returned), k rotated and quantized, v quantized into the cache.

    The same as ``rotary`` of q and of k, then ``kv_append`` at ``slots`` (int32 [T]; -1: a padded row, whose q is still
    rotated).  q, k and v (bf16 [T, heads, head_dim]) may be slices of a fused projection's output; ``out`` may be q
    itself, and otherwise overlaps no other argument.
    """
    c, r, dev = cache._struct, rot._struct, cache._dev
    if rot._dev != dev or r.head_dim != c.head_dim:
        raise ValueError(f"rotary: of head_dim {r.head_dim} on {rot._dev}, the cache of {c.head_dim} on {dev}")
    dim = c.head_dim
    qt, heads, qs = _rows(q, "q", dim, dev)
    kt, kh, ks = _rows(k, "k", dim, dev)
    vt, vh, vs = _rows(v, "v", dim, dev)
    _ints(slots, "slots", 1, dev)
    t, h = slots.shape[0], c.kv_heads
    if kt != t or kh != h or vt != t or vh != h:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)}: expected {(t, h, dim)}")
    if qt != t or heads < 1:
        raise ValueError(f"q {tuple(q.shape)}: expected {t} rows")
    axis = _positions(rot, positions, t)
    out, out_stride = _out(out, q, "q", (t, heads), dim, dev)
    with _on(dev.index):
        st = L.lib().moe_nvfp4_kv_append_rotary(c, r, q.data_ptr(), qs, heads, k.data_ptr(), ks, v.data_ptr(), vs,
                                                positions.data_ptr(), axis, slots.data_ptr(), t, out.data_ptr(),
                                                out_stride, _raw_stream(dev.index))
    if st:
        L.check("moe_nvfp4_kv_append_rotary", st)
    return out
