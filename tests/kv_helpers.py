"""Test-side glue of the key/value cache tests: random caches built by the oracle, the tolerances, and
uploads (never used by the product path)."""

from __future__ import annotations

import numpy as np
import torch

from nvfp4_weight_quantized_amd import kv
from oracle import kv_cache as okv
from oracle import moe as omoe
from oracle import w4a4 as oa4

DEV = "cuda"


def bf16(rng, shape, sigma=1.0) -> np.ndarray:
    """Random values that are bf16-exact, as float64."""
    return omoe.bf16_to_float(oa4.float_to_bf16_bits(rng.normal(0, sigma, shape)))


def to_bf16(values, device=DEV) -> torch.Tensor:
    """bf16-exact float64 values -> a bf16 tensor."""
    t = torch.from_numpy(np.ascontiguousarray(values)).to(torch.bfloat16)
    assert np.array_equal(t.double().numpy(), values, equal_nan=True)
    return t.to(device)


class Case:
    """A cache of random requests: per request (new, old) lengths, shuffled pages, oracle-quantized rows.

    Every byte that belongs to no position of a request (past the lengths, spare pages) is ``fill``:
    0xFF puts NaN scales and -6 codes there.
    """

    def __init__(self, seed, dim, kv_heads, group, page, reqs, window=0, fill=0xFF, spare=2, d_k=0.0371, d_v=0.0113,
                 sigma_k=1.0, sigma_q=1.0, pad=0, width_extra=1):
        rng = np.random.default_rng(seed)
        self.dim, self.kv_heads, self.heads, self.page, self.window = dim, kv_heads, kv_heads * group, page, window
        self.d_k, self.d_v = float(np.float32(d_k)), float(np.float32(d_v))
        new = [n for n, _ in reqs]
        self.lens = np.array([n + o for n, o in reqs], np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.tokens = int(self.offsets[-1]) + pad
        need = [-(-int(n) // page) for n in self.lens]
        total = sum(need) + spare
        perm = rng.permutation(total).astype(np.int32)
        self.table = np.full((len(reqs), max(need + [0]) + width_extra), -7, np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = perm[at:at + n]
            at += n
        self.pages = okv.new_pages(total, page, kv_heads, dim, fill)
        for r in range(len(reqs)):
            if self.lens[r] == 0:
                continue
            slots = okv.slots_of(self.table[r], page, 0, int(self.lens[r]))
            okv.append(self.pages, page, bf16(rng, (len(slots), kv_heads, dim), sigma_k), slots, self.d_k, False)
            okv.append(self.pages, page, bf16(rng, (len(slots), kv_heads, dim)), slots, self.d_v, True)
        self.q = bf16(rng, (self.tokens, self.heads, dim), sigma_q)
        self.scale = float(np.float32(dim ** -0.5))

    def cache(self) -> kv.NvFp4KvCache:
        return kv.NvFp4KvCache(torch.from_numpy(self.pages).to(DEV), self.page, self.d_k, self.d_v)

    def args(self):
        return (torch.from_numpy(self.offsets).to(DEV), torch.from_numpy(self.lens).to(DEV),
                torch.from_numpy(self.table).to(DEV))

    def run(self, cache=None, **kw):
        return kv.kv_attention(cache or self.cache(), to_bf16(self.q), *self.args(), scale=self.scale,
                               window=self.window, return_lse=True, **kw)

    def reference(self):
        return okv.attention(self.q, self.pages, self.page, self.d_k, self.d_v, self.offsets, self.lens, self.table,
                             self.scale, self.window)


def bounds(ref_out, ref_lse, mags, sel, lens_max, dim):
    """Elementwise bounds on |gpu - exact| of (out, lse), from the arithmetic of the kernels.

    Scores: D exact products summed in fp32 (at most D + 8 roundings of partial sums, each at most
    2^-24 of sum|q k|), times the scale and the base-2 constant, minus the running maximum (4 more):
    ds = (D + 12) 2^-24 mag, absolute, in a score; p = exp2 of it (hardware exponential, at most 2 ulp:
    2^-22) is then off by ds + 2^-22 relatively, numerator and denominator alike: 2 (ds + 2^-22).
    p is rounded to fp16 for the value product only: 2^-11 relative down to fp16's smallest normal
    value, below it half a subnormal step, 2^-25; p carries a factor of at least 2^7 at the row's
    largest score, so that step is at most 2^-32 of the largest p, for each position: 2^-32 sum|v| / sum p.  Values are exact; N + 64 fp32
    additions (keys, partial sums, rescales) each lose at most 2^-24 of the sum of magnitudes, in
    numerator and denominator.  out is rounded to bf16 once: 2^-8 relative (half a step).
    """
    ref_out, ref_lse = ref_out[sel], ref_lse[sel]
    terms, plain, mag = (m[sel] for m in mags)
    ds = (dim + 12) * 2.0 ** -24 * mag
    rel = 2.0 ** -11 + 2 * (ds + 2.0 ** -22) + 2 * (lens_max + 64) * 2.0 ** -24
    tol_out = np.abs(ref_out) * 2.0 ** -8 + (1 + 2.0 ** -8) * terms * rel[..., None] + 2.0 ** -32 * plain + 2.0 ** -126
    # lse = ln2 (m + log2 l): ds, the exponential, the additions, and 4 roundings of the result
    finite = np.where(np.isfinite(ref_lse), np.abs(ref_lse), 0.0)
    tol_lse = ds + 2.0 ** -22 + (lens_max + 64) * 2.0 ** -24 + 4 * 2.0 ** -24 * (finite + mag + 1)
    return tol_out, tol_lse


def check_attention(case: Case, out, lse, rows=None):
    """GPU (out, lse) of a case against the oracle, within the derived bounds."""
    ref, ref_lse, mags = case.reference()
    n = int(case.offsets[-1])
    sel = slice(0, n) if rows is None else rows
    got = out.double().cpu().numpy()[sel]
    got_lse = lse.double().cpu().numpy()[sel]
    tol_out, tol_lse = bounds(ref, ref_lse, mags, sel, int(case.lens.max()), case.dim)
    ref, ref_lse = ref[sel], ref_lse[sel]
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    assert np.all(got[empty] == 0.0)
    over = np.abs(got - ref) / tol_out
    assert np.all(over <= 1.0), f"out: {np.nanmax(over)} times the bound"
    lse_over = np.abs(got_lse[~empty] - ref_lse[~empty]) / tol_lse[~empty]
    assert np.all(lse_over <= 1.0), f"lse: {lse_over.max()} times the bound"
