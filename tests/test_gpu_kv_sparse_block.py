"""The sparse operators together, as a serving program runs them: plan, rotating append, index, choice and attention over
several steps of prompts, drafts, single tokens and idle requests against the oracle, and the same captured in a graph."""

import numpy as np
import pytest
import torch

import kv_helpers as kh
import nvfp4_weight_quantized_amd as moe
from oracle import kv_cache as okv
from oracle import kv_sparse as osp

pytestmark = pytest.mark.gpu
DEV = "cuda"

HEADS, KV_HEADS, DIM, PAGE, TOP_K, PAGES = 8, 2, 64, 32, 4, 60


class Block:
    def __init__(self, requests, width=14):
        self.rot = moe.Rotary.from_theta(DIM, 10000.0, sections=(8, 12, 12))
        self.cache = moe.NvFp4KvCache.allocate(PAGES, PAGE, KV_HEADS, DIM, 0.002, 0.002)
        self.index = moe.NvFp4KvIndex.allocate(self.cache)
        self.table = torch.full((requests, width), -1, dtype=torch.int32, device=DEV)

    def step(self, fused, positions3, kv_lens, new_lens, free):
        t = fused.shape[0]
        plan = moe.kv_plan(kv_lens, new_lens, self.table, free, PAGE, PAGES, t)
        q, k, v = fused.split([HEADS, KV_HEADS, KV_HEADS], dim=1)
        # text: every axis holds the plan's positions; images add their own
        q = moe.kv_append_rotary(self.cache, self.rot, q, k, v, plan.positions + positions3, plan.slots)
        args = (plan.query_offsets, plan.seq_lens, self.table)
        moe.kv_index_update(self.cache, self.index, *args, t)
        chosen = moe.kv_select(self.index, q, *args, TOP_K)
        return plan, q, chosen, moe.kv_sparse_attention(self.cache, q, *args, chosen)


def _values(t):
    return t.double().cpu().numpy()


def test_steps_match_the_oracle():
    rng = np.random.default_rng(1)
    block = Block(5)
    order = torch.from_numpy(rng.permutation(PAGES).astype(np.int32)).to(DEV)
    taken, lens = 0, np.zeros(5, np.int32)
    pages = okv.new_pages(PAGES, PAGE, KV_HEADS, DIM)
    codes, scales = np.zeros((PAGES, KV_HEADS, DIM), np.int8), np.zeros((PAGES, KV_HEADS), np.float32)
    for new in ([300, 0, 233, 1, 0], [1, 240, 1, 1, 0], [3, 1, 1, 0, 190], [1, 1, 1, 1, 1], [1, 5, 1, 31, 1]):
        tokens = sum(new) + 2                                  # a padded batch
        fused = kh.to_bf16(kh.bf16(rng, (tokens, HEADS + 2 * KV_HEADS, DIM)))
        extra = torch.from_numpy(rng.integers(0, 16, (3, tokens)).astype(np.int32)).to(DEV)
        plan, q, chosen, out = block.step(fused, extra, torch.from_numpy(lens.copy()).to(DEV),
                                          torch.tensor(new, dtype=torch.int32, device=DEV), order[taken:])
        pos = plan.positions + extra
        assert torch.equal(q, moe.rotary(block.rot, fused[:, :HEADS], pos))
        k = moe.rotary(block.rot, fused[:, HEADS:HEADS + KV_HEADS], pos)
        slots, table = plan.slots.cpu().numpy(), block.table.cpu().numpy()
        okv.append(pages, PAGE, _values(k), slots, 0.002, False)
        okv.append(pages, PAGE, _values(fused[:, HEADS + KV_HEADS:]), slots, 0.002, True)
        assert np.array_equal(block.cache.pages.cpu().numpy(), pages)
        off, after = plan.query_offsets.cpu().numpy(), plan.seq_lens.cpu().numpy()
        osp.index_update(codes, scales, pages, PAGE, off, after, table, tokens)
        assert np.array_equal(block.index.codes.cpu().numpy(), codes)
        assert np.array_equal(block.index.scales.cpu().numpy(), scales)
        want = osp.select(_values(q), codes, scales, PAGE, off, after, table, TOP_K)
        assert np.array_equal(chosen.cpu().numpy(), want)
        ref, lse, mags = osp.attention(_values(q), pages, PAGE, 0.002, 0.002, off, after, table, want, DIM ** -0.5)
        n = int(off[-1])
        tol, _ = kh.bounds(ref, lse, mags, slice(0, n), TOP_K * PAGE, DIM)
        assert np.all(np.abs(_values(out)[:n] - ref[:n]) <= tol)
        assert (out[n:] == 0).all() and (chosen[n:] == -1).all()
        lens, taken = after, taken + int(plan.pages_used)


def test_a_step_captured_once_serves_many():
    """Single tokens over contexts that cross pages, replayed from one graph with eager work between: the eager
    program's lists, rows, pages and index."""
    rng = np.random.default_rng(2)
    base = [kh.to_bf16(kh.bf16(rng, (3, HEADS + 2 * KV_HEADS, DIM))) for _ in range(5)]
    start = kh.to_bf16(kh.bf16(rng, (391, HEADS + 2 * KV_HEADS, DIM)))
    free = torch.arange(PAGES, dtype=torch.int32, device=DEV).flip(0).contiguous()
    ones = torch.ones(3, dtype=torch.int32, device=DEV)
    first = torch.tensor([200, 31, 160], dtype=torch.int32, device=DEV)

    def run(graphed):
        block = Block(3)
        lens = torch.zeros(3, dtype=torch.int32, device=DEV)
        plan, *_ = block.step(start, torch.zeros(3, 391, dtype=torch.int32, device=DEV), lens, first, free)
        lens.copy_(plan.seq_lens)
        head = free.roll(-int(plan.pages_used)).contiguous()
        inp, extra = base[0].clone(), torch.zeros(3, 3, dtype=torch.int32, device=DEV)
        if graphed:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            keep = block.table.clone()
            with torch.cuda.stream(side):
                block.step(inp, extra, lens, ones, head)      # warm up; the first replay writes the same again
                block.table.copy_(keep)
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                res = block.step(inp, extra, lens, ones, head)
        outs = []
        for x in base:
            inp.copy_(x)
            if graphed:
                graph.replay()
                torch.cuda.synchronize()
            else:
                res = block.step(inp, extra, lens, ones, head)
            plan, q, chosen, out = res
            outs.append((q.clone(), chosen.clone(), out.clone()))
            lens.copy_(plan.seq_lens)
            head.copy_(head.roll(-int(plan.pages_used)))
        return outs, block

    eager, b0 = run(False)
    replay, b1 = run(True)
    for x, y in zip(eager, replay):
        assert all(torch.equal(a, b) for a, b in zip(x, y))
    assert torch.equal(b0.table, b1.table) and torch.equal(b0.index.codes, b1.index.codes)
    assert torch.equal(b0.index.scales, b1.index.scales) and torch.equal(b0.cache.pages, b1.cache.pages)
