"""The cache operators together, as a serving program runs them beside the MoE layer: several steps of a
decoder block (plan, append, attention, MoE forward) over prompts, drafts, single tokens and idle
requests, against the oracle's cache and attention; and the same step captured in a graph."""

import numpy as np
import pytest
import torch

import helpers
import kv_helpers as kh
import parity
from nvfp4_weight_quantized_amd import kv, ops
from oracle import kv_cache as okv

pytestmark = pytest.mark.gpu
DEV = "cuda"

HEADS, KV_HEADS, DIM, PAGE = 4, 2, 64, 32
HIDDEN = HEADS * DIM


class Block:
    """A fused query/key/value projection, the cache, and the MoE layer on the attention's output."""

    def __init__(self, requests, num_pages, seed=0):
        rng = np.random.default_rng(seed)
        self.w = torch.randn(HIDDEN, HIDDEN + 2 * KV_HEADS * DIM, device=DEV) * HIDDEN ** -0.5
        self.cache = kv.NvFp4KvCache.allocate(num_pages, PAGE, KV_HEADS, DIM, 0.002, 0.002)
        self.table = torch.full((requests, 12), -1, dtype=torch.int32, device=DEV)
        self.moe = parity.to_gpu_layer(helpers.random_layer(rng, HIDDEN, 128, 8, 2))

    def step(self, x, kv_lens, new_lens, free):
        plan = kv.kv_plan(kv_lens, new_lens, self.table, free, PAGE, self.cache.num_pages, x.shape[0])
        qkv = torch.matmul(x.float(), self.w).to(torch.bfloat16)
        q, k, v = (t.unflatten(1, (-1, DIM)) for t in qkv.split([HIDDEN, KV_HEADS * DIM, KV_HEADS * DIM], dim=1))
        kv.kv_append(self.cache, k, v, plan.slots)
        att = torch.zeros(x.shape[0], HEADS, DIM, dtype=torch.bfloat16, device=DEV)
        kv.kv_attention(self.cache, q, plan.query_offsets, plan.seq_lens, self.table, out=att)
        return plan, (q, k, v), att, ops.forward(self.moe, att.flatten(1))


def _values(t):
    return t.double().cpu().numpy()


def test_steps_of_a_decoder_block_match_the_oracle():
    rng = np.random.default_rng(1)
    block = Block(requests=5, num_pages=40)
    order = torch.from_numpy(rng.permutation(40).astype(np.int32)).to(DEV)
    taken = 0
    lens = np.zeros(5, np.int32)
    pages = okv.new_pages(40, PAGE, KV_HEADS, DIM)
    table = np.full((5, 12), -1, np.int32)
    for step, new in enumerate([[70, 0, 33, 1, 0], [1, 40, 1, 1, 0], [3, 1, 1, 0, 90], [1, 1, 1, 1, 1], [1, 5, 1, 31, 1]]):
        tokens = sum(new) + 2                                  # a padded batch
        x = torch.randn(tokens, HIDDEN, device=DEV).to(torch.bfloat16)
        kv_lens = torch.from_numpy(lens.copy()).to(DEV)
        plan, (q, k, v), att, out = block.step(x, kv_lens, torch.tensor(new, dtype=torch.int32, device=DEV), order[taken:])
        free = order[taken:].cpu().numpy()
        off, after, pos, slots, used, table = okv.plan(lens, new, table, free, PAGE, 40, tokens)
        assert np.array_equal(plan.slots.cpu().numpy(), slots) and np.array_equal(block.table.cpu().numpy(), table)
        okv.append(pages, PAGE, _values(k), slots, 0.002, False)
        okv.append(pages, PAGE, _values(v), slots, 0.002, True)
        assert np.array_equal(block.cache.pages.cpu().numpy(), pages)
        ref, lse, mags = okv.attention(_values(q), pages, PAGE, 0.002, 0.002, off, after, table, DIM ** -0.5)
        n = int(off[-1])
        tol, _ = kh.bounds(ref, lse, mags, slice(0, n), int(after.max()), DIM)
        assert np.all(np.abs(_values(att)[:n] - ref[:n]) <= tol), step
        assert (att[n:] == 0).all() and torch.isfinite(out).all()
        # what the cache hands back is what was stored
        gk, gv = kv.kv_gather(block.cache, plan.slots[:n])
        want = okv.decode(pages, PAGE, slots[:n], 0.002, False)
        assert np.allclose(_values(gk), want, rtol=2.0 ** -8, atol=0)
        lens, taken = after, taken + used


def test_a_step_captured_once_serves_many():
    """Single-token steps replayed from one graph: the plan, the append and the attention read the
    lengths from device tensors; the cache after the replays is the eager program's, byte for byte."""
    x = torch.randn(3, HIDDEN, device=DEV).to(torch.bfloat16)
    free = torch.arange(30, dtype=torch.int32, device=DEV).flip(0).contiguous()
    ones = torch.ones(3, dtype=torch.int32, device=DEV)

    def run(graphed):
        torch.manual_seed(4)
        block = Block(requests=3, num_pages=30)
        kv_lens = torch.tensor([0, 30, 61], dtype=torch.int32, device=DEV)
        block.table[1, 0], block.table[2, :2] = 0, torch.tensor([1, 2], device=DEV)
        inp, head = x.clone(), free.clone()
        outs = []

        def advance(res):
            plan, _, att, out = res
            kv_lens.copy_(plan.seq_lens)
            used = int(plan.pages_used)
            head.copy_(torch.roll(head, -used))
            outs.append((att.clone(), out.clone()))

        if not graphed:
            for i in range(6):
                inp.copy_(x * (i + 1))
                advance(block.step(inp, kv_lens, ones, head))
        else:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):       # warm up on a copy of the state
                keep = block.table.clone()
                block.step(inp, kv_lens, ones, head)
                block.table.copy_(keep)
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                res = block.step(inp, kv_lens, ones, head)
            for i in range(6):
                inp.copy_(x * (i + 1))
                graph.replay()
                torch.cuda.synchronize()
                advance(res)
        return outs, block

    eager, b0 = run(False)
    replay, b1 = run(True)
    for (a, o), (a2, o2) in zip(eager, replay):
        assert torch.equal(a, a2) and torch.equal(o, o2)
    assert torch.equal(b0.table, b1.table)
    # every written position holds the same bytes (the warm-up wrote the first step's rows as well)
    slots = torch.from_numpy(np.concatenate([okv.slots_of(b0.table[r].cpu().numpy(), PAGE, a, a + 6)
                                             for r, a in enumerate((0, 30, 61))]).astype(np.int32)).to(DEV)
    for p, q in zip(kv.kv_gather(b0.cache, slots), kv.kv_gather(b1.cache, slots)):
        assert torch.equal(p, q)
