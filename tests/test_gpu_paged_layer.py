"""The caches in pages as a serving loop uses them: a prompt compressed and appended, forked into samples, decoded token by token
(reserve, compress, append, index scores, selection, attention), a sample dropped, the pool compacted; and a
decode step captured in a graph."""

import math

import numpy as np
import pytest
import torch

from oracle import csa_oracle as O
from oracle import paged_oracle as PO
from tests.parity import check_topk, np64
from tests.test_gpu_attn8 import check_close, reference

pytestmark = pytest.mark.gpu

RATIO, D, DI, HI, H, W, TOPK, PAGE, BLOCK = 4, 512, 128, 64, 128, 32, 24, 16, 8


@pytest.fixture(scope="module")
def ops():
    from long_context_decode_c4a_b200 import ops
    return ops


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """`slots` requests of one layer behind one page table."""

    def __init__(self, ops, slots, num_pages, max_tokens):
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.ops, self.R = ops, slots
        self.book = ops.PageTable.empty(slots, -(-(max_tokens // RATIO + 1) // PAGE), num_pages, PAGE)
        self.main, self.index = ops.PagedCache.e4m3(self.book, BLOCK), ops.PagedCache.bf16(self.book, DI)
        self.cfg, self.icfg = ops.compressor_cfg(RATIO, D), ops.compressor_cfg(RATIO, DI)
        self.state = [torch.empty(slots, 2 * RATIO, 2 * D, **bf) for _ in range(2)] + [torch.empty(slots, 2 * RATIO, 2 * DI, **bf) for _ in range(2)]
        ops.state_reset(self.cfg, *self.state[:2])
        ops.state_reset(self.icfg, *self.state[2:])
        n = max_tokens // RATIO + 1
        self.rows, self.irows = torch.zeros(slots, n, D, **bf), torch.zeros(slots, n, DI, **bf)   # where compress() leaves entries
        self.ring = torch.zeros(slots, W, D, **bf)
        self.gamma, self.igamma = torch.ones(D, **bf), torch.ones(DI, **bf)
        self.ws_i = ops.workspace(ops._lib.CSA_WS_INDEXER_TOPK, slots, 1, self.book.max_entries, TOPK)
        self.ws_a = ops.workspace(ops._lib.CSA_WS_SPARSE_ATTN, slots, 1, 1, 1)

    def take(self, start, S, x):
        """The segment's entries into the pages; x: the compressor's streams."""
        ops = self.ops
        ops.pages_reserve(self.book, torch.div(start.clamp(min=0) + S, RATIO, rounding_mode="floor").to(torch.int32) * (start >= 0))
        ops.compress(self.cfg, start, x["kv"], x["score"], self.gamma, *self.state[:2], self.rows)
        ops.compress(self.icfg, start, x["ikv"], x["iscore"], self.igamma, *self.state[2:], self.irows)
        ops.cache_append(self.main, start, S, self.rows, RATIO)
        ops.cache_append(self.index, start, S, self.irows, RATIO)

    def decode(self, pos, x):
        """One token of every slot (pos < 0: none)."""
        ops = self.ops
        self.take(pos, 1, x)
        live = pos >= 0
        self.ring[torch.arange(self.R, device="cuda"), (pos.clamp(min=0) % W).long()] = torch.where(live[:, None], x["win"], self.ring[:, 0])
        q_pos = pos.view(-1, 1)
        idx = ops.indexer_topk_paged(q_pos, x["q_idx"], x["w"], self.index, TOPK, ws=self.ws_i)
        return idx, ops.sparse_attn8(q_pos, x["q"], self.ring, self.main, idx, x["sink"], W, ws=self.ws_a)


def streams(g, B, S):
    bf = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q = torch.randn(B, 1, H, D, generator=g, device="cuda")
    return dict(kv=bf(B, S, 2 * D), score=bf(B, S, 2 * D), ikv=bf(B, S, 2 * DI), iscore=bf(B, S, 2 * DI), win=bf(B, D), q_idx=bf(B, 1, HI, DI),
                w=torch.randn(B, 1, HI, generator=g, device="cuda") / 8, q=(q * torch.rsqrt(q.square().mean(-1, keepdim=True))).to(torch.bfloat16),
                sink=torch.randn(H, generator=g, device="cuda"))


def test_prompts_samples_and_decode(ops):
    g = torch.Generator(device="cuda").manual_seed(7)
    s = Server(ops, 4, 40, 400)
    # two prompts, in slots 0 and 1, of different lengths: the longer one's segment first, then both
    n = [150, 101]
    x = streams(g, 4, 49)
    s.take(i32([0, -1, -1, -1]), 49, x)
    x2 = streams(g, 4, 101)
    s.take(i32([49, 0, -1, -1]), 101, x2)
    entries = [n[0] // RATIO, n[1] // RATIO, 0, 0]
    assert ops.device_status(s.book.ws) == 0
    # what the pages hold is what the compressor left, quantised as the oracle does
    codes, scales = np.zeros((40, PAGE, D)), np.zeros((40, PAGE // BLOCK))
    table = s.book.table.tolist()
    PO.append(codes, scales, table[0], PAGE, BLOCK, 0, 49 // RATIO, np64(s.rows[0]))
    PO.append(codes, scales, table[0], PAGE, BLOCK, 49 // RATIO, n[0] // RATIO, np64(s.rows[0]))
    PO.append(codes, scales, table[1], PAGE, BLOCK, 0, n[1] // RATIO, np64(s.rows[1]))
    assert np.array_equal(np64(s.main.pages.float()), codes) and np.array_equal(np64(s.main.scales), scales)
    # slot 0 twice more, slot 1 stays: three samples share the first prompt's full pages
    refs = s.book.refs.tolist()
    ref_table = [list(r) for r in table]
    PO.fork(ref_table, refs, PAGE, [0, 1, 0, 0], entries)
    ops.pages_fork(s.book, [s.main, s.index], i32([0, 1, 0, 0]), i32(entries))
    assert s.book.table.tolist() == ref_table and s.book.refs.tolist() == refs
    for t in s.state + [s.rows, s.irows, s.ring]:
        t[2:] = t[0]
    pos = [n[0], n[1], n[0], n[0]]
    for step in range(13):
        if step == 7:   # sample 2 ends; its pages are freed and the pool compacted
            now = [p // RATIO for p in pos]
            ops.pages_fork(s.book, [s.main, s.index], i32([0, 1, -1, 3]), i32([e if r != 2 else 0 for r, e in enumerate(now)]))
            _, live = ops.pages_compact(s.book, [s.main, s.index])
            assert live.item() == len({p for row in s.book.table.tolist() for p in row if p >= 0})
            assert max(p for row in s.book.table.tolist() for p in row) < live.item()
            pos[2] = -1
        x = streams(g, 4, 1)
        idx, out = s.decode(i32(pos), x)
        vis = [(p + 1) // RATIO if p >= 0 else 0 for p in pos]
        E = max(vis)
        want = torch.stack([torch.where(torch.arange(E) < v, torch.arange(E), torch.tensor(-1)) for v in vis]).to(torch.int32).cuda()
        vals, keys = np64(ops.cache_read(s.main, want)), np64(ops.cache_read(s.index, want))
        entry = s.main.scales.repeat_interleave(BLOCK, 1).cpu()
        for r in range(4):
            if pos[r] < 0:
                assert (out[r] == 0).all()
                continue
            # this slot's own entries, whatever it shared: the compressor's rows, within the step of their block
            sc = np.array([entry[s.book.table[r, e // PAGE].item(), e % PAGE].item() for e in range(vis[r])])
            assert np.array_equal(keys[r, : vis[r]], np64(s.irows[r, : vis[r]]))
            rows = np64(s.rows[r, : vis[r]])
            # one rounding of 4 bits (2^-4) or two where the block's step grew, subnormals to 2^-10 of the scale each
            assert (np.abs(vals[r, : vis[r]] - rows) <= 2 * (2.0 ** -4 * np.abs(rows) + 2.0 ** -10 * sc[:, None])).all()
            sel = check_topk(np64(idx[r, 0]), O.indexer_scores(np64(x["q_idx"][r, 0]), np64(x["w"][r, 0]), keys[r], vis[r]), TOPK)
            ref, tol, _ = reference(np64(x["q"][r, 0]), pos[r], W, np64(s.ring[r]), vals[r], sc, sel.tolist(), np64(x["sink"]), 1 / math.sqrt(D), 64, 10000.0)
            check_close(out[r, 0], ref, tol, f"step {step} slot {r}")
        pos = [p + 1 if p >= 0 else p for p in pos]
    for ws in (s.book.ws, s.ws_i, s.ws_a):
        assert ops.device_status(ws) == 0


def test_a_captured_step(ops):
    """The whole decode step in a graph, replayed on new tokens and beside another server's graph, as eager steps would go."""
    g = torch.Generator(device="cuda").manual_seed(8)
    n, steps = 90, 6
    prompt, tokens = streams(g, 3, n), [streams(g, 3, 1) for _ in range(steps)]
    servers, outs = [Server(ops, 3, 60, 200) for _ in range(3)], []
    for s in servers:
        s.take(i32([0, 0, -1]), n, prompt)
    eager = []
    for k in range(steps):
        idx, out = servers[0].decode(i32([n + k, n + k, -1]), tokens[k])
        eager.append((idx.clone(), out.clone()))
    torch.cuda.synchronize()
    graphs = []
    for s in servers[1:]:
        x, pos = {k: v.clone() for k, v in tokens[0].items()}, i32([n, n, -1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = s.decode(pos, x)
        graphs.append((graph, x, pos, res, torch.cuda.Stream()))
    for k in range(steps):
        for graph, x, pos, res, stream in graphs:
            for name, v in x.items():
                v.copy_(tokens[k][name])
            pos.copy_(i32([n + k, n + k, -1]))
        torch.cuda.synchronize()
        for graph, x, pos, res, stream in graphs:   # both at once
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for graph, x, pos, res, stream in graphs:
            assert torch.equal(res[0], eager[k][0]) and torch.equal(res[1], eager[k][1])
    for s in servers[1:]:
        assert torch.equal(s.book.table, servers[0].book.table)
        assert torch.equal(s.main.pages.view(torch.uint8), servers[0].main.pages.view(torch.uint8)) and torch.equal(s.main.scales, servers[0].main.scales)
        for ws in (s.book.ws, s.ws_i, s.ws_a):
            assert ops.device_status(ws) == 0
