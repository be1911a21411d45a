"""Calls back to back on one stream, as a captured step runs them: each grid is
resident while the one before it still writes (programmatic dependent launches),
and must see all that it wrote.  The same calls one at a time, the GPU idle in
between, give the bits to compare with."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from paged_kv_cache_459_b200 import pkv  # noqa: E402
from test_gpu_forget import BF, BT, cuda, new_err, normal, same_bits, tables_for  # noqa: E402

STEPS = 24


class Chain:
    """Per step: a rotary write into shared q and slots, a scored decode over one workspace with the
    scores in place, an eviction by them.  Every step has inputs of its own."""

    def __init__(self, hq, hkv, d, variant, seed):
        lens = [300, 41, 129, 16]
        B = len(lens)
        tables, pool, free = tables_for(lens, seed, spare=20)
        W = tables.shape[1]
        self.hkv, self.d, self.variant = hkv, d, variant
        self.tables, self.lens = cuda(tables), cuda(np.array(lens, np.int32))
        slots = [int(tables[b, (n - 1) // BT]) * BT + (n - 1) % BT for b, n in enumerate(lens)]
        self.slots = cuda(np.array(slots, np.int64))
        self.new_tables = cuda(np.array(free[:4 * B], np.int32).reshape(B, 4))
        self.keep = cuda(np.array([60, 30, 64, 16], np.int32))
        self.kc, self.vc = normal((pool, hkv, BT, d), seed + 1), normal((pool, hkv, BT, d), seed + 2)
        self.qkv = normal((STEPS, B, hq + 2 * hkv, d), seed + 3)
        self.positions = cuda(np.random.default_rng(seed).integers(0, 4096, (STEPS, B)).astype(np.int32))
        self.table = pkv.rope_table(4096, d)
        self.q = torch.zeros((B, hq, d), dtype=BF, device="cuda")
        self.hq = hq
        self.scores = torch.rand((B, hkv, W * BT), device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
        self.ws = torch.zeros(pkv.decode_scored_workspace_bytes(B, hq, hkv, d, W, 64), dtype=torch.uint8, device="cuda")
        self.out = torch.zeros((STEPS, B, hq, d), dtype=BF, device="cuda")
        self.after = torch.zeros((STEPS, B, hkv, 4 * BT), device="cuda")
        self.kept = torch.zeros((STEPS, B, hkv, 4 * BT), dtype=torch.int32, device="cuda")
        self.err = new_err()

    def run(self, between=lambda: None):
        hq, hkv = self.hq, self.hkv
        for i in range(STEPS):
            x = self.qkv[i]
            pkv.rope_kv_write(self.q, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], self.kc, self.vc, self.slots,
                              self.positions[i], self.table, err=self.err)
            between()
            pkv.paged_attention_decode_scored(self.out[i], self.q, self.kc, self.vc, self.tables, self.lens, self.d ** -0.5,
                                              hkv, self.scores, scores_in=self.scores, variant=self.variant,
                                              partition_tokens=64, workspace=self.ws, err=self.err)
            between()
            pkv.evict_tokens(self.kc, self.vc, self.tables, self.lens, self.new_tables, self.keep, self.scores,
                             self.after[i], self.kept[i], sink=2, recent=4, err=self.err)
            between()

    def results(self):
        return [t.clone() for t in (self.out, self.after, self.kept, self.scores, self.kc, self.vc)]


@pytest.mark.parametrize("variant", [pkv.DECODE_SINGLE, pkv.DECODE_SPLIT, pkv.DECODE_CLUSTER])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (14, 2, 128)])
def test_steps_back_to_back_are_the_steps_one_at_a_time(variant, hq, hkv, d):
    one = Chain(hq, hkv, d, variant, seed=3)
    one.run(torch.cuda.synchronize)
    want = one.results()
    assert not same_bits(want[0][0], want[0][1]) and not same_bits(want[1][0], want[1][1])  # no step repeats another
    eager = Chain(hq, hkv, d, variant, seed=3)
    eager.run()
    torch.cuda.synchronize()
    graphed = Chain(hq, hkv, d, variant, seed=3)
    start = [t.clone() for t in (graphed.q, graphed.scores, graphed.kc, graphed.vc)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.run()
    for _ in range(5):
        for t, s in zip((graphed.q, graphed.scores, graphed.kc, graphed.vc), start):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(graphed.results(), want))
    assert all(same_bits(a, b) for a, b in zip(eager.results(), want))
    assert int(one.err.item()) == int(eager.err.item()) == int(graphed.err.item()) == 0


class Prompts:
    """Per step: a scored prefill of other queries into one score buffer, an eviction by them."""

    def __init__(self, lens, hq, hkv, d, steps, seed):
        B = len(lens)
        self.tables_, pool, free = tables_for(lens, seed, spare=2 * B)
        self.tables, self.lens = cuda(self.tables_), cuda(np.array(lens, np.int32))
        self.new_tables = cuda(np.array(free[:2 * B], np.int32).reshape(B, 2))
        self.keep = cuda(np.array([min(n, 27) for n in lens], np.int32))
        self.start = cuda(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))
        self.kc, self.vc = normal((pool, hkv, BT, d), seed + 1), normal((pool, hkv, BT, d), seed + 2)
        self.q = normal((steps, sum(lens), hq, d), seed + 3)
        self.hkv, self.d, self.steps, self.longest = hkv, d, steps, max(lens)
        self.scores = torch.zeros((B, hkv, self.tables.shape[1] * BT), device="cuda")
        n = pkv.prefill_scored_workspace_bytes(sum(lens), B, max(lens), hq, hkv, d, self.tables.shape[1])
        self.ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.after = torch.zeros((steps, B, hkv, 2 * BT), device="cuda")
        self.kept = torch.zeros((steps, B, hkv, 2 * BT), dtype=torch.int32, device="cuda")
        self.err = new_err()

    def run(self, between=lambda: None):
        for i in range(self.steps):
            pkv.paged_attention_prefill_scored(self.out[i], self.q[i], self.kc, self.vc, self.tables, self.lens, self.start,
                                               self.d ** -0.5, self.hkv, self.longest, self.scores, workspace=self.ws,
                                               err=self.err)
            between()
            pkv.evict_tokens(self.kc, self.vc, self.tables, self.lens, self.new_tables, self.keep, self.scores,
                             self.after[i], self.kept[i], sink=1, recent=4, err=self.err)
            between()

    def results(self):
        return [t.clone() for t in (self.out, self.after, self.kept, self.scores, self.kc, self.vc)]


@pytest.mark.parametrize("lens,hq,hkv,steps", [
    ([150, 33, 1], 8, 2, 12),     # the scores joined from ranges of queries, then the eviction
    ([300] * 20, 32, 32, 3),      # the eviction right behind the scores
])
def test_evictions_right_behind_scored_prefills(lens, hq, hkv, steps):
    one = Prompts(lens, hq, hkv, 64, steps, seed=5)
    one.run(torch.cuda.synchronize)
    want = one.results()
    assert not same_bits(want[1][0], want[1][1]) and not same_bits(want[2][0], want[2][1])
    graphed = Prompts(lens, hq, hkv, 64, steps, seed=5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.run()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(graphed.results(), want))
    assert int(one.err.item()) == int(graphed.err.item()) == 0


def test_scored_prefills_on_two_streams_beside_decode_steps():
    """Two captured prompts and the decode chain on streams of their own: tensor memory, the places of
    waiting grids and scratch are shared by nobody to anybody's harm."""
    cases = [Prompts([150, 33, 1], 8, 2, 64, 4, seed=1), Prompts([260, 129], 4, 4, 64, 4, seed=2),
             Chain(14, 2, 128, pkv.DECODE_SPLIT, seed=3)]
    start = [t.clone() for t in (cases[2].q, cases[2].scores, cases[2].kc, cases[2].vc)]
    want = []
    for c in cases:
        c.run(torch.cuda.synchronize)
        want.append(c.results())
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(6):
        for t, s in zip((cases[2].q, cases[2].scores, cases[2].kc, cases[2].vc), start):
            t.copy_(s)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert all(same_bits(a, b) for a, b in zip(c.results(), w)) and int(c.err.item()) == 0
