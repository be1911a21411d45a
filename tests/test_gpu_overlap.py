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
