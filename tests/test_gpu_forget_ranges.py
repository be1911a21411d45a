"""The rotary write, the scored attention and the eviction where the other tests do
not reach: logits far below a row's maximum, tables and bounds wider than the
sequences, rows behind the last one, empty calls, workspaces of the exact size."""
import numpy as np
import pytest
import torch

import forget_ref as ref
from gpu_helpers import check_close

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from paged_kv_cache_459_b200 import pkv  # noqa: E402
from test_gpu_forget import (BF, BT, NAN, cuda, decode_case, f64, new_err, normal, prefill_case,  # noqa: E402
                             same_bits, score_check, tables_for)


# Scale 4 spreads the logits over several hundred powers of two: keys whose weight the exponential
# rounds to nothing (below 2^-125 on the FMA pipe), keys that take a row alone, parts of a row's keys
# whose maxima lie far apart.  The bounds are the formula's own (logit_bound).
@pytest.mark.parametrize("new,old,hq,hkv,d", [
    ([300] * 20, [0] * 20, 32, 32, 64),      # units whole: tiles of 128 queries, no mask but the diagonal's
    ([1000], [0], 8, 2, 64),                 # queries cut into ranges
    ([260, 131], [500, 0], 4, 4, 128),
    ([64, 5], [6000, 3000], 8, 2, 128),      # few rows over long contexts: keys cut into parts
])
def test_scored_prefill_far_logits(new, old, hq, hkv, d):
    prefill_case(new, old, hq, hkv, d, scale=4.0, seed=len(new) + d)


@pytest.mark.parametrize("variant,part", [(0, 512), (1, 512), (2, 64), (4, 64)])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 128), (14, 2, 64), (20, 2, 128)])
def test_scored_decode_table_wider_than_the_sequences(variant, part, hq, hkv, d):
    decode_case([530, 1, 0, 47], hq, hkv, d, True, True, variant, part, seed=hq, width=700)


def test_scored_prefill_wide_table_few_rows():
    prefill_case([9, 40], [700, 0], 8, 2, 64, window=8, seed=2, width=900)


@pytest.mark.parametrize("max_query_len", [150, 1024])
def test_scored_prefill_bounds_and_rows_past_the_last_sequence(max_query_len):
    """max_query_len is a bound, sequences of the batch may be empty, and rows of q behind the last
    sequence's (a padded batch, as a captured call has) are neither read nor written."""
    hq, hkv, d, pad = 8, 2, 64, 45
    new, old = [0, 150, 1, 0, 37, 0], [0, 20, 333, 50, 0, 0]
    lens = [a + b for a, b in zip(new, old)]
    tables, pool, _ = tables_for(lens, 8)
    kc, vc = normal((pool, hkv, BT, d), 1), normal((pool, hkv, BT, d), 2)
    T, B, W = sum(new), len(new), tables.shape[1]
    q = normal((T + pad, hq, d), 3)
    q[T:] = NAN
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    before = np.random.default_rng(4).random((B, hkv, W * BT)).astype(np.float32)
    out = torch.full_like(q, -3.0)
    sout, err = torch.full((B, hkv, W * BT), -7.0, device="cuda"), new_err()
    pkv.paged_attention_prefill_scored(out, q, kc, vc, cuda(tables), cuda(np.array(lens, np.int32)), cuda(qs), 0.125, hkv,
                                       max_query_len, sout, scores_in=cuda(before), err=err)
    assert int(err.item()) == 0
    assert (out[T:] == -3).all()
    q64, k64 = f64(q[:T]), f64(kc)
    check_close(out[:T].view(torch.int16).cpu().numpy().view(np.uint16),
                ref.attention(q64, qs, k64, f64(vc), tables, lens, 0.125), "padded")
    want = ref.scores(q64, qs, k64, tables, lens, 0.125, before.astype(np.float64))
    for b, n in enumerate(old):
        before[b, :, n:] = 0  # not counted
    got = f64(sout)
    score_check(got, want, before.astype(np.float64), ref.logit_bound(q64, k64, 0.125), max(new) * 4)
    assert (got[np.isnan(want)] == -7.0).all()


def test_empty_calls():
    """No tokens, no sequences: nothing is launched, read or written."""
    e16 = lambda *s: torch.zeros(s, dtype=BF, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    kc, vc = e16(4, 2, BT, 64), e16(4, 2, BT, 64)
    pkv.rope_kv_write(e16(0, 4, 64), e16(0, 4, 64), e16(0, 2, 64), e16(0, 2, 64), kc, vc,
                      torch.zeros(0, dtype=torch.int64, device="cuda"), i32(0), pkv.rope_table(8, 64))
    s = torch.zeros((0, 2, 48), device="cuda")
    pkv.paged_attention_decode_scored(e16(0, 4, 64), e16(0, 4, 64), kc, vc, i32(0, 3), i32(0), 0.1, 2, s)
    pkv.paged_attention_prefill_scored(e16(0, 4, 64), e16(0, 4, 64), kc, vc, i32(0, 3), i32(0), i32(1), 0.1, 2, 0, s)
    pkv.evict_tokens(kc, vc, i32(0, 3), i32(0), i32(0, 2), i32(0), s, torch.zeros((0, 2, 32), device="cuda"), i32(0, 2, 32))
    torch.cuda.synchronize()
    assert not kc.any() and not vc.any()


def test_workspaces_of_the_exact_size():
    """The size that is asked for is enough, and 16 bytes less are refused before any launch."""
    lens, hq, hkv, d = [300, 41], 14, 2, 64
    tables, pool, _ = tables_for(lens, 1)
    W = tables.shape[1]
    kc, vc, q = normal((pool, hkv, BT, d), 1), normal((pool, hkv, BT, d), 2), normal((2, hq, d), 3)
    t, ln = cuda(tables), cuda(np.array(lens, np.int32))
    want, got, out = torch.zeros((2, hkv, W * BT), device="cuda"), torch.zeros((2, hkv, W * BT), device="cuda"), torch.empty_like(q)
    pkv.paged_attention_decode_scored(out, q, kc, vc, t, ln, 0.125, hkv, want)
    n = pkv.decode_scored_workspace_bytes(2, hq, hkv, d, W)
    guard = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda")
    pkv.paged_attention_decode_scored(out, q, kc, vc, t, ln, 0.125, hkv, got, workspace=guard[:n])
    assert same_bits(got, want) and (guard[n:] == 77).all()
    with pytest.raises(pkv.PkvError) as e:
        pkv.paged_attention_decode_scored(out, q, kc, vc, t, ln, 0.125, hkv, got, workspace=guard[:n - 16])
    assert e.value.code == pkv.ERR_WORKSPACE
    # few rows over a longer context: parts and ranges in the workspace
    q, qs = normal((30, hq, d), 5), cuda(np.array([0, 20, 30], np.int32))
    out = torch.empty_like(q)
    pkv.paged_attention_prefill_scored(out, q, kc, vc, t, ln, qs, 0.125, hkv, 20, want)
    n = pkv.prefill_scored_workspace_bytes(30, 2, 20, hq, hkv, d, W)
    guard = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda")
    pkv.paged_attention_prefill_scored(out, q, kc, vc, t, ln, qs, 0.125, hkv, 20, got, workspace=guard[:n])
    assert same_bits(got, want) and (guard[n:] == 77).all()
    with pytest.raises(pkv.PkvError) as e:
        pkv.paged_attention_prefill_scored(out, q, kc, vc, t, ln, qs, 0.125, hkv, 20, got, workspace=guard[:n - 16])
    assert e.value.code == pkv.ERR_WORKSPACE


@pytest.mark.parametrize("hq,hkv", [(4, 4), (14, 2)])
def test_a_captured_decode_step_over_a_wide_table_follows_the_lengths(hq, hkv):
    """Tables as wide as the longest a server allows, lengths advanced on the device between replays."""
    d, W, steps, B = 64, 300, 20, 3
    lens = [15, 200, 1]
    tables, pool, _ = tables_for([n + steps for n in lens], 6, width=W)
    kc, vc, table = normal((pool, hkv, BT, d), 1), normal((pool, hkv, BT, d), 2), cuda(tables)
    k2, v2 = kc.clone(), vc.clone()
    q, kn, vn = (torch.empty((B, h, d), dtype=BF, device="cuda") for h in (hq, hkv, hkv))
    ln = cuda(np.array(lens, np.int32))
    s, out, err = torch.zeros((B, hkv, W * BT), device="cuda"), torch.empty_like(q), new_err()
    new = [normal((steps, B, h, d), 9 + i) for i, h in enumerate((hq, hkv, hkv))]

    def step():
        pkv.paged_attention_decode_scored(out, q, kc, vc, table, ln, 0.125, hkv, s, scores_in=s, k_new=kn, v_new=vn, err=err)

    def load(i):
        for x, y in zip((q, kn, vn), new):
            x.copy_(y[i])

    load(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kc.copy_(k2), vc.copy_(v2), s.zero_()
    s2, o2 = torch.zeros_like(s), torch.empty_like(q)
    total = np.zeros((B, hkv, W * BT))
    for i in range(steps):
        load(i)
        graph.replay()
        pkv.paged_attention_decode_scored(o2, q, k2, v2, table, ln, 0.125, hkv, s2, scores_in=s2, k_new=kn, v_new=vn, err=err)
        assert same_bits(out, o2) and same_bits(s, s2) and same_bits(kc, k2) and same_bits(vc, v2)
        n = np.array(lens) + i
        want = ref.scores(f64(q), np.arange(B + 1), f64(kc), tables, n, 0.125, total)
        total = np.nan_to_num(want)
        ln += 1
    assert int(err.item()) == 0
    # every step's weights within the logits' bound, summed
    bound = ref.logit_bound(f64(new[0]), f64(kc), 0.125)
    assert (np.abs(f64(s) - total) <= (bound + steps * (hq // hkv + 1) * 2.0 ** -23) * total + 1e-30).all()


@pytest.mark.parametrize("extra", [1, 2, 6])
def test_evict_score_rows_of_any_alignment(extra):
    """Rows of scores wider than the table, so that they start off 16-byte boundaries."""
    hkv, d, n, keep = 3, 64, 700, 200
    tables, pool, free = tables_for([n, 90], 3, spare=2 * 13)
    W = tables.shape[1]
    r = np.random.default_rng(extra)
    scores = r.random((2, hkv, W * BT + extra)).astype(np.float32)
    scores[:, :, W * BT:] = np.inf  # past the table: never read
    kc, vc = normal((pool, hkv, BT, d), 1), normal((pool, hkv, BT, d), 2)
    kept = torch.full((2, hkv, 13 * BT), -9, dtype=torch.int32, device="cuda")
    after, err = torch.full((2, hkv, 13 * BT), -7.0, device="cuda"), new_err()
    pkv.evict_tokens(kc, vc, cuda(tables), cuda(np.array([n, 90], np.int32)), cuda(free.reshape(2, 13).astype(np.int32)),
                     cuda(np.array([keep, 64], np.int32)), cuda(scores), after, kept, sink=3, recent=9, err=err)
    assert int(err.item()) == 0
    for b, (m, k) in enumerate(((n, keep), (90, 64))):
        for h in range(hkv):
            c = ref.chosen(scores[b, h], m, k, 3, 9)
            assert np.array_equal(kept[b, h, :k].cpu().numpy(), c) and (kept[b, h, k:] == -9).all()
            assert np.array_equal(after[b, h, :k].cpu().numpy(), scores[b, h, c]) and (after[b, h, k:] == -7).all()
