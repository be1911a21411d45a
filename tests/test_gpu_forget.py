"""The rotary write, the scored attention and the eviction on the GPU, against
their formulas in 64 bits (forget_ref.py)."""
import numpy as np
import pytest
import torch

import forget_ref as ref
from gpu_helpers import check_close

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

from paged_kv_cache_459_b200 import pkv  # noqa: E402

BT = 16
BF = torch.bfloat16
NAN = float("nan")


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def same_bits(a, b):
    return torch.equal(bits(a), bits(b))


def normal(shape, seed):
    return torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(BF)


def new_err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def tables_for(lens, seed, spare=6, width=None):
    r = np.random.default_rng(seed)
    need = [-(-int(n) // BT) for n in lens]
    pool = sum(need) + spare
    ids = r.permutation(pool)
    t = np.full((len(lens), width or max(1, max(need))), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = ids[at:at + k]
        at += k
    return t, pool, ids[at:]


def poison_tails(cache, tables, lens):
    """NaN in the slots past each sequence's end, as leftovers may be."""
    for b, n in enumerate(lens):
        if n % BT:
            cache[int(tables[b, n // BT]), :, n % BT:] = NAN


# ------------------------------------------------------------------ rotary write

def rope_case(T, hq, hkv, d, rot, axes, inter, fused, seed, in_place=False):
    r = np.random.default_rng(seed)
    if fused:
        qkv = normal((T, hq + 2 * hkv, d), seed)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = normal((T, hq, d), seed), normal((T, hkv, d), seed + 1), normal((T, hkv, d), seed + 2)
    maxp = 4096
    table = pkv.rope_table(maxp, rot)
    pos = r.integers(0, maxp, (axes, T))
    pair_axis = r.integers(0, axes, rot // 2).tolist()
    pool = -(-T // BT) + 3
    slots = r.permutation(pool * BT)[:T]
    slots[r.random(T) < 0.2] = -1
    kc, vc = normal((pool, hkv, BT, d), seed + 3), normal((pool, hkv, BT, d), seed + 4)
    k0, v0 = f64(kc), f64(vc)
    want_q = ref.rotate(f64(q), pos, table.cpu().numpy(), pair_axis, inter)
    want_k = ref.rotate(f64(k), pos, table.cpu().numpy(), pair_axis, inter)
    q64, k64, v64 = f64(q), f64(k), f64(v)
    out = q if in_place else torch.full((T, hq, d), NAN, dtype=BF, device="cuda")
    err = new_err()
    positions = cuda((pos[0] if axes == 1 else pos).astype(np.int32))
    pkv.rope_kv_write(out, q, k, v, kc, vc, cuda(slots.astype(np.int64)), positions, table,
                      pair_axis=None if axes == 1 else pair_axis, interleaved=inter, err=err)
    assert int(err.item()) == 0
    # bf16 rounding of the result, and fp32 roundings of its two products and their sum
    def close(got, want, x):
        size = np.abs(x).max(-1, keepdims=True) * 2
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -22 * size).all()
    close(f64(out), want_q, q64)
    live = slots >= 0
    blk, off = slots[live] // BT, slots[live] % BT
    got_k, got_v = f64(kc), f64(vc)
    close(got_k[blk, :, off], want_k[live], k64[live])
    assert np.array_equal(got_v[blk, :, off], v64[live])
    # elements past rot are copies, and nothing else in the caches moved
    assert np.array_equal(f64(out)[..., rot:], q64[..., rot:])
    k0[blk, :, off], v0[blk, :, off] = got_k[blk, :, off], got_v[blk, :, off]
    assert np.array_equal(k0, got_k) and np.array_equal(v0, got_v)


@pytest.mark.parametrize("T,hq,hkv,d,rot,axes,inter,fused", [
    (1, 1, 1, 64, 64, 1, False, False),
    (1, 32, 32, 128, 128, 1, False, False),
    (37, 28, 4, 128, 128, 3, False, True),
    (37, 7, 1, 128, 64, 2, True, True),
    (130, 5, 5, 64, 48, 4, False, False),
    (130, 12, 3, 64, 16, 1, True, True),
    (1000, 8, 2, 128, 112, 3, True, False),
    (4099, 32, 8, 128, 128, 1, False, True),
])
def test_rope_write(T, hq, hkv, d, rot, axes, inter, fused):
    rope_case(T, hq, hkv, d, rot, axes, inter, fused, seed=T + rot)


def test_rope_write_in_place():
    rope_case(70, 8, 2, 128, 128, 3, False, True, seed=3, in_place=True)
    rope_case(70, 8, 2, 64, 32, 1, True, False, seed=4, in_place=True)


def test_rope_write_leaves_out_tokens_with_bad_positions_and_slots():
    T, hq, hkv, d = 6, 4, 2, 64
    q, k, v = normal((T, hq, d), 1), normal((T, hkv, d), 2), normal((T, hkv, d), 3)
    kc, vc = normal((2, hkv, BT, d), 4), normal((2, hkv, BT, d), 5)
    k0 = kc.clone()
    table = pkv.rope_table(100, d)
    out = torch.zeros_like(q)
    err = new_err()
    pos = cuda(np.array([0, 99, 100, -1, 5, 6], np.int32))
    slots = cuda(np.array([0, 1, 2, 3, 32, 1 << 40], np.int64))
    pkv.rope_kv_write(out, q, k, v, kc, vc, slots, pos, table, err=err)
    assert int(err.item()) == pkv.DEV_ERR_BAD_POS | pkv.DEV_ERR_BAD_SLOT
    assert not out[2:4].any()            # no q row for a bad position
    assert out[4].any() and out[5].any()  # q is turned where only the slot is bad
    k0[0, :, :2] = kc[0, :, :2]
    assert torch.equal(k0, kc)


def test_rope_write_is_kv_write_at_position_zero():
    """cos 1, sin 0: q and the cache as a plain copy leaves them, bit for bit."""
    T, hq, hkv, d = 50, 4, 4, 128
    q, k, v = normal((T, hq, d), 1), normal((T, hkv, d), 2), normal((T, hkv, d), 3)
    caches = [torch.zeros((5, hkv, BT, d), dtype=BF, device="cuda") for _ in range(4)]
    slots = cuda(np.random.default_rng(0).permutation(80)[:T].astype(np.int64))
    out = torch.empty_like(q)
    pkv.rope_kv_write(out, q, k, v, caches[0], caches[1], slots, torch.zeros(T, dtype=torch.int32, device="cuda"),
                      pkv.rope_table(8, d))
    pkv.paged_kv_write(k, v, caches[2], caches[3], slots)
    assert same_bits(out, q) and same_bits(caches[0], caches[2]) and same_bits(caches[1], caches[3])


# ------------------------------------------------------------------ scored decode

def score_check(got, want, before, bound, tokens):
    """Weights within `bound` of what they are, beside the sums' own fp32 roundings
    (2^-24 for each of up to `tokens` terms and the old score)."""
    there = ~np.isnan(want)
    old = 0 if before is None else np.nan_to_num(before)  # NaN: never read
    added = np.where(there, want, 0) - old
    tol = bound * np.abs(added) + 2.0 ** -23 * np.abs(np.where(there, want, 0)) + tokens * 2.0 ** -24 * np.abs(added)
    bad = there & ~(np.abs(got - np.where(there, want, 0)) <= tol + 1e-30)
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def decode_case(lens, hq, hkv, d, write, with_old, variant=0, part=512, seed=0, scale=None, width=None):
    B = len(lens)
    tables, pool, _ = tables_for(lens, seed, width=width)
    kc, vc = normal((pool, hkv, BT, d), seed + 1), normal((pool, hkv, BT, d), seed + 2)
    poison_tails(kc, tables, lens)
    poison_tails(vc, tables, lens)
    q = normal((B, hq, d), seed + 3)
    new = (normal((B, hkv, d), seed + 4), normal((B, hkv, d), seed + 5)) if write else (None, None)
    scale = scale or d ** -0.5
    W = tables.shape[1]
    r = np.random.default_rng(seed)
    old = r.random((B, hkv, W * BT + 3)).astype(np.float32) * 5 if with_old else None
    if with_old:  # what lies at and past the new token is never read
        for b, n in enumerate(lens):
            old[b, :, max(n - 1, 0):] = np.nan
    sout = torch.full((B, hkv, W * BT + 3), -7.0, device="cuda")
    t, ln = cuda(tables), cuda(np.array(lens, np.int32))
    k2, v2 = kc.clone(), vc.clone()
    out, out2 = torch.full_like(q, NAN), torch.full_like(q, NAN)
    err = new_err()
    pkv.paged_attention_decode_scored(out, q, kc, vc, t, ln, scale, hkv, sout,
                                      scores_in=cuda(old) if with_old else None, k_new=new[0], v_new=new[1],
                                      variant=variant, partition_tokens=part, err=err)
    if write:
        pkv.paged_decode_step(out2, q, *new, k2, v2, t, ln, scale, hkv, variant=variant, partition_tokens=part)
    else:
        pkv.paged_attention_decode(out2, q, k2, v2, t, ln, scale, hkv, variant=variant, partition_tokens=part)
    assert int(err.item()) == 0
    assert same_bits(out, out2) and same_bits(kc, k2) and same_bits(vc, v2)
    q64, k64 = f64(q), f64(kc)
    # a query row for every sequence that has tokens
    live = np.array([n > 0 for n in lens])
    qs = np.concatenate([[0], np.cumsum(live)])
    want = ref.scores(q64[live], qs, k64, tables, lens, scale, None if old is None else old.astype(np.float64)) \
        if with_old else ref.scores(q64[live], qs, k64, tables, lens, scale, np.zeros((B, hkv, W * BT + 3)))
    got = f64(sout)
    score_check(got, want, old, ref.logit_bound(q64, k64, scale), hq // hkv)
    assert (got[np.isnan(want)] == -7.0).all()  # rows past the sequence as they were
    return sout


@pytest.mark.parametrize("lens,hq,hkv,d", [
    ([1], 1, 1, 64), ([16, 17, 0, 1], 4, 4, 128), ([33, 100, 515], 8, 2, 64), ([700, 3], 28, 4, 128),
    ([64, 129], 12, 1, 128), ([40, 250], 17, 1, 64), ([300] * 40, 32, 8, 128), ([1500], 32, 32, 128),
    ([90, 5, 77], 10, 2, 64), ([200, 31], 6, 2, 128),
])
@pytest.mark.parametrize("write", [False, True])
def test_scored_decode(lens, hq, hkv, d, write):
    decode_case(lens, hq, hkv, d, write, with_old=write, seed=len(lens) + hq)


@pytest.mark.parametrize("variant,part", [(1, 512), (2, 32), (2, 512), (4, 64), (4, 512)])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 128), (14, 2, 64), (24, 2, 128)])
def test_scored_decode_variants(variant, part, hq, hkv, d):
    decode_case([530, 1, 0, 47, 16], hq, hkv, d, True, True, variant, part, seed=variant + hq)


def test_scored_decode_far_logits():
    """Keys that a row all but ignores, and one that takes everything."""
    decode_case([400, 50], 4, 4, 64, False, True, scale=4.0, seed=9)


def test_scored_decode_in_place_and_deterministic():
    a = decode_case([700, 65], 14, 2, 128, False, False, seed=2)
    b = decode_case([700, 65], 14, 2, 128, False, False, seed=2)
    assert same_bits(a, b)
    tables, pool, _ = tables_for([100, 30], 1)
    kc, vc, q = normal((pool, 2, BT, 64), 1), normal((pool, 2, BT, 64), 2), normal((2, 4, 64), 3)
    old = torch.rand((2, 2, 7 * BT), device="cuda")
    apart, place, out = torch.zeros_like(old), old.clone(), torch.empty_like(q)
    args = (kc, vc, cuda(tables), cuda(np.array([100, 30], np.int32)), 0.1, 2)
    pkv.paged_attention_decode_scored(out, q, *args, apart, scores_in=old)
    pkv.paged_attention_decode_scored(out, q, *args, place, scores_in=place)
    assert same_bits(apart[0, :, :100], place[0, :, :100]) and same_bits(apart[1, :, :30], place[1, :, :30])
    assert same_bits(place[1, :, 30:], old[1, :, 30:])


def test_scored_decode_bad_blocks_get_no_weight():
    lens = [100, 40]
    tables, pool, _ = tables_for(lens, 1)
    tables[0, 2], tables[1, 0] = pool + 9, -5
    kc, vc, q = normal((pool, 2, BT, 64), 1), normal((pool, 2, BT, 64), 2), normal((2, 4, 64), 3)
    for variant in (1, 2, 4):
        sout = torch.full((2, 2, tables.shape[1] * BT), NAN, device="cuda")
        err, out = new_err(), torch.empty_like(q)
        pkv.paged_attention_decode_scored(out, q, kc, vc, cuda(tables), cuda(np.array(lens, np.int32)), 0.125, 2, sout,
                                          variant=variant, partition_tokens=32, err=err)
        assert int(err.item()) == pkv.DEV_ERR_BAD_BLOCK
        got = f64(sout)
        assert (got[0, :, 32:48] == 0).all() and (got[1, :, :16] == 0).all()
        # the rest of a row's weight is all there is: 2 query heads per KV head
        for b, n in enumerate(lens):
            assert np.abs(got[b, :, :n].sum(-1) - 2).max() < 1e-3


def test_scored_decode_lengths_past_the_table():
    tables, pool, _ = tables_for([32, 20], 1)
    kc, vc, q = normal((pool, 1, BT, 64), 1), normal((pool, 1, BT, 64), 2), normal((2, 1, 64), 3)
    sout = torch.full((2, 1, 32), -7.0, device="cuda")
    err, out = new_err(), torch.empty_like(q)
    pkv.paged_attention_decode_scored(out, q, kc, vc, cuda(tables), cuda(np.array([1000, -3], np.int32)), 0.125, 1, sout,
                                      err=err)
    assert int(err.item()) & pkv.DEV_ERR_BAD_LEN
    assert abs(float(sout[0].sum()) - 1) < 1e-3 and (sout[1] == -7).all() and not out[1].any()


# ------------------------------------------------------------------ scored prefill

def prefill_case(new, old, hq, hkv, d, window=0, with_old=True, seed=0, width=None, scale=None, whole=False):
    B = len(new)
    lens = [a + b for a, b in zip(new, old)]
    tables, pool, _ = tables_for(lens, seed, width=width)
    kc, vc = normal((pool, hkv, BT, d), seed + 1), normal((pool, hkv, BT, d), seed + 2)
    poison_tails(kc, tables, lens)
    poison_tails(vc, tables, lens)
    T = sum(new)
    q = normal((T, hq, d), seed + 3)
    qs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    scale = scale or d ** -0.5
    W = tables.shape[1]
    old_scores = np.random.default_rng(seed).random((B, hkv, W * BT)).astype(np.float32) * 5
    for b in range(B):
        old_scores[b, :, old[b]:] = np.nan
    sout = torch.full((B, hkv, W * BT), -7.0, device="cuda")
    t, ln, st = cuda(tables), cuda(np.array(lens, np.int32)), cuda(qs)
    out, out2 = torch.full_like(q, NAN), torch.full_like(q, NAN)
    err = new_err()
    pkv.paged_attention_prefill_scored(out, q, kc, vc, t, ln, st, scale, hkv, max(new), sout,
                                       scores_in=cuda(old_scores) if with_old else None, window=window, err=err)
    if T:
        pkv.paged_attention_prefill(out2, q, kc, vc, t, ln, st, scale, hkv, max(new))
    assert int(err.item()) == 0
    if whole:  # keys not cut into parts
        assert same_bits(out, out2)
    q64, k64 = f64(q), f64(kc)
    if T:
        want_out = ref.attention(q64, qs, k64, f64(vc), tables, lens, scale)
        check_close(out.view(torch.int16).cpu().numpy().view(np.uint16), want_out, "prefill")
    before = old_scores.astype(np.float64) if with_old else np.zeros(old_scores.shape)
    want = ref.scores(q64, qs, k64, tables, lens, scale, before, window)
    got = f64(sout)
    terms = max(min(n, window) if window else n for n in new) * (hq // hkv)
    score_check(got, want, before, ref.logit_bound(q64, k64, scale) if T else 0, terms)
    assert (got[np.isnan(want)] == -7.0).all()
    return sout


@pytest.mark.parametrize("new,old,hq,hkv,d", [
    ([1], [0], 1, 1, 64), ([1, 17, 0, 130], [0, 0, 40, 3], 4, 4, 128), ([200, 3, 77], [0, 500, 16], 8, 2, 64),
    ([129, 64], [0, 300], 28, 4, 128), ([90], [40], 16, 1, 128), ([33, 5], [0, 129], 17, 1, 64),
    ([1000], [0], 2, 2, 128), ([300, 260], [700, 0], 6, 2, 64), ([0, 0], [20, 0], 4, 2, 64), ([50], [30], 128, 1, 64),
    ([513, 127, 128], [0, 1, 128], 8, 8, 64), ([40, 7], [0, 9], 100, 1, 128),
])
@pytest.mark.parametrize("window", [0, 1, 32])
def test_scored_prefill(new, old, hq, hkv, d, window):
    prefill_case(new, old, hq, hkv, d, window, with_old=window != 1, seed=hq + window)


def test_scored_prefill_unsplit_units():
    """Enough (sequence, head, key tile) units that no unit's queries are cut into ranges, and enough
    items that no item's keys are cut into parts: the bits of the call without scores."""
    prefill_case([300] * 20, [0] * 20, 32, 32, 64, seed=4, whole=True)


@pytest.mark.parametrize("new,old,hq,hkv,d", [
    ([5], [4000], 4, 1, 64), ([129, 1, 0], [3000, 2500, 100], 8, 2, 128), ([300, 40], [1500, 1700], 14, 2, 64),
    ([257], [2300], 12, 1, 128), ([64, 700], [0, 2000], 6, 2, 64), ([1], [130], 3, 3, 128), ([33], [6000], 40, 1, 64),
])
def test_scored_prefill_keys_cut_into_parts(new, old, hq, hkv, d):
    """Few rows over long contexts: parts of every length, some past a tile's or a row's keys."""
    prefill_case(new, old, hq, hkv, d, window=16, seed=sum(new))


def test_scored_prefill_table_wider_than_the_sequences():
    prefill_case([70, 20], [30, 0], 8, 2, 128, seed=6, width=40)


def test_scored_prefill_twice_in_chunks_is_once_whole():
    """Two chunks accumulate what one prompt does, within the sums' rounding."""
    n, hq, hkv, d = 333, 8, 2, 64
    tables, pool, _ = tables_for([n], 3)
    kc, vc, q = normal((pool, hkv, BT, d), 1), normal((pool, hkv, BT, d), 2), normal((n, hq, d), 3)
    t = cuda(tables)
    whole, parts = (torch.full((1, hkv, t.shape[1] * BT), NAN, device="cuda") for _ in range(2))
    i32 = lambda *x: cuda(np.array(x, np.int32))  # noqa: E731
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    pkv.paged_attention_prefill_scored(out, q, kc, vc, t, i32(n), i32(0, n), d ** -0.5, hkv, n, whole)
    pkv.paged_attention_prefill_scored(out2[:200], q[:200], kc, vc, t, i32(200), i32(0, 200), d ** -0.5, hkv, 200, parts)
    pkv.paged_attention_prefill_scored(out2[200:], q[200:], kc, vc, t, i32(n), i32(0, n - 200), d ** -0.5, hkv, n - 200,
                                       parts, scores_in=parts)
    a, b = f64(whole)[..., :n], f64(parts)[..., :n]
    bound = ref.logit_bound(f64(q), f64(kc), d ** -0.5)
    assert (np.abs(a - b) <= (2 * bound + n * 4 * 2.0 ** -23) * a).all()
    check_close(out2.view(torch.int16).cpu().numpy().view(np.uint16), f64(out), "chunks")


def test_scored_prefill_flags_what_does_not_fit():
    hq, hkv, d = 4, 2, 64
    new, lens = [20, 30, 10], [20, 30, 10]
    tables, pool, _ = tables_for(lens, 1)
    kc, vc, q = normal((pool, hkv, BT, d), 1), normal((pool, hkv, BT, d), 2), normal((60, hq, d), 3)
    qs = np.array([0, 20, 50, 60], np.int32)

    def run(lens, qs, maxq):
        sout, err = torch.full((3, hkv, tables.shape[1] * BT), -7.0, device="cuda"), new_err()
        pkv.paged_attention_prefill_scored(torch.empty_like(q), q, kc, vc, cuda(tables), cuda(np.array(lens, np.int32)),
                                           cuda(qs), 0.125, hkv, maxq, sout, err=err)
        return sout, int(err.item())

    good, e = run(lens, qs, 30)
    assert e == 0
    short, e = run([20, 29, 10], qs, 30)      # context shorter than its new tokens
    assert e == pkv.DEV_ERR_BAD_LEN and (short[1] == -7).all()
    assert same_bits(short[0], good[0]) and same_bits(short[2], good[2])
    long, e = run(lens, qs, 25)               # more rows than max_query_len
    assert e == pkv.DEV_ERR_BAD_LEN and (long[1] == -7).all() and same_bits(long[0], good[0])
    t2 = tables.copy()
    t2[0, 1] = pool + 1
    sout, err = torch.full((3, hkv, tables.shape[1] * BT), -7.0, device="cuda"), new_err()
    pkv.paged_attention_prefill_scored(torch.empty_like(q), q, kc, vc, cuda(t2), cuda(np.array(lens, np.int32)),
                                       cuda(qs), 0.125, hkv, 30, sout, err=err)
    assert int(err.item()) == pkv.DEV_ERR_BAD_BLOCK and same_bits(sout[1:], good[1:])


@pytest.mark.parametrize("hq,hkv", [(4, 2), (14, 2), (2, 2)])
def test_scores_of_infinities_and_nan(hq, hkv):
    """An infinity in a key, or NaN in a query or a key, goes where the formula takes it: every weight
    of the rows it meets, and no other row's."""
    d, n, scale = 64, 300, 0.125
    tables, pool, _ = tables_for([n, n], 1)
    for what in ("q", "nan", "inf"):
        kc, vc, q = normal((pool, hkv, BT, d), 1), normal((pool, hkv, BT, d), 2), normal((2 * n, hq, d), 3)
        if what == "q":
            q[200, 1, 3] = NAN          # sequence 0, token 200, query head 1
        else:
            kc[int(tables[0, 250 // BT]), 0, 250 % BT, 5] = NAN if what == "nan" else float("inf")
        i32 = lambda *x: cuda(np.array(x, np.int32))  # noqa: E731
        sout, out = torch.zeros((2, hkv, tables.shape[1] * BT), device="cuda"), torch.empty_like(q)
        pkv.paged_attention_prefill_scored(out, q, kc, vc, cuda(tables), i32(n, n), i32(0, n, 2 * n), scale, hkv, n, sout)
        q64, k64 = f64(q), f64(kc)
        with np.errstate(all="ignore"):
            want = ref.scores(q64, [0, n, 2 * n], k64, tables, [n, n], scale, None)
        got = f64(sout)[:, :, :n]
        want = want[:, :, :n]
        assert np.isnan(want).any() and not np.isnan(want).all()
        assert np.array_equal(np.isnan(got), np.isnan(want)), what
        fine = ~np.isnan(want)
        assert (np.abs(got - want)[fine] <= 1e-3 * want[fine]).all()
        # the same rows one at a time, as decode steps see them
        rows = np.array([[199, 250], [200, 251], [n - 1, n - 1]])
        for pair in rows:
            sout.zero_()
            o = torch.empty((2, hq, d), dtype=BF, device="cuda")
            pkv.paged_attention_decode_scored(o, torch.stack([q[pair[0]], q[n + pair[1]]]).contiguous(), kc, vc, cuda(tables),
                                              i32(pair[0] + 1, pair[1] + 1), scale, hkv, sout)
            with np.errstate(all="ignore"):
                want1 = ref.scores(np.stack([q64[pair[0]], q64[n + pair[1]]]), [0, 1, 2], k64, tables, pair + 1, scale, None)
            got1 = f64(sout)
            for b in range(2):
                assert np.array_equal(np.isnan(got1[b, :, :pair[b] + 1]), np.isnan(want1[b, :, :pair[b] + 1])), (what, pair, b)


def test_scored_prefill_rows_past_the_queries():
    """query_start past the rows of q: the sequence is flagged and left out, nothing of it is read or written."""
    hq, hkv, d = 4, 2, 64
    tables, pool, _ = tables_for([20, 40], 1)
    kc, vc, q = normal((pool, hkv, BT, d), 1), normal((pool, hkv, BT, d), 2), normal((64, hq, d), 3)
    out = torch.full((64, hq, d), NAN, dtype=BF, device="cuda")
    sout, err = torch.full((2, hkv, tables.shape[1] * BT), -7.0, device="cuda"), new_err()
    pkv.paged_attention_prefill_scored(out[:50], q[:50], kc, vc, cuda(tables), cuda(np.array([20, 40], np.int32)),
                                       cuda(np.array([0, 20, 60], np.int32)), 0.125, hkv, 40, sout, err=err)
    assert int(err.item()) == pkv.DEV_ERR_BAD_LEN
    assert out[:20].isfinite().all() and out[20:].isnan().all()
    assert (sout[0, :, :20] > 0).all() and (sout[1] == -7).all()


# ------------------------------------------------------------------ eviction

def evict_case(lens, keep, hkv, d, sink, recent, scores=None, seed=0, width=None):
    B = len(lens)
    r = np.random.default_rng(seed)
    tables, pool, _ = tables_for(lens, seed, width=width)
    m = [min(k, n) for k, n in zip(keep, lens)]
    need = [-(-k // BT) for k in m]
    nt = np.full((B, max(1, max(need))), -1, np.int32)
    fresh = pool + r.permutation(sum(need) + 2)
    at = 0
    for b, k in enumerate(need):
        nt[b, :k] = fresh[at:at + k]
        at += k
    total = pool + sum(need) + 2
    kc, vc = normal((total, hkv, BT, d), seed + 1), normal((total, hkv, BT, d), seed + 2)
    W, NW = tables.shape[1], nt.shape[1]
    if scores is None:
        scores = r.random((B, hkv, W * BT)).astype(np.float32) ** 6
        scores[r.random(scores.shape) < 0.3] = 0.0
        scores[r.random(scores.shape) < 0.2] = 0.25  # ties
    k0, v0 = kc.clone(), vc.clone()
    sout = torch.full((B, hkv, NW * BT + 5), -7.0, device="cuda")
    kept = torch.full((B, hkv, NW * BT), -9, dtype=torch.int32, device="cuda")
    err = new_err()
    pkv.evict_tokens(kc, vc, cuda(tables), cuda(np.array(lens, np.int32)), cuda(nt), cuda(np.array(keep, np.int32)),
                     cuda(scores), sout, kept, sink=sink, recent=recent, err=err)
    assert int(err.item()) == 0
    want_kept = np.full((B, hkv, NW * BT), -9)
    want_s = np.full((B, hkv, NW * BT + 5), -7.0, np.float32)
    for b, n in enumerate(lens):
        for h in range(hkv):
            c = ref.chosen(scores[b, h], n, keep[b], sink, recent)
            want_kept[b, h, :len(c)] = c
            want_s[b, h, :len(c)] = scores[b, h, c]
            i = np.arange(len(c))
            src = [torch.from_numpy(x).cuda() for x in (tables[b, c // BT].astype(np.int64), c % BT)]
            dst = [torch.from_numpy(x).cuda() for x in (nt[b, i // BT].astype(np.int64), i % BT)]
            k0[dst[0], h, dst[1]], v0[dst[0], h, dst[1]] = k0[src[0], h, src[1]], v0[src[0], h, src[1]]
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(sout.cpu().numpy().view(np.int32), want_s.view(np.int32))
    assert same_bits(kc, k0) and same_bits(vc, v0)


@pytest.mark.parametrize("lens,keep,hkv,d,sink,recent", [
    ([1], [1], 1, 64, 0, 0), ([1], [0], 1, 64, 0, 0), ([40, 0, 17], [20, 5, 16], 3, 128, 2, 4),
    ([100, 33], [33, 33], 2, 64, 0, 0), ([500, 16, 250], [499, 1, 100], 4, 128, 4, 32),
    ([300, 200], [50, 60], 2, 64, 100, 200),          # sink and recent ask for more than is kept
    ([1000], [100], 5, 64, 0, 100), ([1000], [100], 2, 128, 100, 0), ([90], [45], 1, 128, 0, 44),
    ([5000, 4097], [700, 4096], 2, 64, 16, 128),
])
def test_evict(lens, keep, hkv, d, sink, recent):
    evict_case(lens, keep, hkv, d, sink, recent, seed=sum(lens))


@pytest.mark.parametrize("width", [256, 257, 513, 1025, 3000])
def test_evict_table_widths(width):
    """One CTA a row, clusters of two and four, and slices of several rounds."""
    evict_case([width * BT - 5, 4000], [2000, 3000], 2, 64, 4, 64, seed=width, width=width)


def test_evict_equal_scores_keep_the_lowest_positions():
    for value in (0.0, 1.5, -np.inf, np.inf):
        evict_case([600, 40], [100, 30], 2, 64, 3, 7, scores=np.full((2, 2, 38 * BT), value, np.float32), seed=1)


def test_evict_odd_scores():
    """Infinities, NaN (below everything), both zeros (equal), subnormal and negative scores."""
    r = np.random.default_rng(2)
    odd = np.array([np.inf, -np.inf, np.nan, 0.0, -0.0, 1e-42, -1e-42, -3.0, 2.0, 3.4e38], np.float32)
    s = odd[r.integers(0, len(odd), (2, 3, 30 * BT))]
    for keep in (20, 250, 470):
        evict_case([480, 300], [keep, 200], 3, 64, 1, 2, scores=s, seed=keep)


def test_evict_bad_lengths_and_blocks():
    tables, pool, _ = tables_for([64, 64, 64], 1)
    nt = np.array([[pool, pool + 1], [pool + 2, pool + 99], [pool + 3, pool + 4]], np.int32)
    kc, vc = normal((pool + 5, 1, BT, 64), 1), normal((pool + 5, 1, BT, 64), 2)
    scores = torch.rand((3, 1, 64), device="cuda")
    k0 = kc.clone()
    sout, kept, err = torch.zeros((3, 1, 32), device="cuda"), torch.full((3, 1, 32), -9, dtype=torch.int32, device="cuda"), new_err()
    pkv.evict_tokens(kc, vc, cuda(tables), cuda(np.array([64, 64, 9999], np.int32)), cuda(nt),
                     cuda(np.array([9999, 32, -1], np.int32)), scores, sout, kept, err=err)
    assert int(err.item()) == pkv.DEV_ERR_BAD_LEN | pkv.DEV_ERR_BAD_BLOCK
    assert (kept[0] >= 0).all() and (kept[2] == -9).all()   # clamped to the new table; nothing kept
    assert same_bits(kc[pool + 3:], k0[pool + 3:])


# ------------------------------------------------------------------ together

def test_a_prompt_its_eviction_and_decode_steps():
    """Rotary write, scored prefill, eviction by those scores into fresh blocks, then decode steps
    that rotate, write and score, with a second eviction; a host copy that holds plain lists of rows
    follows every step."""
    hq, hkv, d, scale = 8, 2, 64, 64 ** -0.5
    prompts, keep, sink, recent = [150, 90, 37], [64, 64, 64], 2, 16
    B, nb, W = 3, 64, 16
    a = pkv.BlockAllocator(nb, np.random.default_rng(0).permutation(nb))
    kc, vc = (torch.full((nb, hkv, BT, d), NAN, dtype=BF, device="cuda") for _ in range(2))
    table = pkv.rope_table(4096, d)
    ids = [10, 11, 12]
    for s in ids:
        a.add_seq(s, 0)
    T = sum(prompts)
    slots = np.concatenate([a.extend(s, n) for s, n in zip(ids, prompts)])
    pos = np.concatenate([np.arange(n) for n in prompts]).astype(np.int32)
    qkv = normal((T, hq + 2 * hkv, d), 1)
    q = torch.empty((T, hq, d), dtype=BF, device="cuda")
    err = new_err()
    pkv.rope_kv_write(q, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kc, vc, cuda(slots), cuda(pos), table, err=err)
    tables, lens = a.export(ids, W)
    qs = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    scores = torch.full((B, hkv, W * BT), NAN, device="cuda")
    out = torch.empty_like(q)
    pkv.paged_attention_prefill_scored(out, q, kc, vc, cuda(tables), cuda(lens), cuda(qs), scale, hkv, max(prompts), scores,
                                       err=err)
    host = [[[ref.rows(f64(c), tables[b], prompts[b], h) for c in (kc, vc)] for h in range(hkv)] for b in range(B)]
    weight = ref.scores(f64(q), qs, f64(kc), tables, lens, scale, None)
    host_w = [[weight[b, h, :prompts[b]] for h in range(hkv)] for b in range(B)]
    next_pos = list(prompts)

    def evict():
        nonlocal scores
        tables, lens = a.export(ids, W)
        m = [min(k, int(n)) for k, n in zip(keep, lens)]
        a.evict(ids, m)
        new_tables, new_lens = a.export(ids, W)
        kept = torch.zeros((B, hkv, W * BT), dtype=torch.int32, device="cuda")
        after = torch.full_like(scores, NAN)
        pkv.evict_tokens(kc, vc, cuda(tables), cuda(lens), cuda(new_tables), cuda(new_lens), scores, after, kept,
                         sink=sink, recent=recent, err=err)
        got = kept.cpu().numpy()
        for b in range(B):
            for h in range(hkv):
                # the choice by the GPU's own scores, the rows by that choice
                c = ref.chosen(scores[b, h].cpu().numpy(), int(lens[b]), keep[b], sink, recent)
                assert np.array_equal(got[b, h, :len(c)], c)
                host[b][h] = [x[c] for x in host[b][h]]
                host_w[b][h] = host_w[b][h][c]
        scores = after

    def check_cache():
        tables, lens = a.export(ids, W)
        for b in range(B):
            for h in range(hkv):
                for c, x in zip((kc, vc), host[b][h]):
                    assert np.array_equal(ref.rows(f64(c), tables[b], int(lens[b]), h), x)
                got = f64(scores)[b, h, :int(lens[b])]
                assert (np.abs(got - host_w[b][h]) <= 1e-3 * np.abs(host_w[b][h]) + 1e-6).all()

    evict()
    check_cache()
    for step in range(6):
        slots = a.append_tokens(ids)
        tables, lens = a.export(ids, W)
        qkv = normal((B, hq + 2 * hkv, d), 50 + step)
        q = torch.empty((B, hq, d), dtype=BF, device="cuda")
        pkv.rope_kv_write(q, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kc, vc, cuda(np.asarray(slots)),
                          cuda(np.array(next_pos, np.int32)), table, err=err)
        out = torch.empty_like(q)
        pkv.paged_attention_decode_scored(out, q, kc, vc, cuda(tables), cuda(lens), scale, hkv, scores, scores_in=scores,
                                          err=err)
        want = np.zeros((B, hq, d))
        for b in range(B):
            for h in range(hkv):
                blk, off = divmod(int(slots[b]), BT)
                host[b][h] = [np.concatenate([x, f64(c)[blk, h, off][None]]) for c, x in zip((kc, vc), host[b][h])]
                n = len(host[b][h][0])
                assert n == lens[b]
                w = ref.weights(f64(q)[b, h * 4:h * 4 + 4], host[b][h][0], scale, np.full(4, n))
                want[b, h * 4:h * 4 + 4] = w @ host[b][h][1]
                host_w[b][h] = np.append(host_w[b][h], 0.0) + w.sum(0)
        check_close(out.view(torch.int16).cpu().numpy().view(np.uint16), want, f"step {step}")
        next_pos = [p + 1 for p in next_pos]
        if step == 3:
            evict()
        check_cache()
    assert int(err.item()) == 0


def _decode_state(seed):
    lens = [300, 41, 128]
    tables, pool, _ = tables_for(lens, seed)
    kc, vc = normal((pool, 2, BT, 128), seed), normal((pool, 2, BT, 128), seed + 1)
    q = normal((3, 14, 128), seed + 2)
    out, s = torch.empty_like(q), torch.zeros((3, 2, tables.shape[1] * BT), device="cuda")
    t, ln = cuda(tables), cuda(np.array(lens, np.int32))
    return lambda: pkv.paged_attention_decode_scored(out, q, kc, vc, t, ln, 0.09, 2, s), (out, s)


def test_two_captured_graphs_and_an_eager_call_share_nothing():
    """Two captured scored decodes replayed on two streams beside an eager one: each has its own
    scratch."""
    runs = [_decode_state(s) for s in (1, 20, 40)]
    for call, _ in runs:
        call()
    torch.cuda.synchronize()
    want = [[x.clone() for x in outs] for _, outs in runs]
    graphs = []
    for call, _ in runs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for _, outs in runs:
        for x in outs:
            x.zero_()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        with torch.cuda.stream(streams[2]):
            runs[2][0]()
    torch.cuda.synchronize()
    for (_, outs), w in zip(runs, want):
        assert all(same_bits(x, y) for x, y in zip(outs, w))


def test_captured_prefill_and_eviction_replay_on_new_inputs():
    hq, hkv, d, n = 8, 2, 64, 260
    tables, pool, free = tables_for([n], 1, spare=8)
    kc, vc, q = normal((pool, hkv, BT, d), 1), normal((pool, hkv, BT, d), 2), normal((n, hq, d), 3)
    t, nt = cuda(tables), cuda(np.array([free[:6]], np.int32))
    ln, st, keep = (cuda(np.array(x, np.int32)) for x in ([n], [0, n], [90]))
    out, s, s2 = torch.empty_like(q), torch.zeros((1, hkv, t.shape[1] * BT), device="cuda"), torch.zeros((1, hkv, 96), device="cuda")
    kept = torch.zeros((1, hkv, 96), dtype=torch.int32, device="cuda")

    def call():
        pkv.paged_attention_prefill_scored(out, q, kc, vc, t, ln, st, d ** -0.5, hkv, n, s)
        pkv.evict_tokens(kc, vc, t, ln, nt, keep, s, s2, kept, sink=2, recent=8)

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    q.copy_(normal((n, hq, d), 77))
    g.replay()
    got = [x.clone() for x in (out, s, s2, kept, kc)]
    for x in (out, s, s2, kept):
        x.zero_()
    call()
    torch.cuda.synchronize()
    assert all(same_bits(x, y) for x, y in zip(got, (out, s, s2, kept, kc)))
