"""The serving operators around a cache that forgets: what is measured.

Four operators, each in its plain form (elementary torch operations in 32 bits)
and, where `own` is true, as a user calls the library:

  rope     rotary positions over one or several axes, fused with the cache write
  decode   one decode step that also accumulates each cached token's attention weight
  prefill  attention of a chunk of new tokens that also accumulates those weights
  evict    the tokens with the most weight kept, copied together into fresh blocks

Caches are [blocks][KV heads][16][d] bf16, reached through int32 block tables;
scores are [sequences][KV heads][row] float32.
"""
import math

import numpy as np
import torch

own = False

BT = 16  # tokens of a block


def listed():
    return [
        # one decode step's 64 new tokens of a multi-head model: the launch is what counts
        dict(name="rope: decode step", op="rope", tokens=64, hq=32, hkv=32, d=128, rot=128, axes=1,
             interleaved=False, cycled=False, fused_qkv=False),
        # prompts with pictures (time, height, width), q, k and v slices of one projection's output
        dict(name="rope: pictures, 3 axes", op="rope", tokens=7411, hq=28, hkv=4, d=128, rot=128, axes=3,
             interleaved=False, cycled=False, fused_qkv=True),
        # a long prompt, half of each head rotated, neighbouring pairs
        dict(name="rope: long, half rotated", op="rope", tokens=32768, hq=32, hkv=8, d=64, rot=32, axes=1,
             interleaved=True, cycled=False, fused_qkv=True),
        # one conversation: latency
        dict(name="decode: one sequence", op="decode", batch=1, lo=1337, hi=1337, hq=32, hkv=32, d=128,
             write=True),
        # a full serving batch, grouped heads
        dict(name="decode: batch 256", op="decode", batch=256, lo=512, hi=4096, hq=28, hkv=4, d=128,
             write=True),
        # few sequences, long contexts
        dict(name="decode: long contexts", op="decode", batch=8, lo=32768, hi=32768, hq=32, hkv=8, d=128,
             write=False),
        # short prompts of odd lengths, every query counted
        dict(name="prefill: short prompts", op="prefill", batch=5, new_lo=1, new_hi=200, old_lo=0, old_hi=0,
             hq=8, hkv=2, d=64, window=0),
        # four prompts, every query counted
        dict(name="prefill: 4 x 2048", op="prefill", batch=4, new_lo=2048, new_hi=2048, old_lo=0, old_hi=0,
             hq=32, hkv=32, d=128, window=0),
        # a chunk after a long cached context, the last 64 queries counted
        dict(name="prefill: chunk, long cache", op="prefill", batch=2, new_lo=1000, new_hi=1024, old_lo=12000,
             old_hi=15000, hq=28, hkv=4, d=128, window=64),
        # a few sequences just over their budget
        dict(name="evict: few sequences", op="evict", batch=4, lo=700, hi=1100, hq=8, hkv=8, d=64, keep=0.6,
             sink=4, recent=64),
        # a serving batch cut to half
        dict(name="evict: batch 64", op="evict", batch=64, lo=512, hi=4096, hq=28, hkv=4, d=128, keep=0.5,
             sink=4, recent=128),
        # long prompts cut to an eighth
        dict(name="evict: long prompts", op="evict", batch=8, lo=32768, hi=32768, hq=32, hkv=8, d=128,
             keep=0.125, sink=16, recent=512),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "decode", "prefill", "evict"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
    group = rng.choice([1, 1, 2, 4, 5, 7, 8, 12] if hkv <= 8 else [1, 2])
    if hkv * group > 32:
        group = max(1, 32 // hkv)
    heads = dict(hq=hkv * group, hkv=hkv, d=d)
    if op == "rope":
        axes = rng.choice([1, 1, 2, 3])
        return dict(op=op, tokens=_log_int(rng, 1, 16384), rot=rng.choice([d, d, d // 2, 48]), axes=axes,
                    interleaved=rng.random() < 0.4, cycled=axes > 1 and rng.random() < 0.5,
                    fused_qkv=rng.random() < 0.5, **heads)
    if op == "decode":
        # at most as many cached values as the largest listed batch holds
        most = 256 * 2300 * 4 * 128
        hi = _log_int(rng, 1, 32768)
        batch = min(_log_int(rng, 1, 256), max(1, most // (hi * hkv * d)))
        return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, spread=rng.randint(1, 1 << 20), write=rng.random() < 0.7, **heads)
    if op == "prefill":
        new = _log_int(rng, 1, 2048)
        old = 0 if rng.random() < 0.4 else _log_int(rng, 1, 12000)
        most = 2 * 28 * 1024 * 15000  # query heads x keys
        batch = min(rng.randint(1, 6), max(1, most // (hkv * group * new * (new + old))))
        return dict(op=op, batch=batch, new_lo=rng.randint(0, new), new_hi=new, old_lo=old // 2, old_hi=old,
                    spread=rng.randint(1, 1 << 20), window=rng.choice([0, 0, 1, 32, 64, 200]), **heads)
    hi = _log_int(rng, 2, 32768)
    most = 8 * 32768 * 8 * 128
    batch = min(_log_int(rng, 1, 64), max(1, most // (hi * hkv * d)))
    return dict(op=op, batch=batch, lo=rng.randint(1, hi), hi=hi, spread=rng.randint(1, 1 << 20), keep=rng.choice([0.125, 0.25, 0.5, 0.9]),
                sink=rng.choice([0, 1, 4, 16]), recent=rng.choice([0, 1, 32, 200, 512]), **heads)


# ------------------------------------------------------------------ inputs

def _blocks(n):
    return -(-int(n) // BT)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, gen, dtype=torch.bfloat16):
    return torch.randn(shape, device="cuda", dtype=torch.float32, generator=gen).to(dtype)


def _tables(lens, width, nprng, pool):
    """Tables over a shuffled pool: row b holds the blocks of lens[b] tokens, -1 after them."""
    ids = nprng.permutation(pool).astype(np.int32)
    t = np.full((len(lens), max(1, width)), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        k = _blocks(n)
        t[b, :k] = ids[at:at + k]
        at += k
    return t, ids[at:]


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _lens(case, seed=None):
    """A case's lengths (for prefill the new tokens and the cached ones): drawn for the case, so that
    work() counts what prepare() makes, and dealt to the sequences by the seed."""
    r = np.random.default_rng([int(case.get("spread", 0)), 7])
    ranges = [("new_lo", "new_hi"), ("old_lo", "old_hi")] if case["op"] == "prefill" else [("lo", "hi")]
    got = [r.integers(case[a], case[b], size=case["batch"], endpoint=True) for a, b in ranges]
    got[0][-1] = case[ranges[0][1]]
    order = np.arange(case["batch"]) if seed is None else np.random.default_rng([int(seed), 11]).permutation(case["batch"])
    return [x[order] for x in got]


def _kept(case, lens):
    return np.minimum(lens, np.maximum(1, (lens * case["keep"]).astype(np.int64)))


def _positions(case, nprng):
    """Positions of the new tokens, one row for each axis. With several axes: stretches of text (all
    axes alike) and pictures (time stands still, height and width walk a grid), as one prompt has them.
    With one axis: prompts of different lengths one after another."""
    T, A = case["tokens"], case["axes"]
    pos = np.zeros((A, T), np.int64)
    t, p = 0, int(nprng.integers(0, 20000))
    while t < T:
        if A == 1 or nprng.random() < 0.5:
            n = min(T - t, int(nprng.integers(1, 2000)))
            pos[:, t:t + n] = p + np.arange(n)
            p = int(nprng.integers(0, 20000)) if A == 1 else p + n
        else:
            h, w = int(nprng.integers(4, 40)), int(nprng.integers(4, 40))
            n = min(T - t, h * w)
            i = np.arange(n)
            grid = [np.zeros(n, np.int64), i // w, i % w]
            for a in range(A):
                pos[a, t:t + n] = p + grid[a if A == 3 else a + 1]
            p += max(h, w)
        t += n
    return pos % 65536


def _pair_axis(case):
    """Which axis turns pair i: contiguous sections, or the axes in turn."""
    half, A = case["rot"] // 2, case["axes"]
    if case["cycled"]:
        return [i % A for i in range(half)]
    if A == 3 and half == 64:
        return [0] * 16 + [1] * 24 + [2] * 24
    return [i * A // half for i in range(half)]


def prepare(case, seed):
    gen, nprng = _gen(seed), np.random.default_rng([int(seed), 3])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    s = dict(case=case, scale=1.0 / math.sqrt(d))
    if case["op"] == "rope":
        T, rot = case["tokens"], case["rot"]
        pool = _blocks(T) + 5
        if case["fused_qkv"]:
            qkv = _normal((T, hq + 2 * hkv, d), gen)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = (_normal((T, h, d), gen) for h in (hq, hkv, hkv))
        ids = nprng.permutation(pool)
        slots = ids[np.arange(T) // BT] * BT + np.arange(T) % BT
        slots[nprng.random(T) < 0.01] = -1  # padding tokens: nothing is written for them
        s["slots"] = _cuda(slots.astype(np.int64))
        s["positions"] = _cuda(_positions(case, nprng).astype(np.int32))
        # the table a program makes once: angles in 64 bits
        freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) / (rot // 2))
        ang = torch.arange(65536, device="cuda", dtype=torch.float64)[:, None] * freq
        s["table"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        s["pair_axis"] = _pair_axis(case)
        s["axis_of"] = torch.tensor(s["pair_axis"], device="cuda")
        s["k_cache"], s["v_cache"] = (_normal((pool, hkv, BT, d), gen) for _ in range(2))
        s["q_out"] = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda")
        return s
    B = case["batch"]
    if case["op"] == "prefill":
        new, old = _lens(case, seed)
        lens = new + old
        s["max_new"] = int(new.max())
        s["query_start"] = _cuda(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
        s["q"] = _normal((int(new.sum()), hq, d), gen)
    else:
        (lens,) = _lens(case, seed)
        s["q"] = _normal((B, hq, d), gen)
    width = max(1, _blocks(lens.max()))
    keep = _kept(case, lens) if case["op"] == "evict" else None
    pool = int(sum(_blocks(n) for n in lens)) + (int(sum(_blocks(n) for n in keep)) if keep is not None else 0) + 9
    t, free = _tables(lens, width, nprng, pool)
    s["tables"], s["lens"] = _cuda(t), _cuda(lens.astype(np.int32))
    s["k_cache"], s["v_cache"] = (_normal((pool, hkv, BT, d), gen) for _ in range(2))
    row = width * BT
    # weights gathered so far: a few tokens hold most of it, many hold none
    w = torch.rand((B, hkv, row), device="cuda", generator=gen)
    scores = torch.where(w < 0.2, torch.zeros_like(w), (w ** 8) * 20)
    s["scores"] = scores
    if case["op"] == "evict":
        nt = np.full((B, max(1, _blocks(keep.max()))), -1, np.int32)
        at = 0
        for b, n in enumerate(keep):
            nt[b, :_blocks(n)] = free[at:at + _blocks(n)]
            at += _blocks(n)
        s["new_tables"], s["keep"] = _cuda(nt), _cuda(keep.astype(np.int32))
        krow = nt.shape[1] * BT
        s["kept"] = torch.full((B, hkv, krow), -1, dtype=torch.int32, device="cuda")
        s["scores_out"] = torch.zeros((B, hkv, krow), device="cuda")
        return s
    s["out"] = torch.empty_like(s["q"])
    s["scores_out"] = torch.zeros_like(scores)
    if case["op"] == "decode" and case["write"]:
        s["k_new"], s["v_new"] = (_normal((B, hkv, d), gen) for _ in range(2))
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if op == "rope":
        return _own_rope(s) if own else _plain_rope(s)
    if op == "decode":
        return _own_decode(s) if own else _plain_decode(s)
    if op == "prefill":
        return _own_prefill(s) if own else _plain_prefill(s)
    return _own_evict(s) if own else _plain_evict(s)


def _own_rope(s):
    from paged_kv_cache_459_b200 import pkv
    pkv.rope_kv_write(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
                      s["table"], pair_axis=s["pair_axis"], interleaved=s["case"]["interleaved"])
    return [s["q_out"], s["k_cache"], s["v_cache"]]


def _own_decode(s):
    from paged_kv_cache_459_b200 import pkv
    pkv.paged_attention_decode_scored(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"],
                                      s["case"]["hkv"], s["scores_out"], scores_in=s["scores"], k_new=s.get("k_new"),
                                      v_new=s.get("v_new"))
    return [s["out"], s["scores_out"]] + ([s["k_cache"], s["v_cache"]] if "k_new" in s else [])


def _own_prefill(s):
    from paged_kv_cache_459_b200 import pkv
    pkv.paged_attention_prefill_scored(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                       s["query_start"], s["scale"], s["case"]["hkv"], s["max_new"], s["scores_out"],
                                       scores_in=s["scores"], window=s["case"]["window"])
    return [s["out"], s["scores_out"]]


def _own_evict(s):
    from paged_kv_cache_459_b200 import pkv
    pkv.evict_tokens(s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["new_tables"], s["keep"], s["scores"],
                     s["scores_out"], s["kept"], sink=s["case"]["sink"], recent=s["case"]["recent"])
    return [s["kept"], s["scores_out"], s["k_cache"], s["v_cache"]]


def _rotated(x, cos, sin, rot, interleaved):
    x = x.float()
    turned, rest = x[..., :rot], x[..., rot:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :rot // 2], turned[..., rot // 2:])
    c, t = cos[:, None, :], sin[:, None, :]
    u, v = a * c - b * t, b * c + a * t
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, rest], -1).to(torch.bfloat16)


def _plain_rope(s):
    rot, inter = s["case"]["rot"], s["case"]["interleaved"]
    half = rot // 2
    pos = s["positions"].long()[s["axis_of"]].T  # [T, rot / 2]
    i = torch.arange(half, device="cuda")
    cos, sin = s["table"][pos, i], s["table"][pos, half + i]
    q_out = _rotated(s["q"], cos, sin, rot, inter)
    k = _rotated(s["k"], cos, sin, rot, inter)
    live = s["slots"] >= 0
    blk, off = s["slots"][live] // BT, s["slots"][live] % BT
    s["k_cache"][blk, :, off] = k[live]
    s["v_cache"][blk, :, off] = s["v"][live]
    return [q_out, s["k_cache"], s["v_cache"]]


def _gathered(cache, tables, hkv, d):
    """The sequences' rows in token order, [B][KV heads][tokens][d], 32 bits."""
    x = cache[tables.clamp(min=0).long()]
    return x.permute(0, 2, 1, 3, 4).reshape(tables.shape[0], hkv, -1, d).float()


def _accumulated(s, weights, first_new):
    """Old weight of the tokens before first_new, plus this pass's; rows past the sequence as they were."""
    p = torch.arange(s["scores"].shape[2], device="cuda")
    before = torch.where(p < first_new[:, None, None], s["scores"], torch.zeros_like(s["scores"]))
    return torch.where(p < s["lens"].long()[:, None, None], before + weights, s["scores_out"])


def _plain_decode(s):
    c = s["case"]
    hq, hkv, d, B = c["hq"], c["hkv"], c["d"], c["batch"]
    lens = s["lens"].long()
    if "k_new" in s:
        live = lens > 0
        at = (lens - 1).clamp(min=0)
        blk = s["tables"].long().gather(1, (at // BT)[:, None])[:, 0][live]
        s["k_cache"][blk, :, (at % BT)[live]] = s["k_new"][live]
        s["v_cache"][blk, :, (at % BT)[live]] = s["v_new"][live]
    k, v = (_gathered(s[n], s["tables"], hkv, d) for n in ("k_cache", "v_cache"))
    p = torch.arange(k.shape[2], device="cuda")
    inside = (p < lens[:, None])[:, None, None, :]
    x = torch.matmul(s["q"].float().view(B, hkv, hq // hkv, d), k.transpose(2, 3)) * s["scale"]
    x = torch.where(inside, x, torch.full_like(x, -math.inf))
    e = torch.where(inside, torch.exp(x - x.amax(-1, keepdim=True)), torch.zeros_like(x))
    w = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    out = torch.matmul(w, v).view(B, hq, d).to(torch.bfloat16)
    scores = _accumulated(s, w.sum(2), lens - 1)
    return [out, scores] + ([s["k_cache"], s["v_cache"]] if "k_new" in s else [])


def _plain_prefill(s):
    c = s["case"]
    hq, hkv, d, B = c["hq"], c["hkv"], c["d"], c["batch"]
    lens, start = s["lens"].long(), s["query_start"].long()
    new = start[1:] - start[:-1]
    i = torch.arange(s["max_new"], device="cuda")
    there = i < new[:, None]
    rows = (start[:-1, None] + i).clamp(max=max(0, s["q"].shape[0] - 1))
    q = s["q"][rows].float().view(B, -1, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)  # [B][KV heads][group][new][d]
    k, v = (_gathered(s[n], s["tables"], hkv, d) for n in ("k_cache", "v_cache"))
    p = torch.arange(k.shape[2], device="cuda")
    at = (lens - new)[:, None] + i
    seen = ((p <= at[:, :, None]) & there[:, :, None])[:, None, None]
    x = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).unflatten(2, (hq // hkv, -1)) * s["scale"]
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    e = torch.where(seen, torch.exp(x - x.amax(-1, keepdim=True)), torch.zeros_like(x))
    w = e / e.sum(-1, keepdim=True).clamp(min=1e-30)
    out = torch.matmul(w.flatten(2, 3), v).unflatten(2, (hq // hkv, -1)).permute(0, 3, 1, 2, 4).reshape(B, -1, hq, d)
    out = out[there].to(torch.bfloat16)
    counted = there & (i >= (new - (c["window"] or s["max_new"]))[:, None])
    scores = _accumulated(s, torch.where(counted[:, None, None, :, None], w, torch.zeros_like(w)).sum((2, 3)), lens - new)
    return [out, scores]


def _plain_evict(s):
    c = s["case"]
    lens, keep = s["lens"].long()[:, None, None], s["keep"].long()[:, None, None]
    p = torch.arange(s["scores"].shape[2], device="cuda")
    recent = torch.clamp(keep, max=c["recent"])
    sink = torch.clamp(keep - recent, max=c["sink"])
    x = torch.where((p < sink) | (p >= lens - recent), torch.full_like(s["scores"], math.inf), s["scores"])
    x = torch.where(p < lens, x, torch.full_like(x, -math.inf))
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    n = s["kept"].shape[2]
    j = torch.arange(n, device="cuda")
    last = torch.full_like(order, s["scores"].shape[2])  # past the budget: sorted to the end
    chosen = torch.where(p < keep, order, last).sort(-1).values[..., :n]
    chosen = torch.nn.functional.pad(chosen, (0, n - chosen.shape[2])) if chosen.shape[2] < n else chosen
    live = (j < keep).expand_as(chosen)
    at = torch.where(live, chosen, torch.zeros_like(chosen))
    kept = torch.where(live, at, torch.full_like(at, -1)).to(torch.int32)
    scores = torch.where(live, s["scores"].gather(2, at), torch.zeros_like(at, dtype=torch.float32))
    b, h, i = live.nonzero(as_tuple=True)
    src = at[b, h, i]
    old, new = s["tables"].long()[b, src // BT], s["new_tables"].long()[b, i // BT]
    s["k_cache"][new, h, i % BT] = s["k_cache"][old, h, src % BT]
    s["v_cache"][new, h, i % BT] = s["v_cache"][old, h, src % BT]
    return [kept, scores, s["k_cache"], s["v_cache"]]


# ------------------------------------------------------------------ the least work

def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        T, rot = case["tokens"], case["rot"]
        # q in and out, k and v in, K and V out, the table's rows, positions and slots
        return {"bytes": T * (2 * hq * d * 2 + 4 * hkv * d * 2 + rot * 4 + 4 * case["axes"] + 8),
                "flops": T * (hq + hkv) * rot * 3}
    if case["op"] == "prefill":
        new, old = (x.astype(np.float64) for x in _lens(case))
        counted = np.minimum(case["window"], new) if case["window"] else new
        pairs = float((new * old + new * (new + 1) / 2).sum())
        again = float((counted * (old + new) - counted * (counted - 1) / 2).sum())
        new, tokens = float(new.sum()), float((new + old).sum())
        return {"bytes": 2 * new * hq * d * 2 + tokens * hkv * (d * 2 * 2 + 8) + tokens / BT * 4,
                "flops": hq * d * (4 * pairs + 2 * again)}
    (lens,) = _lens(case)
    tokens = float(lens.sum())
    if case["op"] == "decode":
        new = case["batch"] * hkv * d * 2 * 2 * 2 if case["write"] else 0
        return {"bytes": tokens * hkv * (d * 2 * 2 + 8) + tokens / BT * 4 + 2 * case["batch"] * hq * d * 2 + new,
                "flops": tokens * hq * d * 4}
    kept = float(_kept(case, lens).sum())
    # every score, the kept tokens' K and V in and out, their scores and indices out
    return {"bytes": tokens * hkv * 4 + kept * hkv * (d * 2 * 2 * 2 + 8), "flops": tokens * hkv}


# ------------------------------------------------------------------ 64 bits

def _rows64(cache, table, n, h):
    """The first n rows of KV head h through one sequence's table, in 64 bits."""
    t = torch.arange(n, device="cuda")
    return cache[table.long()[t // BT], h, t % BT].double()


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "decode": _exact_decode, "prefill": _exact_prefill, "evict": _exact_evict}[case["op"]](s)


def _exact_rope(s):
    c = s["case"]
    half, table = c["rot"] // 2, s["table"].double()
    outs = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
            at = s["positions"][s["pair_axis"][i]].long()
            cos, sin = table[at, i][:, None], table[at, half + i][:, None]
            y[:, :, a] = x[:, :, a].double() * cos - x[:, :, b].double() * sin
            y[:, :, b] = x[:, :, b].double() * cos + x[:, :, a].double() * sin
        outs.append(y)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    t = (s["slots"] >= 0).nonzero()[:, 0]
    for h in range(c["hkv"]):
        kc[s["slots"][t] // BT, h, s["slots"][t] % BT] = outs[1][t, h]
        vc[s["slots"][t] // BT, h, s["slots"][t] % BT] = s["v"][t, h].double()
    return [outs[0], kc, vc]


def _exact_decode(s):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    out = torch.zeros((c["batch"], c["hq"], c["d"]), dtype=torch.float64, device="cuda")
    scores = s["scores_out"].double()
    lens = s["lens"].tolist()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        if "k_new" in s:
            blk = int(s["tables"][b, (n - 1) // BT])
            s["k_cache"][blk, :, (n - 1) % BT] = s["k_new"][b]
            s["v_cache"][blk, :, (n - 1) % BT] = s["v_new"][b]
        for h in range(c["hkv"]):
            k, v = _rows64(s["k_cache"], s["tables"][b], n, h), _rows64(s["v_cache"], s["tables"][b], n, h)
            w = torch.softmax(s["q"][b, h * g:(h + 1) * g].double() @ k.T * s["scale"], -1)
            out[b, h * g:(h + 1) * g] = w @ v
            scores[b, h, :n] = w.sum(0)
            scores[b, h, :n - 1] += s["scores"][b, h, :n - 1].double()
    return [out, scores] + ([s["k_cache"], s["v_cache"]] if "k_new" in s else [])


def _exact_prefill(s):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    scores = s["scores_out"].double()
    lens, start = s["lens"].tolist(), s["query_start"].tolist()
    for b, n in enumerate(lens):
        lo, hi = start[b], start[b + 1]
        new = hi - lo
        pos = torch.arange(n - new, n, device="cuda")
        unseen = torch.arange(n, device="cuda")[None] > pos[:, None]
        first = max(0, new - c["window"]) if c["window"] else 0
        for h in range(c["hkv"]):
            k, v = _rows64(s["k_cache"], s["tables"][b], n, h), _rows64(s["v_cache"], s["tables"][b], n, h)
            total = torch.zeros(n, dtype=torch.float64, device="cuda")
            total[:n - new] = s["scores"][b, h, :n - new].double()
            for m in range(h * g, (h + 1) * g):
                x = (s["q"][lo:hi, m].double() @ k.T * s["scale"]).masked_fill(unseen, -math.inf)
                w = torch.softmax(x, -1)
                out[lo:hi, m] = w @ v
                total += w[first:].sum(0)
            scores[b, h, :n] = total
    return [out, scores]


def _exact_evict(s):
    c = s["case"]
    lens, keep = s["lens"].tolist(), s["keep"].tolist()
    kept, scores = s["kept"].cpu().numpy(), s["scores_out"].double()
    kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
    rows = s["scores"].double().cpu().numpy()
    for b, n in enumerate(lens):
        m = keep[b]
        recent = min(c["recent"], m)
        sink = min(c["sink"], m - recent)
        for h in range(c["hkv"]):
            middle = np.arange(sink, n - recent)
            best = middle[np.lexsort((middle, -rows[b, h, middle]))][:m - recent - sink]
            chosen = np.concatenate([np.arange(sink), np.sort(best), np.arange(n - recent, n)])
            kept[b, h, :m] = chosen
            at, to = torch.from_numpy(chosen).cuda(), torch.arange(m, device="cuda")
            scores[b, h, :m] = s["scores"][b, h, at].double()
            old, new = s["tables"][b].long()[at // BT], s["new_tables"][b].long()[to // BT]
            kc[new, h, to % BT] = s["k_cache"][old, h, at % BT]
            vc[new, h, to % BT] = s["v_cache"][old, h, at % BT]
    return [torch.from_numpy(kept).cuda(), scores, kc, vc]
