"""The rotary write, the scored attention and the eviction on the host: argument
checks that answer before any launch, workspace sizes, and the allocator's
eviction against the reference model."""
import ctypes

import numpy as np
import pytest

from oracle.alloc_model import AllocError as ModelError, BlockManager
from paged_kv_cache_459_b200 import build as pkv_build

pkv_build.build()
from paged_kv_cache_459_b200 import pkv  # noqa: E402

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation rejects first
INVALID, UNSUPPORTED, WORKSPACE = pkv.ERR_INVALID_ARG, pkv.ERR_UNSUPPORTED, pkv.ERR_WORKSPACE


def rope(**kw):
    a = dict(qo=FAKE, q=FAKE, k=FAKE, v=FAKE, sqo=512, sq=512, sk=256, sv=256, kc=FAKE, vc=FAKE, slots=FAKE,
             pos=FAKE, axes=1, pair=None, table=FAKE, maxp=1024, rot=128, inter=0, T=4, Hq=4, Hkv=2, D=128, NB=8)
    a.update(kw)
    return pkv.lib().pkv_rope_kv_write(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
    (dict(rot=8), INVALID), (dict(rot=136), INVALID), (dict(rot=0), INVALID), (dict(rot=72), INVALID),
    (dict(axes=0), INVALID), (dict(axes=5, pair=bytes(64)), INVALID),
    (dict(axes=2), INVALID),                               # several axes need to be told apart
    (dict(axes=2, pair=bytes([2] * 64)), INVALID),         # an axis there is not
    (dict(pair=bytes([1] * 64)), INVALID),
    (dict(inter=2), INVALID), (dict(maxp=0), INVALID), (dict(NB=0), INVALID), (dict(T=-1), INVALID),
    (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(sq=504), INVALID), (dict(sq=516), INVALID), (dict(sqo=8), INVALID), (dict(sk=128), INVALID),
    (dict(sv=250), INVALID),
    (dict(q=None), INVALID), (dict(table=None), INVALID), (dict(slots=None), INVALID), (dict(pos=None), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(kc=FAKE + 2), INVALID), (dict(table=FAKE + 4), INVALID),
    (dict(T=0, q=None, qo=None), pkv.OK),
])
def test_rope_argument_checks(kw, code):
    assert rope(**kw) == code


def decode(**kw):
    a = dict(out=FAKE, q=FAKE, kn=None, vn=None, kc=FAKE, vc=FAKE, tables=FAKE, W=8, lens=FAKE, B=2, Hq=4, Hkv=2,
             D=128, NB=64, scale=0.1, sin=None, sout=FAKE, stride=128, variant=0, part=512, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return pkv.lib().pkv_paged_attention_decode_scored(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(kn=FAKE), INVALID), (dict(vn=FAKE), INVALID), (dict(kn=FAKE + 2, vn=FAKE), INVALID),
    (dict(sout=None), INVALID), (dict(sout=FAKE + 2), INVALID), (dict(sin=FAKE + 1), INVALID),
    (dict(stride=127), INVALID), (dict(D=96), UNSUPPORTED), (dict(Hq=5), INVALID), (dict(variant=3), INVALID),
    (dict(part=40), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=1024), WORKSPACE), (dict(ws=FAKE + 8), WORKSPACE),
    (dict(scale=float("inf")), INVALID), (dict(B=0, out=None), pkv.OK),
])
def test_scored_decode_argument_checks(kw, code):
    assert decode(**kw) == code


def prefill(**kw):
    a = dict(out=FAKE, q=FAKE, T=20, kc=FAKE, vc=FAKE, tables=FAKE, W=8, lens=FAKE, qs=FAKE, B=2, maxq=16, Hq=4,
             Hkv=2, D=128, NB=64, scale=0.1, sin=None, sout=FAKE, stride=128, window=0, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return pkv.lib().pkv_paged_attention_prefill_scored(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVALID), (dict(maxq=-1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(D=32), UNSUPPORTED), (dict(Hq=258), UNSUPPORTED), (dict(Hq=5), INVALID), (dict(sout=None), INVALID),
    (dict(stride=100), INVALID), (dict(qs=None), INVALID), (dict(q=None), INVALID), (dict(q=FAKE + 4), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE), (dict(sin=FAKE + 2), INVALID),
    (dict(W=1 << 25, stride=1 << 40), UNSUPPORTED), (dict(W=1 << 26, stride=1 << 40), INVALID), (dict(B=0), pkv.OK),
])
def test_scored_prefill_argument_checks(kw, code):
    assert prefill(**kw) == code


def evict(**kw):
    a = dict(kc=FAKE, vc=FAKE, tables=FAKE, W=8, lens=FAKE, nt=FAKE + 256, NW=4, keep=FAKE, sin=FAKE, istr=128,
             sout=FAKE + 512, ostr=64, kept=FAKE, sink=1, recent=2, B=2, Hkv=2, D=128, NB=64)
    a.update(kw)
    return pkv.lib().pkv_evict_tokens(*a.values(), None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(sin=None), INVALID), (dict(kept=None), INVALID), (dict(sout=FAKE), INVALID), (dict(nt=FAKE), INVALID),
    (dict(istr=127), INVALID), (dict(ostr=63), INVALID), (dict(sink=-1), INVALID), (dict(recent=-1), INVALID),
    (dict(D=80), UNSUPPORTED), (dict(W=0), INVALID), (dict(NW=0), INVALID), (dict(B=70000), INVALID),
    (dict(kc=FAKE + 8), INVALID), (dict(keep=None), INVALID), (dict(NB=1 << 28), UNSUPPORTED),
    (dict(B=0, kc=None), pkv.OK),
])
def test_evict_argument_checks(kw, code):
    assert evict(**kw) == code


def test_scored_workspace_sizes():
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    base = up(pkv.decode_workspace_bytes_for(pkv.DECODE_AUTO, 3, 28, 4, 128, 33))
    assert pkv.decode_scored_workspace_bytes(3, 28, 4, 128, 33) == base + up(3 * 4 * 8 * 33 * 16 * 4) + up(3 * 28 * 4)
    # one query head per KV head: one logit a token; groups above 8 in chunks
    assert pkv.decode_scored_workspace_bytes(1, 2, 2, 64, 1) >= 2 * 16 * 4 + 8
    assert pkv.decode_scored_workspace_bytes(2, 24, 2, 64, 5) >= 2 * 2 * 2 * 8 * 80 * 4
    assert pkv.decode_scored_workspace_bytes(2, 5, 2, 64, 5) == 0
    assert pkv.prefill_scored_workspace_bytes(-1, 2, 16, 4, 2, 64, 8) == 0
    assert pkv.prefill_scored_workspace_bytes(20, 2, 16, 4, 2, 64, 8) >= 20 * 4 * 4


def _same(a, m):
    assert a.free_blocks() == m.free_blocks()
    assert [a.refcount(b) for b in range(m.num_blocks)] == m.ref
    ids = sorted(m.tables)
    if ids:
        w = max(1, max(len(m.tables[s]) for s in ids))
        for x, y in zip(a.export(ids, w), m.export(ids, w)):
            assert np.array_equal(x, y)


def test_alloc_evict_takes_every_fresh_block_before_returning_one():
    a = pkv.BlockAllocator(8)
    a.add_seq(0, 33)
    a.add_seq(1, 32)  # 3 + 2 blocks, 3 free
    a.evict([0, 1], [17, 5])
    tables, lens = a.export([0, 1], 2)
    assert tables.tolist() == [[5, 6], [7, -1]] and lens.tolist() == [17, 5]
    assert a.free_blocks() == [0, 1, 2, 3, 4]
    with pytest.raises(pkv.AllocError) as e:
        a.evict([0, 0], [1, 1])
    assert e.value.kind == "invalid"
    a.evict([1], [0])
    assert a.export([1], 1)[0].tolist() == [[-1]] and a.free_blocks()[-1] == 7
    a.evict([], [])


def test_alloc_evict_leaves_shared_blocks_to_their_other_holders():
    a = pkv.BlockAllocator(10)
    a.add_seq(0, 40)
    a.fork(0, 1)
    a.evict([0], [20])
    assert a.export([1], 3)[0].tolist() == [[0, 1, 2]] and a.export([0], 3)[0].tolist() == [[3, 4, -1]]
    assert [a.refcount(b) for b in range(5)] == [1, 1, 1, 1, 1]


def test_alloc_evict_against_the_model():
    r = np.random.default_rng(5)
    nb = 60
    order = r.permutation(nb)
    a, m = pkv.BlockAllocator(nb, order), BlockManager(nb, order)
    done = {"evict": 0, "refused": 0}
    for step in range(600):
        ids = sorted(m.tables)
        what = r.integers(0, 6)
        if what == 0 or not ids:
            args = ("add_seq", step, int(r.integers(0, 120)))
        elif what == 1:
            args = ("fork", int(r.choice(ids)), step)
        elif what == 2:
            args = ("append_token", int(r.choice(ids)))
        elif what == 3:
            args = ("free_seq", int(r.choice(ids)))
        else:
            some = [int(x) for x in r.choice(ids, size=int(r.integers(1, 4)))]
            args = ("evict", some, [int(r.integers(0, m.lens[s] + 2)) for s in some])
        got = []
        for side in (a, m):
            try:
                getattr(side, args[0])(*args[1:])
                got.append("ok")
            except (pkv.AllocError, ModelError) as e:
                got.append(e.kind)
        assert got[0] == got[1], args
        if args[0] == "evict":
            done["evict" if got[0] == "ok" else "refused"] += 1
        if args[0] == "append_token":
            a.take_copies(), m.take_copies()
        _same(a, m)
    assert min(done.values()) > 20, done


def test_binding_refuses_what_does_not_fit():
    import torch

    t = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    c = torch.zeros(4, 4, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    s = torch.zeros(2, 4, 16)
    with pytest.raises(ValueError):   # host tensors
        pkv.rope_kv_write(t, t, t, t, c, c, i.long(), i, torch.zeros(8, 64))
    with pytest.raises(ValueError):   # shapes
        pkv.rope_kv_write(t, t, t[:1], t, c, c, i.long(), i, torch.zeros(8, 64))
    with pytest.raises(ValueError):   # one axis entry for each pair
        pkv.rope_kv_write(t, t, t, t, c, c, i.long(), i, torch.zeros(8, 64), pair_axis=[0] * 31)
    with pytest.raises(ValueError):
        pkv.paged_attention_decode_scored(t, t, c, c, i.view(2, 1), i, 1.0, 4, s, k_new=t)
    with pytest.raises(ValueError):   # a score row shorter than the table
        pkv.paged_attention_decode_scored(t, t, c, c, torch.zeros(2, 2, dtype=torch.int32), i, 1.0, 4, s)
    with pytest.raises(ValueError):
        pkv.paged_attention_prefill_scored(t, t, c, c, i.view(2, 1), i, i, 1.0, 4, 1, s)
    with pytest.raises(ValueError):   # kept: new table's tokens
        pkv.evict_tokens(c, c, i.view(2, 1), i, i.view(2, 1), i, s, s, torch.zeros(2, 4, 8, dtype=torch.int32))


@pytest.mark.parametrize("axes,error", [
    (32, TypeError),                                    # a number is not 32 zeros
    (np.zeros(4, dtype=np.int64), "one axis"),          # 4 items, though 32 bytes
    (np.zeros(32, dtype=np.int64), "CUDA"),             # 32 items: refused for the host tensors only
    ([-1] * 32, ValueError), ([256] * 32, ValueError), ([0.0] * 32, TypeError),
])
def test_pair_axis_is_a_sequence_of_ints(axes, error):
    import torch

    t = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    c = torch.zeros(4, 4, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    kind, text = (ValueError, error) if isinstance(error, str) else (error, None)
    with pytest.raises(kind, match=text):
        pkv.rope_kv_write(t, t, t, t, c, c, i.long(), i, torch.zeros(8, 64), pair_axis=axes)


def test_scores_without_dimensions_are_refused():
    import torch

    t = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    c = torch.zeros(4, 4, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="scores"):
        pkv.paged_attention_decode_scored(t, t, c, c, i.view(2, 1), i, 1.0, 4, torch.zeros(()))


def test_rope_table_is_the_cosines_and_sines_of_the_positions():
    import torch

    t = pkv.rope_table(70000, 64, 10000.0, device="cpu")
    assert t.shape == (70000, 64) and t.dtype == torch.float32
    p, i = 69999, 5
    ang = p * 10000.0 ** (-2 * i / 64)
    assert abs(float(t[p, i]) - np.cos(ang)) <= 2.0 ** -24 + 1e-11
    assert abs(float(t[p, 32 + i]) - np.sin(ang)) <= 2.0 ** -24 + 1e-11
    assert ctypes.sizeof(ctypes.c_float) == 4


def test_marshalled_arguments_are_the_headers():
    """marshal.c's letter for every argument of the four calls fits the header's declaration, and
    the binding's names stand at the tensors."""
    import re

    src = open(pkv_build.MARSHAL_SRC).read()
    header = re.sub(r"/\*.*?\*/", "", open(pkv.HEADER).read(), flags=re.S)
    found = re.findall(r'"(\w+)", */\* (pkv_\w+) \*/', src)
    assert [name for _, name in found] == [m[0] for m in pkv._MARSHALLED]
    kinds = dict(b="void", r="void", p="void", i="int32_t", l="int64_t", f="float", s="uint8_t")
    for (spec, name), (_, address, names) in zip(found, pkv._MARSHALLED):
        args = [a.strip() for a in re.search(r"%s\((.*?)\);" % name, header, re.S).group(1).replace("\n", " ").split(",")]
        assert len(args) == len(spec) == len(names) + 1 and address
        for c, arg, n in zip(spec, args, names + ["."]):
            if c in "nqx":
                assert "*" not in arg or "stream" in arg
                assert {"n": "int ", "q": "int64_t ", "x": "float "}[c] in arg or "size_t" in arg or "stream" in arg
                assert n == "."
                continue
            assert "*" in arg and (kinds[c.lower()] in arg or arg == "unsigned int *err_word"), (c, arg)
            assert (n == ".") == (c in "sp")
            if n != ".":
                assert arg.endswith("*" + dict(tables="x").get(n.split(":")[0], n.split(":")[0])) or n.startswith("err")
                assert n.split(":")[1] == c.lower()


def test_marshal_refuses_what_it_cannot_convert():
    from paged_kv_cache_459_b200 import _marshal
    import torch

    _marshal.setup(torch.bfloat16, torch.int32, torch.int64, torch.float32, torch.uint8)
    with pytest.raises(TypeError):
        _marshal.call(9, 1, 0)
    with pytest.raises(TypeError):
        _marshal.call(3, 1, 0, 1, 2)
    t, i, s = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1, 16)
    address = pkv._MARSHALLED[pkv._EVICT][1]
    args = [t, t, i, 1, i, i, 1, i, s, 16, s, 16, i, 0, 0, 1, 1, 64, 2, None, 0]
    # host tensors stand for device -1; every tensor's type, device and layout is looked at
    for at, bad in ((0, t.float()), (0, 5), (2, i.long()), (8, s.double()), (12, "kept"), (1, t.transpose(0, 1).expand(2, 2, 16, 64))):
        a = list(args)
        a[at] = bad
        assert _marshal.call(pkv._EVICT, address, -1, *a) == -(at + 1)
    assert _marshal.call(pkv._EVICT, address, 0, *args) == -1     # another device
    for at, bad, error in ((3, 1 << 40, OverflowError), (3, "w", TypeError), (18, 1 << 70, OverflowError)):
        a = list(args)
        a[at] = bad
        with pytest.raises(error):
            _marshal.call(pkv._EVICT, address, -1, *a)
    # the same tables before and after: the library's own check answers
    assert _marshal.call(pkv._EVICT, address, -1, *args) == pkv.ERR_INVALID_ARG


def test_prefill_workspace_goes_by_the_device_it_is_asked_for(monkeypatch):
    """A device without an index is the current one, and without a CUDA device nothing is remembered:
    the size depends on the SMs of whatever device the library then sees."""
    import torch

    asked = []
    sizes = (20, 2, 16, 4, 2, 64, 8)
    host = pkv.prefill_scored_workspace_bytes(*sizes) if not torch.cuda.is_available() else None
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(pkv, "_prefill_scored_bytes", lambda dev, *s: asked.append((dev, s)) or 7)
    for device in (None, "cuda", torch.device("cuda"), "cuda:1", torch.device("cuda", 2), 5):
        assert pkv.prefill_scored_workspace_bytes(*sizes, window=4, device=device) == 7
    assert [d for d, _ in asked] == [3, 3, 3, 1, 2, 5] and all(s == (*sizes, 4) for _, s in asked)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.prefill_scored_workspace_bytes(*sizes, device="cpu")
    monkeypatch.undo()
    if host is not None:
        before = pkv._prefill_scored_bytes.cache_info()
        assert pkv.prefill_scored_workspace_bytes(*sizes) == host > 0
        assert pkv._prefill_scored_bytes.cache_info() == before


def _python(code, **env):
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    return subprocess.run([sys.executable, "-c", code], cwd=root, env={**os.environ, **env}, capture_output=True, text=True)


def test_calls_without_marshalled_arguments_need_no_marshal_module():
    """The package imports, and its older calls answer, where the marshalling module is missing (another
    interpreter's, no compiler when it was built); the four calls that use it say what to build."""
    r = _python("""
import sys
sys.modules["paged_kv_cache_459_b200._marshal"] = None   # importing it raises ImportError
from paged_kv_cache_459_b200 import pkv
a = pkv.BlockAllocator(4)
a.add_seq(0, 20)
assert pkv.decode_workspace_bytes(2, 4, 64, 8) > 0 and a.export([0], 2)[1].tolist() == [20]
import torch
t = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
c = torch.zeros(4, 4, 16, 64, dtype=torch.bfloat16)
i = torch.zeros(2, dtype=torch.int32)
try:
    pkv.rope_kv_write(t, t, t, t, c, c, i.long(), i, torch.zeros(8, 64))
except ImportError as e:
    assert "paged_kv_cache_459_b200.build" in str(e), e
    print("refused")
""")
    assert r.returncode == 0 and r.stdout.split() == ["refused"], r.stderr


def test_marshal_module_carries_its_interpreters_suffix():
    """Another interpreter does not take the file for its own, and builds one beside it."""
    import sysconfig

    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert pkv_build.MARSHAL.endswith("_marshal" + suffix)
    from paged_kv_cache_459_b200 import _marshal

    assert _marshal.__file__ == pkv_build.MARSHAL
