"""Rules of kernels that overlap on a stream (programmatic dependent launches),
checked on the sources, without a GPU."""
import pathlib
import re

import pytest

ROOT = pathlib.Path(__file__).resolve().parents[1]
CSRC = ROOT / "paged_kv_cache_459_b200" / "csrc"
SOURCES = sorted(p for p in CSRC.iterdir() if p.suffix in (".cu", ".cuh"))


def _code(path):
    text = re.sub(r"/\*.*?\*/", "", path.read_text(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def _functions(code):
    """{name: body} of the device functions and kernels of a file."""
    found = {}
    code = re.sub(r"__launch_bounds__\([^()]*\)", "", code)
    for m in re.finditer(r"(?:__global__|__device__)[^;{}]*?\b(\w+)\((?=[^;{}]*\)\s*(?:const\s*)?\{)", code):
        start = code.index("{", m.end())
        depth, i = 1, start + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(code[i], 0)
            i += 1
        found[m.group(1)] = code[start:i]
    return found


def test_the_functions_are_found():
    assert {"prefill_scores_kernel", "prefill_scores_join_kernel"} <= set(_functions(_code(CSRC / "prefill_scores.cu")))
    assert {"cascade_kernel", "prefix_unit_tc"} <= set(_functions(_code(CSRC / "decode_prefix.cu")))


@pytest.mark.parametrize("path", SOURCES, ids=lambda p: p.name)
def test_dependents_start_only_after_tensor_memory_is_allocated(path):
    """A block holds the right to allocate tensor memory until it gives it up or exits, and a
    dependent's block waits for the whole grid before it does either: started on an SM whose
    block has not allocated yet, the two would wait for each other.  So a kernel lets
    dependents start behind its allocation and the barrier that follows it."""
    if path.name == "tcgen05.cuh":
        return
    functions = _functions(_code(path))
    allocating = {name for name, body in functions.items() if "tc::alloc<" in body}
    for name, body in functions.items():
        starts = [m.start() for m in re.finditer(r"\bpdl_launch_dependents\(\)", body)]
        if name in allocating:
            done = body.index("__syncthreads()", body.index("tc::alloc<"))
            assert all(at > done for at in starts), name
        for callee in allocating - {name}:
            for call in re.finditer(r"\b%s\s*<" % callee, body):
                assert all(at > call.start() for at in starts), f"{name} before {callee}"


# What a kernel may read through the read-only path although the kernel before it on the stream may
# still run: the arrays that include/pkv.h ("Stream order") asks callers not to write from such a kernel.
HOST_WRITTEN = ("seq_lens", "block_tables", "prefix_blocks", "start_blocks", "query_start", "trow", "row + first")


def test_data_of_an_overlapping_kernel_is_not_read_through_the_read_only_path():
    """ld.global.nc is for data that nothing writes while the kernel lives.  A dependent lives while
    the grid before it still writes, so after its wait it reads with plain loads or __ldcg: q, scores,
    log-sum-exps, the order, slots and positions may be that grid's.  (Kernels launched without
    programmatic serialization, kv_write.cu's, start when all before them are done.)"""
    seen = 0
    for path in SOURCES:
        code = _code(path)
        if path.name == "kv_write.cu":
            assert "pdl_" not in code and "launch_dependent" not in code
            continue
        for m in re.finditer(r"__ldg\(", code):
            depth, i = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(code[i], 0)
                i += 1
            arg = code[m.end():i - 1]
            seen += 1
            assert any(name in arg for name in HOST_WRITTEN), f"{path.name}: __ldg({arg})"
        assert "ld.global.nc" not in code, path.name
    assert seen > 10


def _without_one_thread_code(code):
    """The code without what a single thread runs: if (lane == 0) and its like, block or statement."""
    out, at = [], 0
    for m in re.finditer(r"\bif \((?:[^()]*&& )?(?:lane|t|threadIdx\.x) == 0\)\s*", code):
        if m.start() < at:
            continue
        out.append(code[at:m.start()])
        i, depth = m.end(), 0
        while True:
            depth += {"{": 1, "(": 1, "}": -1, ")": -1}.get(code[i], 0)
            if depth == 0 and code[i] in "};":
                break
            i += 1
        at = i + 1
    return "".join(out) + code[at:]


def _statement(code, start):
    """The statement (with its block) that starts at or holds `start`, from there to its end."""
    depth, i = 0, start
    while True:
        depth += {"{": 1, "}": -1}.get(code[i], 0)
        if depth < 0 or (depth == 0 and code[i] in ";}"):
            return code[start:i + 1]
        i += 1


@pytest.mark.parametrize("path", [p for p in SOURCES if p.name != "ptx.cuh"], ids=lambda p: p.name)
def test_no_lane_leaves_its_warp_over_a_wait(path):
    """Lanes that timed out, or saw the abort flag, alone must not leave the others in a warp-wide
    vote, shuffle or tensor-memory access, which would then never end.  A wait that several lanes make
    is decided by a vote of the warp (mbar_wait_warp) or of the block, or it steers no jump: the lane
    only remembers it, and leaves loops by a vote or at their natural end."""
    left = _without_one_thread_code(_code(path))
    for m in re.finditer(r"\bmbar_wait\(", left):
        if left[:m.start()].endswith("__syncthreads_or(!"):
            continue
        then = _statement(left, m.start())
        assert not re.search(r"\b(break|return|continue|goto)\b", then), f"{path.name}: {then}"
    for m in re.finditer(r"warp == kMmaWarp\) \{", left):  # its lanes' `ok` is each lane's own
        role = _statement(left, m.end() - 1)
        loops = re.findall(r"\b(?:for|while) \((?:[^()]|\([^()]*\))*\)", role)
        for loop in loops:
            assert not re.search(r"\bok\b", loop) or "idx = lane" in loop, f"{path.name}: {loop}"
        assert "tc::dealloc" in role or not re.search(r"\b(break|return|goto)\b", role), path.name
