"""Rules of csrc/qdense.cu that no run can show: a fault against them may pass
on one compiler and hang the next.  They are read from the source."""
import os
import re

import pytest

import bit_affine_quantized_gb300.build as build

CSRC = os.path.join(build.HERE, "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|__launch_bounds__\([^)]*\)", "", f.read())


def _functions(code):
    """name -> body of every function at namespace level (the file's braces balance there)."""
    out = {}
    for m in re.finditer(r"^(?:__device__ __forceinline__|__global__)[^;{]*?(\w+)\([^{;]*\)\s*\{", code, re.M):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(code[i], 0)
            i += 1
        out[m.group(1)] = code[m.end():i - 1]
    return out


# instructions that every lane of a warp has to execute together, as qdense.cu writes or calls them
ALIGNED = re.compile(r"\.aligned|bar\.sync|dense::tc_(?:ld32|ld16|alloc|dealloc)\b")


def test_aligned_instructions_follow_a_warp_barrier():
    """Lanes may come apart at any branch that depends on the lane, and only a
    warp barrier brings them together for certain: each wrapper of an aligned
    instruction begins with one, and the kernels use the wrappers alone."""
    functions = _functions(_code("qdense.cu"))
    assert {"qdense_mma_kernel", "qdense_few_kernel", "mm_st32", "cluster_sync_all"} <= set(functions)
    for name, body in functions.items():
        first = ALIGNED.search(body)
        if name.endswith("_kernel"):
            assert not first, f"{name}: {first.group(0)} outside a wrapper"
        elif first:
            assert "__syncwarp();" in body[:first.start()], f"{name}: {first.group(0)} without a warp barrier before it"


def test_few_rows_mma_follows_a_warp_barrier():
    """mma.sync after loads that depend on the lane."""
    body = _functions(_code("qdense.cu"))["qdense_few_kernel"]
    loads, mma = body.index("request(n0, b + kQfAhead);"), body.index("mma_f16(")
    assert "__syncwarp();" in body[loads:mma]


def _branches(body):
    """The bodies of the branches that one lane of a warp takes."""
    for m in re.finditer(r"if \(lane == 0\) \{", body):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(body[i], 0)
            i += 1
        yield m.start(), i


def test_waits_of_whole_warps_have_one_result():
    """A bounded wait that runs out in some lanes only would part the warp
    before its next full-mask vote, which then never ends.  A warp's waits are
    voted on where they stand, or by a vote before the first branch that looks
    at the result; those of one lane are in that lane's branch; waits whose
    result nobody looks at follow the loops."""
    body = _functions(_code("qdense.cu"))["qdense_mma_kernel"]
    alone = list(_branches(body))
    for m in re.finditer(r"mm_wait(?:<[^>]*>)?\(", body):
        if any(a <= m.start() < b for a, b in alone):
            continue
        start = max(body.rfind(c, 0, m.start()) for c in ";{}") + 1
        statement = body[start:body.index(";", m.start())]
        if "ok" not in statement:
            continue
        vote = body.find("__all_sync(", m.start())
        between = body[m.start():vote if vote >= 0 else None]
        parts = r"\b(?:break|continue|return)\b|(?:for|while|if) \((?:[^()]|\([^()]*\))*\bok\b"  # that a lane's own result could part
        voted = "__all_sync(" in statement or (vote >= 0 and not re.search(parts, between))
        assert voted, f"a warp goes on from a lane's own wait: {statement.strip()}"


def test_tensor_memory_is_freed_when_no_warp_uses_it():
    """A wait that ran out lets the warps of a block leave their loops at
    different times, and none may free the tensor memory that another still loads
    or stores: the MMA warp frees it once its own last waits are over, and where
    one of them ran out after the last word of every other warp that uses it; a
    pair behind a barrier of both blocks."""
    body = _functions(_code("qdense.cu"))["qdense_mma_kernel"]
    alone, pair = (m.start() for m in re.finditer("mm_dealloc", body))
    before = body[body.rindex("if (gi > 0)", 0, alone):alone]
    assert before.count("ok = mm_wait") == 2 and before.count("&& ok;") == 2
    assert before.index("__all_sync(0xffffffffu, ok)") < before.index("mm_wait(tdone, 0)")
    words = [m.start() for m in re.finditer(re.escape("if (!kPairs && lane == 0) mm_arrive(tdone);"), body)]
    assert len(words) == 2
    for at, last_use in zip(words, ("cluster_arrive(cluster_map(smem_addr(&dempty[db]), 0));", "mm_st_wait();")):
        assert body.rindex(last_use) < at  # the finish warps, the widen warps
    assert "n = kMmWiden + kMmFin;" in body
    assert "cluster_sync_all();" in body[body.rindex("if (kPairs) {", 0, pair):pair]


def test_arrivals_of_another_block_name_their_scope():
    """An arrival on a barrier of another block is of cluster scope, not of the
    default, the block's own; the forms of the wait differ from one another, and
    the leader's wait for rows, which two blocks' copies write, acquires at that
    scope."""
    code = _code("qdense.cu")
    remote = re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*", code)
    assert remote and all(".cluster.shared::cluster" in r for r in remote)
    waits = re.findall(r"mbarrier\.try_wait[\w.:]*", code)
    assert len(waits) == len(set(waits)) and any(".acquire.cluster" in w for w in waits)
    body = _functions(code)["qdense_mma_kernel"]
    mma = body[body.index("mm_alloc"):body.index("mm_dealloc")]
    assert re.search(r"mm_wait<kPairs \? kClusterAcquire : kBlock>\(&rfull", mma)
