"""Rules of csrc/sample.cu that no run can show: a fault against them may pass on an
idle device and fault on a busy one.  They are read from the source."""
import re

from test_qdense_source import _code


def _kernel():
    code = _code("sample.cu")
    at = code.index("sample_kernel(const SampleArgs a)")
    return code[at:code.index("\n}\n", at)]


def test_other_blocks_run_before_their_memory_is_written():
    """A block may look into another's shared memory only once that block runs: a
    cluster barrier, arrived at after the set-up of what the others write, and
    waited for before the first store."""
    body = _kernel()
    remote = re.search(r"\bsm_(?:put|get|count)\(", body).start()
    arrive, wait = body.index("sm_arrive();"), body.index("sm_wait();")
    assert body.index("s_n = s_own = 0u") < body.index("__syncthreads();") < arrive < wait < remote
    # the barrier's two halves belong together: no other between them
    assert "sm_meet();" not in body[arrive:wait] and "barrier.cluster" not in body[arrive:wait]


def test_a_wait_that_ran_out_ends_the_row():
    """A copy that did not land in time may land later: the block waits for every one
    of its copies again, with a short limit, before the cluster's next barrier, tells
    the others, and all of them leave together, with no token."""
    body = _kernel()
    wait = re.search(r"!mbar_wait\(&s_bar\[q\], 0\)\) \{\s*late = true;\s*break;", body)
    vote = body.index("__syncthreads_or(late)")
    drain = re.search(r"if \(lost\) \{.*?for \(int q = 0; q < chunks; \+\+q\) mbar_wait\(&s_bar\[q\], 0, \d+ull\);", body, re.S)
    told, met = body.index("sm_put(to + 20, told.lost)"), body.index("sm_meet();")
    leave = re.search(r"lanes_max\(of\.lost\) > 0\.f\) \{.*?a\.tokens\[row\] = -1;.*?\n    return;", body, re.S)
    assert wait.start() < vote < drain.start() < body.index("sm_wait();") < told < met < leave.start()
    # nothing between the meeting and the way out asks another block for anything
    assert not re.search(r"sm_(?:put|get|count|far)\(", body[met:leave.end()])
    assert body.count("mbar_wait(") == 2
