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
