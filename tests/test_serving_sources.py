"""CPU tests of two rules that the serving kernels' sources keep, where a run
cannot show a breach: it would need an unlucky moment."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "moe_gemm_gb300", "csrc")
SERVING = ["gate.cu", "paged_kv.cu", "paged_attention.cu", "paged_attention.cuh",
           "paged_attention_tiles.cu", "paged_schedule.cuh"]


def code_of(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", SERVING)
def test_no_read_only_loads(name):
    # A kernel launched early starts while the one before still writes what it will read
    # (logits, q, block tables): after its wait ordinary loads see that, those for data that
    # is read-only for a kernel's whole life need not. The compiler makes such loads of
    # pointers to const that are __restrict__.
    found = re.findall(r"__ldg|ld\.global(?:\.\w+)*\.nc|__restrict__", code_of(name))
    assert found == []


@pytest.mark.parametrize("name", ["paged_attention.cu", "paged_attention_tiles.cu"])
def test_waits_that_give_up_are_voted_on(name):
    # What follows a wait are votes and shuffles of the whole warp. A lane that leaves alone,
    # because the barrier completed for the others just as its own wait ran out, would leave
    # them waiting for it. (The waits with `never` end a warp's work.)
    waits = [s for s in code_of(name).split(";") if re.search(r"\bmbar_wait\(", s)]
    assert waits
    assert [s for s in waits if "__all_sync" not in s and "&never" not in s] == []
