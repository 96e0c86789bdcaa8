"""The verdict of a bounded wait that a whole warp takes (no GPU needed).

Each lane that polls a barrier measures its own time, so near the limit some lanes can see the barrier pass and
others give up. Where votes, shuffles or matrix instructions of the whole warp follow, the warp has to leave or go on
as one: the lanes' verdicts are joined by __all_sync. Looked up in the sources of the kernels whose waiting warps go
on to such instructions: every wait is joined.
"""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "fp8_quant_memory_gb300", "csrc")
JOINED = "__all_sync(0xffffffffu, mbar_wait("
# The exception: waits after which a lane only leaves a loop of further waits, for copies already issued to land before
# the block ends.
DRAIN = re.compile(r"^if \(!mbar_wait\(kWaitLimitNs, &(sm\.)?full\[\w+ % [\w.:]+\], .*\) break;$")


@pytest.mark.parametrize("name, fewest", [("fq_attention.cu", 4), ("fq_append.cu", 3)])
def test_every_warp_takes_one_verdict(name, fewest):
    with open(os.path.join(CSRC, name)) as f:
        code = [line.split("//")[0].strip() for line in f]
    waits = [(n, line) for n, line in enumerate(code, 1) if "mbar_wait(" in line]
    assert len(waits) >= fewest
    bad = [w for w in waits if JOINED not in w[1] and not DRAIN.match(w[1])]
    assert not bad, bad
