"""Waits of the attention over shared prefixes, from its source: each lane of a warp comes to
the same end of a wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_mla_decode_04_gb300", "csrc")


@pytest.fixture(scope="module")
def source():
    with open(os.path.join(CSRC, "shared_decode.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_waits_that_may_give_up_are_a_warps_or_a_threads(source):
    """mbar_wait ends for each lane by itself. Where the others would meet lanes that have given up (at a shuffle
    or a barrier of the warp), the lanes vote; a wait without a flag to give up for is one lane's alone."""
    waits = [m.start() for m in re.finditer(r"\bmbar_wait\s*\(", source)]
    assert waits
    for at in waits:
        depth, end = 1, source.index("(", at) + 1
        while depth:
            depth += {"(": 1, ")": -1}.get(source[end], 0)
            end += 1
        if "abort_flag" in source[at:end]:
            assert re.search(r"__all_sync\(0xffffffffu, $", source[:at]), source[at:end]
        else:
            assert "nullptr" in source[at:end]
