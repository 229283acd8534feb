"""How the attention's warps wait on one another, read from the kernels' source: a
wait that gives up is reached by no valid input, and no input may be made to hang a
GPU to reach it.

Tensor-memory instructions, full-mask shuffles and named barriers are executed by a
warp as a whole.  A wait whose answer differs between lanes would send some lanes of a
warp to the end of the block and leave the others in such an instruction for ever, so
every wait of a role gives one answer to its whole warp."""

import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "confidence_scheduled_speculative_gb300", "csrc")


def source(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["attend.cu", "fewrows.cuh", "schedule.cuh", "tensor.cuh"])
def test_a_lane_waits_with_its_warp(name):
    """A look at a barrier by one lane stands only inside a vote of all lanes."""
    text = source(name)
    calls = [m.start() for m in re.finditer(r"\brole_wait\(", text)]
    definition = re.search(r"bool role_wait\(", text)
    if definition:
        calls.remove(definition.end() - len("role_wait("))
    for at in calls:
        vote = text.rfind("__all_sync(", 0, at)
        assert vote >= 0 and ";" not in text[vote:at], text[at - 60:at + 60]


def test_every_role_waits():
    """The check above has something to look at: five roles' waits."""
    assert len(re.findall(r"\bwarp_wait\(", source("attend.cu"))) == 5


def test_weights_are_written_before_the_columns_are_freed():
    """A warp that gives up after storing weights to tensor memory waits for the store
    first: once all warps have come to the end the columns go to another block."""
    text = source("attend.cu")
    for m in re.finditer(r"tmem_store_pairs16\(", text):
        leave = text.index("if (!ok) break;", m.end())
        assert "tmem_wait_store();" in text[m.end():leave]
