"""How the warps of the latent cache's and the prompts' kernels wait on one another, read from
their source, as test_window_waits does for the window's: a wait that gives up is reached by
no valid input."""

import re

import pytest

from test_window_waits import source


@pytest.mark.parametrize("name,waits", [("latent_attend.cu", 1), ("prompt.cu", 1)])
def test_every_wait_is_the_whole_warps(name, waits):
    """Roles wait through warp_wait alone, in one place each."""
    text = source(name)
    assert not re.search(r"\brole_wait\(", text) and len(re.findall(r"\bwarp_wait\(", text)) == waits


@pytest.mark.parametrize("name,barriers", [("latent_attend.cu", ["key_full", "value_full"]),
                                           ("prompt.cu", ["q_full", "key_full", "value_full"])])
def test_copies_end_before_the_block_does(name, barriers):
    """A copying warp that gives up waits for each barrier that its tensor copies complete on."""
    text = source(name)
    at = text.index("CopyWarp) {")
    asked = set(re.findall(r"first_cta\(&ctl\.(\w+)\[", text[at:text.index("MatrixWarp) {", at)]))
    drains = [m for m in re.finditer(r"if \(!ok && rank == 0 [^{]*\{", text)]
    assert asked == set(barriers) and len(drains) == 1
    drain = text[drains[0].end():text.index("} else if", drains[0].end())]
    assert set(re.findall(r"mbar_wait\(smem_addr\(&ctl\.(\w+)\[", drain)) == asked


def test_prompt_weights_are_written_before_the_columns_are_freed():
    """As in the window's kernel: no warp leaves between a store to tensor memory and its end."""
    text = source("prompt.cu")
    at = text.index("tmem_store16(scores")
    assert "break" not in text[at:text.index("tmem_wait_store();", at)]
