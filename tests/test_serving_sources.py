"""Serving many samples of one prompt without a GPU: what the kernels' sources and host code say."""
import re

import pytest

from test_target_sources import _host_check, _source


def test_what_a_prefix_launch_spoils(tmp_path):
    """Where a wait gives up: the groups of the CTA's run, and all of their rows in the workspace."""
    _host_check(tmp_path, "paged_give_up_check.cpp", "-fsanitize=undefined", "-fno-sanitize-recover")


def test_rows_that_overlap(tmp_path):
    _host_check(tmp_path, "rows_apart_check.cpp")


@pytest.mark.parametrize("name", ["paged_chunk.cu", "paged_prefix.cu"])
def test_no_output_is_announced_after_a_failed_wait(name):
    """The products' warp: the one commit on which a unit's rows are written hangs on all of its waits so far, and comes after
    those of the tile's values and weights."""
    text = _source(name)
    assert re.findall(r"mma_commit\(([^,]+), o_done", text) == ["go & fine"]
    outputs = text[text.index("auto outputs = [&]"):text.index("mma_commit(go & fine, o_done")]
    assert outputs.count("fine &= mbar_wait_warp(") == 3
