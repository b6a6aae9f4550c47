"""Serving many samples of one prompt without a GPU: what the kernels' host code says."""
from test_target_sources import _host_check


def test_what_a_prefix_launch_spoils(tmp_path):
    """Where a wait gives up: the groups of the CTA's run, and all of their rows in the workspace."""
    _host_check(tmp_path, "paged_give_up_check.cpp", "-fsanitize=undefined", "-fno-sanitize-recover")
