"""The target's side without a GPU: what the sources and their host code say about it, beyond the refusals
and layouts of test_target_host.py."""
import glob
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_drafter_pos_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


@pytest.mark.parametrize("name", sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu"))
                                        if "fence.mbarrier_init" in open(p).read()))
def test_barriers_are_initialised_once(name):
    """Initialising a barrier that is in use is undefined, so every kernel does it in one place, before its fence."""
    text = _source(name)
    assert text.count("fence.mbarrier_init") == 1
    before, after = text.split("fence.mbarrier_init")
    assert "mbar_init_count(" in before and "mbar_init_count(" not in after
