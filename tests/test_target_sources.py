"""The target's side without a GPU: what the sources and their host code say about it, beyond the refusals
and layouts of test_target_host.py."""
import glob
import os
import shutil
import subprocess

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


def _host_check(tmp_path, name, *flags):
    gxx, inc = shutil.which("g++"), "/usr/local/cuda/include"
    if gxx is None or not os.path.exists(os.path.join(inc, "cuda.h")):
        pytest.skip("g++ or the CUDA headers are missing")
    exe = str(tmp_path / "check")
    subprocess.run([gxx, "-std=c++17", "-O2", *flags, "-I", CSRC, "-I", inc, os.path.join(ROOT, "tests", name), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.startswith("ok "), out.stdout


def test_requests_of_a_run(tmp_path):
    """Those that a CTA flags when one of its waits gives up."""
    _host_check(tmp_path, "paged_run_check.cpp")


def test_the_longest_caches_stay_in_32_bits(tmp_path):
    _host_check(tmp_path, "paged_limits_check.cpp", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover")


def test_a_wait_that_gives_up_spoils_its_whole_run():
    """Every role marks its CTA (none flags one request alone), the joining kernel flags the run, and partials that never
    come are NaN."""
    text, join = _source("paged_chunk.cu"), _source("paged_attention.cu")
    assert text.count("a.desc[8 * c + 6] = 1;") == 3 and "status[cc.r]" not in text and "status[cs.r]" not in text
    assert text.count("a.desc[8 * c + 6] = 0;") == 1 and text.index("make_float2(NAN, NAN)") < text.index("tcgen05.alloc")
    combine = join[join.index("paged_combine_kernel("):]
    assert combine.index("flag_run(a, blockIdx.x)") < combine.index("if (d0.x < 0) return;") and "paged_in_run(" in join
