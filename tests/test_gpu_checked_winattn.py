"""The checked build (SS_BOUNDS_CHECK) on the window attention, its cache and the rotation.

In that build every global index that these kernels form is compared with its tensor's
extent before the access, but for tiles that TMA fetches, which clips them itself.  The
small and odd shapes run against libssscan_checked.so in a child process, each test
followed by a look at the error word.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SELECTION = ["tests/test_gpu_winattn.py::test_" + n for n in (
    "widths", "masks", "strided_shared_heads", "sinks_of_a_long_row", "rows_behind_a_length_are_neither_read_nor_written",
    "broadcast_and_reversed_operands", "many_heads", "the_end_of_a_strided_operand")] + [
    "tests/test_gpu_winattn_cache.py::test_" + n for n in (
        "widths_and_lengths", "pages", "several_tokens", "long_rows_cut_between_blocks",
        "lengths_out_of_range_and_pages_that_are_none", "entries_that_no_visible_token_lies_in_are_not_followed",
        "strided_queries_and_shared_pages", "rotate", "rotate_strided_in_place_and_counts", "append",
        "append_without_queries_and_in_place", "a_dialogue")]


def test_under_the_checked_build():
    from selective_state_space_ss_b200 import build as B

    lib = B.build_checked()
    env = dict(os.environ, SSSCAN_LIBRARY=lib, SS_CHECK_ERROR_WORD="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        *SELECTION], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=1800)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
