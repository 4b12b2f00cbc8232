"""The checked build (SS_BOUNDS_CHECK) on the linear attention and the state pool.

In that build every global index that these kernels form is compared with its tensor's
extent (for a strided operand what its strides reach) before the access, but for tiles that
TMA fetches, which clips them itself.  The small and odd shapes, rows of no tokens, plain
loads, segments, heads cut between CTAs and padding slots run against libssscan_checked.so
in a child process, each test followed by a look at the error word.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SELECTION = [
    "tests/test_gpu_linattn.py::test_fwd",
    "tests/test_gpu_linattn.py::test_fwd_strided_shared_heads",
    "tests/test_gpu_linattn.py::test_fwd_segments",
    "tests/test_gpu_linattn.py::test_more_heads_than_sms",
    "tests/test_gpu_linattn.py::test_fwd_lengths_and_rows_behind",
    "tests/test_gpu_linattn.py::test_fwd_broadcast_decay_and_no_state",
    "tests/test_gpu_linattn.py::test_fwd_state_in_place_and_pieces",
    "tests/test_gpu_linattn.py::test_bwd",
    "tests/test_gpu_linattn.py::test_bwd_strided_shared_heads",
    "tests/test_gpu_linattn.py::test_bwd_segments_and_anchors",
    "tests/test_gpu_linattn.py::test_bwd_lengths",
    "tests/test_gpu_linattn.py::test_step",
    "tests/test_gpu_linattn.py::test_step_slots_padding_and_doubles",
    "tests/test_gpu_linattn.py::test_prompt_pool_prompt_steps",
    "tests/test_gpu_linattn_decay_grad.py::test_lengths_of_a_chunk",
    "tests/test_gpu_linattn_decay_grad.py::test_strided_rows_and_a_token_that_forgets",
    "tests/test_gpu_linattn_cuts.py::test_more_heads_than_sms",
    "tests/test_gpu_state_pool.py",
]


def test_under_the_checked_build():
    from selective_state_space_ss_b200 import build as B

    lib = B.build_checked()
    env = dict(os.environ, SSSCAN_LIBRARY=lib, SS_CHECK_ERROR_WORD="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        *SELECTION], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=1800)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
