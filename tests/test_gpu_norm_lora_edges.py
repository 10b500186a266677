"""Layer norm and low-rank adapters at sizes and in orders of calls where the launch itself, or the
hand-over of a buffer inside a kernel, can go wrong.  The results are compared as in the operators'
own tests, whose tolerances are derived there."""
import os
import subprocess
import sys

import pytest

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("M,L", [(1000, 383), (993, 381), (512, 767), (481, 762), (256, 1535), (225, 1524)])
def test_first_plan_of_a_process(M, L):
    """Counters of just under 48 KB beside the kernel's static arrays, with no larger plan before them in the process."""
    need_gpu()
    p = subprocess.run([sys.executable, "-c", f"from tests.test_gpu_lora import test_plan; test_plan({M}, {L})"],
                       cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-2000:]
