"""The operators between the serving calls where their sizes and values end (64-bit forms of
tests/step_reference.py)."""
import os
import subprocess
import sys

import pytest

from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


# ------------------------------------------------------------------ logits
FRESH = """
import sys
sys.path.insert(0, {here!r})
sys.path.insert(0, {root!r})
import test_gpu_step as S
x, kw = S.logits_case(1, 1, {V}, 40, {nb}, 5)
for probs in (True, False):
    S.check_logits(x, kw, probabilities=probs)
print("fine")
"""


@pytest.mark.parametrize("V,nb", [(50257, 286), (50257, 300), (50257, 341), (65536, 342), (32769, 1024)])
def test_biases_that_end_near_the_default_limit_of_shared_memory(V, nb):
    """16 values a thread and 286 to 341 biases ask for just less than 48 KB.  Each in a process of
    its own: a larger call before would have raised the kernel's limit for good."""
    code = FRESH.format(here=HERE, root=os.path.dirname(HERE), V=V, nb=nb)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
