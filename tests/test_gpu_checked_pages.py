"""The page operators through the checked build (tests/test_gpu_checked.py): its in-kernel bounds checks cover the
records that the key bounds and the page scores read and write, the copies of the remap and the compaction, the copies
and stages of the attention over selected pages and the warp states that its merge lays over them.  The tests of
these operators run against that library in a child process; every one of them requires the status word that it
expects, so a check that fires fails them."""
import os
import subprocess
import sys

import pytest

from test_gpu_checked import ROOT, _checked_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_page_operators_through_the_checked_build():
    lib = _checked_library()
    env = dict(os.environ, KVQ3_LIBRARY=lib)
    files = [os.path.join(ROOT, "tests", f) for f in ("test_gpu_pages.py", "test_gpu_pages_range.py",
                                                      "test_gpu_pages_accuracy.py", "test_gpu_pages_lists.py", "test_gpu_stop.py")]
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", *files]
    p = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    print(p.stdout[-2000:])
    assert p.returncode == 0, p.stdout[-4000:] + p.stderr[-2000:]
    probe = subprocess.run([sys.executable, "-c", "import hadamard_rotated_bit_kvq3_gb300 as K; print(K.LIB_PATH)"],
                           cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert probe.stdout.strip() == lib
