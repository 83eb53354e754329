"""The 4-bit products and the norm under the bounds-checked library (MOE_CHECKED): every fetch of codes, scales and
activations and every store of a tile is tested against its tensor's size, and the experts' tests require a clean
status word.  The tests run in a child process, which loads the checked build."""
import subprocess
import sys

import pytest

from test_gpu_checked import ROOT, _checked_env

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("files,select", [
    (["tests/test_gpu_w4.py"], "not 4_gib"),
    (["tests/test_gpu_w4_tables.py", "tests/test_gpu_w4_expert_parallel.py"], ""),
    (["tests/test_gpu_norm.py"], "not 2_31_elements"),
])
def test_checked_build_runs_clean(files, select):
    r = subprocess.run([sys.executable, "-m", "pytest", *files, "-q", "-m", "gpu", "-x", "-p", "no:cacheprovider",
                        "-k", select], cwd=ROOT, env=_checked_env(), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and " failed" not in r.stdout
