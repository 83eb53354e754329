"""The layer norm and the gradient calls under the bounds-checked library (MOE_CHECKED), in a child process."""
import subprocess
import sys

import pytest

from test_gpu_checked import ROOT, _checked_env

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("files,select", [
    (["tests/test_gpu_norm_bwd.py"], "not 2_31_elements and not row_counts"),
    (["tests/test_gpu_token_bwd.py", "tests/test_gpu_block_grad.py"], "not 2_31_elements"),
])
def test_checked_build_runs_clean(files, select):
    r = subprocess.run([sys.executable, "-m", "pytest", *files, "-q", "-m", "gpu", "-x", "-p", "no:cacheprovider",
                        "-k", select], cwd=ROOT, env=_checked_env(), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and " failed" not in r.stdout
