"""The norms and clipping of lists under the self-checking debug library: no access leaves its extent or alignment."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_grad_clip_suites_record_no_violation_under_the_debug_build():
    from fsdp_sharded_mixed_flatparameter_gb300 import build
    build.build(debug=True)
    env = dict(os.environ, ZERO_SHARD_DEBUG="1")
    p = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_gpu_grad_clip.py", "tests/test_gpu_grad_clip_steps.py"], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=1800)
    assert p.returncode == 0, p.stdout[-4000:] + p.stderr[-2000:]
