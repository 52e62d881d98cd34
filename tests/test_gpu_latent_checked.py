"""The latent-row operators through the bounds-checked build (see tests/test_gpu_checked_build.py): positions in lists and page
tables, pool rows, output and workspace positions.  Every case must give its usual results, and no kernel may record a
violation (checked after every test by the fixture in conftest.py)."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_latent_operators_in_the_checked_build():
    from sparse_mla_kv_gb300 import _build

    _build.build(variant="checked")
    env = dict(os.environ, HS_LIB_VARIANT="checked")
    probe = subprocess.run([sys.executable, "-c", "import sparse_mla_kv_gb300 as hs; print(hs.check_status())"],
                           cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert probe.returncode == 0 and probe.stdout.strip() == "0", probe.stdout + probe.stderr   # not -1: checked
    p = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "-k", "not cold_caches and not beyond_32_bit and not large_row", "tests/test_gpu_latent.py",
                        "tests/test_gpu_latent_edges.py"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert p.returncode == 0, p.stdout[-3000:] + p.stderr[-2000:]
    assert " passed" in p.stdout and "failed" not in p.stdout
