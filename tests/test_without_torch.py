"""Host test of a build without torch: the other tests are still collected."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_collection(tmp_path):
    (tmp_path / "torch.py").write_text("raise ModuleNotFoundError('no torch')\n")
    env = {**os.environ, "PYTHONPATH": str(tmp_path)}
    r = subprocess.run([sys.executable, "-m", "pytest", "tests", "--collect-only", "-q", "-m", "not gpu", "-p", "no:cacheprovider"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=110)
    assert r.returncode == 0, r.stdout[-2000:]
    assert "tests/test_host.py::" in r.stdout and "tests/test_ops.py::" not in r.stdout
