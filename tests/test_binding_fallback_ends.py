"""The operators at the ends of a language model through ctypes, where the package
stands without its extension module."""
import os
import shutil
import subprocess
import sys

from test_binding_fallback import PACKAGE, ROOT


def test_refusals_without_the_extension_module(tmp_path):
    copy = tmp_path / "matmul_selection_gb300"
    (copy / "_build").mkdir(parents=True)
    shutil.copy(os.path.join(PACKAGE, "__init__.py"), copy)
    os.symlink(os.path.join(PACKAGE, "_build", "libmm_gb300.so"), copy / "_build" / "libmm_gb300.so")
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(tmp_path), ROOT]))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_ends_cpu.py")], cwd=tmp_path, env=env,
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
