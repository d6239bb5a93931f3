"""The package without its extension module: the operators' calls go through
ctypes, with the same checks."""
import os
import shutil
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "matmul_selection_gb300")


def test_import_and_refusals_without_the_extension_module(tmp_path):
    copy = tmp_path / "matmul_selection_gb300"
    (copy / "_build").mkdir(parents=True)
    shutil.copy(os.path.join(PACKAGE, "__init__.py"), copy)
    os.symlink(os.path.join(PACKAGE, "_build", "libmm_gb300.so"), copy / "_build" / "libmm_gb300.so")
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([str(tmp_path), ROOT]))
    r = subprocess.run([sys.executable, "-c", "import matmul_selection_gb300 as mm; print(mm.__file__); "
                        "print(mm._fast.__name__)"], cwd=tmp_path, env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == [str(copy / "__init__.py"), "_Ctypes"]
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_operators_cpu.py")], cwd=tmp_path, env=env,
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
