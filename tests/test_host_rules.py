"""Host-side rules of the library that need no GPU, in small C++ programs."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "matmul_selection_gb300", "csrc")


def run(name, tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    exe = str(tmp_path / name)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread", "-I", CSRC,
                    os.path.join(HERE, "cpp", name + ".cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


def test_scratch_outlives_the_graphs_that_hold_it(tmp_path):
    run("scratch_test", tmp_path)


def test_set_up_is_kept_for_each_device(tmp_path):
    run("per_device_test", tmp_path)


def test_e4m3_product_chooses_a_form_that_takes_the_size(tmp_path):
    run("q8_choice_test", tmp_path)
