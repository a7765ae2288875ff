"""The build without torch: the C library needs hipcc alone.  A stand-in compiler writes the
files that it is asked for, so what is looked at is the order of the steps, not the code."""
import os
import shutil
import stat
import subprocess
import sys

import pytest

PACKAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       "tile_gemm_communication_amd")

COMPILER = """#!/bin/sh
while [ $# -gt 0 ]; do
  if [ "$1" = -o ]; then echo built > "$2"; fi
  shift
done
"""


@pytest.fixture
def package(tmp_path):
    """The build script beside one source, and a compiler for it."""
    (tmp_path / "pkg" / "csrc").mkdir(parents=True)
    shutil.copy(os.path.join(PACKAGE, "build.py"), tmp_path / "pkg" / "build.py")
    (tmp_path / "pkg" / "csrc" / "one.hip").write_text("")
    (tmp_path / "pkg" / "csrc" / "fm_python.cpp").write_text("")
    hipcc = tmp_path / "hipcc"
    hipcc.write_text(COMPILER)
    hipcc.chmod(hipcc.stat().st_mode | stat.S_IXUSR)
    return tmp_path


def _build(package, path=None):
    env = dict(os.environ, HIPCC=str(package / "hipcc"))
    env.pop("PYTHONPATH", None)
    if path:
        env["PYTHONPATH"] = str(path)
    return subprocess.run([sys.executable, "-S", str(package / "pkg" / "build.py")], env=env,
                          capture_output=True, text=True, timeout=60)   # -S: no installed packages


def test_the_library_is_built_without_torch(package):
    r = _build(package)
    assert r.returncode == 0, r.stderr
    assert (package / "pkg" / "libfluxmi.so").exists()
    assert not (package / "pkg" / "_fluxmi.so").exists()
    assert "_fluxmi.so" in r.stderr and "torch" in r.stderr      # says what is left out, and why


def test_a_module_that_does_not_build_leaves_the_library(package):
    (package / "lib" / "torch").mkdir(parents=True)
    (package / "lib" / "torch" / "__init__.py").write_text("")   # a torch without its headers
    r = _build(package, package / "lib")
    assert r.returncode != 0
    assert (package / "pkg" / "libfluxmi.so").exists()
