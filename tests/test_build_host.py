"""What the build runs, with the compilers replaced by a record of their command lines."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import importlib.util, os, sys
if sys.argv[1] == "without":
    sys.modules["torch"] = None  # as where it is not installed
spec = importlib.util.spec_from_file_location("b", os.path.join(%r, "allreduce_compatible_gradient_gb300", "_build.py"))
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.PKG = b.OBJ_DIR = sys.argv[2]
b.LIB = os.path.join(sys.argv[2], "libgq.so")
seen = []

def run(command, **kw):
    seen.append(os.path.basename(command[0]))
    open(command[command.index("-o") + 1], "w").close()

class Popen:
    returncode = 0

    def __init__(self, command):
        run(command)

    def wait(self):
        return 0
b.subprocess.run, b.subprocess.Popen = run, Popen
assert b.build_library(force=True) == b.LIB and os.path.exists(b.LIB)
print(seen.count("nvcc"), seen.count("g++"), len(b.UNITS))
"""


def commands(which, folder):
    r = subprocess.run([sys.executable, "-c", SCRIPT % ROOT, which, str(folder)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return [int(v) for v in r.stdout.split()]


def test_the_library_needs_nvcc_alone(tmp_path):
    nvcc, gxx, units = commands("without", tmp_path)
    assert nvcc == units + 1 and gxx == 0


def test_the_extension_is_built_beside_it(tmp_path):
    nvcc, gxx, units = commands("with", tmp_path)
    assert nvcc == units + 1 and gxx == 1
