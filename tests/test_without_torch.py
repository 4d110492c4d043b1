"""The package is imported and the C library built without torch, which only
the calls on tensors and the extension over emu_layers.h need."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HIDE = """
import importlib.metadata as md, sys
class No:
    def find_spec(self, name, path=None, target=None):
        if name.split('.')[0] == 'torch':
            raise ModuleNotFoundError("No module named 'torch'", name='torch')
sys.meta_path.insert(0, No())
version = md.version
def without(name):
    if name == 'torch':
        raise md.PackageNotFoundError(name)
    return version(name)
md.version = without
"""


def _run(code):
    r = subprocess.run([sys.executable, "-c", HIDE + code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_import_and_load():
    from fp32_emulated_gemm_split_gb300 import _build
    _build.build()
    assert _run("import fp32_emulated_gemm_split_gb300 as e; print(e.emu_version() > 0, 'torch' in sys.modules)"
                ).split() == ["True", "False"]


def test_build_makes_the_library_and_leaves_the_extension_out():
    """(with the compilers' commands recorded in place of running them)"""
    out = _run("""
from fp32_emulated_gemm_split_gb300 import _build as b
import subprocess, os
ran = []
class Done:
    returncode, stdout, stderr = 0, '', ''
subprocess.run = lambda cmd, **kw: ran.append(cmd) or Done()
moved = []
os.replace = lambda a, to: moved.append(to)
print(b.build(force=True) == b.LIB_PATH, len(ran) == len(b.SOURCES) + 1, moved == [b.LIB_PATH],
      any(b.BIND_SOURCE in x for cmd in ran for x in cmd))
""")
    assert out.split() == ["True", "True", "True", "False"]


def test_the_layers_say_what_is_missing():
    assert "torch" in _run("""
import fp32_emulated_gemm_split_gb300 as e
try:
    e.emu_gated
except ModuleNotFoundError as err:
    print(err)
""")
