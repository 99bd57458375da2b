"""The library is a C ABI without torch: building it needs no torch, which only the binding's call module is compiled against."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HIDE = """
import sys
class Hide:
    def find_spec(self, name, path=None, target=None):
        if name == "torch" or name.startswith("torch."):
            raise ModuleNotFoundError(f"No module named {name!r}", name=name)
sys.meta_path.insert(0, Hide())
"""


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)


def test_the_library_builds_without_torch():
    import __graft_entry__
    __graft_entry__.build()  # so that nothing is left to compile below
    r = run(HIDE + "from chunked_prefill_causal_gb300 import build\nprint(build.build())")
    assert r.returncode == 0, r.stderr
    assert os.path.exists(r.stdout.strip())


def test_a_torch_that_is_there_gets_its_call_module():
    from chunked_prefill_causal_gb300 import build
    build.build()
    assert os.path.exists(build.call_module_path())


def test_a_broken_torch_is_not_taken_for_a_missing_one():
    """Only an absent torch leaves the call module out; any other failure to import it is an error of the build."""
    r = run("import sys\nclass Broken:\n    def find_spec(self, name, path=None, target=None):\n        if name == 'torch':\n"
            "            raise ImportError('broken', name=name)\nsys.meta_path.insert(0, Broken())\n"
            "from chunked_prefill_causal_gb300 import build\nbuild.build()")
    assert r.returncode != 0 and "broken" in r.stderr


def test_the_call_module_names_its_python(monkeypatch):
    """Its binary interface is that of one Python and one torch: another of either never loads it."""
    import sysconfig

    from chunked_prefill_causal_gb300 import build
    mine = build.call_module_path()
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: ".cpython-399-some-os.so" if name == "EXT_SUFFIX" else None)
    assert build.call_module_path() != mine
    monkeypatch.undo()
    import torch
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    assert build.call_module_path() != mine
