"""The package without torch: its binding needs none."""
import subprocess
import sys

import pytest

from conftest import ROOT

BLOCKED = """
import sys
class NoTorch:
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ModuleNotFoundError(f"No module named {name!r}", name=name)
sys.meta_path.insert(0, NoTorch())
"""


def run(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_all_names_without_torch():
    out = run(BLOCKED + "from scale_factor_layout_b200 import *\nprint(mx_rearranged_size.__name__, rearrange.__name__, 'expert_sort' in globals())")
    assert out.split() == ["mx_rearranged_size", "rearrange", "False"]


def test_an_operator_without_torch_says_what_is_missing():
    out = run(BLOCKED + "import scale_factor_layout_b200 as m\ntry:\n    m.expert_sort\nexcept ModuleNotFoundError as e:\n    print(e.name)")
    assert out.split() == ["torch"]


def test_all_names_with_torch():
    pytest.importorskip("torch")
    out = run("from scale_factor_layout_b200 import *\nprint(expert_sort.__module__, grouped_matmul_k.__name__, rearrange.__name__)")
    assert out.split() == ["scale_factor_layout_b200.moe", "grouped_matmul_k", "rearrange"]


def test_importing_the_package_imports_no_torch():
    assert run("import sys, scale_factor_layout_b200\nprint('torch' in sys.modules)").split() == ["False"]
