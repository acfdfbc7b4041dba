"""The package without its C++ module: everything but the paged cache's calls is there."""
import os
import subprocess
import sys
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = "int4_block_quantized_matmulnbits_b200"

# each puts something in the way of the module before the package is imported
NO_MODULE = """
import sys
class Finder:
    def find_spec(self, name, path=None, target=None):
        if name == "{pkg}._binding":
            raise ImportError("libtorch_python.so: cannot open shared object file")
sys.meta_path.insert(0, Finder())
"""
OTHER_TORCH = """
import sys, types
m = types.ModuleType("{pkg}._binding")
m.torch_version = "1.0"
sys.modules["{pkg}._binding"] = m
"""
NO_COMPILER = """
import importlib.util, os, sys, types
spec = importlib.util.spec_from_file_location("{pkg}.build", os.path.join("{pkg}", "build.py"))
class Finder:
    def find_spec(self, name, path=None, target=None):
        if name == "{pkg}.build":
            return spec
spec.loader.exec_module, run = None, spec.loader.exec_module
def exec_module(m):
    run(m)
    def fails(*a):
        raise FileNotFoundError("g++")
    m.build_binding = fails
spec.loader.exec_module = exec_module
sys.meta_path.insert(0, Finder())
"""
USE = """
import torch
import {pkg} as mnb
from {pkg} import step
print(mnb.mnb_packed_sizes(64, 64, 32, torch.float16, True))
i = torch.zeros(4, dtype=torch.int32)
try:
    mnb.mnb_paged_tables(i, i, i.view(4, 1), 16, 3, i, i[:1], i, i, i, i, i[:1])
except ImportError as e:
    print(e)
"""


@pytest.mark.parametrize("way,why", [(NO_MODULE, "cannot open"), (OTHER_TORCH, "built for torch 1.0"),
                                     (NO_COMPILER, "FileNotFoundError: g++")],
                         ids=["no module", "other torch", "no compiler"])
def test_the_rest_runs_without_the_module(way, why):
    r = subprocess.run([sys.executable, "-c", (way + USE).format(pkg=PKG)], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    sizes, told = r.stdout.strip().split("\n")
    assert sizes == "(2048, 256, 64)"
    assert "the paged cache's calls need" in told and why in told


def test_the_module_is_this_pythons_and_this_torchs():
    import torch

    import int4_block_quantized_matmulnbits_b200 as mnb

    assert os.path.basename(mnb._binding.__file__) == "_binding" + sysconfig.get_config_var("EXT_SUFFIX")
    assert mnb._binding.torch_version == str(torch.__version__)
