"""The compiled binding is built for one Python and one torch, and is not loaded under others (no GPU
needed)."""
import os
import subprocess
import sys

import torch

import mamba_ssd_scan_03_b200 as ssd
from mamba_ssd_scan_03_b200 import build as ssd_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def call_under(version):
    """What a first call says under a torch of that version."""
    code = ("import torch\n"
            f"torch.__version__ = {version!r}\n"
            "import mamba_ssd_scan_03_b200 as ssd\n"
            "try:\n"
            "    ssd.group_norm_gate(torch.zeros(2, 8), torch.zeros(8))\n"
            "except Exception as e:\n"
            "    print(type(e).__name__, e)\n")
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, capture_output=True,
                          text=True).stdout


def test_binding_is_of_this_python_and_torch():
    ssd_build.build()
    assert os.path.exists(ssd.BINDING_PATH)
    name = os.path.basename(ssd.BINDING_PATH)
    assert sys.implementation.cache_tag in name and torch.__version__ in name
    said = call_under(str(torch.__version__))
    assert said.startswith("ValueError") and "CUDA" in said  # loaded: it refuses host tensors


def test_binding_of_another_torch_is_not_loaded():
    ssd_build.build()
    said = call_under("0.1.2")
    assert said.startswith("RuntimeError") and "0.1.2" in said and "is missing" in said
