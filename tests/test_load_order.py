"""One HIP runtime in the process, whichever of the library and torch a program loads first."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
COUNT = "print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))"


@pytest.mark.parametrize("first,then", [("import moe_lora_adapter_amd as m; m.align_capacity(4, 2, 8, 16)", "import torch"),
                                        ("import torch", "import moe_lora_adapter_amd as m; m.lib()")])
def test_one_hip_runtime(first, then):
    out = subprocess.run([sys.executable, "-c", "\n".join([first, then, COUNT])], cwd=ROOT, capture_output=True,
                         text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-500:]
    assert out.stdout.split()[-1] == "1"
