"""The training calls' Python side, without a GPU."""
import os
import subprocess
import sys

from ternary_weight_linear_fwd_b200 import build as blbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_sizes_and_layouts_need_no_torch():
    """The package, its library, the layouts and the workspace queries work where torch cannot be imported, and do not
    import it where it can."""
    blbuild.build()
    code = """
import sys
{block}
import ternary_weight_linear_fwd_b200 as bl
assert bl.packed_layout(64, 256)[0] == 64 and bl.layout_version() > 0 and bl.lib()
assert bl.norm_backward_workspace_bytes(100, 2560) > 0
assert bl.backward_weight_workspace_bytes(100, 641, 2560) > 0
w = bl.PackedWeights(640, 2560, 0, 0, None, None, None)
assert bl.backward_input_workspace_bytes(w, 16) == 0
assert not sys.modules.get("torch")
"""
    for block in ("sys.modules['torch'] = None", ""):
        r = subprocess.run([sys.executable, "-c", code.format(block=block)], capture_output=True, text=True, cwd=ROOT)
        assert r.returncode == 0, (block, r.stderr[-2000:])
