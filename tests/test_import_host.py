"""The binding without torch: the library builds, opens and refuses without it (no GPU)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys

class NoTorch:
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ImportError("no torch here")

sys.meta_path.insert(0, NoTorch())
import __graft_entry__
__graft_entry__.build()
from moe_task_scheduling_gb300 import etmoe as E
assert E.load().et_version() > 0
assert E.et_moe_workspace_bytes(16, 256, 512, 8, 2) > 0 and E.et_w4_gemv_workspace_bytes(1, 8, 32, 32) > 0
assert E.load().et_w4_gemv(None, 16, 16, 16, 1, None, 1, 8, 32, 32, 256, 256, None) == E.ET_ERR_INVALID
assert E._ptr(4096) == 4096 and E._stream(7) == 7
assert "torch" not in sys.modules
print("ok")
"""


def test_the_library_opens_without_torch():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
