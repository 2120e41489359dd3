"""What the build needs and when it builds again (no GPU, and no compiler is run)."""
from __future__ import annotations

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT_TORCH = """
import sys
sys.modules["torch"] = None                                     # importing it raises ImportError
from paged_kv_decode_slot_gb300 import build
commands = []

class Compiler:
    returncode = 0
    def __init__(self, cmd, **kw):
        commands.append(cmd)
    def communicate(self):
        return b"", None

build.subprocess.Popen = Compiler
build.subprocess.check_call = lambda cmd: open(cmd[cmd.index("-o") + 1], "wb").close()
build.nvcc_path = lambda: "nvcc"
build.ARGS_PATH = build.LIB_PATH = sys.argv[1] + "/lib.so"
build.BUILD_DIR = sys.argv[1]
assert build.build_library() == build.LIB_PATH
assert len(commands) == len(build.SOURCES) and all(cmd[0] == "nvcc" for cmd in commands)
print("BUILT")
"""


def test_the_library_builds_without_torch(tmp_path):
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH, str(tmp_path)], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "BUILT" in r.stdout, r.stderr[-2000:]
    assert "tensor_args is not built (no torch" in r.stderr
