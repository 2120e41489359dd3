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


def test_the_extension_is_built_for_this_python_and_torch(tmp_path, monkeypatch):
    """It is built again where its source, Python or torch changed since, or where that is asked for; not otherwise."""
    import torch
    from paged_kv_decode_slot_gb300 import build
    started = []

    class Compiler:
        returncode = 0

        def __init__(self, cmd, **kw):
            started.append(cmd)
            open(cmd[cmd.index("-o") + 1], "wb").close()

        def communicate(self):
            return b"", None
    monkeypatch.setattr(build.subprocess, "Popen", Compiler)
    monkeypatch.setattr(build, "ARGS_PATH", str(tmp_path / "tensor_args.so"))

    def builds(force=False):
        before = len(started)
        build.finish_tensor_args(build.start_tensor_args(force))
        return len(started) > before
    assert builds() and not builds() and builds(force=True) and not builds()
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert builds() and not builds()
    assert any("99.0" in arg for arg in started[-1])
    monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    assert builds() and not builds()
    monkeypatch.setattr(sys, "version", "4.0.0 (elsewhere)")
    assert builds() and not builds()
    source = os.path.getmtime(build.ARGS_SOURCE)
    os.utime(tmp_path / "tensor_args.so", (source - 9, source - 9))
    assert builds() and not builds()


ANOTHER_TORCH = """
from paged_kv_decode_slot_gb300 import build
build.build_library()
from paged_kv_decode_slot_gb300 import tensor_args
real = build.args_built_for
import torch
assert tensor_args.built_for == real(torch)
build.args_built_for = lambda torch: real(torch) + " of another day"
from paged_kv_decode_slot_gb300 import binding
assert binding._calls is None and binding._arg is binding._arg_py and binding._maybe is binding._maybe_py
print("PYTHON")
"""


def test_an_extension_built_for_others_is_not_used():
    r = subprocess.run([sys.executable, "-c", ANOTHER_TORCH], cwd=ROOT, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and "PYTHON" in r.stdout, r.stderr[-2000:]


def test_the_package_gives_what_the_binding_has_now(monkeypatch):
    """An entry point replaced in the binding (a wrapper, a stand-in) is seen through the package, used before or not."""
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    import paged_kv_decode_slot_gb300 as pkv
    from paged_kv_decode_slot_gb300 import binding
    before = pkv.pkv_verify_draft
    assert before is binding.pkv_verify_draft
    monkeypatch.setattr(binding, "pkv_verify_draft", len)
    assert pkv.pkv_verify_draft is len
    monkeypatch.undo()
    assert pkv.pkv_verify_draft is before
    monkeypatch.setattr(binding, "_f32", binding._f32)          # what the package does not offer stays the binding's
    assert not hasattr(pkv, "_f32") and not hasattr(pkv, "pkv_nothing")
    from paged_kv_decode_slot_gb300 import step                 # another module's names are its own
    assert pkv.step is step and not hasattr(pkv, "SparseDecodeStep")


def test_plans_of_any_list_are_calls_that_the_library_takes():
    """Partitions of selected-block lists cover them and fit the merge for every group of query heads that attention takes."""
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    from paged_kv_decode_slot_gb300 import binding
    from paged_kv_decode_slot_gb300.step import plan_blocks_attention
    for seqs in (1, 2, 5, 8, 20, 64, 1000, 65535):
        for heads in (1, 2, 8, 40):
            for most in (1, 8, 9, 128, 250, 513, 1000, 16384, 131072, 131073, 1 << 20, 1 << 26):
                p = plan_blocks_attention(seqs, heads, most, 152)
                if p.mode == "split":
                    assert p.partition_blocks * p.max_partitions >= most > p.partition_blocks * (p.max_partitions - 1)
                    assert 8 * p.max_partitions <= binding.IN_KERNEL_MERGE_WEIGHTS, (seqs, heads, most)


def test_clusters_of_a_plan_run_at_once():
    """CTAs of three per SM that fit in clusters of a size on 152 SMs (cudaOccupancyMaxActiveClusters on a GB300)."""
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    from paged_kv_decode_slot_gb300.step import plan_blocks_attention
    fit = {1: 456, 2: 228, 3: 148, 4: 110, 5: 87, 6: 74, 7: 59, 8: 51, 9: 46, 10: 43, 11: 36, 12: 36, 13: 28, 14: 26, 15: 26, 16: 21}
    for units in range(1, 115):
        for most in (9, 40, 128, 250, 257, 500, 512):
            p = plan_blocks_attention(units, 1, most, 152)
            assert p.mode == "split" and fit[p.max_partitions] >= units, (units, most, p)
