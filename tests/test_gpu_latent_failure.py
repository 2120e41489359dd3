"""Expiring in-kernel waits of attention over a latent cache: no fault, no hang, the context stays usable.

As in test_gpu_failure.py: a test build of the library (-DPKV_TEST_HOOKS) withholds one tile of every sequence (from it on
nothing is loaded or signalled in that CTA) under a limit of 1 ms, so the waits on it expire in every role, and in both CTAs of
a pair; copies already issued have to land, MMAs to finish and tensor memory to be released before the CTAs leave.  Only
PKV_FLAG_TIMEOUT may be flagged, and it must be.  The same call then runs with the defaults and must give what it gave before."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
for _p in (ROOT, HERE):
    if _p not in sys.path:
        sys.path.insert(0, _p)

from test_gpu_failure import hooks_lib  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# heads, new tokens, lengths
CASES = {
    "16 rows": (16, 1, [900, 70, 3000]),
    "32 rows": (8, 4, [900, 70, 3000]),
    "pairs": (128, 1, [900, 70, 3000]),
    "pairs, one of them with rows": (40, 1, [2000] * 100),
    "pairs, several chunks": (100, 3, [500, 129, 1000]),
    "48 rows": (24, 2, [900, 70, 3000]),
    "pairs, the second CTA without rows": (60, 1, [2000] * 100),
}


@pytest.mark.parametrize("case", CASES)
def test_latent_attention_survives_expired_waits_and_recovers(hooks_lib, case):  # noqa: F811
    env = dict(os.environ, PKV_LIBRARY=hooks_lib)
    r = subprocess.run([sys.executable, os.path.abspath(__file__), case], env=env, cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "RECOVERED" in r.stdout, (r.stdout[-4000:], r.stderr[-4000:])


def expired_waits_case(case: str) -> None:
    """One case, in a process whose library is the test build (PKV_LIBRARY)."""
    import paged_kv_decode_slot_gb300 as pkv
    from paged_kv_decode_slot_gb300 import binding
    from test_gpu_latent import Case
    assert binding.HAS_TEST_HOOKS, "the child must load the -DPKV_TEST_HOOKS build"
    N, T, ctx = CASES[case]
    c = Case(len(case), ctx, N, T).poison()

    def run(flag=0):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = c.run(pkv, err=err)
        torch.cuda.synchronize()
        assert pkv.pkv_read_err_flag(err)[1] == flag, f"flags {pkv.pkv_read_err_flag(err)[1]:#x}"
        return out, lse
    want = run()
    c.check(*want)
    for tile in (0, 1, 2, 5):
        prev, off = pkv.pkv_set_wait_limit_ns(1_000_000), pkv.pkv_debug_withhold_tile(tile)
        run(pkv.PKV_FLAG_TIMEOUT)
        pkv.pkv_debug_withhold_tile(off)
        pkv.pkv_set_wait_limit_ns(prev)
        got = run()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got)), f"tile {tile}"


if __name__ == "__main__":
    expired_waits_case(sys.argv[1])
    print("RECOVERED", flush=True)
