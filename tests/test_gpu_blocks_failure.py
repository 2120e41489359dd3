"""Expiring in-kernel waits of attention over selected blocks: no fault, no hang, the context and the workspace stay usable.

As in test_gpu_failure.py: a test build of the library (-DPKV_TEST_HOOKS) withholds one tile of every CTA (no load, no arrival on
its barrier) under a limit of 1 ms, so the consumer's bounded wait on it expires and the producers' waits behind it are
given up while other tiles of the same batch were issued already -- each of those copies has to be waited for before the ring is
used again.  Only PKV_FLAG_TIMEOUT may be flagged, and it must be.  The same call then runs with the defaults and must give
what it gave before."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
for _p in (ROOT, HERE):
    if _p not in sys.path:
        sys.path.insert(0, _p)

from test_gpu_failure import hooks_lib  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# kind of pools, head size, sequences, KV heads, list entries, entries a partition (0: whole lists)
CASES = {
    "whole lists, eight warps": ("bf16", 128, 2, 4, 60, 0),
    "whole lists, four warps": ("bf16", 128, 20, 8, 40, 0),
    "whole lists, H = 64": ("bf16", 64, 3, 2, 60, 0),
    "whole lists, e4m3": ("e4m3_block", 128, 2, 4, 100, 0),
    "whole lists, e4m3, four warps": ("e4m3_head", 128, 40, 8, 60, 0),
    "clusters": ("bf16", 128, 3, 2, 90, 30),
    "clusters, e4m3": ("e4m3_block", 128, 3, 2, 120, 60),
    "workspace": ("bf16", 128, 3, 2, 400, 20),
    "workspace, e4m3": ("e4m3_head", 128, 2, 2, 800, 40),
}


@pytest.mark.parametrize("case", CASES)
def test_block_attention_survives_expired_waits_and_recovers(hooks_lib, case):  # noqa: F811
    env = dict(os.environ, PKV_LIBRARY=hooks_lib)
    r = subprocess.run([sys.executable, os.path.abspath(__file__), case], env=env, cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "RECOVERED" in r.stdout, (r.stdout[-4000:], r.stderr[-4000:])


def expired_waits_case(case: str) -> None:
    """One case, in a process whose library is the test build (PKV_LIBRARY)."""
    import ops_ref as R
    import paged_kv_decode_slot_gb300 as pkv
    from devutil import bf16_dev, i32_dev, out_f64
    from paged_kv_decode_slot_gb300 import binding
    assert binding.HAS_TEST_HOOKS, "the child must load the -DPKV_TEST_HOOKS build"
    kv, H, B, K, M, pb = CASES[case]
    N, r = 2 * K, np.random.default_rng(len(case))
    ctx = [16 * M - 5] * B
    tab, pool = R.tables(r, ctx)
    q = bf16_dev(R.to_bf16(r.standard_normal((B, N, H))))
    sel = torch.arange(M, dtype=torch.int32, device="cuda").expand(B, K, M).contiguous()
    out, lse = torch.zeros_like(q), torch.zeros(B, N, device="cuda")
    parts = -(-M // pb) if pb else 0
    ws = torch.zeros(pkv.pkv_splitk_workspace_bytes(B, N, H, parts), dtype=torch.uint8, device="cuda") if pb else None
    if kv == "bf16":
        pools = [torch.randn(pool, 16, K, H, device="cuda").bfloat16() for _ in range(2)]
    else:
        pools = [torch.randint(0, 0x50, (pool, 16, K, H), device="cuda").to(torch.uint8) for _ in range(2)]
        pools += [torch.rand(*((pool, K) if kv == "e4m3_block" else (K,)), device="cuda") + 0.1 for _ in range(2)]
    attend = pkv.pkv_decode_attn_blocks if kv == "bf16" else pkv.pkv_decode_attn_blocks_fp8

    def run(flag=0):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pkv.check(attend(q, *pools, i32_dev(tab), i32_dev(ctx), sel, H ** -0.5, out, lse, pb, parts, ws, err))
        torch.cuda.synchronize()
        assert pkv.pkv_read_err_flag(err)[1] == flag, f"flags {pkv.pkv_read_err_flag(err)[1]:#x}"
        return out.clone(), lse.clone()
    want = run()
    assert np.isfinite(out_f64(want[0])).all()
    for tile in (0, 1, 3, 6):
        prev, off = pkv.pkv_set_wait_limit_ns(1_000_000), pkv.pkv_debug_withhold_tile(tile)
        run(pkv.PKV_FLAG_TIMEOUT)
        pkv.pkv_debug_withhold_tile(off)
        pkv.pkv_set_wait_limit_ns(prev)
        got = run()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got)), f"tile {tile}"


if __name__ == "__main__":
    expired_waits_case(sys.argv[1])
    print("RECOVERED", flush=True)
