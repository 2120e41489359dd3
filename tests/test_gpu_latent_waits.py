"""The limit of a wait inside latent attention is of one step of its pipeline, however long a CTA's run is: under a limit well
above a step's time and well below a run's, nothing expires."""
from __future__ import annotations

import pytest
import torch

from test_gpu_latent import pkv, same  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [16, 32, 128])
def test_a_long_run_under_a_short_limit(pkv, N):  # noqa: F811
    """A long sequence for every CTA, each ending inside a block; the sequences share their blocks."""
    B, ctx = torch.cuda.get_device_properties(0).multi_processor_count, 65533
    torch.manual_seed(N)
    cache = torch.randn(4096, 16, 576, device="cuda").bfloat16()
    tab = torch.arange(4096, dtype=torch.int32, device="cuda").expand(B, 4096).contiguous()
    lens = torch.full((B,), ctx, dtype=torch.int32, device="cuda")
    q = torch.randn(B, 1, N, 576, device="cuda").bfloat16()
    ws = torch.zeros(pkv.pkv_latent_workspace_bytes(B, 1, N), dtype=torch.uint8, device="cuda")

    def run():
        out, lse, err = torch.zeros(B, 1, N, 512, device="cuda").bfloat16(), torch.zeros(B, 1, N, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        pkv.check(pkv.pkv_decode_attn_latent(q, cache, tab, lens, 0.05, out, lse, ws, err))
        b.record()
        torch.cuda.synchronize()
        return out, lse, int(err), a.elapsed_time(b)
    run()
    want = run()
    assert want[2] == 0 and want[3] > 0.9                    # (ms)
    prev = pkv.pkv_set_wait_limit_ns(300_000)
    try:
        got = run()
    finally:
        pkv.pkv_set_wait_limit_ns(prev)
    assert got[2] == 0 and same(got[0], want[0]) and same(got[1], want[1])
