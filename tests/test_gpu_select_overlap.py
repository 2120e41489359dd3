"""A workspace that something else writes while a selection runs (calls that share one must not overlap): what comes out is
meaningless, but every call ends, writes within its outputs, and leaves the next one as it should be."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ops_ref as R
from devutil import bf16_dev, i32_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    import paged_kv_decode_slot_gb300 as pkv
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return pkv


@pytest.mark.parametrize("alike", [True, False], ids=["equal blocks", "random blocks"])
@pytest.mark.parametrize("B,K,nb,M", [(40, 5, 1500, 128), (8, 2, 9000, 300)])
def test_selection_ends_while_its_workspace_is_written(pkv, B, K, nb, M, alike):
    r = np.random.default_rng(nb)
    ctx = [16 * nb - int(x) for x in r.integers(0, 3000, B)]
    pool, H = 4000, 64                                          # sequences share blocks: only the tables are long
    tab = r.integers(0, pool, (B, nb)).astype(np.int32)
    q = bf16_dev(R.to_bf16(r.standard_normal((B, 2 * K, H))))
    bounds = torch.randn(pool, K, 2, H, device="cuda").sort(2).values.bfloat16()
    if alike:                                                   # every score is undecided: lists and sums in the workspace
        bounds[:] = bounds[:1]
    tables, lens = i32_dev(tab), i32_dev(ctx)
    sel = torch.full((B + 2, K, M), -9, dtype=torch.int32, device="cuda")
    ws = torch.zeros(pkv.pkv_select_workspace_bytes(B, K, nb), dtype=torch.uint8, device="cuda")

    def run():
        pkv.check(pkv.pkv_select_blocks(q, bounds, tables, lens, sel[1:-1], ws, 1, 1))
    run()
    torch.cuda.synchronize()
    want = sel.clone()
    assert bool((want[1:-1] >= 0).all())
    side, noise = torch.cuda.Stream(), torch.randint(0, 256, (3, ws.numel()), device="cuda").to(torch.uint8)
    torch.cuda.synchronize()
    for i in range(60):
        run()
        with torch.cuda.stream(side):
            ws.copy_(noise[i % 3]) if i % 2 else ws.zero_()
    torch.cuda.synchronize()
    assert bool((sel[0] == -9).all()) and bool((sel[-1] == -9).all())
    assert bool(((sel[1:-1] >= -9) & (sel[1:-1] < nb)).all())
    run()
    torch.cuda.synchronize()
    assert torch.equal(sel, want)
