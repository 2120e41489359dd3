"""Key bounds, selection and attention over selected blocks where a pool's elements lie past 2^31 and its bytes past 2^32: the
blocks in use are the pool's last ones, and what the same blocks give in a small pool is what they give there."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ops_ref as R
from devutil import bf16_dev, i32_dev

pytestmark = pytest.mark.gpu
K, H, N = 8, 128, 16
CTX = [640, 100, 4001]


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    import paged_kv_decode_slot_gb300 as pkv
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return pkv


def at_the_end(small, blocks):
    """A pool of `blocks` blocks of zeros that ends with the small pool's."""
    big = torch.zeros(blocks, *small.shape[1:], dtype=small.dtype, device="cuda")
    big[blocks - len(small):] = small
    return big


@pytest.fixture
def case():
    r = np.random.default_rng(1)
    tab, pool = R.tables(r, CTX)
    return r, tab, pool, i32_dev(CTX)


# elements of a pool: 140,000 x 16 x 1,024 = 2.3e9 (bf16, 4.6 GB); 280,000 x 16 x 1,024 = 4.6e9 (e4m3, 4.6 GB)
BLOCKS = {"bf16": 140_000, "e4m3": 280_000}


def pools(kv, pool, n):
    if kv == "bf16":
        return [torch.randn(pool, 16, K, H, device="cuda").bfloat16() for _ in range(n)], []
    return ([torch.randint(0, 0x70, (pool, 16, K, H), device="cuda").to(torch.uint8) for _ in range(n)],
            [torch.rand(pool, K, device="cuda") + 0.1 for _ in range(n)])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_key_bounds(pkv, case, kv):
    r, tab, pool, ctx = case
    (k,), scale = pools(kv, pool, 1)
    bounds = pkv.pkv_key_bounds if kv == "bf16" else pkv.pkv_key_bounds_fp8
    small = torch.zeros(pool, K, 2, H, dtype=torch.bfloat16, device="cuda")
    pkv.check(bounds(k, *scale, i32_dev(tab), ctx, 5000, small))
    nb = BLOCKS[kv]
    big = torch.zeros(nb, K, 2, H, dtype=torch.bfloat16, device="cuda")
    pkv.check(bounds(at_the_end(k, nb), *(at_the_end(s, nb) for s in scale), i32_dev(np.where(tab < 0, -1, tab + nb - pool)), ctx, 5000, big))
    assert torch.equal(big[nb - pool:], small) and not bool(big[:nb - pool].any()) and bool(small.any())


def test_selection_from_bounds_past_32_bits(pkv, case):
    r, tab, pool, ctx = case
    nb = 1_060_000                                              # x 8 x 2 x 128 elements: 2.2e9, 4.3 GB
    mid, half = torch.randn(pool, K, H, device="cuda"), torch.rand(pool, K, H, device="cuda")
    small = torch.stack([mid - half, mid + half], 2).bfloat16()
    q = bf16_dev(R.to_bf16(r.standard_normal((len(CTX), N, H))))
    got = []
    for bounds, shift in ((small, 0), (at_the_end(small, nb), nb - pool)):
        sel = torch.full((len(CTX), K, 30), -9, dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        ws = torch.empty(pkv.pkv_select_workspace_bytes(len(CTX), K, tab.shape[1]), dtype=torch.uint8, device="cuda")
        pkv.check(pkv.pkv_select_blocks(q, bounds, i32_dev(np.where(tab < 0, -1, tab + shift)), ctx, sel, ws, 1, 1, err))
        assert pkv.pkv_read_err_flag(err)[1] == 0
        got.append(sel.cpu().numpy())
    assert np.array_equal(*got)
    want = R.select(R.bf16_values(q.view(torch.int16).cpu().numpy().view(np.uint16)), small.double().cpu().numpy(), tab, CTX, 30, 1, 1)
    assert np.array_equal(got[0], want)


@pytest.mark.parametrize("pb", [0, 8])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_attention(pkv, case, kv, pb):
    r, tab, pool, ctx = case
    kv_pools, scales = pools(kv, pool, 2)
    attend = pkv.pkv_decode_attn_blocks if kv == "bf16" else pkv.pkv_decode_attn_blocks_fp8
    q = bf16_dev(R.to_bf16(r.standard_normal((len(CTX), N, H))))
    M, nb = 40, BLOCKS[kv]
    sel = np.full((len(CTX), K, M), -1, dtype=np.int32)
    for b, c in enumerate(CTX):
        for h in range(K):
            pick = np.sort(r.permutation(-(-c // 16))[:M])
            sel[b, h, :len(pick)] = pick
    sel = torch.from_numpy(sel).cuda()
    got = []
    for big in (False, True):
        p = [at_the_end(t, nb) for t in (*kv_pools, *scales)] if big else [*kv_pools, *scales]
        out, lse = torch.zeros_like(q), torch.zeros(len(CTX), N, device="cuda")
        parts = -(-M // pb) if pb else 0
        ws = torch.zeros(pkv.pkv_splitk_workspace_bytes(len(CTX), N, H, parts), dtype=torch.uint8, device="cuda") if pb else None
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        table = i32_dev(np.where(tab < 0, -1, tab + nb - pool) if big else tab)
        pkv.check(attend(q, *p, table, ctx, sel, H ** -0.5, out, lse, pb, parts, ws, err))
        assert pkv.pkv_read_err_flag(err)[1] == 0
        got.append((out.view(torch.int16), lse))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and bool(got[0][0].any())
