"""Block selection where scores are decided far below 32 bits: operands of every magnitude side by side.  A score counts as
its real value rounded once to 64 bits (math.fsum in the reference), so selections have to be equal."""
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


def check(pkv, q, bounds, tab, ctx, M, first=1, last=1):
    """q [B, N, H] and bounds [pool, K, 2, H] float64 that bf16 holds (or that are rounded to it here)."""
    q, bounds = R.to_bf16(q), R.to_bf16(bounds)
    B, K = len(ctx), bounds.shape[1]
    with np.errstate(invalid="ignore"):
        want = R.select(R.bf16_values(q), R.bf16_values(bounds), tab, ctx, M, first, last)
    sel = torch.full((B, K, M), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkv.pkv_select_workspace_bytes(B, K, tab.shape[1]), dtype=torch.uint8, device="cuda")
    pkv.check(pkv.pkv_select_blocks(bf16_dev(q), bf16_dev(bounds), i32_dev(tab), i32_dev(ctx), sel, ws, first, last, err))
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_OK, 0)
    got = sel.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


def case(seed, N, K, H, ctx):
    r = np.random.default_rng(seed)
    tab, pool = R.tables(r, ctx)
    mid, half = r.standard_normal((pool, K, H)), np.abs(r.standard_normal((pool, K, H)))
    return r, r.standard_normal((len(ctx), N, H)), np.stack([mid - half, mid + half], 2), tab, pool


SHAPES = [(1, 1, 64), (4, 1, 128), (8, 1, 64), (6, 3, 128)]
CTX = [16 * 70, 16 * 300 + 5, 40]


@pytest.mark.parametrize("power", [20, 40, 60, 80, 100, 126])
@pytest.mark.parametrize("N,K,H", SHAPES)
def test_a_large_bound_where_the_query_is_zero(pkv, N, K, H, power):
    """One element of the bounds is 2^power, but the query has nothing there: the others decide."""
    r, q, bounds, tab, _ = case(power + N, N, K, H, CTX)
    q[..., 5] = 0.0
    bounds[:, :, 1, 5] = 2.0 ** power
    bounds[::3, :, 0, 5] = -2.0 ** power
    check(pkv, q, bounds, tab, CTX, 25)


@pytest.mark.parametrize("power", [20, 60, 100, 120])
@pytest.mark.parametrize("N,K,H", [(4, 1, 128), (8, 1, 64), (6, 3, 128)])
def test_a_large_query_head_that_does_not_decide(pkv, N, K, H, power):
    """One head of each group is 2^power at an element whose bounds are negative: its score never is the largest."""
    r, q, bounds, tab, _ = case(power + N + 1, N, K, H, CTX)
    q[:, ::N // K] = 0.0
    q[:, ::N // K, 9] = 2.0 ** power
    bounds[:, :, 1, 9] = -np.abs(bounds[:, :, 1, 9]) - 0.25
    bounds[:, :, 0, 9] = bounds[:, :, 1, 9] - 1.0
    check(pkv, q, bounds, tab, CTX, 25)


@pytest.mark.parametrize("low,high", [(-133, -100), (-60, 60), (-133, 0), (0, 126), (-120, 126)])
@pytest.mark.parametrize("N,K,H", SHAPES)
def test_operands_of_every_magnitude(pkv, N, K, H, low, high):
    """Exponents uniform between low and high for queries and bounds alike, subnormal numbers among them."""
    r, q, bounds, tab, pool = case(high - low + H, N, K, H, CTX)
    power = lambda shape: 2.0 ** r.integers(low, high + 1, shape)
    q = r.choice([-1.0, 1.0], q.shape) * r.uniform(1, 2, q.shape) * power(q.shape)
    a, b = (r.choice([-1.0, 1.0], (pool, K, H)) * r.uniform(1, 1.9, (pool, K, H)) * power((pool, K, H)) for _ in range(2))
    check(pkv, q, np.stack([np.minimum(a, b), np.maximum(a, b)], 2), tab, CTX, 25)


@pytest.mark.parametrize("power", [-30, -70, -120])
@pytest.mark.parametrize("N,K,H", SHAPES)
def test_large_terms_that_cancel_and_a_rest_far_below(pkv, N, K, H, power):
    """Terms of 2^60 and more cancel exactly; what is left, of 2^power, decides, with equal blocks among them."""
    r, q, bounds, tab, pool = case(300 - power + N, N, K, H, CTX)
    q[...] = 0.0
    q[..., :16], q[..., 16:32] = 2.0 ** 20, 2.0 ** 20
    q[..., 40:44] = 2.0 ** (power // 2)
    k = np.zeros((pool, K, H))
    big = r.integers(1, 200, (pool, K, 16)) * 2.0 ** r.integers(40, 90, (pool, K, 16))
    k[..., :16], k[..., 16:32] = big, -big
    k[..., 40:44] = r.integers(-9, 10, (pool, K, 4)) * 2.0 ** (power - power // 2)
    check(pkv, q, np.stack([k, k], 2), tab, CTX, 25)


def test_finite_scores_beside_infinite_ones_and_at_the_ends_of_the_range(pkv):
    """Numbers at bf16's ends (exponents that no scale reaches), and heads with infinite bounds beside finite heads."""
    N, K, H = 4, 1, 64
    r, q, bounds, tab, _ = case(77, N, K, H, CTX)
    check(pkv, np.clip(q, -1.9, 1.9) * 2.0 ** 126, np.clip(bounds, -1.9, 1.9) * 2.0 ** 126, tab, CTX, 25)
    q[:, :, 7] = 0.25
    q[:, 0, 7] = 2.0 ** -100                                    # every head meets the infinities
    bounds[tab[1, 20:40], 0, 1, 7] = np.inf
    bounds[tab[1, 50:60], 0, :, 7] = -np.inf                    # scores of -inf
    bounds[:, 0, 1, 9] = 2.0 ** 100
    q[..., 9] = 0.0
    check(pkv, q, bounds, tab, CTX, 12)
    check(pkv, q, bounds, tab, CTX, 60)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_no_logit_exceeds_its_blocks_score(pkv, kv):
    """Scores of the bounds that the library wrote against the keys' products: bf16 bounds bound them; e4m3 bounds, half a step
    of bf16 and a rounding to fp32 off, up to 1/254 of sum |q| |bound|."""
    r = np.random.default_rng(5)
    K, H, ctx = 2, 128, [16 * 40, 333]
    tab, pool = R.tables(r, ctx)
    bounds = torch.zeros(pool, K, 2, H, dtype=torch.bfloat16, device="cuda")
    if kv == "bf16":
        k = R.to_bf16(r.standard_normal((pool, 16, K, H)))
        keys = R.bf16_values(k)
        pkv.check(pkv.pkv_key_bounds(bf16_dev(k), i32_dev(tab), i32_dev(ctx), 640, bounds))
    else:
        k = (r.integers(0, 0x70, (pool, 16, K, H)) | r.integers(0, 2, (pool, 16, K, H)) << 7).astype(np.uint8)
        scale = r.uniform(0.01, 0.1, (pool, K)).astype(np.float32)
        keys = R.e4m3_table()[k] * scale.astype(np.float64)[:, None, :, None]
        pkv.check(pkv.pkv_key_bounds_fp8(torch.from_numpy(k).cuda(), torch.from_numpy(scale).cuda(), i32_dev(tab), i32_dev(ctx), 640, bounds))
    box, q = bounds.double().cpu().numpy(), R.bf16_values(R.to_bf16(r.standard_normal((K, 3, H))))
    for b, c in enumerate(ctx):
        for j in range(-(-c // 16)):
            rows, (lo, hi) = keys[tab[b, j], :min(16, c - 16 * j)], box[tab[b, j]].transpose(1, 0, 2)
            for h in range(K):
                score = np.where(q[h] > 0, q[h] * hi[h], q[h] * lo[h]).sum(-1)
                slack = 1e-12 if kv == "bf16" else (np.abs(q[h]) * np.where(q[h] > 0, np.abs(hi[h]), np.abs(lo[h]))).sum(-1) / 254
                assert np.all((rows[:, h] @ q[h].T).max(0) <= score + slack)
