"""Key bounds and block selection on the GPU against float64: bounds bit for bit, selections equal.

bf16 bounds are minima and maxima of bf16 numbers: no rounding.  e4m3 bounds round code * scale once to fp32 and once
to bf16: half a bf16 step, 2^-8 of the value, and 2^-24.  Selections are whole numbers and have to be equal, whatever
the scores' rounding: near ties are decided by the sums in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ops_ref as R
from devutil import bf16_dev, bf16_host, i32_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    import paged_kv_decode_slot_gb300 as pkv
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return pkv


CTX = [0, 1, 15, 16, 17, 40, 255, 300]


@pytest.mark.parametrize("num_new", [1, 2, 16, 17, 33, 100000])
@pytest.mark.parametrize("K,H", [(1, 64), (3, 128), (40, 128)])
def test_key_bounds_bf16(pkv, K, H, num_new):
    r = np.random.default_rng(K + num_new)
    tab, pool = R.tables(r, CTX)
    keys = R.to_bf16(r.standard_normal((pool, 16, K, H)))
    for b, c in enumerate(CTX):                                # what lies behind a context is not looked at
        if c % 16:
            keys[tab[b, c // 16], c % 16:] = 0x7FC0 if b % 2 else 0x7F80
    kept = np.full((pool, K, 2, H), 0x1234, dtype=np.uint16)
    want = R.to_bf16(R.key_bounds(R.bf16_values(keys), tab, CTX, num_new, R.bf16_values(kept)))
    got, err = bf16_dev(kept), torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.check(pkv.pkv_key_bounds(bf16_dev(keys), i32_dev(tab), i32_dev(CTX), num_new, got, err))
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_OK, 0)
    assert np.array_equal(bf16_host(got), want)


@pytest.mark.parametrize("blocks", [False, True], ids=["head", "block"])
@pytest.mark.parametrize("H", [64, 128])
def test_key_bounds_e4m3(pkv, blocks, H):
    r = np.random.default_rng(H + blocks)
    K, num_new = 5, 20
    tab, pool = R.tables(r, CTX)
    codes = r.integers(0, 256, (pool, 16, K, H)).astype(np.uint8)
    codes[(codes & 127) == 127] = 3
    sc = (2.0 ** r.uniform(-9, 3, (pool, K) if blocks else K)).astype(np.float32)
    val = R.e4m3_table()[codes] * (sc.astype(np.float64)[:, None, :, None] if blocks else sc.astype(np.float64)[None, None, :, None])
    want = R.key_bounds(val, tab, CTX, num_new, np.zeros((pool, K, 2, H)))
    got = torch.zeros(pool, K, 2, H, dtype=torch.bfloat16, device="cuda")
    pkv.check(pkv.pkv_key_bounds_fp8(torch.from_numpy(codes).cuda(), torch.from_numpy(sc).cuda(), i32_dev(tab), i32_dev(CTX), num_new, got))
    out = got.double().cpu().numpy()
    assert np.all(np.abs(out - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want))
    assert np.all((want == 0) == (out == 0))


def test_key_bounds_nan_keys_bad_blocks_and_nothing_to_do(pkv):
    K, H = 2, 64
    keys = torch.randn(4, 16, K, H, device="cuda").bfloat16()
    keys[1, 3, 1, 7] = float("nan")
    tab = torch.tensor([[1, 9, 2], [0, 3, -1]], dtype=torch.int32, device="cuda")
    err, got = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(4, K, 2, H, dtype=torch.bfloat16, device="cuda")
    pkv.check(pkv.pkv_key_bounds(keys, tab, i32_dev([48, 32]), 48, got, err))
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_ERR_RANGE, pkv.PKV_FLAG_BLOCK_RANGE)
    nan = torch.isnan(got)
    assert bool(nan[1, 1, :, 7].all()) and int(nan.sum()) == 2
    for blk in (0, 2, 3):
        assert torch.equal(got[blk, :, 0], keys[blk].amin(0)) and torch.equal(got[blk, :, 1], keys[blk].amax(0))
    before = got.clone()
    err.zero_()
    pkv.check(pkv.pkv_key_bounds(keys, tab, i32_dev([48, 49]), 0, got, err))          # no new tokens
    pkv.check(pkv.pkv_key_bounds(keys, tab[:0], i32_dev([]), 5, got, err))            # no sequences
    assert pkv.pkv_read_err_flag(err)[1] == 0
    pkv.check(pkv.pkv_key_bounds(keys, tab, i32_dev([-1, 49]), 16, got, err))         # lengths outside the table
    assert pkv.pkv_read_err_flag(err)[1] == pkv.PKV_FLAG_CTX_RANGE
    assert torch.equal(got.view(torch.int16), before.view(torch.int16))


# ------------------------------------------------------------------------------------ selection
def run_select(pkv, q, bounds, tab, ctx, M, first, last, err=None, fill=None, stream=None):
    B, K = len(ctx), bounds.shape[1]
    sel = torch.full((B, K, M), -9, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkv.pkv_select_workspace_bytes(B, K, tab.shape[1]), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF if fill is None else fill)                   # the workspace's contents do not matter
    pkv.check(pkv.pkv_select_blocks(q, bounds, i32_dev(tab), i32_dev(ctx), sel, ws, first, last, err, stream))
    return sel


def case(seed, ctx, N, K, H, spread=1.0, width=None):
    r = np.random.default_rng(seed)
    tab, pool = R.tables(r, ctx, width)
    q = R.to_bf16(r.standard_normal((len(ctx), N, H)))
    mid, half = spread * r.standard_normal((pool, K, H)), np.abs(r.standard_normal((pool, K, H)))
    return q, R.to_bf16(np.stack([mid - half, mid + half], 2)), tab, pool


def check(pkv, q, bounds, tab, ctx, M, first, last, **kw):
    want = R.select(R.bf16_values(q), R.bf16_values(bounds), tab, ctx, M, first, last)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_select(pkv, bf16_dev(q), bf16_dev(bounds), tab, ctx, M, first, last, err, **kw).cpu().numpy()
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_OK, 0)
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("N,K,H", [(1, 1, 64), (8, 4, 128), (4, 1, 128), (16, 2, 64), (5, 5, 128)])
@pytest.mark.parametrize("M,first,last", [(1, 0, 1), (1, 1, 0), (1, 0, 0), (4, 1, 1), (7, 0, 3), (3, 1, 2), (37, 2, 1), (200, 1, 1)])
def test_selection_matches_float64(pkv, N, K, H, M, first, last):
    ctx = [0, 1, 16, 17, 16 * M, 16 * M + 1, 16 * (M + 1) + 3, 900, 3000]
    q, bounds, tab, _ = case(M + N + H, ctx, N, K, H, width=400)
    check(pkv, q, bounds, tab, ctx, M, first, last)


@pytest.mark.parametrize("nb,M", [(257, 64), (2049, 100), (8192, 128), (8193, 128), (9001, 500)])
def test_selection_of_long_contexts(pkv, nb, M):
    """Around the number of scores the choosing CTA keeps in shared memory, and beyond it."""
    ctx = [16 * nb, 16 * nb - 5, 100]
    q, bounds, tab, _ = case(nb, ctx, 2, 1, 64)
    check(pkv, q, bounds, tab, ctx, M, 1, 2)


@pytest.mark.parametrize("N,H", [(1, 64), (4, 128), (8, 128)])
@pytest.mark.parametrize("step", [-20, -30, -47, -55])
def test_scores_that_differ_far_below_32_bits(pkv, N, H, step):
    """score_j = 1 + k_j 2^step with k a permutation: equal in 32 bits, told apart by the sums that follow."""
    nb, M = 250, 30
    r = np.random.default_rng(N - step)
    tab, pool = R.tables(r, [16 * nb])
    q, bounds = np.zeros((1, N, H)), np.zeros((pool, 1, 2, H))
    q[0, :, 3], q[0, :, H - 2] = 1.0, 2.0 ** (step // 2)
    q[0, :-1, 3] = 0.5                                          # the last head decides
    bounds[:, :, :, 3] = 1.0
    bounds[tab[0], 0, :, H - 2] = (r.permutation(nb) * 2.0 ** (step - step // 2))[:, None]
    check(pkv, R.to_bf16(q), R.to_bf16(bounds), tab, [16 * nb], M, 1, 1)


@pytest.mark.parametrize("eq,eb", [(-70, -65), (-60, -60), (-120, -10), (70, 66), (100, 27)])
def test_scores_that_leave_the_range_of_32_bits(pkv, eq, eb):
    """Products and sums that under- or overflow in 32 bits: the choice is that of the real values all the same."""
    ctx = [16 * 300, 16 * 40 + 1]
    q, bounds, tab, _ = case(eq + eb + 400, ctx, 4, 2, 64)
    q, bounds = R.to_bf16(R.bf16_values(q) * 2.0 ** eq), R.to_bf16(R.bf16_values(bounds) * 2.0 ** eb)
    assert np.isfinite(R.bf16_values(q)).all() and np.isfinite(R.bf16_values(bounds)).all()
    check(pkv, q, bounds, tab, ctx, 20, 1, 1)


def test_ties_go_to_the_lowest_index(pkv):
    """Equal blocks, a query of zeros, and equal scores of different blocks."""
    ctx = [16 * 700, 16 * 90, 16 * 20]
    q, bounds, tab, pool = case(3, ctx, 8, 2, 128)
    bounds[:] = bounds[0]                                       # every block alike: more ties than are ranked pairwise
    check(pkv, q, bounds, tab, ctx, 33, 1, 1)
    q2, bounds2, _, _ = case(4, ctx, 8, 2, 128)
    q2[:] = 0
    check(pkv, q2, bounds2, tab, ctx, 33, 1, 1)
    # a few kinds of blocks: ties within each
    bounds3 = bounds2[np.random.default_rng(0).integers(0, 3, pool)]
    q3 = R.to_bf16(np.random.default_rng(1).standard_normal((3, 8, 128)))
    for M in (5, 20, 300):
        check(pkv, q3, bounds3, tab, ctx, M, 0, 1)


@pytest.mark.parametrize("nb,M", [(300, 40), (2000, 600), (9000, 1000)])
def test_scores_that_32_bits_cannot_tell_apart(pkv, nb, M):
    """Large terms that cancel to the last bit, with small ones beneath the fp32 sums' rounding: what is left decides.
    Terms are powers of two and small integers times 2^-14, so that the sums are exact in 64 bits."""
    r = np.random.default_rng(nb)
    ctx = [16 * nb, 16 * (nb // 2)]
    tab, pool = R.tables(r, ctx)
    H = 128
    q = np.zeros((2, 2, H))
    q[..., :64] = 2.0 ** r.integers(6, 9, (2, 2, 64))
    q[..., 64:] = 2.0 ** -7
    k = np.zeros((pool, 1, H))
    big = 2.0 ** r.integers(6, 9, (pool, 1, 32))
    k[..., :32], k[..., 32:64] = big, -big
    k[..., 64:] = r.integers(-100, 100, (pool, 1, 64)) * 2.0 ** -7
    q[..., 32:64] = q[..., :32]                                 # q . (big, -big) = 0 exactly
    bounds = np.stack([k, k], 2)                                # one key per block: the bound is its logit
    check(pkv, R.to_bf16(q), R.to_bf16(bounds), tab, ctx, M, 1, 1)


def test_forced_blocks_need_no_bounds_and_nan_bounds_are_chosen(pkv):
    ctx = [16 * 60]
    q, bounds, tab, _ = case(6, ctx, 4, 1, 64)
    clean = bounds.copy()
    bounds[tab[0, [0, 1, 58, 59]]] = 0x7FC0                     # first two, last two: never looked at
    want = R.select(R.bf16_values(q), R.bf16_values(clean), tab, ctx, 10, 2, 2)
    got = run_select(pkv, bf16_dev(q), bf16_dev(bounds), tab, ctx, 10, 2, 2).cpu().numpy()
    assert np.array_equal(got, want)
    bounds = clean.copy()
    bounds[tab[0, 33], 0, 0, 5] = 0x7FC0                        # NaN in one element's lower bound
    q[0, :, 5] = 0xBF80                                         # -1: the lower bound counts
    check(pkv, q, bounds, tab, ctx, 3, 1, 1)
    bounds[tab[0, 20:40], 0] = 0x7FC0                           # more NaN blocks than places: the lowest indices
    check(pkv, q, bounds, tab, ctx, 9, 1, 1)


def test_infinite_bounds_come_first(pkv):
    ctx = [16 * 50]
    q, bounds, tab, _ = case(7, ctx, 2, 2, 64)
    q[0, :, 3] = 0x3F80                                         # 1: the upper bound counts
    bounds[tab[0, 30], :, 1, 3] = 0x7F80
    bounds[tab[0, 31], :, 1, 3] = 0xFF80
    bounds[tab[0, 31], :, 0, 3] = 0xFF80
    check(pkv, q, bounds, tab, ctx, 4, 1, 1)
    check(pkv, q, bounds, tab, ctx, 49, 1, 1)


def test_bad_blocks_and_lengths_are_flagged(pkv):
    ctx = [16 * 40, 16 * 40]
    q, bounds, tab, pool = case(8, ctx, 2, 1, 64)
    tab[0, 7], tab[0, 9] = pool, -1
    want = R.select(R.bf16_values(q), R.bf16_values(bounds), tab, ctx, 12, 1, 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run_select(pkv, bf16_dev(q), bf16_dev(bounds), tab, ctx, 12, 1, 1, err).cpu().numpy()
    assert pkv.pkv_read_err_flag(err)[1] == pkv.PKV_FLAG_BLOCK_RANGE
    assert np.array_equal(got, want) and not set((7, 9)) & set(got[0, 0])
    err.zero_()
    got = run_select(pkv, bf16_dev(q), bf16_dev(bounds), tab, [16 * 40 + 1, -3], 12, 1, 1, err).cpu().numpy()
    assert pkv.pkv_read_err_flag(err)[1] == pkv.PKV_FLAG_CTX_RANGE and np.all(got == -1)


def test_selection_repeats_on_any_workspace_stream_and_in_a_graph(pkv):
    ctx = list(np.random.default_rng(9).integers(0, 12000, 70))
    q, bounds, tab, _ = case(9, ctx, 8, 4, 128)
    qd, bd = bf16_dev(q), bf16_dev(bounds)
    a = run_select(pkv, qd, bd, tab, ctx, 40, 1, 1, fill=0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b = run_select(pkv, qd, bd, tab, ctx, 40, 1, 1, fill=0x7F)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    sel = torch.zeros_like(a)
    ws = torch.empty(pkv.pkv_select_workspace_bytes(70, 4, tab.shape[1]), dtype=torch.uint8, device="cuda")
    t, c = i32_dev(tab), i32_dev(ctx)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.check(pkv.pkv_select_blocks(qd, bd, t, c, sel, ws, 1, 1))
    for _ in range(3):
        sel.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, sel)
    want = R.select(R.bf16_values(q[:3]), R.bf16_values(bounds), tab[:3], ctx[:3], 40, 1, 1)
    assert np.array_equal(a[:3].cpu().numpy(), want)


def test_many_sequences_and_no_sequence(pkv):
    """More sequences than a warp's lanes look up at once, most of them too short to be scored."""
    r = np.random.default_rng(10)
    ctx = [int(c) for c in np.where(r.random(1000) < 0.03, r.integers(100, 400, 1000), r.integers(0, 64, 1000))]
    q, bounds, tab, _ = case(10, ctx, 2, 2, 64, width=30)
    check(pkv, q, bounds, tab, ctx, 4, 1, 1)
    sel = run_select(pkv, bf16_dev(q[:0]), bf16_dev(bounds), tab[:0], [], 4, 1, 1)
    assert sel.numel() == 0
