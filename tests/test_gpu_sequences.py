"""Rows of a batch and the blocks they hold, on the GPU: forks, extensions with copies on write, compaction and the copies in
many pools, each equal to the same done row by row on the host."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import latent_ref as L
from devutil import i32_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    import paged_kv_decode_slot_gb300 as pkv
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return pkv


def host(t):
    return t.cpu().numpy()


def err_of(err):
    return int(err.cpu()[0])


def flag():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def workspace(pkv, num_blocks):
    return torch.full((pkv.pkv_blocks_workspace_bytes(num_blocks),), 0x7B, dtype=torch.uint8, device="cuda")


def run_extend(pkv, tables, ctx, num_new, ref, stream=None):
    d = [i32_dev(x) for x in (tables, ctx, num_new, ref)]
    copies, err = torch.full((len(ctx), 2), 77, dtype=torch.int32, device="cuda"), flag()
    pkv.check(pkv.pkv_extend_sequences(d[0], d[1], d[2], d[3], copies, workspace(pkv, len(ref)), err, stream))
    return (*(host(x) for x in (d[0], d[1], d[3], copies)), err_of(err))


# rows, table width, blocks: one row; few; more rows than one CTA's threads; more blocks than one step of every warp
SIZES = [(1, 1, 1), (1, 5, 4), (7, 9, 40), (64, 20, 1000), (300, 6, 1500), (1100, 3, 2500), (5, 700, 3000), (40, 40, 70001)]


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("rows,width,blocks", SIZES)
def test_extend(pkv, rows, width, blocks, seed):
    r = np.random.default_rng(seed)
    tables, ctx, ref = L.random_rows(r, rows, width, blocks, [0.3, 0.6, 0.95][seed])
    num_new = r.integers(0, [2, 20, 16 * width + 1][seed], rows).astype(np.int32)
    num_new = np.minimum(num_new, 16 * width - ctx)
    num_new[r.random(rows) < 0.2] = 0
    want = L.extend(tables, ctx, num_new, ref)
    got = run_extend(pkv, tables, ctx, num_new, ref)
    for g, w, name in zip(got, want, ("tables", "lengths", "counts", "copies")):
        np.testing.assert_array_equal(g, w, name)
    assert got[4] == (pkv.PKV_FLAG_NO_BLOCKS if want[4] else 0)
    nb = -(-got[1] // 16)
    assert np.array_equal(L.counts(got[0], got[1], blocks), got[2]) and np.all(got[0][np.arange(width) >= nb[:, None]] == -1)


def test_last_of_the_rows_that_share_a_block_keeps_it(pkv):
    tables = np.array([[3, 5], [3, 5], [3, 5], [3, 5]], dtype=np.int32)
    ctx, ref = np.full(4, 20, dtype=np.int32), np.array([0, 0, 0, 4, 0, 4, 0, 0], dtype=np.int32)
    t, c, f, copies, err = run_extend(pkv, tables, ctx, np.ones(4, dtype=np.int32), ref)
    assert err == 0 and copies.tolist() == [[5, 0], [5, 1], [5, 2], [-1, -1]] and t[:, 1].tolist() == [0, 1, 2, 5]
    assert f.tolist() == [1, 1, 1, 4, 0, 1, 0, 0]
    # one of them stays as it is: all three that grow leave
    t, c, f, copies, err = run_extend(pkv, tables, ctx, np.array([1, 0, 1, 1], dtype=np.int32), ref)
    assert err == 0 and copies.tolist() == [[5, 0], [-1, -1], [5, 1], [5, 2]] and f[5] == 1 and c.tolist() == [21, 20, 21, 21]


def test_rows_behind_the_first_refused_one_stay(pkv):
    tables = np.full((4, 4), -1, dtype=np.int32)
    tables[:, 0] = [0, 1, 2, 2]
    ctx, ref = np.array([16, 10, 5, 5], dtype=np.int32), np.array([1, 1, 2, 0, 0], dtype=np.int32)
    # row 0 takes one of the two free blocks, row 1 needs two: it, and the sharing rows behind it, are left alone
    t, c, f, copies, err = run_extend(pkv, tables, ctx, np.array([3, 30, 1, 1], dtype=np.int32), ref)
    assert err == pkv.PKV_FLAG_NO_BLOCKS and c.tolist() == [19, 10, 5, 5] and f.tolist() == [1, 1, 2, 1, 0]
    assert t[0, :2].tolist() == [0, 3] and np.array_equal(t[1:], tables[1:]) and np.all(copies == -1)


def test_extend_refuses_rows_with_bad_values(pkv):
    tables = np.array([[0, -1], [9, -1], [2, -1], [3, -1]], dtype=np.int32)
    ctx, ref = np.array([5, 5, -1, 16], dtype=np.int32), np.array([1, 1, 1, 1, 0, 0], dtype=np.int32)
    t, c, f, copies, err = run_extend(pkv, tables, ctx, np.array([-3, 1, 1, 17], dtype=np.int32), ref)
    assert err == pkv.PKV_FLAG_CTX_RANGE | pkv.PKV_FLAG_BLOCK_RANGE
    assert np.array_equal(t, tables) and np.array_equal(c, ctx) and np.array_equal(f, ref) and np.all(copies == -1)
    # a row that fills its table to the last token is no such row (the impossible length is flagged though it does not
    # grow); a sum that would pass 32 bits is one
    t, c, f, copies, err = run_extend(pkv, tables, ctx, np.array([0, 0, 0, 16], dtype=np.int32), ref)
    assert err == pkv.PKV_FLAG_CTX_RANGE and c[3] == 32 and t[3].tolist() == [3, 4]
    _, c, _, _, err = run_extend(pkv, tables, ctx, np.array([2 ** 31 - 1, 0, 0, 0], dtype=np.int32), ref)
    assert err == pkv.PKV_FLAG_CTX_RANGE and np.array_equal(c, ctx)


@pytest.mark.parametrize("what", ["counts of zero", "counts too high", "counts below zero"])
def test_counts_that_disagree_end_in_bounds(pkv, what):
    r = np.random.default_rng(3)
    tables, ctx, ref = L.random_rows(r, 50, 12, 900, 0.7)
    bad = np.zeros_like(ref) if what == "counts of zero" else ref + 3 if what == "counts too high" else ref - 2
    t, c, f, copies, err = run_extend(pkv, tables, ctx, np.minimum(9, 192 - ctx).astype(np.int32), bad)
    assert np.all((t >= -1) & (t < 900)) and np.all((c >= ctx) & (c <= ctx + 9)) and err & ~(512 | 1024) == 0


@pytest.mark.parametrize("rows,width,blocks", SIZES)
@pytest.mark.parametrize("rows_out", ["same", "fewer", "more"])
def test_fork(pkv, rows, width, blocks, rows_out):
    r = np.random.default_rng(rows + width)
    tables, ctx, ref = L.random_rows(r, rows, width, blocks)
    n = rows if rows_out == "same" else rows // 2 if rows_out == "fewer" else 3 * rows + 1
    parents = r.integers(-1, rows, n).astype(np.int32)
    want = L.fork(tables, ctx, parents, blocks)
    d = [i32_dev(x) for x in (tables, ctx, parents, ref)]
    out, lens, err = (torch.full((n, width), 77, dtype=torch.int32, device="cuda"),
                      torch.full((n,), 77, dtype=torch.int32, device="cuda"), flag())
    pkv.check(pkv.pkv_fork_sequences(*d, out, lens, err))
    assert err_of(err) == 0
    for g, w in zip((out, lens, d[3]), want):
        np.testing.assert_array_equal(host(g), w)
    np.testing.assert_array_equal(host(d[0]), tables)      # the old rows are left as they were


def test_fork_flags_bad_values(pkv):
    tables, ctx = np.array([[0, 1], [2, 99], [1, 1]], dtype=np.int32), np.array([20, 20, 1000], dtype=np.int32)
    out, lens = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    cases = [([0, 3, -2, 0], pkv.PKV_FLAG_SEQ_RANGE), ([1, 1, 0, -1], pkv.PKV_FLAG_BLOCK_RANGE), ([2, 1, 0, -1], pkv.PKV_FLAG_CTX_RANGE)]
    for parents, want in cases:
        err, ref = flag(), i32_dev([1, 1, 1])
        rows = tables if want != pkv.PKV_FLAG_CTX_RANGE else np.where(tables == 99, 2, tables).astype(np.int32)
        lengths = ctx if want == pkv.PKV_FLAG_CTX_RANGE else np.minimum(ctx, 20).astype(np.int32)
        if want == pkv.PKV_FLAG_SEQ_RANGE:
            rows = np.where(tables == 99, 2, tables).astype(np.int32)
        pkv.check(pkv.pkv_fork_sequences(i32_dev(rows), i32_dev(lengths), i32_dev(parents), ref, out, lens, err))
        # (the third row's block 1 loses a holder it has too few of in the first two cases)
        assert err_of(err) & ~pkv.PKV_FLAG_REF_RANGE == want, (parents, err_of(err))
    assert lens.tolist() == [0, 20, 20, 0]                 # a parent of an impossible length counts as empty


@pytest.mark.parametrize("rows,width,blocks", SIZES)
@pytest.mark.parametrize("share", [1.0, 0.3, 0.0], ids=["all moves", "some", "one move"])
def test_compact(pkv, rows, width, blocks, share):
    r = np.random.default_rng(rows * width)
    tables, ctx, ref = L.random_rows(r, rows, width, blocks)
    most = max(1, int(share * (blocks // 2)))
    want = L.compact(tables, ctx, ref, most)
    d = [i32_dev(x) for x in (tables, ctx, ref)]
    moves, n, err = (torch.full((most, 2), 77, dtype=torch.int32, device="cuda"), torch.full((1,), 77, dtype=torch.int32, device="cuda"),
                     flag())
    pkv.check(pkv.pkv_compact_blocks(*d, moves, n, workspace(pkv, blocks), err))
    assert err_of(err) == 0 and int(n) == want[3]
    for g, w in zip((d[0], d[2], moves), want):
        np.testing.assert_array_equal(host(g), w)
    if share == 1.0:
        used = host(d[2]) > 0
        assert not used[int(used.sum()):].any()


def test_compact_without_rows_and_with_stray_entries(pkv):
    # counts alone (no rows): the moves are the same; entries behind a row's blocks are not looked at
    moves, n, err = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"), flag()
    ref = i32_dev([0, 1, 0, 2, 0, 1])
    pkv.check(pkv.pkv_compact_blocks(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"),
                                     ref, moves, n, workspace(pkv, 6), err))
    assert moves.tolist() == [[5, 0], [3, 2], [-1, -1]] and int(n) == 2 and ref.tolist() == [1, 1, 2, 0, 0, 0] and err_of(err) == 0
    tables, ref = i32_dev([[5, 3, 5, 777]]), i32_dev([0, 0, 0, 1, 0, 1])
    pkv.check(pkv.pkv_compact_blocks(tables, i32_dev([30]), ref, moves, n, workspace(pkv, 6), err))
    assert tables.tolist() == [[0, 1, 5, 777]] and err_of(err) == 0
    # a row that holds a block no count speaks of, and one outside the pool
    tables, ref = i32_dev([[4, 3], [9, 3]]), i32_dev([0, 0, 0, 2, 0, 0])
    pkv.check(pkv.pkv_compact_blocks(tables, i32_dev([30, 30]), ref, moves, n, workspace(pkv, 6), err))
    assert err_of(err) == pkv.PKV_FLAG_REF_RANGE | pkv.PKV_FLAG_BLOCK_RANGE and tables.tolist() == [[4, 0], [9, 0]]


@pytest.mark.parametrize("dtype,shape", [(torch.bfloat16, (16, 576)), (torch.uint8, (16, 1, 64)), (torch.bfloat16, (16, 5, 128)),
                                         (torch.float32, (4,)), (torch.uint8, (16 * 4097,))])
@pytest.mark.parametrize("num_pools", [1, 3, 64])
def test_copies_in_many_pools(pkv, dtype, shape, num_pools):
    r = np.random.default_rng(num_pools)
    blocks = 90
    pools = [torch.randint(0, 255, (blocks, *shape), device="cuda", dtype=torch.uint8).to(dtype) for _ in range(num_pools)]
    want = [p.clone() for p in pools]
    ids = r.permutation(blocks)
    pairs = np.full((200, 2), -1, dtype=np.int32)
    at = r.permutation(200)[:40]
    pairs[at, 0], pairs[at, 1] = ids[:40], ids[40:80]
    for a, b in pairs[at]:
        for p in want:
            p[int(b)] = p[int(a)]
    err = flag()
    pkv.check(pkv.pkv_copy_blocks_pools(pools, i32_dev(pairs), err))
    assert err_of(err) == 0 and all(torch.equal(a, b) for a, b in zip(pools, want))
    pairs[:4] = [[0, 90], [-1, 3], [2, -1], [5, 5]]
    pairs[4:] = -1
    pkv.check(pkv.pkv_copy_blocks_pools(pools, i32_dev(pairs), err))
    assert err_of(err) == pkv.PKV_FLAG_BLOCK_RANGE and all(torch.equal(a, b) for a, b in zip(pools, want))


def test_copies_past_2_to_the_32_bytes(pkv):
    """A pool of 4.8 GB: the last block to the first and back to the one before the last."""
    blocks = 262_144
    pool = torch.zeros(blocks, 16, 576, dtype=torch.bfloat16, device="cuda")
    pool[-1] = torch.randn(16, 576, device="cuda").bfloat16()
    pkv.check(pkv.pkv_copy_blocks_pools([pool], i32_dev([[blocks - 1, 0]])))
    pkv.check(pkv.pkv_copy_blocks_pools([pool], i32_dev([[0, blocks - 2]])))
    assert torch.equal(pool[0], pool[-1]) and torch.equal(pool[-2], pool[-1]) and not pool[1:-2].any()


def test_in_a_graph_on_another_stream_and_with_a_workspace_in_use_elsewhere(pkv):
    """A captured tick (extend, copies, compact, copies) replayed from saved states equals the eager one."""
    r = np.random.default_rng(5)
    tables, ctx, ref = L.random_rows(r, 30, 10, 400, 0.6)
    num_new = np.minimum(r.integers(0, 40, 30), 160 - ctx).astype(np.int32)
    now = [i32_dev(x) for x in (tables, ctx, ref)]
    then = [t.clone() for t in now]
    new = i32_dev(num_new)
    copies, moves, n = (torch.zeros(30, 2, dtype=torch.int32, device="cuda"), torch.zeros(200, 2, dtype=torch.int32, device="cuda"),
                        torch.zeros(1, dtype=torch.int32, device="cuda"))
    pool, ws, err = torch.randn(400, 16, 576, device="cuda").bfloat16(), workspace(pkv, 400), flag()
    saved = pool.clone()

    def tick():
        for a, b in zip(now, then):
            a.copy_(b)
        pool.copy_(saved)
        pkv.check(pkv.pkv_extend_sequences(now[0], now[1], new, now[2], copies, ws, err))
        pkv.check(pkv.pkv_copy_blocks_pools([pool], copies, err))
        pkv.check(pkv.pkv_compact_blocks(now[0], now[1], now[2], moves, n, ws, err))
        pkv.check(pkv.pkv_copy_blocks_pools([pool], moves, err))
    tick()
    want = [t.clone() for t in (*now, copies, moves, n, pool)]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        tick()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        tick()
    for _ in range(3):
        pool.zero_(), copies.zero_(), moves.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*now, copies, moves, n, pool), want))
    # what the host does with the same rows
    t, c, f, cp, _ = L.extend(tables, ctx, num_new, ref)
    t, f, mv, k = L.compact(t, c, f, 200)
    for g, w in zip((*now, copies, moves), (t, c, f, cp, mv)):
        np.testing.assert_array_equal(host(g), w)
    p = saved.clone()
    for a, b in [x for x in cp if x[0] >= 0]:
        p[int(b)] = p[int(a)]
    for a, b in mv[:k]:
        p[int(b)] = p[int(a)]
    assert torch.equal(p, pool)


@pytest.mark.parametrize("new", [1, 100, 0])
def test_extend_more_rows_than_threads(pkv, new):
    """Several rows a thread: their states are kept in `copies` between the passes."""
    r = np.random.default_rng(new)
    rows, width, blocks = 9001, 9, 60000
    tables, ctx, ref = L.random_rows(r, rows, width, blocks, 0.6)
    num_new = np.minimum(r.integers(0, new + 1, rows), 16 * width - ctx).astype(np.int32)
    now = [i32_dev(x) for x in (tables, ctx, ref)]
    copies, err = torch.full((rows, 2), -2147483648, dtype=torch.int32, device="cuda"), flag()
    pkv.check(pkv.pkv_extend_sequences(now[0], now[1], i32_dev(num_new), now[2], copies, workspace(pkv, blocks), err))
    t, c, f, cp, refused = L.extend(tables, ctx, num_new, ref)
    assert err_of(err) == (pkv.PKV_FLAG_NO_BLOCKS if refused else 0)
    for g, w in zip((*now, copies), (t, c, f, cp)):
        np.testing.assert_array_equal(host(g), w)


def test_what_copies_held_before_does_not_matter(pkv):
    """Values as the call itself leaves them meanwhile for its warps."""
    r = np.random.default_rng(8)
    tables, ctx, ref = L.random_rows(r, 60, 30, 4000, 0.5)
    num_new = np.minimum(r.choice([0, 1, 3, 200], 60), 480 - ctx).astype(np.int32)
    t, c, f, cp, _ = L.extend(tables, ctx, num_new, ref)
    for fill in (-2147483648, -2147483648 + 5, -3, 0, 7):
        now = [i32_dev(x) for x in (tables, ctx, ref)]
        copies, err = torch.full((60, 2), fill, dtype=torch.int32, device="cuda"), flag()
        pkv.check(pkv.pkv_extend_sequences(now[0], now[1], i32_dev(num_new), now[2], copies, workspace(pkv, 4000), err))
        assert err_of(err) == 0
        for g, w in zip((*now, copies), (t, c, f, cp)):
            np.testing.assert_array_equal(host(g), w)
