"""Rows of a batch through steps that not all of them take part in: rows that were refused or asked for nothing keep their
cached tokens, and those of the rows that share their blocks."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import latent_ref as L
import ops_ref as R
from devutil import bf16_dev, bf16_host, i32_dev, out_f64
from test_gpu_latent import INV, pkv, same  # noqa: F401
from test_gpu_sequences import SIZES, err_of, flag, host, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,width,blocks", SIZES + [(9001, 9, 60000)])
@pytest.mark.parametrize("new", [1, 100])
def test_lengths_for_the_step(pkv, rows, width, blocks, new):  # noqa: F811
    r = np.random.default_rng(rows + new)
    tables, ctx, ref = L.random_rows(r, rows, width, blocks, 0.8)
    num_new = np.minimum(r.integers(0, new + 1, rows), 16 * width - ctx).astype(np.int32)
    bad = r.random(rows) < 0.05
    num_new[bad] = -1
    want = L.extend(tables, ctx, num_new, ref)
    d = [i32_dev(x) for x in (tables, ctx, num_new, ref)]
    copies, lens, err = torch.zeros(rows, 2, dtype=torch.int32, device="cuda"), torch.full((rows,), 77, dtype=torch.int32, device="cuda"), flag()
    pkv.check(pkv.pkv_extend_sequences(*d, copies, workspace(pkv, blocks), err, step_lens=lens))
    assert err_of(err) == (pkv.PKV_FLAG_NO_BLOCKS if want[4] else 0) | (pkv.PKV_FLAG_CTX_RANGE if bad.any() else 0)
    for g, w in zip((d[0], d[1], d[3], copies), want):
        np.testing.assert_array_equal(host(g), w)
    np.testing.assert_array_equal(host(lens), np.where(want[1] != ctx, want[1], 0))


@pytest.mark.parametrize("N,T", [(16, 1), (128, 1), (4, 3)])
def test_rows_that_do_not_grow_keep_their_tokens(pkv, N, T):  # noqa: F811
    """Few free blocks: the rows from the first that needs one too many are refused; some ask for none.  Their blocks are shared."""
    from paged_kv_decode_slot_gb300.step import LatentDecodeStep, SequenceBlocks
    r = np.random.default_rng(N)
    err = flag()
    seqs = SequenceBlocks(8, 6, 12, err_flag=err)
    cache = bf16_dev(R.to_bf16(r.standard_normal((12, 16, 576))))
    seqs.extend(i32_dev([20, 16, 30, 0, 0, 0, 0, 0]), [cache])         # 5 blocks
    seqs.fork(i32_dev([0, 1, 0, 2, 1, 1, 0, 2]))
    before, lens_before = cache.clone(), host(seqs.context_lens).copy()
    # a copy on write or a new block for rows 0, 2, 3 and 4 (row 6, the last, keeps its own): seven are free; then row 7 asks for four
    new = np.array([T, 0, T, T, T, 0, T, 52], dtype=np.int32)
    want = L.extend(host(seqs.block_tables), lens_before, new, host(seqs.ref_counts))
    assert want[4]
    seqs.extend(i32_dev(new), [cache])
    assert err_of(err) == pkv.PKV_FLAG_NO_BLOCKS
    grew = np.array([1, 0, 1, 1, 1, 0, 1, 0], dtype=bool)
    lens = host(seqs.context_lens)
    np.testing.assert_array_equal(lens, np.where(grew, lens_before + T, lens_before))
    np.testing.assert_array_equal(host(seqs.step_lens), np.where(grew, lens, 0))
    held = cache.clone()                                               # with the copies on write
    new_q = lambda *s: bf16_dev(R.to_bf16(r.standard_normal(s)))
    q, kv = new_q(8, T, N, 576), new_q(8, T, 576)
    step = LatentDecodeStep(kv, new_q(8, T, N, 64), q, cache, seqs.block_tables, seqs.step_lens, 0.07, torch.from_numpy(INV).cuda())
    step.run()
    tab = host(seqs.block_tables)
    # nothing but the new tokens' rows has changed
    written = np.zeros((12, 16), dtype=bool)
    for b in np.flatnonzero(grew):
        for p in range(int(lens[b]) - T, int(lens[b])):
            written[tab[b, p // 16], p % 16] = True
    assert written.sum() == grew.sum() * T
    changed = (bf16_host(cache) != bf16_host(held)).any(-1)
    np.testing.assert_array_equal(changed, written)
    for b in range(8):                                                 # every row's old tokens are what they were
        old = lambda c, t: bf16_host(c)[t[b, :-(-int(lens_before[b]) // 16)]].reshape(-1, 576)[:lens_before[b]]
        np.testing.assert_array_equal(old(cache, tab), old(before, tab) if not grew[b] else old(held, tab))
    ref, _, spread, size = L.attention(R.bf16_values(bf16_host(q)), out_f64(cache), tab, np.where(grew, lens, 0), 0.07)
    tol = (2.0 ** -8 + 2 * 576 * 2.0 ** -23 * 0.07 * size[..., None] + 1e-4) * spread + 2.0 ** -7 * np.abs(ref) + 1e-30
    assert np.all(np.abs(out_f64(step.out) - ref) <= tol)
    assert bool((step.out[torch.from_numpy(~grew).cuda()] == 0).all())


def test_a_captured_loop_with_beams(pkv):  # noqa: F811
    """Beams that choose their parents, grow (with copies on write) and step, all in one graph over tensors and a step that were
    there before: every replay starts from what the last one left."""
    from paged_kv_decode_slot_gb300.step import LatentDecodeStep, SequenceBlocks
    r = np.random.default_rng(11)
    rows, width, blocks, N = 12, 6, 60, 8
    err = flag()
    cache = bf16_dev(R.to_bf16(r.standard_normal((blocks, 16, 576))))
    SequenceBlocks(rows, width, blocks).fork(torch.zeros(rows, dtype=torch.int32, device="cuda"))   # (first use of the kernels)
    seqs = SequenceBlocks(rows, width, blocks, err_flag=err)
    kept = (seqs.block_tables, seqs.context_lens)
    seqs.extend(i32_dev([37, 5, 16, 30] + [0] * 8), [cache])
    parents, new = i32_dev(np.zeros(rows)), i32_dev(np.ones(rows))
    fresh = lambda *s: bf16_dev(R.to_bf16(r.standard_normal(s)))
    step = LatentDecodeStep(fresh(rows, 1, 576), fresh(rows, 1, N, 64), fresh(rows, 1, N, 576), cache, seqs.block_tables, seqs.step_lens, 0.07,
                            torch.from_numpy(INV).cuda(), err_flag=err)
    step.run()                                                         # (no row has a step yet: nothing is written)
    tab, ctx, ref = (host(x).copy() for x in (seqs.block_tables, seqs.context_lens, seqs.ref_counts))
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        seqs.fork(parents, stream)
        seqs.extend(new, [cache], stream)
        step.run(stream)
    for k in range(8):
        parents.copy_(i32_dev(r.integers(-1 if k else 0, rows if k else 4, rows)))
        new.copy_(i32_dev(r.integers(0, 2, rows)))
        step.kv_new.copy_(fresh(rows, 1, 576))
        graph.replay()
        torch.cuda.synchronize()
        tab, ctx, ref = L.fork(tab, ctx, host(parents), blocks)
        old = ctx
        tab, ctx, ref, _, refused = L.extend(tab, ctx, host(new), ref)
        assert not refused and err_of(err) == 0
        for g, w in zip((seqs.block_tables, seqs.context_lens, seqs.ref_counts), (tab, ctx, ref)):
            np.testing.assert_array_equal(host(g), w, f"replay {k}")
        want, _, spread, size = L.attention(R.bf16_values(bf16_host(step.q)), out_f64(cache), tab, np.where(ctx > old, ctx, 0), 0.07)
        tol = (2.0 ** -8 + 2 * 576 * 2.0 ** -23 * 0.07 * size[..., None] + 1e-4) * spread + 2.0 ** -7 * np.abs(want) + 1e-30
        assert np.all(np.abs(out_f64(step.out) - want) <= tol), f"replay {k}"
    assert kept[0] is seqs.block_tables and kept[1] is seqs.context_lens
