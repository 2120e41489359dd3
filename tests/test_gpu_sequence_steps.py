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


def shortened(tab, kept, blocks):
    tab = tab.copy()
    for b, n in enumerate(kept):
        tab[b, -(-int(n) // 16):] = -1
    return tab, L.counts(tab, kept, blocks)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("rows,width,blocks", SIZES)
def test_shorten(pkv, rows, width, blocks, seed):  # noqa: F811
    """Rows of every kind (some share blocks) keep all, some or none of their tokens."""
    from paged_kv_decode_slot_gb300.step import SequenceBlocks
    r = np.random.default_rng(seed)
    tables, ctx, ref = L.random_rows(r, rows, width, blocks, 0.8)
    kept = [ctx.copy(), np.zeros_like(ctx), r.integers(0, ctx + 1).astype(np.int32), np.maximum(0, ctx - r.integers(0, 20, rows)).astype(np.int32)][seed]
    err = flag()
    seqs = SequenceBlocks(rows, width, blocks, err_flag=err)
    for t, x in ((seqs.block_tables, tables), (seqs.context_lens, ctx), (seqs.ref_counts, ref)):
        t.copy_(i32_dev(x))
    seqs.shorten(i32_dev(kept))
    tab, counts = shortened(tables, kept, blocks)
    assert err_of(err) == 0
    for g, w in zip((seqs.block_tables, seqs.context_lens, seqs.ref_counts), (tab, kept, counts)):
        np.testing.assert_array_equal(host(g), w)


def test_shorten_refuses_the_rows_own_lengths(pkv):  # noqa: F811
    from paged_kv_decode_slot_gb300.step import SequenceBlocks
    seqs = SequenceBlocks(3, 2, 9)
    with pytest.raises(ValueError, match="context_lens"):
        seqs.shorten(seqs.context_lens)
    for bad in (i32_dev([0, 0]), torch.zeros(3, dtype=torch.int64, device="cuda"), None):
        with pytest.raises((TypeError, ValueError)):
            seqs.shorten(bad)


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
def test_a_loop_of_drafts_and_verifications_loses_no_block(pkv, captured):  # noqa: F811
    """Samples of one prompt each draft T tokens, step over all T + 1, and keep what the verification accepts, across block
    borders and in shared last blocks: after every tick the counts are what the tables say, and no other row's token changed."""
    from paged_kv_decode_slot_gb300.step import LatentDecodeStep, SequenceBlocks
    r = np.random.default_rng(captured)
    rows, width, blocks, N, T, V = 6, 12, 80, 4, 5, 40
    err = flag()
    cache = bf16_dev(R.to_bf16(r.standard_normal((blocks, 16, 576))))
    seqs = SequenceBlocks(rows, width, blocks, err_flag=err)
    seqs.extend(i32_dev([45, 0, 0, 30, 0, 0]), [cache])
    seqs.fork(i32_dev([0, 0, 0, 3, 3, -1]))
    fresh = lambda *s: bf16_dev(R.to_bf16(r.standard_normal(s)))
    step = LatentDecodeStep(fresh(rows, T + 1, 576), fresh(rows, T + 1, N, 64), fresh(rows, T + 1, N, 576), cache, seqs.block_tables, seqs.step_lens,
                            0.07, torch.from_numpy(INV).cuda(), err_flag=err)
    ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    new, drafted, lens, kept = i32_dev([T + 1] * 5 + [0]), ints(rows, T), i32_dev([T] * 5 + [0]), ints(rows)
    probs, u, s = torch.rand(rows, T + 1, V, device="cuda"), torch.rand(rows, T, device="cuda"), torch.rand(rows, device="cuda")
    accepted, tokens, ws = ints(rows), ints(rows, T + 1), torch.zeros(pkv.pkv_verify_workspace_bytes(rows, V), dtype=torch.uint8, device="cuda")
    u.fill_(0.3)

    def tick(stream=None):
        seqs.extend(new, [cache], stream)
        step.run(stream)
        pkv.check(pkv.pkv_verify_draft(probs, None, drafted, u, s, accepted, tokens, ws, draft_lens=lens, context_lens=seqs.context_lens,
                                       context_lens_out=kept, err_flag=err, stream=stream))
        seqs.shorten(kept, stream)
    if captured:
        state = (seqs.block_tables, seqs.context_lens, seqs.ref_counts, cache, step.q)
        saved = [t.clone() for t in state]
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            tick(stream)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            tick(stream)
        for t, x in zip(state, saved):
            t.copy_(x)
        torch.cuda.synchronize()
    seen, most = set(), 0
    for k in range(40):
        tab, ctx, ref = (host(x).copy() for x in (seqs.block_tables, seqs.context_lens, seqs.ref_counts))
        rows_of = lambda t, n: [bf16_host(cache)[t[b, :-(-int(n[b]) // 16)]].reshape(-1, 576)[:n[b]] for b in range(rows)]
        old = rows_of(tab, ctx)
        probs.copy_(torch.rand(rows, T + 1, V, device="cuda") ** 3)
        drafted.copy_(torch.randint(0, V, (rows, T), device="cuda", dtype=torch.int32))
        step.kv_new.copy_(fresh(rows, T + 1, 576))
        graph.replay() if captured else tick()
        torch.cuda.synchronize()
        assert err_of(err) == 0
        tab, ctx, ref, _, refused = L.extend(tab, ctx, host(new), ref)
        kept_want = ctx - host(lens) + host(accepted)
        tab, ref = shortened(tab, kept_want, blocks)
        assert not refused
        for g, w in zip((seqs.block_tables, seqs.context_lens, seqs.ref_counts), (tab, kept_want, ref)):
            np.testing.assert_array_equal(host(g), w, f"tick {k}")
        for b, now in enumerate(rows_of(tab, kept_want)):
            np.testing.assert_array_equal(now[:len(old[b])], old[b])
        seen |= set(host(accepted).tolist())
        most = max(most, int(kept_want.max()))
        if most > 16 * width - 2 * (T + 1):
            break
    assert len(seen) > 3 and most > 100
    seqs.fork(i32_dev([-1] * rows))
    assert not seqs.ref_counts.any()


def test_a_step_that_grows_its_rows_is_captured_without_a_run(pkv):  # noqa: F811
    """The first step run eagerly, the others replayed: what the same number of eager steps gives."""
    from paged_kv_decode_slot_gb300.step import LatentDecodeStep, SequenceBlocks, StepGraph
    r = np.random.default_rng(2)
    fresh = lambda *s: bf16_dev(R.to_bf16(r.standard_normal(s)))
    base, kv, rope, absorbed = fresh(40, 16, 576), fresh(4, 1, 576), fresh(4, 1, 8, 64), fresh(4, 1, 8, 576)

    class Tick:
        def __init__(self):
            self.seqs, self.cache, self.ones = SequenceBlocks(4, 6, 40), base.clone(), i32_dev([1] * 4)
            self.seqs.extend(i32_dev([5, 31, 0, 47]), [self.cache])
            q = absorbed.clone()
            q[..., 512:] = rope                                        # turned in place
            self.step = LatentDecodeStep(kv, q[..., 512:], q, self.cache, self.seqs.block_tables, self.seqs.step_lens, 0.07, torch.from_numpy(INV).cuda())
            self.out = self.step.out

        def run(self, stream=None):
            self.seqs.extend(self.ones, [self.cache], stream)
            self.step.run(stream)
    one, other = Tick(), Tick()
    one.run()
    graph = StepGraph(one, warm_up=False)
    for _ in range(4):
        graph.replay()
    for _ in range(5):
        other.run()
    torch.cuda.synchronize()
    assert one.seqs.context_lens.tolist() == [10, 36, 5, 52]
    for a, b in ((one.seqs.block_tables, other.seqs.block_tables), (one.seqs.context_lens, other.seqs.context_lens),
                 (one.seqs.ref_counts, other.seqs.ref_counts), (one.cache, other.cache), (one.step.q, other.step.q), (one.out, other.out)):
        assert same(a, b)


@pytest.mark.parametrize("count", [0, -1, -7])
@pytest.mark.parametrize("blocks", [6, 40000], ids=["one CTA", "cluster"])
def test_counts_too_low_are_flagged(pkv, count, blocks):  # noqa: F811
    """A row that grows into a partly filled block whose count knows no holder; one that grows into a fresh block does not look at
    its others' counts; a fork that gives up a block without holders."""
    ref = np.zeros(blocks, dtype=np.int32)
    ref[:3] = [1, count, 1]
    tables = np.array([[0, -1], [1, -1], [2, -1]], dtype=np.int32)
    for ctx, new, want in (([5, 5, 5], [1, 1, 1], pkv.PKV_FLAG_REF_RANGE), ([5, 5, 5], [1, 0, 1], 0), ([5, 16, 5], [1, 0, 1], 0)):
        d, copies, err = [i32_dev(x) for x in (tables, ctx, new, ref)], torch.zeros(3, 2, dtype=torch.int32, device="cuda"), flag()
        pkv.check(pkv.pkv_extend_sequences(*d, copies, workspace(pkv, blocks), err))
        assert err_of(err) == want, (ctx, new)
    out, lens = torch.zeros(3, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    for parents, want in (([0, -1, 2], pkv.PKV_FLAG_REF_RANGE), ([0, 1, 2], 0)):
        err = flag()
        pkv.check(pkv.pkv_fork_sequences(i32_dev(tables), i32_dev([5, 5, 5]), i32_dev(parents), i32_dev(ref), out, lens, err))
        assert err_of(err) == want, parents


def test_the_binding_names_what_is_wrong_with_the_lengths_for_the_step(pkv):  # noqa: F811
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    tab, ctx, new, ref, copies, ws = i32(2, 4), i32(2), i32(2), i32(9), i32(2, 2), workspace(pkv, 9)
    call = lambda lens: pkv.pkv_extend_sequences_step(tab, ctx, new, ref, copies, lens, ws)
    assert call(i32(2)) == 0 and call(None) == 0 and call(torch.zeros(2, dtype=torch.int32).pin_memory()) == 0
    assert call(ctx) == pkv.PKV_ERR_SHAPE and call(new) == pkv.PKV_ERR_SHAPE
    for bad in (i32(3), i32(2, 1), i32(2).long(), torch.zeros(2, dtype=torch.int32), i32(4)[::2]):
        with pytest.raises((TypeError, ValueError), match="step_lens"):
            call(bad)
