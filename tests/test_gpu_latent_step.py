"""The latent cache and the operators on sequences' blocks together, as a serving loop uses them: prompts, forks, steps with
copies on write, sequences that end, compaction, and attention after each, against float64 over a plain record of every
sequence's rows; a captured step; the binding's refusals."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import latent_ref as L
import ops_ref as R
from devutil import bf16_dev, bf16_host, i32_dev, out_f64
from test_gpu_latent import INV, pkv, same  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,T", [(16, 1), (8, 3), (128, 1)])
def test_a_serving_loop(pkv, N, T):  # noqa: F811
    from paged_kv_decode_slot_gb300.step import LatentDecodeStep, SequenceBlocks
    r = np.random.default_rng(N + T)
    rows, blocks, layers = 12, 160, 2
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    seqs = SequenceBlocks(rows, 12, blocks, err_flag=err)
    caches = [torch.full((blocks, 16, 576), float("nan"), device="cuda").bfloat16() for _ in range(layers)]
    inv, w = torch.from_numpy(INV).cuda(), bf16_dev(R.to_bf16(1 + 0.1 * r.standard_normal(512)))
    record = [[np.zeros((0, 576)) for _ in range(rows)] for _ in range(layers)]   # every row's cached rows, as values

    def check_blocks():
        ctx, tab, ref = (x.cpu().numpy() for x in (seqs.context_lens, seqs.block_tables, seqs.ref_counts))
        assert ctx.tolist() == [len(x) for x in record[0]]
        assert np.array_equal(L.counts(tab, ctx, blocks), ref)
        for b in range(rows):
            for la in range(layers):
                if ctx[b]:
                    got = out_f64(caches[la])[tab[b, :-(-ctx[b] // 16)]].reshape(-1, 576)[:ctx[b]]
                    np.testing.assert_array_equal(got, record[la][b])

    def step(live):
        """T more tokens for the rows `live`, in every layer; attention checked."""
        new = np.where(live, T, 0).astype(np.int32)
        seqs.extend(i32_dev(new), caches)
        for la in range(layers):
            q = bf16_dev(R.to_bf16(r.standard_normal((rows, T, N, 576))))
            s = LatentDecodeStep(bf16_dev(R.to_bf16(r.standard_normal((rows, T, 576)))), bf16_dev(R.to_bf16(r.standard_normal((rows, T, N, 192))))[..., 128:],
                                 q, caches[la], seqs.block_tables, torch.where(i32_dev(new) > 0, seqs.context_lens, 0), 0.07, inv, w,
                                 interleaved=True, err_flag=err)
            s.run()
            slots = s.slot_mapping.cpu().numpy()
            values = out_f64(caches[la]).reshape(-1, 576)
            for b in np.flatnonzero(live):
                record[la][b] = np.concatenate([record[la][b], values[slots[b]]])
            lens = np.where(live, [len(x) for x in record[la]], 0)
            ref, _, spread, size = L.attention(R.bf16_values(bf16_host(q)), np.nan_to_num(out_f64(caches[la])), seqs.block_tables.cpu().numpy(),
                                               lens, 0.07)
            tol = (2.0 ** -8 + 2 * 576 * 2.0 ** -23 * 0.07 * size[..., None] + 1e-4) * spread + 2.0 ** -8 * np.abs(ref) + 1e-30
            assert np.all(np.abs(out_f64(s.out) - ref) <= tol)

    def fork(parents):
        seqs.fork(i32_dev(parents))
        for la in range(layers):
            record[la] = [record[la][p] if p >= 0 else np.zeros((0, 576)) for p in parents]

    # prompts of three sequences, of odd lengths
    prompt = np.zeros(rows, dtype=np.int32)
    prompt[[0, 4, 5]] = [37, 64, 90]
    seqs.extend(i32_dev(prompt), caches)
    for la in range(layers):
        for b in (0, 4, 5):
            n = int(prompt[b])
            q = torch.zeros(n, 1, 576, device="cuda").bfloat16()
            pos = torch.arange(n, dtype=torch.int32, device="cuda")
            slots = (seqs.block_tables[b].long()[pos.long() // 16] * 16 + pos % 16)
            pkv.check(pkv.pkv_latent_append(bf16_dev(R.to_bf16(r.standard_normal((n, 576)))), q[..., 512:], pos, inv, slots, caches[la], q, w,
                                            interleaved=True, err_flag=err))
            record[la][b] = out_f64(caches[la]).reshape(-1, 576)[slots.cpu().numpy()]
    check_blocks()
    fork([0, 0, 0, -1, 4, 5, 5, 4, 4, -1, -1, 0])
    for k in range(4):
        live = np.array([len(x) > 0 for x in record[0]]) & (r.random(rows) < 0.8)
        step(live)
        check_blocks()
    fork([-1, 1, 1, -1, 5, -1, 6, -1, 8, -1, 11, 11])     # some end, some fork, some move
    check_blocks()
    seqs.compact(caches)
    check_blocks()
    used = seqs.ref_counts.cpu().numpy() > 0
    assert not used[int(used.sum()):].any() and int(seqs.num_moves) > 0
    step(np.array([len(x) > 0 for x in record[0]]))
    check_blocks()
    assert int(err) == 0
    fork([-1] * rows)
    assert int(seqs.ref_counts.abs().sum()) == 0 and bool((seqs.block_tables == -1).all())


@pytest.mark.parametrize("N", [16, 128])
def test_a_captured_step_replays_with_new_inputs(pkv, N):  # noqa: F811
    from paged_kv_decode_slot_gb300.step import LatentDecodeStep, LayerStack, StepGraph
    r = np.random.default_rng(N)
    ctx = [100, 1, 700]
    tab, pool = R.tables(r, ctx)
    inv = torch.from_numpy(INV).cuda()
    new = lambda *shape: bf16_dev(R.to_bf16(r.standard_normal(shape)))
    base = [new(pool, 16, 576) for _ in range(2)]
    make = lambda caches: [LatentDecodeStep(new(3, 1, 576), new(3, 1, N, 64), new(3, 1, N, 576), c, i32_dev(tab), i32_dev(ctx), 0.07, inv)
                           for c in caches]
    steps = make([b.clone() for b in base])
    stack = LayerStack(steps)
    graph = StepGraph(stack)
    for _ in range(3):
        for s in steps:
            s.q.copy_(new(3, 1, N, 576)), s.kv_new.copy_(new(3, 1, 576)), s.q_rope.copy_(new(3, 1, N, 64))
        qs = [s.q.clone() for s in steps]
        graph.replay()
        torch.cuda.synchronize()
        for s, q in zip(steps, qs):
            eager = LatentDecodeStep(s.kv_new, s.q_rope, q, s.latent_cache.clone(), s.block_tables, s.context_lens, 0.07, inv)
            eager.run()
            assert same(s.out, eager.out) and same(s.lse, eager.lse) and same(s.latent_cache, eager.latent_cache) and same(s.q, q)
    assert stack.launches_per_step() == 6


def test_two_streams_side_by_side(pkv):  # noqa: F811
    """Two batches' steps at once on two streams, each with its own workspace."""
    from paged_kv_decode_slot_gb300.step import LatentDecodeStep
    r = np.random.default_rng(0)
    new = lambda *shape: bf16_dev(R.to_bf16(r.standard_normal(shape)))
    inv, steps = torch.from_numpy(INV).cuda(), []
    for N, ctx in ((16, [3000, 20, 500]), (128, [900] * 7)):
        tab, pool = R.tables(r, ctx)
        steps.append(LatentDecodeStep(new(len(ctx), 1, 576), new(len(ctx), 1, N, 64), new(len(ctx), 1, N, 576), new(pool, 16, 576), i32_dev(tab),
                                      i32_dev(ctx), 0.07, inv))
    want = []
    for s in steps:
        s.run()
        want.append((s.out.clone(), s.lse.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(50):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.out.zero_()
                s.run(st)
    torch.cuda.synchronize()
    assert all(same(s.out, o) and same(s.lse, l) for s, (o, l) in zip(steps, want))


def test_the_binding_names_what_is_wrong(pkv):  # noqa: F811
    bf, i32 = lambda *s: torch.zeros(*s, device="cuda").bfloat16(), lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    cache, q, out = bf(4, 16, 576), bf(2, 1, 8, 576), bf(2, 1, 8, 512)
    tab, ctx = i32(2, 2), i32(2)
    ws = torch.zeros(pkv.pkv_latent_workspace_bytes(2, 1, 8), dtype=torch.uint8, device="cuda")
    attend = lambda **k: pkv.pkv_decode_attn_latent(*[k.get(n, d) for n, d in (("q", q), ("cache", cache), ("tab", tab), ("ctx", ctx), ("scale", 0.1),
                                                                                  ("out", out), ("lse", None), ("ws", ws))])
    assert attend() == 0
    for name, bad, what in (("cache", bf(4, 16, 512), "latent_cache"), ("cache", bf(4, 16, 1, 576), "latent_cache"), ("q", bf(2, 8, 576), "q"),
                            ("q", q.float(), "q"), ("q", q.cpu().pin_memory(), "q"), ("out", bf(2, 1, 8, 576), "out"), ("tab", i32(3, 2), "block_tables"),
                            ("ctx", i32(3), "context_lens"), ("ctx", ctx.long(), "context_lens"), ("ws", ws[:-1], None)):
        if what is None:
            assert attend(**{name: bad}) == pkv.PKV_ERR_WORKSPACE
        else:
            with pytest.raises((TypeError, ValueError), match=what):
                attend(**{name: bad})
    inv, kv, slots = torch.zeros(32, dtype=torch.float64, device="cuda"), bf(2, 1, 576), torch.zeros(2, 1, dtype=torch.int64, device="cuda")
    put = lambda **k: pkv.pkv_latent_append_multi(*[k.get(n, d) for n, d in (("kv", kv), ("qr", q[..., 512:]), ("tab", tab), ("ctx", ctx), ("inv", inv),
                                                                                ("cache", cache), ("q", q), ("slots", slots))])
    assert put() == 0
    for name, bad, what in (("qr", q, "q_rope"), ("qr", q[..., 512:].float(), "q_rope"), ("qr", q[..., 512:].cpu(), "q_rope"),
                            ("qr", q[..., ::9], "q_rope"), ("kv", bf(2, 1, 512), "kv_new"), ("inv", inv[:16].contiguous(), "inv_freq"),
                            ("slots", slots.int(), "slot_mapping")):
        with pytest.raises((TypeError, ValueError), match=what):
            put(**{name: bad})
    assert put(qr=bf(2, 1, 8, 68)[..., :64]) == pkv.PKV_ERR_ALIGN         # heads 68 elements apart
    with pytest.raises(ValueError):
        pkv.pkv_copy_blocks_pools([], i32(1, 2))
    with pytest.raises((TypeError, ValueError)):
        pkv.pkv_copy_blocks_pools([bf(4, 16, 576), bf(5, 16, 576)], i32(1, 2))
    assert pkv.pkv_copy_blocks_pools([bf(4, 4)], i32(1, 2)) == pkv.PKV_ERR_UNSUPPORTED
    assert pkv.pkv_fork_sequences(tab, ctx, i32(2), i32(9), tab, i32(2)) == pkv.PKV_ERR_SHAPE
    # no tokens, no sequences, no pairs
    empty = lambda *s: torch.zeros(*s, device="cuda").bfloat16()
    assert pkv.pkv_decode_attn_latent(empty(0, 1, 8, 576), cache, i32(0, 2), i32(0), 0.1, empty(0, 1, 8, 512)) == 0
    assert pkv.pkv_copy_blocks_pools([cache], i32(0, 2)) == 0
    assert pkv.pkv_extend_sequences(i32(0, 2), i32(0), i32(0), i32(9), i32(0, 2), ws) == 0


@pytest.mark.parametrize("N", [16, 128])
def test_a_captured_tick_grows_its_sequences(pkv, N):  # noqa: F811
    """Extension with copies, append and attention in one graph, each launch ahead of its predecessor's end, replayed over many
    steps: what the same calls give one at a time, each after the end of the last."""
    from paged_kv_decode_slot_gb300.step import LatentDecodeStep, SequenceBlocks, StepGraph
    r = np.random.default_rng(N)
    rows, blocks, ticks = 40, 400, 40
    inv, new = torch.from_numpy(INV).cuda(), lambda *shape: bf16_dev(R.to_bf16(r.standard_normal(shape)))
    base, q_rope, absorbed = new(blocks, 16, 576), new(rows, 1, N, 64), new(rows, 1, N, 576)
    kv = new(ticks, rows, 1, 576)
    parents = i32_dev(r.integers(0, 12, rows))

    class Tick:
        def __init__(self):
            self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
            self.seqs = SequenceBlocks(rows, 16, blocks, err_flag=self.err)
            self.cache = base.clone()
            first = np.zeros(rows, dtype=np.int32)
            first[:12] = np.random.default_rng(1).integers(1, 100, 12)
            self.seqs.extend(i32_dev(first), [self.cache])
            self.seqs.fork(parents)
            self.ones = torch.ones(rows, dtype=torch.int32, device="cuda")
            self.step = LatentDecodeStep(kv[0].clone(), q_rope, absorbed.clone(), self.cache, self.seqs.block_tables, self.seqs.context_lens, 0.05,
                                         inv, err_flag=self.err)
            self.out = self.step.out

        def run(self, stream=None):
            self.seqs.extend(self.ones, [self.cache], stream)
            self.step.run(stream)

        def state(self):
            return (self.seqs.block_tables, self.seqs.context_lens, self.seqs.ref_counts, self.seqs.copies, self.cache, self.step.q, self.step.out,
                    self.step.lse, self.err)
    one, other = Tick(), Tick()
    saved = [t.clone() for t in one.state()]
    graph = StepGraph(one)                                    # (runs the step while it warms up)
    for t, s in zip(one.state(), saved):
        t.copy_(s)
    for k in range(ticks):
        one.step.kv_new.copy_(kv[k])
        graph.replay()
        other.step.kv_new.copy_(kv[k])
        torch.cuda.synchronize()
        s = other.step
        other.seqs.extend(other.ones, ())
        torch.cuda.synchronize()
        other.seqs._copy([other.cache], other.seqs.copies, None)
        torch.cuda.synchronize()
        pkv.check(pkv.pkv_latent_append_multi(s.kv_new, s.q_rope, s.block_tables, s.context_lens, inv, s.latent_cache, s.q, s.slot_mapping, None,
                                              s.eps, False, s.err_flag))
        torch.cuda.synchronize()
        pkv.check(pkv.pkv_decode_attn_latent(s.q, s.latent_cache, s.block_tables, s.context_lens, s.scale, s.out, s.lse, s.workspace, s.err_flag))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(one.state(), other.state())), f"tick {k}"
    assert int(one.err) == 0 and int(one.seqs.context_lens.min()) > ticks


def test_blocks_of_more_pools_than_one_call_takes(pkv):  # noqa: F811
    from paged_kv_decode_slot_gb300.step import SequenceBlocks
    seqs = SequenceBlocks(2, 2, 5)
    pools = [torch.zeros(5, 16, 8, device="cuda") for _ in range(600)]
    seqs.extend(i32_dev([7, 0]), pools)
    for k, p in enumerate(pools):
        p[0] = k + 1
    seqs.fork(i32_dev([0, 0]))
    seqs.extend(i32_dev([1, 1]), pools)
    assert seqs.copies.tolist() == [[0, 1], [-1, -1]]
    assert all(bool((p[:2] == k + 1).all()) and not p[2:].any() for k, p in enumerate(pools))


def test_arguments_in_pinned_host_memory(pkv):  # noqa: F811
    """What the kernels read and write with plain loads and stores may lie in pinned host memory: the same results."""
    r = np.random.default_rng(4)
    new = lambda *shape: bf16_dev(R.to_bf16(r.standard_normal(shape)))
    pin = lambda t: t.cpu().pin_memory()
    inv, w, ctx = torch.from_numpy(INV).cuda(), new(512), [700, 0, 33]
    for N in (16, 128):
        tab, pool = R.tables(r, ctx)
        cache, q, kv, rope = new(pool, 16, 576), new(3, 1, N, 576), new(3, 1, 576), new(3, 1, N, 64)
        results = []
        for move in (lambda t: t, pin):
            c, qq = cache.clone(), q.clone()
            slots, out, lse = (move(torch.zeros(3, 1, dtype=torch.int64, device="cuda")), move(torch.zeros(3, 1, N, 512, device="cuda").bfloat16()),
                               move(torch.zeros(3, 1, N, device="cuda")))
            ws = torch.zeros(pkv.pkv_latent_workspace_bytes(3, 1, N), dtype=torch.uint8, device="cuda")
            t, l = move(i32_dev(tab)), move(i32_dev(ctx))
            pkv.check(pkv.pkv_latent_append_multi(move(kv), move(rope), t, l, move(inv), c, qq, slots, move(w), 1e-6, True))
            pkv.check(pkv.pkv_decode_attn_latent(qq, c, t, l, 0.05, out, lse, ws))
            torch.cuda.synchronize()
            results.append([x.cpu() for x in (c, qq, slots, out, lse)])
        assert all(same(a, b) for a, b in zip(*results))
    tables, lens, ref = L.random_rows(r, 20, 12, 200, 0.5)
    num_new = np.minimum(r.integers(0, 90, 20), 192 - lens).astype(np.int32)
    results = []
    for move in (lambda t: t, pin):
        t, l, f = move(i32_dev(tables)), move(i32_dev(lens)), i32_dev(ref)
        copies, moves, n = (move(torch.zeros(k, 2, dtype=torch.int32, device="cuda")) for k in (20, 100, 1))
        to, lo = move(torch.zeros(30, 12, dtype=torch.int32, device="cuda")), move(torch.zeros(30, dtype=torch.int32, device="cuda"))
        n = n.view(-1)[:1]
        ws = torch.zeros(pkv.pkv_blocks_workspace_bytes(200), dtype=torch.uint8, device="cuda")
        pool = torch.arange(200 * 16, device="cuda", dtype=torch.float32).view(200, 16).clone()
        pkv.check(pkv.pkv_extend_sequences(t, l, move(i32_dev(num_new)), f, copies, ws))
        pkv.check(pkv.pkv_copy_blocks_pools([pool], copies))
        pkv.check(pkv.pkv_fork_sequences(t, l, move(i32_dev(np.arange(30) % 17)), f, to, lo))
        pkv.check(pkv.pkv_compact_blocks(to, lo, f, moves, n, ws))
        pkv.check(pkv.pkv_copy_blocks_pools([pool], moves))
        torch.cuda.synchronize()
        results.append([x.cpu() for x in (t, l, f, copies, to, lo, moves, n, pool)])
    assert all(torch.equal(a, b) for a, b in zip(*results))
