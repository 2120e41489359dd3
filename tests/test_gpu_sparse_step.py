"""The operators in a run, as a serving loop uses them: a prompt rotated and appended, the bounds of its blocks, decode steps
over selected blocks (SparseDecodeStep), and speculative steps (rotating append of several tokens, multi-token attention,
verification, the context that remains).  Each stage is compared with float64 on the state that the stages before it left."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ops_ref as R
from devutil import bf16_dev, bf16_host, i32_dev, out_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    import paged_kv_decode_slot_gb300 as pkv
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return pkv


N, K, H = 8, 2, 128
INV = np.array([10000.0 ** (-j / 32) for j in range(32)])      # half of each head is turned


class Serving:
    """A batch with prompts in the cache (rotated, appended) and the bounds of their blocks."""

    def __init__(self, pkv, seed, prompts, room, kv="bf16"):
        r = self.r = np.random.default_rng(seed)
        self.pkv, self.kv, self.B = pkv, kv, len(prompts)
        self.tab, self.pool = R.tables(r, [p + room for p in prompts])
        self.tables = i32_dev(self.tab)
        self.lens = np.array(prompts, dtype=np.int32)
        kind = torch.bfloat16 if kv == "bf16" else torch.uint8
        self.kc, self.vc = (torch.zeros(self.pool, 16, K, H, dtype=kind, device="cuda") for _ in range(2))
        self.bounds = torch.zeros(self.pool, K, 2, H, dtype=torch.bfloat16, device="cuda")
        self.inv = torch.from_numpy(INV).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scales = ()
        if kv != "bf16":
            self.scales = tuple(torch.from_numpy((2.0 ** r.uniform(-7, -6, (self.pool, K))).astype(np.float32)).cuda() for _ in range(2))
        n = int(sum(prompts))
        seq = np.repeat(np.arange(self.B), prompts)
        pos = np.concatenate([np.arange(p) for p in prompts])
        slots = self.tab[seq, pos // 16].astype(np.int64) * 16 + pos % 16
        q, k, v = (bf16_dev(R.to_bf16(r.standard_normal((n, h, H)))) for h in (N, K, K))
        rope = pkv.pkv_rope_append if kv == "bf16" else pkv.pkv_rope_append_fp8
        pkv.check(rope(q, k, v, i32_dev(pos), self.inv, *self.scales, torch.from_numpy(slots).cuda(), self.kc, self.vc, q, err_flag=self.err))
        self.refresh(int(max(prompts)))

    def refresh(self, num_new):
        if self.kv == "bf16":
            self.pkv.check(self.pkv.pkv_key_bounds(self.kc, self.tables, i32_dev(self.lens), num_new, self.bounds, self.err))
        else:
            self.pkv.check(self.pkv.pkv_key_bounds_fp8(self.kc, self.scales[0], self.tables, i32_dev(self.lens), num_new, self.bounds, self.err))

    def pools(self):
        """float64 values of the pools."""
        if self.kv == "bf16":
            return R.bf16_values(bf16_host(self.kc)), R.bf16_values(bf16_host(self.vc))
        t = R.e4m3_table()
        return tuple(t[c.cpu().numpy()] * s.double().cpu().numpy()[:, None, :, None] for c, s in zip((self.kc, self.vc), self.scales))

    def check_bounds(self):
        want = R.key_bounds(self.pools()[0], self.tab, self.lens, 10 ** 6, np.zeros((self.pool, K, 2, H)))
        got = R.bf16_values(bf16_host(self.bounds))
        assert np.all(np.abs(got - want) <= (0 if self.kv == "bf16" else 2.0 ** -8 + 2.0 ** -23) * np.abs(want))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_sparse_decode_steps(pkv, kv, graph):
    from paged_kv_decode_slot_gb300.step import SparseDecodeStep, StepGraph
    s = Serving(pkv, 1, [700, 33, 15, 16, 400], 40, kv)
    s.check_bounds()
    M = 12
    q, k, v = (torch.zeros(s.B, h, H, dtype=torch.bfloat16, device="cuda") for h in (N, K, K))
    lens = i32_dev(s.lens)
    lens += 1
    scales = dict(k_scale=s.scales[0], v_scale=s.scales[1]) if s.scales else {}
    step = SparseDecodeStep(q, k, v, s.kc, s.vc, s.bounds, s.tables, lens, 0.1, s.inv, M, last_blocks=2, err_flag=s.err, **scales)
    lens -= 1
    run = StepGraph(step).replay if graph else step.run         # (the graph's own first run: the last prompt token's slot)
    for i in range(20):
        new = [R.to_bf16(s.r.standard_normal((s.B, h, H))) for h in (N, K, K)]
        for t, bits in zip((q, k, v), new):
            t.copy_(bf16_dev(bits))
        lens += 1
        s.lens += 1
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert pkv.pkv_read_err_flag(s.err) == (pkv.PKV_OK, 0)
        if i % 6:
            continue
        pos = s.lens - 1
        slots = s.tab[np.arange(s.B), pos // 16] * 16 + pos % 16
        assert np.array_equal(step.slot_mapping.cpu().numpy()[:, 0], slots)
        keys, values = s.pools()
        turned = R.bf16_values(bf16_host(step.q_turned))
        x = R.bf16_values(new[0])
        ref = R.rope(x, pos, INV, False)
        assert np.all(np.abs(turned - ref) <= 2.0 ** -8 * np.abs(ref) + 2e-6 * np.abs(x).max())
        if kv == "bf16":
            row = keys.reshape(-1, K, H)[slots]
            kx = R.bf16_values(new[1])
            kref = R.rope(kx, pos, INV, False)
            assert np.all(np.abs(row - kref) <= 2.0 ** -8 * np.abs(kref) + 2e-6 * np.abs(kx).max())
        s.check_bounds()
        sel = step.selected.cpu().numpy()
        assert np.array_equal(sel, R.select(turned, R.bf16_values(bf16_host(s.bounds)), s.tab, s.lens, M, 1, 2))
        out, lse, spread = R.blocks_attention(turned, keys, values, s.tab, s.lens, sel, 0.1)
        w = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
        assert np.all(np.abs(out_f64(step.out) - out) <= (w + 1e-4) * spread + 2.0 ** -8 * np.abs(out) + 1e-30)
        assert np.abs(step.lse.double().cpu().numpy() - lse).max() <= 1e-4
        full = (-(-s.lens // 16) <= M)                          # short sequences are attended in full
        assert full.any() and not full.all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_calls_made_by_the_extension_and_from_python_are_alike(pkv, kv, monkeypatch):
    """Plain arguments go through the compiled calls, every one of them; without the extension the results are the same bits."""
    from paged_kv_decode_slot_gb300 import binding as B
    from paged_kv_decode_slot_gb300.step import SparseDecodeStep
    assert B._calls is not None
    taken = {}

    class Recorder:
        def __getattr__(self, name):
            def call(*args):
                status = getattr(compiled, name)(*args)
                taken.setdefault(name, []).append(status)
                return status
            return call
    compiled, results = B._calls, []
    for calls in (Recorder(), None):
        monkeypatch.setattr(B, "_calls", calls)
        s = Serving(pkv, 3, [300, 20], 20, kv)
        q, k, v = (bf16_dev(R.to_bf16(s.r.standard_normal((s.B, h, H)))) for h in (N, K, K))
        scales = dict(k_scale=s.scales[0], v_scale=s.scales[1]) if s.scales else {}
        step = SparseDecodeStep(q, k, v, s.kc, s.vc, s.bounds, s.tables, i32_dev(s.lens + 1), 0.1, s.inv, 9, err_flag=s.err, **scales)
        step.run(torch.cuda.current_stream())
        p = torch.softmax(torch.from_numpy(s.r.standard_normal((s.B, 3, 77))).cuda(), -1).float()
        tok, u = torch.zeros(s.B, 2, dtype=torch.int32, device="cuda"), torch.from_numpy(s.r.random((s.B, 2)).astype(np.float32)).cuda()
        acc, out = torch.empty(s.B, dtype=torch.int32, device="cuda"), torch.empty(s.B, 3, dtype=torch.int32, device="cuda")
        ws = torch.zeros(pkv.pkv_verify_workspace_bytes(s.B, 77), dtype=torch.uint8, device="cuda")
        for V in (None, 70):
            pkv.check(pkv.pkv_verify_draft(p, None, tok, u, u[:, 0].contiguous(), acc, out, ws, vocab_size=V))
        assert pkv.pkv_read_err_flag(s.err) == (pkv.PKV_OK, 0)
        results.append([t.cpu().view(torch.uint8) for t in (s.kc, s.vc, s.bounds, step.q_turned, step.slot_mapping, step.selected, step.out,
                                                           step.lse, acc, out)])
    fp8 = "" if kv == "bf16" else "_fp8"
    assert sorted(taken) == sorted(["rope_append" + fp8, "rope_append_multi" + fp8, "key_bounds" + fp8, "select_blocks",
                                    "decode_attn_blocks" + fp8, "verify_draft"])
    assert all(x == 0 for seen in taken.values() for x in seen)
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_launches_behind_copies_other_streams_and_each_other(pkv, kv):
    """The launches start early behind whatever is ahead of them and wait for it: new inputs written by copies (from the host
    too), by kernels and on another stream just before a step, eager and captured, many steps without a pause."""
    from paged_kv_decode_slot_gb300.step import SparseDecodeStep
    steps, M, ctx0 = 24, 6, [200, 90, 17]
    r = np.random.default_rng(5)
    news = [[R.to_bf16(r.standard_normal((len(ctx0), h, H))) for h in (N, K, K)] for _ in range(steps)]
    pinned = [[bf16_dev(x).cpu().pin_memory() for x in new] for new in news]
    outs = []
    for mode in ("one by one", "behind each other", "captured"):
        s = Serving(pkv, 4, ctx0, steps + 1, kv)
        q, k, v = (torch.zeros(s.B, h, H, dtype=torch.bfloat16, device="cuda") for h in (N, K, K))
        lens = i32_dev(s.lens)
        kept = torch.zeros(steps, s.B, N, H, dtype=torch.bfloat16, device="cuda")
        scales = dict(k_scale=s.scales[0], v_scale=s.scales[1]) if s.scales else {}
        step = SparseDecodeStep(q, k, v, s.kc, s.vc, s.bounds, s.tables, lens, 0.1, s.inv, M, err_flag=s.err, **scales)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()

        def one(i):
            here = torch.cuda.current_stream()
            side.wait_stream(here)
            q.copy_(pinned[i][0], non_blocking=True)           # a copy right ahead of the first launch
            with torch.cuda.stream(side):
                k.copy_(pinned[i][1], non_blocking=True)
                v.copy_(pinned[i][2], non_blocking=True)
            lens.add_(1)
            here.wait_stream(side)                             # ahead of it: two streams
            step.run()
            kept[i].copy_(step.out)

        if mode == "captured":
            g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.graph(g, stream=st):
                for i in range(steps):
                    one(i)
            assert int(lens[0]) == ctx0[0]
            g.replay()
        else:
            for i in range(steps):
                one(i)
                if mode == "one by one":
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert pkv.pkv_read_err_flag(s.err) == (pkv.PKV_OK, 0)
        outs.append((kept.clone(), s.kc.clone(), s.bounds.clone()))
    for other in outs[1:]:
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(outs[0], other))
    assert all(bool((outs[0][0][i] != outs[0][0][i + 1]).any()) for i in range(steps - 1))


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_two_streams_at_once(pkv, graph):
    """Two batches' steps and verifications side by side on two streams (clusters, persistent grids and early launches of both
    share the SMs), many times: the results of one after the other."""
    from paged_kv_decode_slot_gb300.step import SparseDecodeStep
    work = []
    for seed, prompts, kv in ((6, [900, 300, 77], "bf16"), (7, [2000], "e4m3")):
        s = Serving(pkv, seed, prompts, 2, kv)
        q, k, v = (bf16_dev(R.to_bf16(s.r.standard_normal((s.B, h, H)))) for h in (N, K, K))
        scales = dict(k_scale=s.scales[0], v_scale=s.scales[1]) if s.scales else {}
        step = SparseDecodeStep(q, k, v, s.kc, s.vc, s.bounds, s.tables, i32_dev(s.lens + 1), 0.1, s.inv, 40, err_flag=s.err, **scales)
        p = torch.softmax(torch.from_numpy(s.r.standard_normal((s.B, 4, 60001))).cuda().float() * 3, -1)
        d = torch.softmax(torch.from_numpy(s.r.standard_normal((s.B, 3, 60001))).cuda().float() * 3, -1)
        tok = d.argmax(-1).int()
        u, sam = torch.from_numpy(s.r.random((s.B, 3)).astype(np.float32)).cuda(), torch.from_numpy(s.r.random(s.B).astype(np.float32)).cuda()
        acc, out = torch.empty(s.B, dtype=torch.int32, device="cuda"), torch.empty(s.B, 4, dtype=torch.int32, device="cuda")
        ws = torch.zeros(pkv.pkv_verify_workspace_bytes(s.B, 60001), dtype=torch.uint8, device="cuda")

        def run(step=step, args=(p, d, tok, u, sam, acc, out, ws)):
            step.run()
            pkv.check(pkv.pkv_verify_draft(*args))
        run()
        torch.cuda.synchronize()
        results = (step.out, step.lse, step.selected, s.kc, s.vc, acc, out)
        work.append((run, results, [t.clone() for t in results], torch.cuda.Stream(), s.err))
    if graph:
        graphs = []
        for run, _, _, st, _ in work:
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g, stream=st):
                for _ in range(5):
                    run()
            graphs.append(g)
        eager = work                                            # (it holds the tensors that the graphs read)
        work = [(g.replay, *w[1:]) for g, w in zip(graphs, eager)]
    for _ in range(4):
        for _, results, _, _, _ in work:
            for t in results[:3] + results[5:]:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for run, _, _, st, _ in work:
                with torch.cuda.stream(st):
                    run()
        torch.cuda.synchronize()
        for _, results, want, _, err in work:
            assert pkv.pkv_read_err_flag(err) == (pkv.PKV_OK, 0)
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(results, want))


def test_speculative_steps_over_one_cache(pkv):
    """T drafted tokens and the one before them: rotating append, multi-token attention, verification against the target's
    probabilities, and the next step from the context that remains -- refused tokens' slots are written over."""
    s = Serving(pkv, 2, [50, 16, 31, 200], 64)
    T, V = 3, 501
    r = s.r
    w = torch.from_numpy(r.standard_normal((N * H, V))).cuda() * 0.3
    from paged_kv_decode_slot_gb300.step import MultiTokenStep
    ctx = i32_dev(s.lens)                                       # contexts kept so far, on the device
    written = [dict() for _ in range(s.B)]                      # position -> v row of the token last written there
    ws = torch.zeros(pkv.pkv_verify_workspace_bytes(s.B, V), dtype=torch.uint8, device="cuda")
    kept_before = s.lens.copy()
    seen = set()
    for i in range(6):
        q, k, v = (bf16_dev(R.to_bf16(r.standard_normal((s.B, T + 1, h, H)))) for h in (N, K, K))
        full = ctx + (T + 1)
        turned, slots = torch.empty_like(q), torch.empty(s.B, T + 1, dtype=torch.int64, device="cuda")
        pkv.check(pkv.pkv_rope_append_multi(q, k, v, s.tables, full, s.inv, s.kc, s.vc, turned, slots, err_flag=s.err))
        step = MultiTokenStep(turned, k, v, s.kc, s.vc, s.tables, full, 0.1, err_flag=s.err, fused=False)
        step.attention()
        p = torch.softmax(step.out.double().view(s.B, T + 1, -1) @ w, -1).float()
        d = torch.softmax(torch.log(p[:, :T]) + 0.5 * torch.randn(s.B, T, V, device="cuda", generator=torch.Generator("cuda").manual_seed(i)), -1)
        tok = torch.from_numpy(np.stack([[r.choice(V, p=row / row.sum()) for row in b] for b in d.double().cpu().numpy()])).int().cuda()
        u, sam = torch.from_numpy(r.random((s.B, T)).astype(np.float32)).cuda(), torch.from_numpy(r.random(s.B).astype(np.float32)).cuda()
        acc, out = torch.empty(s.B, dtype=torch.int32, device="cuda"), torch.empty(s.B, T + 1, dtype=torch.int32, device="cuda")
        pkv.check(pkv.pkv_verify_draft(p, d, tok, u, sam, acc, out, ws, context_lens=full, context_lens_out=ctx, err_flag=s.err))
        assert pkv.pkv_read_err_flag(s.err) == (pkv.PKV_OK, 0)
        a = acc.cpu().numpy()
        want = R.verify(p.double().cpu().numpy(), d.double().cpu().numpy(), tok.cpu().numpy(), u.cpu().numpy(), sam.cpu().numpy())
        assert np.array_equal(a, want[0]) and np.array_equal(out.cpu().numpy(), want[1])
        assert np.array_equal(ctx.cpu().numpy(), kept_before + 1 + a)
        # attention of the step, on the cache as it is
        keys, values = s.pools()
        tq, lens = R.bf16_values(bf16_host(turned)), full.cpu().numpy()
        for t in range(T + 1):
            c = lens - T + t
            sel = np.full((s.B, K, s.tab.shape[1]), -1, dtype=np.int32)
            for b in range(s.B):
                sel[b, :, :-(-int(c[b]) // 16)] = np.arange(-(-int(c[b]) // 16))
            ref, _, spread = R.blocks_attention(tq[:, t], keys, values, s.tab, c, sel, 0.1)
            assert np.all(np.abs(out_f64(step.out[:, t]) - ref) <= 2 * (2.0 ** -8 + 1e-4) * spread + 2.0 ** -8 * np.abs(ref) + 1e-30)
        vb = bf16_host(v)
        for b in range(s.B):
            for t in range(T + 1):
                written[b][int(kept_before[b]) + t] = vb[b, t]
        kept_before = ctx.cpu().numpy().copy()
        seen |= set(a.tolist())
    assert len(seen) > 1
    rows = bf16_host(s.vc).reshape(-1, K, H)
    for b in range(s.B):
        for p_, row in written[b].items():
            assert np.array_equal(rows[s.tab[b, p_ // 16] * 16 + p_ % 16], row)


def test_sparse_step_refusals(pkv):
    from paged_kv_decode_slot_gb300.step import SparseDecodeStep
    s = Serving(pkv, 3, [20], 4)
    t = lambda h: torch.zeros(1, h, H, dtype=torch.bfloat16, device="cuda")
    args = (t(N), t(K), t(K), s.kc, s.vc, s.bounds, s.tables, i32_dev([21]), 0.1, s.inv, 4)
    with pytest.raises(ValueError):
        SparseDecodeStep(*args, last_blocks=0)
    with pytest.raises(ValueError):
        SparseDecodeStep(*args, k_scale=torch.ones(K, device="cuda"))
    step = SparseDecodeStep(*args, first_blocks=2, last_blocks=3)   # more forced blocks than places
    with pytest.raises(pkv.PkvError):
        step.run()
