"""The latent cache on the GPU against float64: the append (norm, rotary key, queries) and decode attention.

Append: a value is computed in fp32 and rounded once to bf16, half a step, 2^-8 of it.  Before that the norm's factor is off
by the fp32 sum of 512 squares (512 2^-24, all of one sign), a division, a square root and two products: below 2^-14; a turned
element a cos - b sin by the angle's 2^-32 turns and sincospif's error, below 2^-20 of |a| + |b|.

Attention: a weight enters the product rounded to bf16 (2^-8 of it) while the sum does not, so sum w |v| / l times 2^-8
bounds what that moves; the result's own rounding is 2^-8 of it; a logit's fp32 sum of 576 exact products, done in any order, is
off by at most 576 2^-23 scale sum |q c| = d, which moves weights by 2 d of themselves and lse by d; exponentials, their
arguments (up to 2^7 in steps of 2^-24) and the fp32 sums add less than 1e-4 of sum w |v| / l, and 2e-6 (1 + |lse|) to lse."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import latent_ref as L
import ops_ref as R
from devutil import bf16_dev, bf16_host, i32_dev, out_f64

pytestmark = pytest.mark.gpu
INV = 10000.0 ** (-np.arange(32) / 32)


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    import paged_kv_decode_slot_gb300 as pkv
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return pkv


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------------------------------------ append
def rows_tol(kv, ref, weight):
    """Per element of a cached row."""
    tol = 2.0 ** -8 * np.abs(ref) + 1e-30
    tol[:, :512] += 2.0 ** -14 * np.abs(ref[:, :512]) * (weight is not None)
    rope = np.abs(kv[:, 512:])
    tol[:, 512:] += 2.0 ** -20 * rope.max(-1, keepdims=True) * 2
    return tol


@pytest.mark.parametrize("N", [1, 5, 16, 31, 32, 33, 64, 100, 128])
@pytest.mark.parametrize("norm,inter", [(True, True), (True, False), (False, True), (False, False)])
def test_append(pkv, N, norm, inter):
    r = np.random.default_rng(N)
    n = 37
    kv = R.to_bf16(r.standard_normal((n, 576)) * 2.0 ** r.integers(-6, 7, (n, 1)))
    kv[3, :512] = 0                                        # a latent vector of zeros: eps alone under the root
    qr, q0 = R.to_bf16(r.standard_normal((n, N, 192))), R.to_bf16(r.standard_normal((n, N, 576)))
    pos = r.integers(0, [10, 3000, 200000, 2 ** 31 - 1][N % 4], n).astype(np.int32)
    slots = r.permutation(5 * 16)[:n].astype(np.int64)
    slots[[5, 20]] = -1
    w = R.to_bf16(1 + 0.2 * r.standard_normal(512)) if norm else None
    eps = 1e-5
    cache, q, err = torch.full((5, 16, 576), 7.0, device="cuda").bfloat16(), bf16_dev(q0), torch.zeros(1, dtype=torch.int32, device="cuda")
    view = bf16_dev(qr)[..., 128:]                         # strides of a wider projection
    pkv.check(pkv.pkv_latent_append(bf16_dev(kv), view, i32_dev(pos), torch.from_numpy(INV).cuda(), torch.from_numpy(slots).cuda(),
                                    cache, q, None if w is None else bf16_dev(w), eps, inter, err))
    assert int(err) == 0
    kvf, wf = R.bf16_values(kv), None if w is None else R.bf16_values(w)
    ref = L.append_rows(kvf, pos, INV, inter, wf, eps)
    live = slots >= 0
    got = out_f64(cache).reshape(-1, 576)
    assert np.all(np.abs(got[slots[live]] - ref[live]) <= rows_tol(kvf, ref, w)[live])
    if not norm:
        np.testing.assert_array_equal(bf16_host(cache).reshape(-1, 576)[slots[live], :512], kv[live, :512])
    untouched = np.setdiff1d(np.arange(80), slots)
    assert np.all(got[untouched] == 7.0)
    qf = R.bf16_values(qr[..., 128:])
    want = R.rope(qf, pos, INV, inter)
    gotq = out_f64(q)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * 2 * np.abs(qf).max(-1, keepdims=True) + 1e-30
    assert np.all(np.abs(gotq[live][..., 512:] - want[live]) <= tol[live])
    np.testing.assert_array_equal(bf16_host(q)[..., :512], q0[..., :512])
    np.testing.assert_array_equal(bf16_host(q)[~live], q0[~live])


@pytest.mark.parametrize("B,T,N", [(1, 1, 1), (3, 1, 16), (5, 4, 33), (70, 3, 8), (2, 64, 5)])
def test_append_of_the_newest_tokens(pkv, B, T, N):
    """Slots from the tables; in place (q_rope is q's own part) as from a separate tensor; contexts shorter than T."""
    r = np.random.default_rng(B + T)
    ctx = r.integers(0, 90, B).astype(np.int32)
    ctx[0] = max(0, T - 1)
    tab, pool = R.tables(r, ctx, 7)
    kv, q0 = R.to_bf16(r.standard_normal((B, T, 576))), R.to_bf16(r.standard_normal((B, T, N, 576)))
    w, inv = bf16_dev(R.to_bf16(1 + 0.2 * r.standard_normal(512))), torch.from_numpy(INV).cuda()
    results = []
    for place in ("separate", "in place", "given slots"):
        cache, q = torch.full((pool, 16, 576), 7.0, device="cuda").bfloat16(), bf16_dev(q0)
        slots = torch.full((B, T), 99, dtype=torch.int64, device="cuda")
        src = q[..., 512:] if place == "in place" else bf16_dev(q0)[..., 512:]
        if place != "given slots":
            pkv.check(pkv.pkv_latent_append_multi(bf16_dev(kv), src, i32_dev(tab), i32_dev(ctx), inv, cache, q, slots, w, 1e-6, True))
        else:
            pkv.check(pkv.pkv_slot_mapping_multi(i32_dev(tab), i32_dev(ctx), pool, slots))
            pos = torch.clamp(i32_dev(ctx)[:, None] - T + torch.arange(T, device="cuda", dtype=torch.int32), min=0)
            pkv.check(pkv.pkv_latent_append(bf16_dev(kv).view(B * T, 576), src.reshape(B * T, N, 64), pos.view(-1).contiguous(), inv,
                                            slots.view(-1), cache, q.view(B * T, N, 576), w, 1e-6, True))
        results.append((cache, q, slots))
    for got in results[1:]:
        assert all(same(a, b) for a, b in zip(got, results[0]))
    pos = ctx[:, None] - T + np.arange(T)
    live = pos >= 0
    slots = results[0][2].cpu().numpy()
    assert np.all(slots[~live] == -1)
    want = np.take_along_axis(tab, np.maximum(pos, 0) // 16, 1) * 16 + pos % 16
    np.testing.assert_array_equal(slots[live], want[live])
    ref = L.append_rows(R.bf16_values(kv).reshape(-1, 576), np.maximum(pos, 0).reshape(-1), INV, True, R.bf16_values(bf16_host(w)), 1e-6)
    got = out_f64(results[0][0]).reshape(-1, 576)[slots[live]]
    tol = rows_tol(R.bf16_values(kv).reshape(-1, 576), ref, w)
    assert np.all(np.abs(got - ref[live.reshape(-1)]) <= tol[live.reshape(-1)])


def test_append_flags_and_leaves_out(pkv):
    kv, inv = torch.randn(3, 1, 576, device="cuda").bfloat16(), torch.from_numpy(INV).cuda()
    q0 = torch.randn(3, 1, 2, 576, device="cuda").bfloat16()
    q, cache, err = q0.clone(), torch.zeros(4, 16, 576, device="cuda").bfloat16(), torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.zeros(3, 1, dtype=torch.int64, device="cuda")
    tab, ctx = i32_dev([[0, 9], [1, 2], [3, 3]]), i32_dev([20, 33, 5])
    pkv.check(pkv.pkv_latent_append_multi(kv, q0[..., 512:], tab, ctx, inv, cache, q, slots, err_flag=err))
    assert int(err) == pkv.PKV_FLAG_BLOCK_RANGE | pkv.PKV_FLAG_CTX_RANGE and slots.view(-1).tolist() == [-1, -1, 3 * 16 + 4]
    assert same(q[:2], q0[:2]) and not same(q[2], q0[2]) and int((cache != 0).any(-1).sum()) == 1
    err.zero_(), cache.zero_()
    pkv.check(pkv.pkv_latent_append(kv[:, 0], q0[:, 0, :, 512:], i32_dev([1, 2, 3]), inv, torch.tensor([64, -5, 63], device="cuda"), cache,
                                    q[:, 0], err_flag=err))
    assert int(err) == pkv.PKV_FLAG_SLOT_RANGE and int((cache != 0).any(-1).sum()) == 1 and bool((cache[3, 15] != 0).any())


# --------------------------------------------------------------------------------------- attention
class Case:
    def __init__(self, seed, ctx, N, T=1, width=None, spread=1.0):
        self.r = r = np.random.default_rng(seed)
        self.ctx, self.N, self.T = np.asarray(ctx, dtype=np.int32), N, T
        self.tab, self.pool = R.tables(r, ctx, width)
        self.q = R.to_bf16(spread * r.standard_normal((len(ctx), T, N, 576)))
        self.cache = R.to_bf16(r.standard_normal((self.pool, 16, 576)))
        self.scale = 192 ** -0.5

    def poison(self):
        """Infinities and NaN in every row that no sequence holds."""
        keep = np.zeros((self.pool, 16), dtype=bool)
        for b, c in enumerate(self.ctx):
            for j in range(-(-int(c) // 16)):
                if 0 <= self.tab[b, j] < self.pool:
                    keep[self.tab[b, j], :min(16, int(c) - 16 * j)] = True
        self.cache[~keep] = np.where(self.r.random((int((~keep).sum()), 576)) < 0.5, 0x7FC0, 0xFF80).astype(np.uint16)
        return self

    def run(self, pkv, stream=None, lse=True, err=None, ws=None):
        B = len(self.ctx)
        out = torch.full((B, self.T, self.N, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
        l = torch.full((B, self.T, self.N), float("nan"), device="cuda") if lse else None
        if ws is None:
            ws = torch.full((pkv.pkv_latent_workspace_bytes(B, self.T, self.N),), 0x7F, dtype=torch.uint8, device="cuda")
        pkv.check(pkv.pkv_decode_attn_latent(bf16_dev(self.q), bf16_dev(self.cache), i32_dev(self.tab), i32_dev(self.ctx), self.scale, out, l,
                                             ws, err, stream))
        return out, l

    def check(self, out, lse, what=""):
        ref, ref_lse, spread, size = L.attention(R.bf16_values(self.q), np.nan_to_num(R.bf16_values(self.cache), nan=0.0, posinf=0.0, neginf=0.0),
                                                 self.tab, self.ctx, self.scale)
        d = (576 * 2.0 ** -23 * abs(self.scale) * size)[..., None]
        got = out_f64(out)
        bad = np.argwhere(~np.isfinite(got).all(-1))
        assert len(bad) == 0, f"{what}: {len(bad)} rows are not finite, (sequence, token, head) {bad[:4].tolist()} .. {bad[-1].tolist()}"
        tol = (2.0 ** -8 + 2 * d + 1e-4) * spread + 2.0 ** -8 * np.abs(ref) + 1e-30
        assert np.all(np.abs(got - ref) <= tol), f"{what}: {(np.abs(got - ref) / tol).max():.2f} of the bound"
        if lse is not None:
            l = lse.double().cpu().numpy()
            fin = np.isfinite(ref_lse)
            assert np.array_equal(np.isneginf(l), ~fin), what
            assert np.all(np.abs(l[fin] - ref_lse[fin]) <= d[..., 0][fin] + 2e-6 * (1 + np.abs(ref_lse[fin]))), what
        # far below the bound on average: what a mistake in a few rows or elements would not be
        n = np.abs(ref).mean()
        assert n == 0 or np.abs(got - ref).mean() <= 2.0 ** -8 * spread.mean(), what


CTX = [0, 1, 2, 15, 16, 17, 47, 48, 49, 64, 65, 127, 128, 129, 144, 255, 256, 257, 400, 1000]


@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("N", [1, 3, 8, 16, 17, 32, 33, 40, 64, 65, 128, 130])
def test_matches_float64(pkv, N, T):
    c = Case(N + T, CTX, N, T).poison()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(pkv, err=err)
    c.check(out, lse)
    assert int(err) == 0


@pytest.mark.parametrize("N", [4, 20, 48, 128])
@pytest.mark.parametrize("ctx", [[3000], [5, 9000, 0, 17], [1] * 400, [700, 1300] * 40, [40000, 3]], ids=str)
def test_lengths_and_batches(pkv, ctx, N):
    """One sequence over the whole GPU, very uneven ones, many short ones (several of them a CTA), an empty one."""
    c = Case(len(ctx), ctx, N).poison()
    c.check(*c.run(pkv))


@pytest.mark.parametrize("N", [16, 32, 128])
def test_single_token_gives_its_row(pkv, N):
    c = Case(1, [1] * 9, N).poison()
    out, lse = c.run(pkv)
    want = bf16_dev(c.cache)[torch.from_numpy(c.tab[:, 0].astype(np.int64)).cuda(), 0, :512]
    assert same(out, want[:, None, None].expand(9, 1, N, 512))


@pytest.mark.parametrize("N", [16, 32, 100])
@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0, 30.0])
def test_scales_and_growing_maxima(pkv, N, scale):
    """Logits that keep rising (the maximum moves in every tile) and falling ones; none (a mean); weights of one token alone."""
    c = Case(7, [600, 600, 333], N)
    ramp = np.linspace(0.05, 4.0, 600)
    rows = R.bf16_values(c.cache)
    for b, up in ((0, ramp), (1, ramp[::-1])):
        direction = R.bf16_values(c.q[b, 0, 0])
        for j in range(38):
            n = min(16, 600 - 16 * j)
            rows[c.tab[b, j], :n] = 0.1 * rows[c.tab[b, j], :n] + up[16 * j:16 * j + n, None] * np.sign(direction)
    c.cache, c.scale = R.to_bf16(rows), scale
    c.poison().check(*c.run(pkv), what=f"scale {scale}")


@pytest.mark.parametrize("N", [16, 128])
def test_infinite_and_nan_values_stay_in_their_rows(pkv, N):
    """A sequence whose cache or queries hold NaN does not touch the others', in whatever CTA they are."""
    c = Case(3, [300, 200, 17, 900], N).poison()
    want = c.run(pkv)
    c.cache[c.tab[1, 3], 2] = 0x7FC0
    c.q[2] = 0x7F80
    out, lse = c.run(pkv)
    for b in (0, 3):
        assert same(out[b], want[0][b]) and same(lse[b], want[1][b])
    assert bool(out[1].isnan().all()) and bool(out[2].isnan().any())


@pytest.mark.parametrize("N", [16, 32, 128])
def test_bad_blocks_and_lengths(pkv, N):
    c = Case(5, [400, 400, 400, 100, 64], N, width=25)
    c.tab[0, 3], c.tab[1, 0], c.tab[2, 24], c.tab[3, :7] = -1, 10 ** 6, c.pool, -5
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(pkv, err=err)
    assert int(err) == pkv.PKV_FLAG_BLOCK_RANGE
    c.check(out, lse)
    assert bool((out[3] == 0).all()) and bool(torch.isneginf(lse[3]).all())
    c = Case(6, [100, 100, 100], N, width=7)
    c.ctx[:2] = [113, -1]
    err.zero_()
    out, lse = c.run(pkv, err=err)
    assert int(err) == pkv.PKV_FLAG_CTX_RANGE and bool((out[:2] == 0).all()) and bool(torch.isneginf(lse[:2]).all())
    c.check(out, lse)


@pytest.mark.parametrize("N,T", [(16, 1), (24, 3), (128, 1)])
def test_same_result_again_on_other_streams_in_graphs_and_without_lse(pkv, N, T):
    c = Case(9, [2000, 100, 0, 777, 3333], N, T).poison()
    out, lse = c.run(pkv)
    again = c.run(pkv)
    assert same(out, again[0]) and same(lse, again[1])
    assert same(out, c.run(pkv, lse=False)[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = c.run(pkv)
    s.synchronize()
    assert same(out, other[0])
    # two graphs with workspaces of their own, replayed at once on two streams
    B = len(c.ctx)
    q, cache, tab, ctx = bf16_dev(c.q), bf16_dev(c.cache), i32_dev(c.tab), i32_dev(c.ctx)
    graphs, outs = [], []
    for _ in range(2):
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        ws = torch.zeros(pkv.pkv_latent_workspace_bytes(B, T, N), dtype=torch.uint8, device="cuda")
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=st):
            pkv.check(pkv.pkv_decode_attn_latent(q, cache, tab, ctx, c.scale, o, l, ws))
        graphs.append((g, st, ws))
        outs.append((o, l))
    for _ in range(4):
        for o, l in outs:
            o.zero_(), l.zero_()
        torch.cuda.synchronize()
        for g, st, _ in graphs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        assert all(same(out, o) and same(lse, l) for o, l in outs)


def test_a_batchs_workspace_serves_fewer_sequences(pkv):
    ws = torch.full((pkv.pkv_latent_workspace_bytes(60, 1, 32),), 0xFF, dtype=torch.uint8, device="cuda")
    for ctx in ([900] * 60, [5000], [100, 7], [3000] * 20):
        c = Case(len(ctx), ctx, 32).poison()
        c.check(*c.run(pkv, ws=ws))


@pytest.mark.parametrize("N", [16, 128])
def test_pool_past_2_to_the_32_bytes(pkv, N):
    """The blocks in use are the last of 262,144 (4.8 GB): the same result as in a small pool."""
    c = Case(2, [1000, 3, 500], N)
    want = c.run(pkv)
    nb = 262_144
    big = torch.full((nb, 16, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    big[nb - c.pool:] = bf16_dev(c.cache)
    tab = i32_dev(np.where(c.tab < 0, -1, c.tab + nb - c.pool))
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    ws = torch.zeros(pkv.pkv_latent_workspace_bytes(3, 1, N), dtype=torch.uint8, device="cuda")
    pkv.check(pkv.pkv_decode_attn_latent(bf16_dev(c.q), big, tab, i32_dev(c.ctx), c.scale, out, lse, ws))
    assert same(out, want[0]) and same(lse, want[1])
    # and an append into its last block
    kv, q = torch.randn(1, 576, device="cuda").bfloat16(), torch.zeros(1, N, 576, device="cuda").bfloat16()
    pkv.check(pkv.pkv_latent_append(kv, q[..., 512:], i32_dev([0]), torch.from_numpy(INV).cuda(), torch.tensor([16 * nb - 1], device="cuda"), big, q))
    assert same(big[-1, -1], kv[0])


@pytest.mark.parametrize("N,T,ctx", [(1, 64, [70, 3, 200, 64, 0, 65]), (3, 64, [130, 64, 1, 900]), (128, 64, [300, 63]), (130, 33, [31, 257])], ids=str)
def test_up_to_64_new_tokens(pkv, N, T, ctx):
    """Many chunks of rows a sequence; lengths below the number of new tokens."""
    c = Case(N, ctx, N, T).poison()
    c.check(*c.run(pkv))


@pytest.mark.parametrize("N", [1, 40])
def test_a_large_batch_of_short_sequences(pkv, N):
    r = np.random.default_rng(N)
    c = Case(N, r.integers(0, 40, 5000), N, spread=0.5).poison()
    c.check(*c.run(pkv))


@pytest.mark.parametrize("N,T", [(48, 1), (16, 3), (24, 2), (47, 1), (11, 4), (49, 1), (60, 1)])
def test_around_48_rows(pkv, N, T):
    """The widest a CTA takes alone, and the first that a pair of CTAs shares."""
    c = Case(N, CTX, N, T).poison()
    c.check(*c.run(pkv))
    c = Case(N, [9000, 70, 0, 3333], N, T).poison()
    c.check(*c.run(pkv))


@pytest.mark.parametrize("N,T", [(128, 1), (70, 1), (40, 5), (16, 1), (32, 1)])
@pytest.mark.parametrize("ctx", [[5000, 700, 129, 40, 300], [257, 256, 384, 1], [12000]], ids=str)
def test_logits_that_jump_far_above_the_maximum_so_far(pkv, N, T, ctx):
    """Now and then a token's logits exceed all before it by hundreds, for some rows and not for others: sums already made are
    scaled down, again and again, in the first tile, the last, and where a sequence is cut."""
    c = Case(N + len(ctx), ctx, N, T, spread=0.02)
    r = c.r
    q, cache = R.bf16_values(c.q).copy(), R.bf16_values(c.cache).copy() * 0.5
    q[..., 0] = r.choice([0.0, 1.0, 1.0, -1.0, 0.25], q.shape[:-1])
    q[..., 1] = r.choice([0.0, 0.0, 1.0], q.shape[:-1])
    for b, n in enumerate(ctx):
        level, side = -400.0, -300.0
        for j in range(n):
            level += (r.random() < 0.01) * r.integers(20, 200)
            side += (r.random() < 0.004) * r.integers(20, 200)
            row = cache[c.tab[b, j // 16], j % 16]
            row[0], row[1] = level, side
        cache[c.tab[b, (n - 1) // 16], (n - 1) % 16, 0] = 2000.0           # the very last token above all
    c.q, c.cache, c.scale = R.to_bf16(q), R.to_bf16(cache), 1.0
    c.poison()
    first = c.run(pkv)
    c.check(*first)
    again = c.run(pkv)
    assert same(first[0], again[0]) and same(first[1], again[1])
