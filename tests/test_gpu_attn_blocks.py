"""Attention over selected blocks on the GPU against float64.

Tolerance of an output element: the weights enter the product rounded to bf16 (half a step: 2^-8 of each weight; e4m3
pools: f16, 2^-11) while their sum does not, so sum w |v| / l times 2^-8 bounds what that moves; the result's own rounding is
2^-8 of it; the fp32 sums, exponentials (2^-22) and logits (below) add less than 1e-4 of sum w |v| / l.  lse: a logit's fp32 sum of H
exact products is off by at most H 2^-23 sum |q k| scale, and so is lse, plus 1e-6 of the sums and 2^-22 of the exponentials."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ops_ref as R
from devutil import assert_close, bf16_dev, i32_dev, out_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    import paged_kv_decode_slot_gb300 as pkv
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return pkv


class Case:
    def __init__(self, seed, ctx, N, K, H, kv="bf16", width=None):
        r = np.random.default_rng(seed)
        self.ctx, self.N, self.K, self.H, self.kv, self.r = ctx, N, K, H, kv, r
        self.tab, self.pool = R.tables(r, ctx, width)
        self.q = R.to_bf16(r.standard_normal((len(ctx), N, H)))
        self.scale = 1.0 / H ** 0.5
        shape = (self.pool, 16, K, H)
        if kv == "bf16":
            self.k, self.v = R.to_bf16(r.standard_normal(shape)), R.to_bf16(r.standard_normal(shape))
            self.kf, self.vf = R.bf16_values(self.k), R.bf16_values(self.v)
        else:
            codes = lambda: np.where(((c := r.integers(0, 256, shape).astype(np.uint8)) & 127) >= 0x50, c & 0xBF, c)
            self.k, self.v = codes(), codes()
            sc = lambda: (2.0 ** r.uniform(-4, 1, (self.pool, K) if kv == "e4m3_block" else K)).astype(np.float32)
            self.ks, self.vs = sc(), sc()
            wide = lambda s: s.astype(np.float64)[:, None, :, None] if s.ndim == 2 else s.astype(np.float64)[None, None, :, None]
            self.kf, self.vf = R.e4m3_table()[self.k] * wide(self.ks), R.e4m3_table()[self.v] * wide(self.vs)

    def lists(self, M, holes=False):
        """A random choice of min(M, blocks) blocks per (sequence, KV head); holes: some entries -1, random order."""
        out = np.full((len(self.ctx), self.K, M), -1, dtype=np.int32)
        for b, c in enumerate(self.ctx):
            nb = -(-int(c) // 16)
            for k in range(self.K):
                pick = self.r.permutation(nb)[:min(M, nb)]
                if holes:
                    pick[self.r.random(len(pick)) < 0.3] = -1
                    out[b, k, :len(pick)] = pick
                else:
                    out[b, k, :len(pick)] = np.sort(pick)
        return out

    def poison(self, selected):
        """NaN in every row that no list entry covers (bf16 pools: infinities too; e4m3: the NaN code)."""
        keep = np.zeros((self.pool, 16, self.K), dtype=bool)
        for b, c in enumerate(self.ctx):
            nb = -(-int(c) // 16)
            for k in range(self.K):
                for j in selected[b, k, :min(nb, selected.shape[2])]:
                    if 0 <= j < nb:
                        keep[self.tab[b, j], :min(16, int(c) - 16 * int(j)), k] = True
        self.k[~keep] = 0x7FC0 if self.kv == "bf16" else 0x7F
        self.v[~keep] = 0x7F80 if self.kv == "bf16" else 0xFF

    def run(self, pkv, selected, pb=0, err=None, lse=True, stream=None):
        B, M = len(self.ctx), selected.shape[2]
        q = bf16_dev(self.q)
        out = torch.full_like(q, float("nan"))
        l = torch.full((B, self.N), float("nan"), device="cuda") if lse else None
        parts = -(-M // pb) if pb else 0
        ws = torch.zeros(pkv.pkv_splitk_workspace_bytes(B, self.N, self.H, parts), dtype=torch.uint8, device="cuda") if pb else None
        sel, tab, ctx = torch.from_numpy(selected).cuda(), i32_dev(self.tab), i32_dev(self.ctx)
        if self.kv == "bf16":
            st = pkv.pkv_decode_attn_blocks(q, bf16_dev(self.k), bf16_dev(self.v), tab, ctx, sel, self.scale, out, l, pb, parts, ws, err, stream)
        else:
            st = pkv.pkv_decode_attn_blocks_fp8(q, torch.from_numpy(self.k).cuda(), torch.from_numpy(self.v).cuda(),
                                                torch.from_numpy(self.ks).cuda(), torch.from_numpy(self.vs).cuda(), tab, ctx, sel,
                                                self.scale, out, l, pb, parts, ws, err, stream)
        pkv.check(st)
        if pb:
            torch.cuda.synchronize()
            off = pkv.pkv_splitk_workspace_bytes(B, self.N, self.H, parts) - B * self.N * 4
            assert int(ws[off:].view(torch.int32).abs().sum()) == 0, "the merge counters are not back at zero"
        return out, l

    def check(self, out, lse, selected, what):
        ref, ref_lse, spread = R.blocks_attention(R.bf16_values(self.q), self.kf, self.vf, self.tab, self.ctx, selected, self.scale)
        got = out_f64(out)
        w = 2.0 ** -8 if self.kv == "bf16" else 2.0 ** -11
        tol = (w + 1e-4) * spread + 2.0 ** -8 * np.abs(ref) + 1e-30
        assert np.all(np.isfinite(got)), what
        assert np.all(np.abs(got - ref) <= tol), f"{what}: {(np.abs(got - ref) / tol).max():.2f} of the bound"
        if lse is not None:
            top = self.scale * np.abs(R.bf16_values(self.q)).sum(-1) * np.nan_to_num(np.abs(self.kf)).max()
            l = lse.double().cpu().numpy()
            fin = np.isfinite(ref_lse)
            assert np.array_equal(np.isneginf(l), ~fin), what
            err = np.abs(l[fin] - ref_lse[fin])
            assert np.all(err <= self.H * 2.0 ** -23 * top[fin] + 2e-6 * (1 + np.abs(ref_lse[fin]))), f"{what}: lse off by {err.max():.2e}"


CTX = [0, 1, 15, 16, 17, 31, 33, 100, 400, 1000]
HEADS = [(1, 1, 64), (8, 4, 128), (4, 1, 128), (16, 2, 64), (8, 1, 128)]


@pytest.mark.parametrize("holes", [False, True], ids=["sorted", "holes"])
@pytest.mark.parametrize("M,pb", [(1, 0), (5, 0), (5, 1), (20, 0), (20, 7), (64, 8), (70, 70)])
@pytest.mark.parametrize("N,K,H", HEADS)
def test_matches_float64_bf16(pkv, N, K, H, M, pb, holes):
    c = Case(N + H + M, CTX, N, K, H)
    sel = c.lists(M, holes)
    c.poison(sel)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(pkv, sel, pb, err)
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_OK, 0)
    c.check(out, lse, sel, f"N={N} K={K} H={H} M={M} pb={pb}")


@pytest.mark.parametrize("kv", ["e4m3_head", "e4m3_block"])
@pytest.mark.parametrize("M,pb", [(1, 0), (20, 0), (20, 7), (64, 8), (70, 33)])
@pytest.mark.parametrize("N,K", [(1, 1), (8, 4), (16, 2)])
def test_matches_float64_e4m3(pkv, kv, N, K, M, pb):
    c = Case(N + M, CTX, N, K, 128, kv)
    sel = c.lists(M, holes=pb == 7)
    c.poison(sel)
    out, lse = c.run(pkv, sel, pb)
    c.check(out, lse, sel, f"{kv} N={N} K={K} M={M} pb={pb}")


@pytest.mark.parametrize("kv", ["bf16", "e4m3_block"])
def test_every_block_selected_is_dense_attention(pkv, kv):
    """All blocks listed: what pkv_decode_attn gives, within both kernels' rounding (the tests' tolerance)."""
    c = Case(11, [700, 33, 1, 512], 8, 2, 128, kv)
    sel = c.lists(44)
    out, _ = c.run(pkv, sel)
    dense, lse = torch.empty_like(out), torch.empty(4, 8, device="cuda")
    q, tab, ctx = bf16_dev(c.q), i32_dev(c.tab), i32_dev(c.ctx)
    if kv == "bf16":
        pkv.check(pkv.pkv_decode_attn(q, bf16_dev(c.k), bf16_dev(c.v), tab, ctx, c.scale, dense, lse))
    else:
        pkv.check(pkv.pkv_decode_attn_fp8(q, torch.from_numpy(c.k).cuda(), torch.from_numpy(c.v).cuda(), torch.from_numpy(c.ks).cuda(),
                                          torch.from_numpy(c.vs).cuda(), tab, ctx, c.scale, dense, lse))
    _, _, spread = R.blocks_attention(R.bf16_values(c.q), c.kf, c.vf, c.tab, c.ctx, sel, c.scale)
    assert np.all(np.abs(out_f64(out) - out_f64(dense)) <= 2 * (2.0 ** -8 + 1e-4) * spread + 2.0 ** -7 * np.abs(out_f64(dense)) + 1e-30)


@pytest.mark.parametrize("pb", [0, 4])
def test_entries_out_of_range_twice_and_behind_the_blocks(pkv, pb):
    c = Case(12, [100, 100, 40], 4, 2, 128)
    sel = c.lists(12)
    sel[0, 0, 2], sel[0, 1, 0] = 7, -2                         # not a block of 100 tokens; not -1
    sel[1, 0, :7] = [3, 3, 3, 0, 6, -1, -1]                     # a block three times counts three times
    sel[2, :, 3:] = 99                                          # behind the three blocks: not read
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = c.run(pkv, sel, pb, err)
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_ERR_RANGE, pkv.PKV_FLAG_BLOCK_RANGE)
    c.check(out, lse, sel, "entries")
    c.tab[0, 1] = c.pool                                        # a block id outside the pool
    err.zero_()
    sel = c.lists(12)
    out, lse = c.run(pkv, sel, pb, err)
    assert pkv.pkv_read_err_flag(err)[1] == pkv.PKV_FLAG_BLOCK_RANGE
    c.check(out, lse, sel, "block id")
    err.zero_()
    c2 = Case(13, [100, 100], 4, 2, 128)
    good, c2.ctx = c2.lists(12), [-1, 113]
    out, lse = c2.run(pkv, good, pb, err)
    assert pkv.pkv_read_err_flag(err)[1] == pkv.PKV_FLAG_CTX_RANGE
    assert np.all(out_f64(out) == 0) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("kv,N,K,H", [("bf16", 8, 1, 128), ("bf16", 6, 3, 64), ("e4m3_block", 8, 2, 128)])
@pytest.mark.parametrize("parts", [2, 3, 8, 9, 15, 16, 17, 40])
def test_partitions_that_merge_in_clusters_and_through_the_workspace(pkv, kv, N, K, H, parts):
    """Lists in two to sixteen partitions (a cluster each) and more, lists that end in any of them, some without a key."""
    M = 3 * parts - 1
    c = Case(parts + N, [16 * n for n in range(0, M + 4, max(1, M // 7))] + [16 * M - 3, 1, 17], N, K, H, kv)
    sel = c.lists(M, holes=True)
    sel[0], sel[-3, :, :3], sel[-3, :, 6:9] = -1, -1, -1
    c.poison(sel)
    c.check(*c.run(pkv, sel, 3), sel, f"{parts} partitions")


@pytest.mark.parametrize("kv", ["bf16", "e4m3_head"])
@pytest.mark.parametrize("parts", [1, 2, 3, 5])
def test_more_partitions_than_run_at_once(pkv, kv, parts):
    c = Case(21 + parts, [int(x) for x in np.random.default_rng(parts).integers(0, 16 * 11, 90)], 8, 8, 128, kv)
    sel = c.lists(10)
    c.check(*c.run(pkv, sel, -(-10 // parts)), sel, f"{parts} partitions of {90 * 8} lists")


@pytest.mark.parametrize("kv,H", [("bf16", 64), ("bf16", 128), ("e4m3_block", 128)])
@pytest.mark.parametrize("B", [18, 20, 37, 40, 55, 59])
def test_whole_lists_around_what_runs_at_once(pkv, kv, H, B):
    """Eight lists a sequence: about one, two and three for each SM, where the number of warps a list changes."""
    c = Case(B + H, [int(x) for x in np.random.default_rng(B).integers(0, 16 * 22, B)], 8, 8, H, kv)
    sel = c.lists(20)
    c.check(*c.run(pkv, sel), sel, f"{B * 8} lists")


@pytest.mark.parametrize("pb", [0, 3])
def test_nothing_selected(pkv, pb):
    c = Case(14, [100, 3, 0], 4, 2, 64)
    out, lse = c.run(pkv, np.full((3, 2, 9), -1, dtype=np.int32), pb)
    assert np.all(out_f64(out) == 0) and bool(torch.isneginf(lse).all())
    out, lse = c.run(pkv, np.full((3, 2, 9), -1, dtype=np.int32), pb, lse=False)
    assert np.all(out_f64(out) == 0)


def test_large_logits_and_v_scales_far_apart(pkv):
    """Logits of several tens (one key takes all), blocks whose V scales lie 2^60 apart."""
    c = Case(15, [900, 640], 8, 2, 128)
    c.scale = 2.0
    sel = c.lists(30)
    c.check(*c.run(pkv, sel, 8), sel, "large logits")
    e = Case(16, [900, 640], 8, 2, 128, "e4m3_block")
    e.vs = (2.0 ** e.r.uniform(-40, 20, e.vs.shape)).astype(np.float32)
    e.vf = R.e4m3_table()[e.v] * e.vs.astype(np.float64)[:, None, :, None]
    out, lse = e.run(pkv, sel, 8)
    ref, _, _ = R.blocks_attention(R.bf16_values(e.q), e.kf, e.vf, e.tab, e.ctx, sel, e.scale)
    # weights relative to the largest scale round in f16 at 2^-24 of the unit: of the largest |v| there is
    big = np.abs(e.vf).max()
    assert np.all(np.abs(out_f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 1e-4) * big)


def test_repeats_on_another_stream_in_a_graph_and_long_lists(pkv):
    c = Case(17, [5000, 4000, 16], 8, 2, 128, width=320)
    sel = c.lists(300)
    a, la = c.run(pkv, sel, 16)
    c.check(a, la, sel, "long lists")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        b, lb = c.run(pkv, sel, 16)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16)) and torch.equal(la, lb)
    q, k, v, tab, ctx, s = bf16_dev(c.q), bf16_dev(c.k), bf16_dev(c.v), i32_dev(c.tab), i32_dev(c.ctx), torch.from_numpy(sel).cuda()
    ws = torch.zeros(pkv.pkv_splitk_workspace_bytes(3, 8, 128, 19), dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(q), torch.zeros(3, 8, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.check(pkv.pkv_decode_attn_blocks(q, k, v, tab, ctx, s, c.scale, out, lse, 16, 19, ws))
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.view(torch.int16), out.view(torch.int16)) and torch.equal(la, lse)
    assert pkv.pkv_decode_attn_blocks(q[:0], k, v, tab[:0], ctx[:0], s[:0], c.scale, out[:0]) == pkv.PKV_OK


def test_one_workspace_for_batches_of_every_size(pkv):
    """A batch that shrinks and grows on the workspace of its largest size: the counters stay where no partial reaches."""
    c = Case(19, [900, 640, 33, 0, 500, 480], 8, 2, 128)
    sel = c.lists(40)
    q, k, v, tab, ctx, s = bf16_dev(c.q), bf16_dev(c.k), bf16_dev(c.v), i32_dev(c.tab), i32_dev(c.ctx), torch.from_numpy(sel).cuda()
    ws = torch.zeros(pkv.pkv_splitk_workspace_bytes(6, 8, 128, 7) + 12, dtype=torch.uint8, device="cuda")
    first = None
    for n in (6, 2, 1, 5, 6, 3, 6):
        out, lse = torch.full_like(q[:n], float("nan")), torch.zeros(n, 8, device="cuda")
        pkv.check(pkv.pkv_decode_attn_blocks(q[:n], k, v, tab[:n], ctx[:n], s[:n], c.scale, out, lse, 6, 7, ws))
        first = out if first is None else first
        assert torch.equal(out.view(torch.int16), first[:n].view(torch.int16))
    c.check(first, None, sel, "shrinking batch")


def test_blocks_past_four_gigabytes(pkv):
    nb = 70000                                                  # 70,000 x 16 x 8 x 128 x 2 bytes: 2.3 GB a pool, 4.6 in all
    c = Case(18, [640, 100], 16, 8, 128)
    c.tab[c.tab >= 0] += nb - c.pool
    k, v = (torch.zeros(nb, 16, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[nb - c.pool:], v[nb - c.pool:] = bf16_dev(c.k), bf16_dev(c.v)
    sel = c.lists(12)
    q = bf16_dev(c.q)
    out, lse = torch.empty_like(q), torch.empty(2, 16, device="cuda")
    pkv.check(pkv.pkv_decode_attn_blocks(q, k, v, i32_dev(c.tab), i32_dev(c.ctx), torch.from_numpy(sel).cuda(), c.scale, out, lse))
    c.tab[c.tab >= 0] -= nb - c.pool
    c.check(out, lse, sel, "big pool")
