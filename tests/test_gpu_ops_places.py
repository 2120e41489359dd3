"""Calls of the operators around the step that are allowed and rarely made: arguments in pinned host memory, the largest batch,
the most drafted tokens, more partitions than a list has, sizes of one."""
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


def same(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_arguments_in_pinned_host_memory(pkv, kv):
    """Everything but the pools, scales, bounds, workspaces and the rotation's inputs may lie there, inputs and outputs alike."""
    r = np.random.default_rng(1)
    B, N, K, H, M = 3, 8, 2, 128, 6
    ctx = [300, 17, 90]
    tab, pool = R.tables(r, ctx)
    dt = torch.bfloat16 if kv == "bf16" else torch.uint8
    sc = [] if kv == "bf16" else [torch.rand(pool, K, device="cuda") * 0.02 + 0.01 for _ in range(2)]
    fn = lambda name: getattr(pkv, name + ("" if kv == "bf16" else "_fp8"))
    q, k, v = (bf16_dev(R.to_bf16(r.standard_normal((B, 1, h, H)))) for h in (N, K, K))
    inv = torch.from_numpy(10000.0 ** (-np.arange(64) / 64))
    p = torch.from_numpy(r.dirichlet(np.ones(333), (B, 3)).astype(np.float32))
    d = torch.from_numpy(r.dirichlet(np.ones(333), (B, 2)).astype(np.float32))
    tok, u, s = torch.from_numpy(r.integers(0, 333, (B, 2)).astype(np.int32)), torch.rand(B, 2), torch.rand(B)
    results = []
    for place in (lambda t: t.cuda(), lambda t: t.cpu().pin_memory()):
        new = lambda *shape, dtype=torch.bfloat16: place(torch.zeros(*shape, dtype=dtype))
        kc, vc = (torch.full((pool, 16, K, H), 3, dtype=dt, device="cuda") for _ in range(2))
        bounds = torch.zeros(pool, K, 2, H, dtype=torch.bfloat16, device="cuda")
        tables, lens, err = place(torch.from_numpy(tab)), place(torch.tensor(ctx, dtype=torch.int32)), new(1, dtype=torch.int32)
        turned, slots = new(B, 1, N, H), new(B, 1, dtype=torch.int64)
        pkv.check(fn("pkv_rope_append_multi")(q, k, v, tables, lens, place(inv), *sc, kc, vc, turned, slots, err_flag=err))
        given, pos = new(B, N, H), place(torch.tensor(ctx, dtype=torch.int32) - 1)
        pkv.check(fn("pkv_rope_append")(q[:, 0], k[:, 0], v[:, 0], pos, place(inv), *sc, slots.view(-1), kc, vc, given, err_flag=err))
        pkv.check(fn("pkv_key_bounds")(kc, *sc[:1], tables, lens, 400, bounds, err))
        sel = new(B, K, M, dtype=torch.int32)
        ws = torch.zeros(pkv.pkv_select_workspace_bytes(B, K, tab.shape[1]), dtype=torch.uint8, device="cuda")
        pkv.check(pkv.pkv_select_blocks(turned[:, 0], bounds, tables, lens, sel, ws, err_flag=err))
        out, lse = new(B, N, H), new(B, N, dtype=torch.float32)
        pkv.check(fn("pkv_decode_attn_blocks")(turned[:, 0], kc, vc, *sc, tables, lens, sel, 0.1, out, lse, err_flag=err))
        acc, tokens, after = new(B, dtype=torch.int32), new(B, 3, dtype=torch.int32), new(B, dtype=torch.int32)
        ws = torch.zeros(pkv.pkv_verify_workspace_bytes(B, 333), dtype=torch.uint8, device="cuda")
        pkv.check(pkv.pkv_verify_draft(place(p), place(d), place(tok), place(u), place(s), acc, tokens, ws, context_lens=lens,
                                       context_lens_out=after, err_flag=err))
        torch.cuda.synchronize()
        assert int(err) == 0 and same(turned[:, 0], given) and bool((sel >= 0).any()) and bool(out.any())
        results.append([t.cpu() for t in (kc, vc, bounds, turned, slots, sel, out, lse, acc, tokens, after)])
    assert all(same(a, b) for a, b in zip(*results))


def test_the_largest_batch(pkv):
    """65,535 sequences, most of them empty or short: bounds, selection and attention of the few that are not."""
    r = np.random.default_rng(2)
    B, N, K, H, M, width = 65535, 2, 1, 64, 3, 8
    ctx = np.where(r.random(B) < 0.002, r.integers(60, 128, B), 0).astype(np.int32)
    ctx[[0, 1, B - 1]] = 128, 0, 127
    live = np.nonzero(ctx)[0]
    pool = 16 * len(live)
    tab = np.full((B, width), -1, dtype=np.int32)
    for i, b in enumerate(live):
        tab[b] = r.permutation(16)[:width] + 16 * i
    keys, values = (R.to_bf16(r.standard_normal((pool, 16, K, H))) for _ in range(2))
    kc, vc = bf16_dev(keys), bf16_dev(values)
    bounds = torch.zeros(pool, K, 2, H, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.check(pkv.pkv_key_bounds(kc, i32_dev(tab), i32_dev(ctx), 200, bounds, err))
    q = torch.randn(B, N, H, device="cuda").bfloat16()
    sel = torch.full((B, K, M), -9, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkv.pkv_select_workspace_bytes(B, K, width), dtype=torch.uint8, device="cuda")
    pkv.check(pkv.pkv_select_blocks(q, bounds, i32_dev(tab), i32_dev(ctx), sel, ws, 1, 1, err))
    outs = []
    for pb, parts in ((0, 0), (1, 3)):
        out, lse = torch.full_like(q, float("nan")), torch.zeros(B, N, device="cuda")
        ws2 = torch.zeros(pkv.pkv_splitk_workspace_bytes(B, N, H, parts), dtype=torch.uint8, device="cuda") if pb else None
        pkv.check(pkv.pkv_decode_attn_blocks(q, kc, vc, i32_dev(tab), i32_dev(ctx), sel, 0.125, out, lse, pb, parts, ws2, err))
        outs.append(out)
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_OK, 0)
    dead = torch.from_numpy(ctx == 0).cuda()
    assert bool((sel[dead] == -1).all()) and all(bool((o[dead] == 0).all()) for o in outs)
    got = sel[torch.from_numpy(live).cuda()].cpu().numpy()
    qv = R.bf16_values(bf16_host(q[torch.from_numpy(live).cuda()]))
    assert np.array_equal(got, R.select(qv, R.bf16_values(bf16_host(bounds)), tab[live], ctx[live], M, 1, 1))
    ref, _, spread = R.blocks_attention(qv, R.bf16_values(keys), R.bf16_values(values), tab[live], ctx[live], got, 0.125)
    for o in outs:
        o = o[torch.from_numpy(live).cuda()].double().cpu().numpy()
        assert np.all(np.abs(o - ref) <= (2.0 ** -15 + 1e-4) * spread + 2.0 ** -8 * np.abs(ref))


@pytest.mark.parametrize("B,V", [(1, 7), (70, 50), (3, 5000)])
def test_the_most_drafted_tokens(pkv, B, V):
    """1,024 of them, all but a few accepted: refused early, in the middle, at the last one and never."""
    r = np.random.default_rng(B)
    T = 1024
    p, q = r.dirichlet(np.ones(V), (B, T + 1)), r.dirichlet(np.ones(V), (B, T))
    tok = r.integers(0, V, (B, T))
    u = np.zeros((B, T), np.float32)                            # accepted wherever p is not zero
    for b in range(B):
        at = (0, 31, 32, 600, T - 1, T)[b % 6]
        if at < T:
            p[b, at, tok[b, at]] = 0.0
    s = r.random(B).astype(np.float32)
    P, Q = (torch.from_numpy(x.astype(np.float32)).cuda() for x in (p, q))
    acc, out = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, T + 1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(pkv.pkv_verify_workspace_bytes(B, V), dtype=torch.uint8, device="cuda")
    pkv.check(pkv.pkv_verify_draft(P, Q, i32_dev(tok), torch.from_numpy(u).cuda(), torch.from_numpy(s).cuda(), acc, out, ws))
    want = R.verify(P.double().cpu().numpy(), Q.double().cpu().numpy(), tok, u, s)
    assert np.array_equal(acc.cpu().numpy(), want[0]) and np.array_equal(out.cpu().numpy(), want[1])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("parts", [2, 5, 16, 17, 60])
def test_more_partitions_than_a_list_has(pkv, kv, parts):
    """A grid for longer lists than these: the partitions behind a list's end take no part."""
    r = np.random.default_rng(parts)
    ctx, N, K, H, M = [100, 16, 0, 33], 4, 2, 128, 7
    tab, pool = R.tables(r, ctx)
    if kv == "bf16":
        pools = [bf16_dev(R.to_bf16(r.standard_normal((pool, 16, K, H)))) for _ in range(2)]
    else:
        pools = [torch.from_numpy(r.integers(0, 0x50, (pool, 16, K, H)).astype(np.uint8)).cuda() for _ in range(2)]
        pools += [torch.rand(K, device="cuda") + 0.1 for _ in range(2)]
    attend = pkv.pkv_decode_attn_blocks if kv == "bf16" else pkv.pkv_decode_attn_blocks_fp8
    sel = np.full((4, K, M), -1, dtype=np.int32)
    for b, c in enumerate(ctx):
        sel[b, :, :min(M, -(-c // 16))] = np.arange(min(M, -(-c // 16)))
    q, sel = bf16_dev(R.to_bf16(r.standard_normal((4, N, H)))), torch.from_numpy(sel).cuda()
    outs = []
    for pb, most in ((0, 0), (4, 2), (4, parts)):
        out, lse = torch.full_like(q, float("nan")), torch.zeros(4, N, device="cuda")
        ws = torch.zeros(pkv.pkv_splitk_workspace_bytes(4, N, H, most), dtype=torch.uint8, device="cuda") if pb else None
        pkv.check(attend(q, *pools, i32_dev(tab), i32_dev(ctx), sel, 0.1, out, lse, pb, most, ws))
        outs.append((out.double().cpu(), lse.double().cpu()))
    for out, lse in outs[1:]:
        assert bool((out[2] == 0).all()) and bool(torch.isneginf(lse[2]).all())
        fin = [0, 1, 3]
        assert bool(((out - outs[0][0]).abs() <= 2.0 ** -7 * outs[0][0].abs() + 1e-4).all())
        assert bool(((lse[fin] - outs[0][1][fin]).abs() <= 1e-5 * (1 + outs[0][1][fin].abs())).all())
