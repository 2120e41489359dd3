"""Verification of drafted tokens on the GPU: whole numbers, equal to the definition in 64 bits."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import ops_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    import paged_kv_decode_slot_gb300 as pkv
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return pkv


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def run(pkv, p, q, tokens, u, r, lens=None, V=None, err=None, ctx=None, ws=None, stream=None):
    B, T = tokens.shape
    V_ = p.shape[2] if V is None else V
    acc = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    out = torch.full((B, T + 1), -9, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = torch.zeros(pkv.pkv_verify_workspace_bytes(B, V_), dtype=torch.uint8, device="cuda")
    ctx_out = None if ctx is None else torch.empty_like(ctx)
    pkv.check(pkv.pkv_verify_draft(p, q, dev(tokens, torch.int32), dev(u, torch.float32), dev(r, torch.float32), acc, out, ws,
                                   draft_lens=None if lens is None else dev(lens, torch.int32), context_lens=ctx,
                                   context_lens_out=ctx_out, vocab_size=V, err_flag=err, stream=stream))
    return acc.cpu().numpy(), out.cpu().numpy(), ctx_out


def draw(seed, B, T, V, dtype, near=0.5):
    """(p, q) device tensors and drafted tokens that follow q."""
    r = np.random.default_rng(seed)
    a = 2.5 * r.standard_normal((B, T + 1, V))
    b = a[:, :T] + near * r.standard_normal((B, T, V))
    soft = lambda x: (e := np.exp(x - x.max(-1, keepdims=True))) / e.sum(-1, keepdims=True)
    tok = (b + r.gumbel(size=b.shape)).argmax(-1) if T else np.zeros((B, 0), np.int64)
    return dev(soft(a), dtype), dev(soft(b), dtype), tok, r


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("onehot", [False, True], ids=["draft", "onehot"])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (2, 1, 2), (3, 0, 17), (5, 2, 7), (4, 3, 255), (4, 3, 256), (4, 3, 257), (7, 8, 1000),
                                   (33, 4, 5003), (3, 40, 300), (2, 2, 32000), (1, 3, 131071), (300, 1, 64)])
def test_matches_the_definition(pkv, B, T, V, onehot, dtype):
    p, q, tok, r = draw(B + T + V, B, T, V, dtype)
    if onehot:
        q = None
    u, s = r.random((B, T)).astype(np.float32), r.random(B).astype(np.float32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc, out, _ = run(pkv, p, q, tok, u, s, err=err)
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_OK, 0)
    want = R.verify(p.double().cpu().numpy(), None if q is None else q.double().cpu().numpy(), tok, u, s)
    assert np.array_equal(acc, want[0]) and np.array_equal(out, want[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("B,T,V", [(700, 1, 40001), (1, 2, 300001), (2, 1, 524287)])
def test_runs_of_many_entries_and_rows_of_many_runs(pkv, B, T, V, dtype):
    """One CTA a row, so that the draw goes through a run in several steps; rows cut into as many runs as there may be."""
    p, q, tok, r = draw(B + T + V, B, T, V, dtype)
    u, s = r.random((B, T)).astype(np.float32), r.random(B).astype(np.float32)
    acc, out, _ = run(pkv, p, q, tok, u, s)
    want = R.verify(p.double().cpu().numpy(), q.double().cpu().numpy(), tok, u, s)
    assert np.array_equal(acc, want[0]) and np.array_equal(out, want[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_ragged_drafts_padded_rows_and_shorter_contexts(pkv, dtype):
    """Draft lengths from 0 to T, rows wider than the vocabulary (with values that must not count), contexts kept."""
    B, T, V = 40, 5, 1001
    p, q, tok, r = draw(3, B, T, V, dtype)
    wide = lambda x, w: torch.nn.functional.pad(x, (0, w - V), value=0.9)
    lens = r.integers(0, T + 1, B)
    for b in range(B):                                          # behind a draft's length nothing is read
        tok[b, lens[b]:] = -77
    u, s = r.random((B, T)).astype(np.float32), r.random(B).astype(np.float32)
    u[:, :2] = 0.0                                              # the first tokens stand
    ctx = dev(r.integers(T + 1, 5000, B), torch.int32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc, out, after = run(pkv, wide(p, 1040), wide(q, 1003), tok, u, s, lens=lens, V=V, err=err, ctx=ctx)
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_OK, 0)
    want = R.verify(p.double().cpu().numpy(), q.double().cpu().numpy(), tok, u, s, lens)
    assert np.array_equal(acc, want[0]) and np.array_equal(out, want[1])
    assert len(set(acc.tolist())) > 2
    assert np.array_equal(after.cpu().numpy(), ctx.cpu().numpy() - lens + acc)
    # in place
    ws = torch.zeros(pkv.pkv_verify_workspace_bytes(B, V), dtype=torch.uint8, device="cuda")
    a, o = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, T + 1, dtype=torch.int32, device="cuda")
    same = ctx.clone()
    pkv.check(pkv.pkv_verify_draft(p, q, dev(tok, torch.int32), dev(u, torch.float32), dev(s, torch.float32), a, o, ws,
                                   draft_lens=dev(lens, torch.int32), context_lens=same, context_lens_out=same))
    assert torch.equal(same, after)


def test_draws_on_the_borders(pkv):
    """Weights that are multiples of 2^-16 and random numbers on the running sums: an entry is drawn when its running sum
    exceeds r times the total, not when it equals it; entries of weight 0 never are."""
    r = np.random.default_rng(5)
    V, B = 3001, 400
    w = r.multinomial(65536, r.dirichlet(np.full(V, 0.05))).astype(np.float64) / 65536
    run_ = np.cumsum(w)
    assert run_[-1] == 1.0
    cut = np.concatenate([[0.0], run_[w > 0][:-1]])
    s = r.choice(cut, B)
    s[:2] = 0.0, np.float32(1.0 - 2.0 ** -24)
    below = np.maximum(0.0, np.nextafter(s.astype(np.float32), np.float32(0.0)).astype(np.float64))
    for rr in (s, below):
        rr = rr.astype(np.float32)
        p = dev(np.tile(w, (B, 1, 1)), torch.float32)
        _, out, _ = run(pkv, p, None, np.zeros((B, 0), np.int64), np.zeros((B, 0)), rr)
        want = np.searchsorted(run_, rr.astype(np.float64), side="right")
        assert np.array_equal(out[:, 0], want) and np.all(w[out[:, 0]] > 0)


def test_acceptance_at_equality_and_at_zeros(pkv):
    """u q < p decides: equality refuses, q = 0 accepts unless p = 0, u = 0 accepts unless p = 0."""
    V = 8
    p = np.zeros((6, 2, V)); q = np.zeros((6, 1, V))
    p[:, :, 0] = 0.25; p[:, :, 1] = 0.75
    q[:, :, 0] = 0.5; q[:, :, 2] = 0.5
    tok = np.array([[0], [0], [0], [1], [2], [3]])
    u = np.array([[0.5], [np.nextafter(np.float32(0.5), np.float32(0))], [0.0], [0.9], [0.0], [0.0]], dtype=np.float32)
    s = np.zeros(6, np.float32)
    acc, out, _ = run(pkv, dev(p, torch.float32), dev(q, torch.float32), tok, u, s)
    # 0.5 * 0.5 = 0.25 is not below 0.25; one ulp less is; token 1 has q = 0; tokens 2 and 3 have p = 0
    assert acc.tolist() == [0, 1, 1, 1, 0, 0]
    assert out[:, 0].tolist() == [1, 0, 0, 1, 1, 1]            # residual max(p - q, 0): only entry 1
    assert out[1:4, 1].tolist() == [0, 0, 0]
    want = R.verify(p, q, tok, u, s)
    assert np.array_equal(acc, want[0]) and np.array_equal(out, want[1])


def test_values_that_are_no_probabilities(pkv):
    """Negative, NaN, infinite and huge entries count as clamped; rows need not add up to one."""
    r = np.random.default_rng(6)
    B, T, V = 64, 2, 777
    p, q = r.random((B, T + 1, V)) * 0.01, r.random((B, T, V)) * 0.01
    for x in (p, q):
        x[r.random(x.shape) < 0.05] *= -1
        x[r.random(x.shape) < 0.02] = math.nan
        x[r.random(x.shape) < 0.01] = math.inf
        x[r.random(x.shape) < 0.01] = -math.inf
        x[r.random(x.shape) < 0.01] = 37.0
    tok, u, s = r.integers(0, V, (B, T)), r.random((B, T)).astype(np.float32), r.random(B).astype(np.float32)
    P, Q = dev(p, torch.float32), dev(q, torch.float32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    acc, out, _ = run(pkv, P, Q, tok, u, s, err=err)
    want = R.verify(P.double().cpu().numpy(), Q.double().cpu().numpy(), tok, u, s)
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_OK, 0)
    assert np.array_equal(acc, want[0]) and np.array_equal(out, want[1])


def test_no_mass_bad_tokens_bad_lengths_and_odd_random_numbers(pkv):
    V, T = 50, 2
    p, q = np.zeros((5, 3, V)), np.zeros((5, 2, V))
    p[0, :, 3] = 1.0                                            # sequence 0: a token outside the vocabulary, refused
    p[1, :, 4], q[1, :, 4] = 0.5, 0.75                          # 1: refused without residual: drawn from p
    q[2, :, 5] = 1.0                                            # 2: a row of zeros
    p[3, :, 6] = 0.3                                            # 3: a draft length outside [0, T]
    p[4, :, 7], p[4, :, 8] = 0.5, 0.5                           # 4: sample numbers outside [0, 1)
    tok = np.array([[V, 0], [4, 0], [5, 0], [6, 6], [0, 0]])
    u = np.array([[0.0, 0], [0.9, 0], [0.5, 0], [0.0, 0], [0, 0]], dtype=np.float32)
    s = np.array([0, 0, 0, 0.5, 1.5], dtype=np.float32)
    P, Q = dev(p, torch.float32), dev(q, torch.float32)
    for lens, flag in (([2, 2, 0, 2, 0], pkv.PKV_FLAG_TOKEN_RANGE | pkv.PKV_FLAG_NO_MASS), ([0, 2, 0, 9, 0], pkv.PKV_FLAG_TOKEN_RANGE | pkv.PKV_FLAG_NO_MASS),
                       ([0, 2, 0, -4, 0], pkv.PKV_FLAG_TOKEN_RANGE | pkv.PKV_FLAG_NO_MASS)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        acc, out, _ = run(pkv, P, Q, tok, u, s, lens=lens, err=err)
        assert pkv.pkv_read_err_flag(err) == (pkv.PKV_ERR_RANGE, flag)
        assert acc[0] == 0 and out[0].tolist() == [3, -1, -1]
        assert acc[1] == 0 and out[1].tolist() == [4, -1, -1]
        assert acc[2] == 0 and out[2].tolist() == [-1, -1, -1]
        n = min(max(lens[3], 0), T)
        assert acc[3] == n and out[3].tolist() == [6] * (n + 1) + [-1] * (T - n)
        assert out[4].tolist() == [8, -1, -1]
    # one-hot drafts outside the vocabulary: refused, drawn from p
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in (-5, V, 2 ** 31 - 1):
        acc, out, _ = run(pkv, P, None, np.full((5, 2), bad), u, s, lens=[1, 1, 0, 1, 1], err=err)
        assert acc.tolist() == [0] * 5 and out[:, 0].tolist() == [3, 4, -1, 6, 8]


def test_the_sampled_tokens_follow_the_target(pkv):
    """Accepted and redrawn tokens together are distributed as the target, whatever the draft: 60,000 sequences, 8 tokens.  A
    count of n p is off by more than 5.5 sigma once in 10^7."""
    B, V = 60000, 8
    r = np.random.default_rng(8)
    p, q = r.dirichlet(np.ones(V)), r.dirichlet(np.ones(V))
    tok = r.choice(V, size=(B, 1), p=q)
    P, Q = dev(np.tile(p, (B, 2, 1)), torch.float32), dev(np.tile(q, (B, 1, 1)), torch.float32)
    acc, out, _ = run(pkv, P, Q, tok, r.random((B, 1)).astype(np.float32), r.random(B).astype(np.float32))
    got = np.bincount(out[:, 0], minlength=V)
    assert np.all(np.abs(got - B * p) <= 5.5 * np.sqrt(B * p * (1 - p)))
    rate = np.minimum(p, q).sum()
    assert abs(acc.sum() - B * rate) <= 5.5 * math.sqrt(B * rate * (1 - rate))


def test_one_workspace_for_batches_and_vocabularies_of_every_size(pkv):
    B, T, V = 12, 2, 9000
    p, q, tok, r = draw(10, B, T, V, torch.float32)
    u, s = r.random((B, T)).astype(np.float32), r.random(B).astype(np.float32)
    ws = torch.zeros(pkv.pkv_verify_workspace_bytes(B, V) + 5, dtype=torch.uint8, device="cuda")
    for n, v in ((12, 9000), (1, 9000), (12, 300), (5, 8999), (12, 9000), (11, 17), (12, 9000)):
        t = np.minimum(tok[:n], v - 1)
        acc, out, _ = run(pkv, p[:n], q[:n], t, u[:n], s[:n], V=v, ws=ws)
        want = R.verify(p[:n].double().cpu().numpy(), q[:n].double().cpu().numpy(), t, u[:n], s[:n], V=v)
        assert np.array_equal(acc, want[0]) and np.array_equal(out, want[1])


def test_repeats_on_one_workspace_another_stream_and_in_a_graph(pkv):
    B, T, V = 9, 4, 50001
    p, q, tok, r = draw(9, B, T, V, torch.float32)
    u, s = r.random((B, T)).astype(np.float32), r.random(B).astype(np.float32)
    ws = torch.zeros(pkv.pkv_verify_workspace_bytes(B, V), dtype=torch.uint8, device="cuda")
    a = run(pkv, p, q, tok, u, s, ws=ws)
    assert int(ws[-4 * B:].view(torch.int32).abs().sum()) == 0, "the counters are not back at zero"
    b = run(pkv, p, q, tok, u, s, ws=ws)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        c = run(pkv, p, q, tok, u, s)
    torch.cuda.synchronize()
    for x in (b, c):
        assert np.array_equal(a[0], x[0]) and np.array_equal(a[1], x[1])
    args = (dev(tok, torch.int32), dev(u, torch.float32), dev(s, torch.float32))
    acc, out = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, T + 1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.check(pkv.pkv_verify_draft(p, q, *args, acc, out, ws))
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(a[0], acc.cpu().numpy()) and np.array_equal(a[1], out.cpu().numpy())
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    assert pkv.pkv_verify_draft(p[:0], q[:0], args[0][:0], args[1][:0], args[2][:0], e, out[:0], ws) == pkv.PKV_OK


def test_a_batch_that_shrinks_between_clusters_and_the_workspace(pkv):
    """Forty long rows share out through the workspace, a few of them in clusters: calls in turn on one workspace, repeated
    and captured, give the same tokens and leave the counters at zero."""
    B, T, V = 40, 1, 70001
    p, q, tok, r = draw(31, B, T, V, torch.float32)
    u, s = r.random((B, T)).astype(np.float32), r.random(B).astype(np.float32)
    want = R.verify(p.double().cpu().numpy(), q.double().cpu().numpy(), tok, u, s)
    ws = torch.zeros(pkv.pkv_verify_workspace_bytes(B, V), dtype=torch.uint8, device="cuda")
    for n in (40, 3, 40, 1, 9, 39, 40):
        acc, out, _ = run(pkv, p[:n], q[:n], tok[:n], u[:n], s[:n], ws=ws)
        assert np.array_equal(acc, want[0][:n]) and np.array_equal(out, want[1][:n])
        assert int(ws[-4 * B:].view(torch.int32).abs().sum()) == 0, "the counters are not back at zero"
    args = (dev(tok, torch.int32), dev(u, torch.float32), dev(s, torch.float32))
    acc, out = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, T + 1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        for _ in range(2):
            pkv.check(pkv.pkv_verify_draft(p, q, *args, acc, out, ws))
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(acc.cpu().numpy(), want[0]) and np.array_equal(out.cpu().numpy(), want[1])
