"""Verification where the weights to draw from are tiny: rows that are far from normalised, and residuals that lie in the
distributions' tails alone.  Tokens are whole numbers and equal to the definition in 64 bits: a weight is off by 2^-45 of the
row's largest, so a draw differs only where r times the total comes that near to a running sum."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ops_ref as R

pytestmark = pytest.mark.gpu
DTYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    import paged_kv_decode_slot_gb300 as pkv
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return pkv


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def check(pkv, p, q, tok, u, s, flag=0, ws=None):
    B, T = tok.shape
    V = p.shape[2]
    acc, out = torch.full((B,), -9, dtype=torch.int32, device="cuda"), torch.full((B, T + 1), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(pkv.pkv_verify_workspace_bytes(B, V), dtype=torch.uint8, device="cuda") if ws is None else ws
    pkv.check(pkv.pkv_verify_draft(p, q, dev(tok, torch.int32), dev(u, torch.float32), dev(s, torch.float32), acc, out, ws, err_flag=err))
    assert pkv.pkv_read_err_flag(err)[1] == flag
    assert int(ws[-4 * B:].view(torch.int32).abs().sum()) == 0, "the counters are not back at zero"
    want = R.verify(p.double().cpu().numpy(), None if q is None else q.double().cpu().numpy(), tok, u, s)
    assert np.array_equal(acc.cpu().numpy(), want[0])
    assert np.array_equal(out.cpu().numpy(), want[1]), np.argwhere(out.cpu().numpy() != want[1])[:5]
    return out.cpu().numpy()


NONE = lambda B: (np.zeros((B, 0), np.int64), np.zeros((B, 0), np.float32))


@DTYPES
@pytest.mark.parametrize("power", [-7, -9, -25, -50, -100, -140])
@pytest.mark.parametrize("B,V", [(1, 1), (3, 17), (5, 1000), (33, 5003), (2, 70001), (200, 3001)])
def test_rows_far_from_normalised(pkv, B, V, power, dtype):
    """Distributions times 2^power (subnormal numbers from 2^-126 on): the draw is that of the distribution.  bf16's smallest
    number is 2^-133: at 2^-140 a row may hold nothing any more, and then there is nothing to draw."""
    r = np.random.default_rng(B + V - power)
    w = r.dirichlet(np.full(V, 0.3), (B, 1)) * 2.0 ** power
    w[:, :, r.integers(0, V)] = 2.0 ** (power - 2)              # some weight at least
    P = dev(w, dtype)
    empty = bool((P == 0).all(-1).any())
    assert not empty or (power == -140 and dtype is torch.bfloat16)
    check(pkv, P, None, *NONE(B), r.random(B).astype(np.float32), flag=pkv.PKV_FLAG_NO_MASS if empty else 0)


@DTYPES
@pytest.mark.parametrize("onehot", [False, True], ids=["draft", "onehot"])
@pytest.mark.parametrize("tail", [2.0 ** -20, 2.0 ** -44, 2.0 ** -60, 2.0 ** -120])
@pytest.mark.parametrize("B,V", [(4, 200), (9, 20001), (300, 4000), (40, 70001)])
def test_residuals_in_the_tail(pkv, B, V, tail, onehot, dtype):
    """Target and draft agree but in their tails, where the target has a little more at some entries: after a refusal the token is
    one of those."""
    r = np.random.default_rng(B + V + int(-np.log2(tail)))
    p = np.zeros((B, 2, V))
    head = max(2, V // 10)
    if onehot:
        tok = r.integers(0, head, (B, 1))
        p[np.arange(B), 0, tok[:, 0]] = 1.0                     # all of it where the draft has all of it
        u = np.full((B, 1), 1.0, np.float32)                    # refused: 1 * 1 < 1 does not hold
    else:
        p[:, :, :head] = r.dirichlet(np.full(head, 0.5), (B, 2))
        tok = r.integers(head, V, (B, 1))                       # drafted where the target has nothing
        u = r.uniform(0.1, 1, (B, 1)).astype(np.float32)
    q = None if onehot else p[:, :1].copy()
    more = np.where(r.random((B, V - head)) < 0.3, r.uniform(0.1, 1, (B, V - head)) * tail, 0.0)
    more[:, 0] = tail
    p[:, 0, head:] = more
    if onehot:
        p[np.arange(B), 0, tok[:, 0]] = 1.0
    else:
        b = np.arange(B)
        p[b, 0, tok[:, 0]] = 0.0
        p[b, 0, head + (tok[:, 0] == head)] = tail
        q[b, 0, tok[:, 0]] = tail
    P, Q = dev(p, dtype), None if q is None else dev(q, dtype)
    out = check(pkv, P, Q, tok, u, r.random(B).astype(np.float32))
    rest = P[:, 0].double().cpu().numpy() - (0 if Q is None else Q[:, 0].double().cpu().numpy())
    assert np.all(rest[np.arange(B), out[:, 0]] > 0) and np.all(out[:, 0] >= head)


@DTYPES
def test_a_single_smallest_number_and_none(pkv, dtype):
    """One entry of the type's smallest number; a residual that is zero falls back to p, tiny as p may be; no entry at all."""
    V, B = 3001, 6
    least = 2.0 ** (-149 if dtype is torch.float32 else -133)
    p, q = np.zeros((B, 2, V)), np.zeros((B, 1, V))
    p[0, 0, 2999] = least                                       # the draft has nothing: the residual is this number
    p[1, 0, 17], q[1, 0, 17] = 2 * least, least
    p[2, 0, 5], p[2, 0, 9], q[2, 0, 5], q[2, 0, 9] = least, 3 * least, 2 * least, 3 * least   # no residual: from p
    q[3, 0, 8] = 0.5                                            # nothing anywhere
    p[4, 0, 0], q[4, 0, 0], p[4, 0, V - 1] = 1.0, 1.0, least    # beside a certainty that the draft shares
    p[5, 0, :] = least
    tok = np.array([[1], [2], [5], [8], [3], [4]])
    u = np.array([[0.5], [0.5], [0.75], [0.5], [0.5], [1.0]], np.float32)
    q[5, 0, 4] = 1.0
    for s in (0.0, 0.3, 0.99):
        out = check(pkv, dev(p, dtype), dev(q, dtype), tok, u, np.full(B, s, np.float32), flag=pkv.PKV_FLAG_NO_MASS)
        assert out[[0, 1, 3, 4], 0].tolist() == [2999, 17, -1, V - 1] and out[2, 0] in (5, 9)


def test_many_equal_tiny_weights_on_the_borders(pkv):
    """2^k equal weights of 2^-40, under random numbers on the running sums: exact, as for large weights."""
    V = 4096
    w = np.full((64, 1, V), 2.0 ** -40)
    s = np.random.default_rng(3).integers(0, V, 64) / V
    out = check(pkv, dev(w, torch.float32), None, *NONE(64), s.astype(np.float32))
    assert np.array_equal(out[:, 0], (s * V).astype(np.int64))


def test_tiny_and_ordinary_rows_in_turn_and_in_a_graph(pkv):
    """A batch of both on one workspace, repeated and replayed."""
    r = np.random.default_rng(4)
    B, V = 40, 70001
    w = r.dirichlet(np.full(V, 0.3), (B, 1)) * np.where(np.arange(B) % 3 == 0, 1.0, 2.0 ** -30)[:, None, None]
    P, s = dev(w, torch.float32), r.random(B).astype(np.float32)
    ws = torch.zeros(pkv.pkv_verify_workspace_bytes(B, V), dtype=torch.uint8, device="cuda")
    want = check(pkv, P, None, *NONE(B), s, ws=ws)
    check(pkv, P[:3], None, *NONE(3), s[:3])
    tok, u, sam = dev(np.zeros((B, 0)), torch.int32), dev(np.zeros((B, 0)), torch.float32), dev(s, torch.float32)
    acc, out = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.check(pkv.pkv_verify_draft(P, None, tok, u, sam, acc, out, ws))
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), want)
