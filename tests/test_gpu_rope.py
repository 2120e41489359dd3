"""The rotating append on the GPU against float64: turned queries and keys, unturned values, slots, both pair layouts,
partial rotation, far positions, bf16 and e4m3 pools.

Tolerances.  bf16 results: half a step, 2^-8 of the value, plus the fp32 arithmetic: the angle's fraction of a turn has
32 bits (off by 2^-33 turns: 7.4e-10 rad) and is rounded to 24 (2^-25 turns: 1.9e-7 rad), sincospif is off by at most
2 ulp (2.4e-7), two products and a sum round to 2^-24 each: together below 6e-7 (|a| + |b|); 1e-6 is taken.  e4m3: half a
step, 2^-4 of the value (2^-10 scale below the normal codes), plus the same.  Values are compared bit for bit with
pkv_append / pkv_append_fp8."""
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


def freqs(R_, base=500000.0):
    return np.array([base ** (-2.0 * j / R_) for j in range(R_ // 2)])


def f64_dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64)).cuda()


def near(got, ref, a_abs, what):
    tol = 2.0 ** -8 * np.abs(ref) + 1e-6 * a_abs + 2.0 ** -133
    bad = np.abs(got - ref) - tol
    assert np.all(bad <= 0), f"{what}: off by {np.abs(got - ref).max():.3e} at {np.unravel_index(bad.argmax(), bad.shape)}"


def pair_sums(x):
    """A bound of |a| + |b| for every element of a head."""
    return 2 * np.abs(x).max(-1, keepdims=True) * np.ones_like(x)


class Case:
    def __init__(self, seed, n, N, K, H, R_, inter, pool=None, positions=None):
        r = np.random.default_rng(seed)
        self.N, self.K, self.H, self.inter, self.n = N, K, H, inter, n
        self.q, self.k, self.v = (R.to_bf16(r.standard_normal((n, h, H))) for h in (N, K, K))
        self.f = freqs(R_)
        self.pos = (r.integers(0, 5000, n) if positions is None else np.resize(positions, n)).astype(np.int32)
        self.pool = pool or -(-n // 16) + 2
        self.slots = r.permutation(self.pool * 16)[:n].astype(np.int64)
        if n > 3:
            self.slots[[1, n - 1]] = -1
        self.live = self.slots >= 0
        self.q_ref = R.rope(R.bf16_values(self.q), self.pos, self.f, inter)
        self.k_ref = R.rope(R.bf16_values(self.k), self.pos, self.f, inter)

    def dev(self):
        return (bf16_dev(self.q), bf16_dev(self.k), bf16_dev(self.v), i32_dev(self.pos), f64_dev(self.f))

    def slots_dev(self):
        return torch.from_numpy(self.slots).cuda()

    def check_q(self, q_out, what):
        got = bf16_host(q_out)
        assert np.array_equal(got[~self.live], np.full_like(got[~self.live], 0x1234)), f"{what}: a left-out row was written"
        x = R.bf16_values(self.q)
        near(R.bf16_values(got)[self.live], self.q_ref[self.live], pair_sums(x)[self.live], what)


def marked(shape):
    return bf16_dev(np.full(shape, 0x1234, dtype=np.uint16))


FAR = [0, 1, 2, 1000, 131071, 999983, 16777217, 2 ** 31 - 1, -3]


@pytest.mark.parametrize("n,N,K,H,R_,inter,positions", [
    (1, 1, 1, 64, 64, False, None), (1, 1, 1, 128, 16, True, None), (5, 8, 2, 64, 32, False, None),
    (17, 32, 8, 128, 128, False, FAR), (17, 4, 4, 128, 64, True, FAR), (9, 5, 5, 128, 96, False, FAR),
    (300, 16, 2, 64, 48, True, None), (40, 100, 50, 128, 128, False, None), (33, 129, 43, 64, 64, True, None),
])
def test_rope_append_matches_float64(pkv, n, N, K, H, R_, inter, positions):
    c = Case(n + N + H, n, N, K, H, R_, inter, positions=positions)
    q, k, v, pos, f = c.dev()
    kc, vc, out = marked((c.pool, 16, K, H)), marked((c.pool, 16, K, H)), marked((n, N, H))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.check(pkv.pkv_rope_append(q, k, v, pos, f, c.slots_dev(), kc, vc, out, interleaved=inter, err_flag=err))
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_OK, 0)
    c.check_q(out, "q")
    rows_k, rows_v = bf16_host(kc).reshape(-1, K, H), bf16_host(vc).reshape(-1, K, H)
    at = c.slots[c.live]
    near(R.bf16_values(rows_k[at]), c.k_ref[c.live], pair_sums(R.bf16_values(c.k))[c.live], "k")
    assert np.array_equal(rows_v[at], c.v[c.live])
    rest = np.setdiff1d(np.arange(c.pool * 16), at)
    assert np.all(rows_k[rest] == 0x1234) and np.all(rows_v[rest] == 0x1234)
    if R_ < H:  # elements behind the rotation are copied bit for bit
        assert np.array_equal(bf16_host(out)[c.live][..., R_:], c.q[c.live][..., R_:])
        assert np.array_equal(rows_k[at][..., R_:], c.k[c.live][..., R_:])


def test_position_zero_changes_nothing_and_in_place_equals_out_of_place(pkv):
    c = Case(5, 600, 8, 2, 128, 128, False)
    q, k, v, pos, f = c.dev()
    kc, vc, out = marked((c.pool, 16, 2, 128)), marked((c.pool, 16, 2, 128)), q.clone()
    pkv.check(pkv.pkv_rope_append(q, k, v, torch.zeros_like(pos), f, c.slots_dev(), kc, vc, out))
    assert torch.equal(out.view(torch.int16), q.view(torch.int16))
    pkv.check(pkv.pkv_rope_append(q, k, v, pos, f, c.slots_dev(), kc, vc, out))
    same = q.clone()
    pkv.check(pkv.pkv_rope_append(same, k, v, pos, f, c.slots_dev(), kc, vc, same))
    assert torch.equal(same.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_multi_form_equals_given_slots(pkv, oracle, T, kv):
    """Slots and positions from the tables: the same results, bit for bit, as pkv_slot_mapping_multi's slots
    given with the positions -- with empty sequences and ones shorter than T."""
    r = np.random.default_rng(T)
    ctx = np.array([0, 1, 2, 4, 5, 15, 16, 17, 33, 64, 250], dtype=np.int32)
    B, N, K, H = len(ctx), 8, 4, 128
    tab, pool = R.tables(r, ctx)
    q, k, v = (bf16_dev(R.to_bf16(r.standard_normal((B, T, h, H)))) for h in (N, K, K))
    f = f64_dev(freqs(64))
    slots = torch.full((B, T), -7, dtype=torch.int64, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kind = torch.uint8 if kv == "e4m3" else torch.bfloat16
    new = lambda: torch.zeros(pool, 16, K, H, dtype=kind, device="cuda")
    sc = [torch.rand(pool, K, device="cuda") * 0.02 + 0.005 for _ in range(2)]
    kc, vc, out = new(), new(), torch.zeros_like(q)
    if kv == "e4m3":
        st = pkv.pkv_rope_append_multi_fp8(q, k, v, i32_dev(tab), i32_dev(ctx), f, *sc, kc, vc, out, slots, err_flag=err)
    else:
        st = pkv.pkv_rope_append_multi(q, k, v, i32_dev(tab), i32_dev(ctx), f, kc, vc, out, slots, err_flag=err)
    pkv.check(st)
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_OK, 0)
    want = oracle.slot_mapping_multi(tab, ctx, T)
    assert np.array_equal(slots.cpu().numpy(), want)
    pos = i32_dev((ctx[:, None] - T + np.arange(T)).reshape(-1))
    flat = [x.view(B * T, *x.shape[2:]) for x in (q, k, v)]
    kc2, vc2, out2 = new(), new(), torch.zeros_like(flat[0])
    given = torch.from_numpy(want.reshape(-1)).cuda()
    if kv == "e4m3":
        pkv.check(pkv.pkv_rope_append_fp8(*flat, pos, f, *sc, given, kc2, vc2, out2))
    else:
        pkv.check(pkv.pkv_rope_append(*flat, pos, f, given, kc2, vc2, out2))
    eq = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert eq(kc, kc2) and eq(vc, vc2) and eq(out.view(-1, N, H), out2)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("blocks", [False, True], ids=["head", "block"])
def test_e4m3_values_bitwise_and_keys_to_half_a_step(pkv, blocks, inter):
    c = Case(40 + inter, 211, 6, 3, 128, 96, inter)
    r = np.random.default_rng(1)
    ks, vs = (torch.from_numpy((2.0 ** r.uniform(-9, -5, (c.pool, 3) if blocks else 3)).astype(np.float32)).cuda() for _ in range(2))
    if not blocks:
        vs[0] = 2.0 ** -6                                     # a power of two: quotients fall on ties
    q, k, v, pos, f = c.dev()
    new = lambda: torch.zeros(c.pool, 16, 3, 128, dtype=torch.uint8, device="cuda")
    kc, vc, kc2, vc2, out = new(), new(), new(), new(), marked((211, 6, 128))
    pkv.check(pkv.pkv_rope_append_fp8(q, k, v, pos, f, ks, vs, c.slots_dev(), kc, vc, out, interleaved=inter))
    pkv.check(pkv.pkv_append_fp8(k, v, ks, vs, c.slots_dev(), kc2, vc2))
    assert torch.equal(vc, vc2)
    c.check_q(out, "q")
    at = c.slots[c.live]
    sc = ks.double().cpu().numpy()
    sc = sc[at // 16][:, :, None] if blocks else sc[None, :, None]
    got = R.e4m3_table()[kc.cpu().numpy().reshape(-1, 3, 128)[at]] * sc
    ref = np.clip(c.k_ref[c.live], -448 * sc, 448 * sc)
    tol = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * sc) + 1e-6 * pair_sums(R.bf16_values(c.k))[c.live]
    assert np.all(np.abs(got - ref) <= tol), np.abs(got - ref).max()


@pytest.mark.parametrize("scale", [1.0, 0.0123, 3.0, 2.0 ** -7, 1e-30, 1e-38, 3e33, 1.7e38])
def test_e4m3_quotients_of_extreme_values(pkv, scale):
    """Signed zeros, subnormals, infinities, NaN, values at and beyond the codes' end, ties and their neighbours under
    scales from 1e-38 to 1.7e38: the codes pkv_append_fp8 gives, bit for bit (values, and keys at position 0)."""
    r = np.random.default_rng(3)
    K, H, n = 2, 128, 64
    table = R.e4m3_table()
    fine = np.sort(table[~np.isnan(table)])
    with np.errstate(over="ignore"):
        ties = R.to_bf16((((fine[1:] + fine[:-1]) / 2) * scale).astype(np.float32))
    bits = np.concatenate([np.array([0, 0x8000, 1, 0x8001, 0x7F7F, 0xFF7F, 0x7F80, 0xFF80, 0x7FC0], dtype=np.uint16),
                           ties, ties + 1, ties - 1, r.integers(0, 65536, 4096).astype(np.uint16)])
    x = bf16_dev(np.resize(bits, (n, K, H)))
    q = torch.zeros(n, K, H, dtype=torch.bfloat16, device="cuda")
    sc = torch.full((K,), scale, device="cuda")
    slots, pos = torch.arange(n, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    new = lambda: torch.zeros(n // 16, 16, K, H, dtype=torch.uint8, device="cuda")
    kc, vc, kc2, vc2 = new(), new(), new(), new()
    pkv.check(pkv.pkv_rope_append_fp8(q, x, x, pos, f64_dev(freqs(64)), sc, sc, slots, kc, vc, q))
    pkv.check(pkv.pkv_append_fp8(x, x, sc, sc, slots, kc2, vc2))
    nan = (vc2 & 0x7F) == 0x7F
    assert torch.equal(((vc & 0x7F) == 0x7F), nan) and torch.equal(vc[~nan], vc2[~nan])
    # keys: the unturned half of each head, where position 0 leaves even infinities and NaN to themselves
    assert torch.equal(kc[..., 64:][~nan[..., 64:]], kc2[..., 64:][~nan[..., 64:]])


def test_e4m3_codes_of_every_bf16_value_over_many_scales(pkv):
    """All 65,536 bit patterns over 96 scales (mantissas of zeros, of ones, next to powers of two, random; exponents from 2^-102
    to 2^102): the codes of pkv_append_fp8, which divides."""
    K, H, n = 96, 128, 512
    r = np.random.default_rng(6)
    mant = np.concatenate([[0, 1, 0x7FFFFF, 0x7FFFFE, 0x400000, 0x3FFFFF, 0x2AAAAA, 0x555555], r.integers(0, 1 << 23, K - 8)])
    expo = np.concatenate([np.repeat(127, 8), r.integers(25, 230, 8), r.integers(100, 140, K - 16)])
    sc = torch.from_numpy((expo.astype(np.uint32) << 23 | mant.astype(np.uint32)).view(np.float32)).cuda()
    bits = np.arange(65536, dtype=np.uint16).reshape(n, 1, H)
    kv = bf16_dev(np.ascontiguousarray(np.broadcast_to(bits, (n, K, H))))
    pools = [torch.zeros(n // 16, 16, K, H, dtype=torch.uint8, device="cuda") for _ in range(4)]
    slots = torch.arange(n, dtype=torch.int64, device="cuda")
    pkv.check(pkv.pkv_append_fp8(kv, kv, sc, sc, slots, pools[0], pools[1]))
    q = torch.zeros(n, 1, H, dtype=torch.bfloat16, device="cuda")
    pkv.check(pkv.pkv_rope_append_fp8(q, kv, kv, i32_dev(np.zeros(n)), torch.ones(8, dtype=torch.float64, device="cuda"), sc, sc, slots,
                                      pools[2], pools[3], q))
    nan = (pools[1] & 0x7F) == 0x7F
    assert torch.equal((pools[3] & 0x7F) == 0x7F, nan) and torch.equal(pools[3][~nan], pools[1][~nan])
    assert torch.equal(pools[2][..., 16:][~nan[..., 16:]], pools[0][..., 16:][~nan[..., 16:]])


def test_bad_slots_tables_and_lengths_are_flagged_and_left_out(pkv):
    c = Case(6, 20, 4, 2, 64, 64, False)
    q, k, v, pos, f = c.dev()
    slots = c.slots_dev()
    slots[5] = c.pool * 16
    c.live[5] = False
    kc, vc, out = marked((c.pool, 16, 2, 64)), marked((c.pool, 16, 2, 64)), marked((20, 4, 64))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.check(pkv.pkv_rope_append(q, k, v, pos, f, slots, kc, vc, out, err_flag=err))
    assert pkv.pkv_read_err_flag(err) == (pkv.PKV_ERR_RANGE, pkv.PKV_FLAG_SLOT_RANGE)
    c.check_q(out, "q")
    for ctx, entry, flag in ((40, 9, pkv.PKV_FLAG_BLOCK_RANGE), (40, -1, pkv.PKV_FLAG_BLOCK_RANGE), (49, 1, pkv.PKV_FLAG_CTX_RANGE)):
        err.zero_()
        tab = torch.tensor([[0, 1, entry]], dtype=torch.int32, device="cuda")
        got = torch.full((1, 1), 5, dtype=torch.int64, device="cuda")
        kc, vc, out = marked((3, 16, 2, 64)), marked((3, 16, 2, 64)), marked((1, 1, 4, 64))
        pkv.check(pkv.pkv_rope_append_multi(q[:1, None], k[:1, None], v[:1, None], tab, i32_dev([ctx]), f, kc, vc, out, got,
                                            err_flag=err))
        assert pkv.pkv_read_err_flag(err) == (pkv.PKV_ERR_RANGE, flag) and int(got) == -1
        assert np.all(bf16_host(kc) == 0x1234) and np.all(bf16_host(vc) == 0x1234) and np.all(bf16_host(out) == 0x1234)


def test_more_units_than_ctas_twice_on_another_stream_and_in_a_graph(pkv):
    """Rows of several units a token, many times the grid; replayed calls and calls on a side stream agree bit for bit."""
    c = Case(8, 3001, 70, 30, 64, 64, False)
    q, k, v, pos, f = c.dev()
    slots = c.slots_dev()

    def fresh():
        return marked((c.pool, 16, 30, 64)), marked((c.pool, 16, 30, 64)), marked((3001, 70, 64))
    a = fresh()
    pkv.check(pkv.pkv_rope_append(q, k, v, pos, f, slots, *a))
    c.check_q(a[2], "q")
    b, st = fresh(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    pkv.check(pkv.pkv_rope_append(q, k, v, pos, f, slots, *b, stream=st))
    g = torch.cuda.CUDAGraph()
    d = fresh()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.check(pkv.pkv_rope_append(q, k, v, pos, f, slots, *d))
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, d):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16)) and torch.equal(x.view(torch.int16), z.view(torch.int16))
    pkv.check(pkv.pkv_rope_append(q[:0], k[:0], v[:0], pos[:0], f, slots[:0], a[0], a[1], a[2][:0]))


def test_slots_past_32_bits(pkv):
    """A pool whose rows lie past 2^31 elements: the last block's rows."""
    nb, K, H = 140000, 8, 128                                  # 140,000 x 16 x 1,024 elements: 2.3e9, 4.6 GB a pool
    kc = torch.zeros(nb, 16, K, H, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    c = Case(9, 3, 8, K, H, 128, False, pool=nb)
    slots = torch.tensor([nb * 16 - 1, nb * 16 - 16, 7], device="cuda")
    q, k, v, pos, f = c.dev()
    out = torch.empty_like(q)
    pkv.check(pkv.pkv_rope_append(q, k, v, pos, f, slots, kc, vc, out))
    got = torch.stack([kc.view(-1, K, H)[int(s)] for s in slots])
    near(R.bf16_values(bf16_host(got)), c.k_ref, pair_sums(R.bf16_values(c.k)), "k")
    assert torch.equal(torch.stack([vc.view(-1, K, H)[int(s)] for s in slots]), v)
    assert int((vc.view(torch.int16) != 0).any(-1).any(-1).sum()) == 3
