"""How exact attention over selected blocks is: its output carries its own rounding to bf16 and no rounding of the
softmax weights to 16 bits.

Queries pick one element of the keys and the softmax scale is 1, so logits are exact.  What is left: a weight enters the
product P V as a pair of 16-bit numbers (bf16: 2^-16 of it is lost; f16: 2^-22, or 2^-25 of the unit that the list's
largest V scale sets), exponentials and their arguments are off by less than 2^-20, the fp32 sums over up to 64 tokens by
64 2^-24 = 2^-18: 2^-15 of sum w |v| / l bounds them all, beside half a step of bf16, 2^-8 of the result."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ops_ref as R
from devutil import bf16_dev, i32_dev, out_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    from paged_kv_decode_slot_gb300.build import build_library
    build_library()
    import paged_kv_decode_slot_gb300 as pkv
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return pkv


CTX = [1, 2, 3, 5, 16, 17, 31, 40, 64]
E4M3 = R.e4m3_table()


class Case:
    """Lists of up to 64 tokens; every query is `unit` at one element, 0 elsewhere."""

    def __init__(self, seed, kv, N, K, H, unit=1.0):
        self.r = r = np.random.default_rng(seed)
        self.kv, self.N, self.K, self.H = kv, N, K, H
        self.tab, self.pool = R.tables(r, CTX)
        self.scale = 1.0
        q = np.zeros((len(CTX), N, H))
        q[np.arange(len(CTX))[:, None], np.arange(N)[None], r.integers(0, H, (len(CTX), N))] = unit
        self.q = R.to_bf16(q)
        shape = (self.pool, 16, K, H)
        if kv == "bf16":
            self.k, self.v = R.to_bf16(r.uniform(-3, 3, shape)), R.to_bf16(r.standard_normal(shape))
            self.scales = ()
        else:
            # codes of magnitude below 8, scales within a factor of eight of each other
            codes = lambda: (r.integers(0, 0x50, shape) | r.integers(0, 2, shape) << 7).astype(np.uint8)
            self.k, self.v = codes(), codes()
            by = (self.pool, K) if kv == "e4m3_block" else (K,)
            self.scales = tuple((2.0 ** r.uniform(-3, 0, by)).astype(np.float32) for _ in range(2))
        self.sel = np.full((len(CTX), K, 4), -1, dtype=np.int32)
        for b, c in enumerate(CTX):
            self.sel[b, :, :-(-c // 16)] = np.arange(-(-c // 16))

    def values(self):
        if self.kv == "bf16":
            return R.bf16_values(self.k), R.bf16_values(self.v)
        wide = lambda s: s.astype(np.float64)[:, None, :, None] if s.ndim == 2 else s.astype(np.float64)[:, None]
        return E4M3[self.k] * wide(self.scales[0]), E4M3[self.v] * wide(self.scales[1])

    def run(self, pkv, pb):
        q, out = bf16_dev(self.q), torch.full((len(CTX), self.N, self.H), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(len(CTX), self.N, device="cuda")
        parts = -(-4 // pb) if pb else 0
        ws = torch.zeros(pkv.pkv_splitk_workspace_bytes(len(CTX), self.N, self.H, parts), dtype=torch.uint8, device="cuda") if pb else None
        tail = (i32_dev(self.tab), i32_dev(CTX), torch.from_numpy(self.sel).cuda(), self.scale, out, lse, pb, parts, ws)
        if self.kv == "bf16":
            pkv.check(pkv.pkv_decode_attn_blocks(q, bf16_dev(self.k), bf16_dev(self.v), *tail))
        else:
            pkv.check(pkv.pkv_decode_attn_blocks_fp8(q, *(torch.from_numpy(x).cuda() for x in (self.k, self.v, *self.scales)), *tail))
        return out_f64(out), lse.double().cpu().numpy()


KINDS = [("bf16", 4, 2, 64), ("bf16", 8, 1, 128), ("bf16", 5, 5, 128), ("e4m3_head", 8, 2, 128), ("e4m3_block", 8, 1, 128),
         ("e4m3_block", 3, 3, 128)]


def check(c, out, lse):
    keys, values = c.values()
    ref, ref_lse, spread = R.blocks_attention(R.bf16_values(c.q), keys, values, c.tab, CTX, c.sel, c.scale)
    unit = 2.0 ** -25 * 64 * 8 * (c.scales[1].max() if c.scales else 0.0)
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -15 * spread + unit
    assert np.all(np.abs(out - ref) <= tol), f"{(np.abs(out - ref) / tol).max():.2f} of the bound"
    assert np.all(np.abs(lse - ref_lse) <= 2.0 ** -18 * (1 + np.abs(ref_lse)))


@pytest.mark.parametrize("pb", [0, 1, 2])
@pytest.mark.parametrize("kv,N,K,H", KINDS)
def test_output_is_off_by_its_own_rounding_alone(pkv, kv, N, K, H, pb):
    c = Case(N + H + pb, kv, N, K, H)
    check(c, *c.run(pkv, pb))


@pytest.mark.parametrize("pb", [0, 1])
@pytest.mark.parametrize("kv,N,K,H", KINDS)
def test_the_average_of_a_constant_is_that_constant(pkv, kv, N, K, H, pb):
    """Values that every token shares, of all 128 mantissas (e4m3: all its codes below NaN, times a power of two): an average
    that is off by 2^-15 of them rounds back to them."""
    c = Case(7 + N + H + pb, kv, N, K, H)
    if kv == "bf16":
        row = (c.r.integers(0, 2, (K, H)) << 15 | c.r.integers(110, 140, (K, H)) << 7 | np.resize(np.arange(128), (K, H))).astype(np.uint16)
        want = R.bf16_values(row)
    else:
        row = (np.resize(np.arange(0x7F), (K, H)) | c.r.integers(0, 2, (K, H)) << 7).astype(np.uint8)
        c.scales = (c.scales[0], np.full_like(c.scales[1], 2.0 ** -5))
        want = E4M3[row] * 2.0 ** -5
    c.v = np.broadcast_to(row, c.v.shape).copy()
    out, _ = c.run(pkv, pb)
    assert np.array_equal(out, np.broadcast_to(np.repeat(want, N // K, 0), out.shape))


@pytest.mark.parametrize("kv,power", [(kv, p) for kv in ("e4m3_head", "e4m3_block") for p in (-120, -100, -30, -14, 15, 16, 40, 100, 120)] +
                         [("bf16", p) for p in (-100, 16, 100)])
def test_queries_of_any_magnitude(pkv, kv, power):
    """Queries of 2^power under a softmax scale of 2^-power, whose logits are ordinary; and one head of a group whose logits are
    2^power times the others', which attends to its largest logits alone, or to all tokens alike (K scales are powers of
    two there: logits are equal, or apart by 2^-8 of themselves)."""
    c = Case(power + 200, kv, 8, 2, 128, unit=2.0 ** power)
    c.scale = 2.0 ** -power
    check(c, *c.run(pkv, 0))
    c = Case(power + 300, kv, 8, 2, 128)
    q = R.bf16_values(c.q)
    q[:, 3] *= 2.0 ** power
    c.q = R.to_bf16(q)
    if c.scales:
        c.scales = ((2.0 ** np.round(np.log2(c.scales[0]))).astype(np.float32), c.scales[1])
    check(c, *c.run(pkv, 2))
