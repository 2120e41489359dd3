"""Special cases of latent attention whose results are known to the bit.

Equal values.  Where all tokens of a sequence have the same latent vector v, softmax weights summing to one give out = v whatever
the logits, which the rotary keys alone set.  The weights enter the product rounded to bf16, so they have to be normalised by the
sum of the rounded ones.  Then out / v is the ratio of two fp32 sums of the same n positive terms, each off by at most 2^-23 a
term (rounded or cut off), and a few products of a join: below 2^-9 for n < 10,000, the least half step of a bf16 number, so that
the result is v itself."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import ops_ref as R
from devutil import bf16_dev, bf16_host
from test_gpu_latent import Case, pkv, same  # noqa: F401

pytestmark = pytest.mark.gpu


class EqualValues(Case):
    """One latent vector a sequence; rotary keys of growing size, some tokens far above all before them."""

    def __init__(self, seed, ctx, N, T=1):
        super().__init__(seed, ctx, N, T)
        r, B = self.r, len(ctx)
        self.v = R.to_bf16(r.standard_normal((B, 512)) * 2.0 ** r.integers(-3, 4, (B, 1)))
        rows = R.bf16_values(self.cache)
        for b, n in enumerate(ctx):
            size = np.linspace(0.3, 4.0, n) * np.where(r.random(n) < 0.01, 8.0, 1.0)
            if n > 300:
                size[n // 2] = size[n - 2] = 40.0           # some rows' one token that counts, behind their first tile
            for j in range(-(-n // 16)):
                k = min(16, n - 16 * j)
                rows[self.tab[b, j], :k, 512:] *= size[16 * j:16 * j + k, None]
        self.cache = R.to_bf16(rows)
        for b, n in enumerate(ctx):
            for j in range(-(-n // 16)):
                self.cache[self.tab[b, j], :min(16, n - 16 * j), :512] = self.v[b]
        q = R.bf16_values(self.q)
        q[..., :512] = 0                                    # (their logits would be one number for all tokens)
        self.q = R.to_bf16(q)
        self.poison()


@pytest.mark.parametrize("N,T", [(1, 1), (16, 1), (5, 3), (20, 1), (32, 1), (11, 3), (40, 1), (64, 1), (128, 1), (65, 3)])
@pytest.mark.parametrize("ctx", [[1, 16, 47, 49, 128, 130, 257, 700, 1000], [9000, 5, 0, 333], [3000]], ids=str)
def test_equal_values_come_back(pkv, N, T, ctx):  # noqa: F811
    c = EqualValues(N + T, ctx, N, T)
    out, lse = c.run(pkv)
    got = bf16_host(out)
    for b, n in enumerate(ctx):
        for t in range(T):
            want = c.v[b] if n - T + t >= 0 else np.zeros(512, dtype=np.uint16)
            wrong = (got[b, t] != want).any(-1)
            assert not wrong.any(), f"sequence {b} of {n} tokens, token {t}: heads {np.flatnonzero(wrong).tolist()} differ"
    c.check(out, lse)


@pytest.mark.parametrize("N", [16, 32, 128])
@pytest.mark.parametrize("above", [3, 7, 11, 30])
def test_a_token_that_outweighs_the_reference(pkv, N, above):  # noqa: F811
    """A token 2^above 1.0039 times the reference that the first tile set: its weight lies between two bf16 numbers, and next to
    nothing else counts.  (So many sequences that most are one CTA's alone: a part that began at the token would weigh it 1.)"""
    c = Case(3, [400, 390] * 100, N)
    q, rows = np.zeros(c.q.shape), np.zeros(c.cache.shape)
    q[..., 512:514] = 1.0
    v = R.bf16_values(R.to_bf16(c.r.standard_normal((200, 512))))
    for b, n in enumerate(c.ctx):
        at = rows.reshape(-1, 576)
        slots = c.tab[b, np.arange(n) // 16] * 16 + np.arange(n) % 16
        at[slots, :512], at[slots, 512] = v[b], -20.0
        at[slots[0], 512], at[slots[300], 512], at[slots[300], 513] = 0.0, above, 0.0056
    c.q, c.cache, c.scale = R.to_bf16(q), R.to_bf16(rows), float(np.log(2.0))
    c.poison()
    out, lse = c.run(pkv)
    assert same(out, bf16_dev(R.to_bf16(v))[:, None, None].expand(200, 1, N, 512))
    c.check(out, lse)
