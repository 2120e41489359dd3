"""Latent attention at the borders of how its work is dealt out: batches that each warp deals out for itself and larger ones
(whose sums lie in shared memory where the first loads then land), on both sides of a thread a sequence; the most rows that
one CTA takes alone, and the first that a pair of CTAs shares."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from test_gpu_latent import CTX, Case, pkv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [16, 32, 40])
@pytest.mark.parametrize("B", [127, 128, 129, 352, 353, 385])
def test_batches_around_the_borders_of_the_deal(pkv, B, N):  # noqa: F811
    c = Case(B + N, np.random.default_rng(B).integers(0, 150, B), N).poison()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = c.run(pkv, err=err)
    c.check(*first)
    for _ in range(20):
        again = c.run(pkv, err=err)
        assert torch.equal(first[0].view(torch.int16), again[0].view(torch.int16)) and torch.equal(first[1], again[1])
    assert int(err) == 0


@pytest.mark.parametrize("N,T", [(15, 1), (16, 1), (17, 1), (31, 1), (8, 4), (16, 2), (32, 1), (33, 1), (11, 3), (17, 2)])
def test_rows_around_the_widths_of_a_cta(pkv, N, T):  # noqa: F811
    for ctx in (CTX, [9000, 70, 0, 3333]):
        c = Case(N, ctx, N, T).poison()
        c.check(*c.run(pkv))
