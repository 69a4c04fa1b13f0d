"""Sampling from long rows of equal weights: the exact kernel's sums, and how it finds
a cut among them."""

import numpy as np
import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab,rows", [(151936, 512), (1 << 20, 480)])
def test_borders_between_long_runs_of_equal_weights(vocab, rows):
    """Rows of two values, each filling one half, and one heavier element; u beside the border between the halves (2^-38
    to both sides).  A thread adds up to `vocab` / 1024 equal pairs of numbers: roundings of one sign, which a running
    pair left as it is lets grow with the square of their number (n^2 2^-53 of the sum: 2^-38.6 and 2^-33).  The
    border is known to 2^-48 here (weights in 64 bits, counts exact), the draw's is to be within 2^-40 of the sum."""
    g = torch.Generator("cuda").manual_seed(vocab)
    half = vocab // 2
    a, b = (torch.rand(rows, generator=g, device="cuda") * 2 - 3 for _ in range(2))
    x = torch.empty(rows, vocab, device="cuda")
    x[:, :half], x[:, half:] = a[:, None], b[:, None]
    x[:, 0] = 0.0
    wa, wb = (np.exp(v.double().cpu().numpy()) for v in (a, b))
    ahead = (1 + (half - 1) * wa).astype(np.longdouble)
    share = (ahead / (ahead + (vocab - half) * wb)).astype(np.float64)
    side = np.where(np.arange(rows) % 2 == 0, -1, 1)
    u = share * (1 + side * 2.0 ** -38)
    # min-p cuts nothing off, but takes the rows through the cut's sums (a CTA each, so many pairs a thread)
    token, _, _, kept = fp8rl.sample(x, torch.tensor(u, device="cuda"), 1.0, 0, 1.0, 1e-6)
    assert (kept == vocab).all()
    assert int((token.cpu().numpy() != np.where(side < 0, half - 1, half)).sum()) == 0
