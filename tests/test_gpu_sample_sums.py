"""Sampling from long rows of equal weights: the exact kernel's sums, and how it finds
a cut among them."""
import math

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


def time_of(x, u, top_p):
    out = fp8rl.sample(x, u, 1.0, 0, top_p)
    best = math.inf
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        fp8rl.sample(x, u, 1.0, 0, top_p, out=out)
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best, out


def two_values(n, rows=1):
    """50 logits of 0, n of -10: each of the latter is 2^-0.83 / 16 = 7902 / 8192 of its bin's heaviest."""
    x = torch.full((rows, 50 + n), -10.0, device="cuda")
    x[:, 1000:1050] = 0.0
    return x


def test_a_cut_behind_more_elements_than_32_bits_of_mass_hold():
    # 543530 x 7902 is 2^32 and 4764 more: a bin that wraps looks empty, and the cut is then sought bin by bin (230 of
    # them, a pass each).  The tokens are the same either way; the time is not.
    u = torch.tensor([0.9], device="cuda", dtype=torch.float64)
    fits, _ = time_of(two_values(500000), u, 0.9)
    n = 543530
    took, (token, lp, lp_kept, kept) = time_of(two_values(n), u, 0.9)
    w = math.exp(-10.0)
    want = math.ceil((0.9 * (50 + n * w) - 50) / w)  # of the light ones, the lowest ids first
    assert abs(int(kept) - 50 - want) <= 1  # (top_p is fp32: 2^-25 of the mass is 0.04 of a token)
    goal, light = 0.9 * (50 + (int(kept) - 50) * w), (0.9 * (50 + (int(kept) - 50) * w) - 50) / w
    assert abs(int(token) - (50 + math.floor(light))) <= 1 and goal > 50
    assert took <= 4 * fits, (took, fits)


@pytest.mark.parametrize("vocab", [1 << 20, (1 << 21) + 77])
@pytest.mark.parametrize("top_p", [0.3, 0.95])
def test_flat_rows_of_millions(vocab, top_p):
    x = torch.full((2, vocab), 1.5, device="cuda")
    u = torch.tensor([0.25, 1 - 2.0 ** -53], device="cuda", dtype=torch.float64)
    token, _, lp_kept, kept = fp8rl.sample(x, u, 1.0, 0, top_p)
    p = torch.tensor(top_p).double().item()
    n = math.ceil(p * vocab)
    assert kept.tolist() == [n, n] and token.tolist() == [math.floor(0.25 * n), n - 1]
    assert (lp_kept + math.log(n)).abs().max() <= 2.0 ** -21 * math.log(n)
