"""Log probabilities and their gradient at the ends of the temperature's range
with masked logits, against the formulas in fp64 with the bounds of
test_gpu_logprob.py."""
import math

import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl
from test_gpu_logprob import check, forward64, grad64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8rl.load_library(build_if_missing=True)


def make(rows, vocab, dtype, spread, seed=0, pad=0, offset=0):
    """Rows with a third of their logits -inf; the tokens are not."""
    g = torch.Generator("cuda").manual_seed(seed)
    buf = torch.full((rows * (vocab + pad) + offset,), -math.inf, dtype=dtype, device="cuda")
    x = buf[offset:].as_strided((rows, vocab), (vocab + pad, 1), storage_offset=offset)
    x.copy_((torch.randn(rows, vocab, generator=g, device="cuda") * spread).to(dtype))
    x[torch.rand(rows, vocab, generator=g, device="cuda") < 1 / 3] = -math.inf
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda").int()
    x.scatter_(1, t.long()[:, None], 0.25 * spread)
    return x, t


LAYOUTS = [(0, 0), (3, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,offset", LAYOUTS)
@pytest.mark.parametrize("temperature", [1e20, 1e26, 1.4e27, 1.5e27, 5e27, 1e28, 1e30, 3e38])
@pytest.mark.parametrize("rows,vocab", [(3, 501), (4, 40001)])
def test_high_temperatures_keep_masked_logits_out(rows, vocab, temperature, pad, offset, dtype):
    for spread in (2.0, temperature / 8):
        x, t = make(rows, vocab, dtype, spread, seed=vocab, pad=pad, offset=offset)
        _, ent, stats = check(x, t, temperature=temperature, topk=5)
        if spread == 2.0:  # the type's lowest value beside them counts for what it is
            y = x.clone()
            y[:, 1::7] = torch.finfo(dtype).min
            y.scatter_(1, t.long()[:, None], 0.25 * spread)
            check(y, t, temperature=temperature)
        g = torch.full((rows,), temperature, device="cuda").clamp(max=1e30)
        got = fp8rl.logprobs_backward(x, t, stats, ent, g, g, temperature=temperature)
        d, tol = grad64(x, t, g, g, temperature)
        assert bool(((got.double() - d).abs() <= tol).all())
        assert bool((got[x == -math.inf] == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,offset", LAYOUTS)
@pytest.mark.parametrize("temperature", [1e-1, 1e-3, 1e-4, 1e-5, 2e-6, 1e-6])
@pytest.mark.parametrize("gh", [0.01, -1.0, 300.0, 1e6])
def test_gradient_of_masked_logits_at_low_temperatures(gh, temperature, pad, offset, dtype):
    """The entropy's gradient has a factor 1 / T beside exponents of its own 1 / T."""
    rows, vocab = 4, 5003
    for spread in (2.0, 3 * temperature):
        x, t = make(rows, vocab, dtype, spread, seed=5, pad=pad, offset=offset)
        _, ent, stats = check(x, t, temperature=temperature)
        g = torch.tensor([1.0, -0.5, 0.0, 2.0], device="cuda")
        gg = torch.full((rows,), gh, device="cuda")
        got = fp8rl.logprobs_backward(x, t, stats, ent, g, gg, temperature=temperature)
        d, tol = grad64(x, t, g, gg, temperature)
        # exponentials below 2^-126 are flushed: such an element is its value, or 0
        tol += torch.where(forward64(x, t, temperature)[1] < 2.0 ** -125, d.abs(), 0.0)
        assert not bool(got.isnan().any())
        assert bool(((got.double() - d).abs() <= tol).all())
        assert bool((got[x == -math.inf] == 0).all())
