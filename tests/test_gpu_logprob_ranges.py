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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("temperature", [1e-39, 2.5e-39, 4e-39, 8e-39])
def test_temperatures_whose_inverse_overflows(temperature, dtype):
    """The largest logits share the probability, the others have none."""
    x = torch.full((3, 1001), -1.0, dtype=dtype, device="cuda")
    x[:, 500:] = -math.inf
    x[0, 7], x[1, 100:104], x[2, ::100] = 2.0, 0.0, 1.0
    most = torch.tensor([1.0, 4.0, 11.0], device="cuda", dtype=torch.float64)
    t = torch.tensor([7, 103, 900], dtype=torch.int32, device="cuda")
    lp, ent, stats, ids, top_lp = fp8rl.logprobs(x, t, temperature=temperature, topk=2)
    assert fp8rl.fp8rl_sync_status() == 0
    assert bool(((lp.double() + most.log()).abs() <= 2.0 ** -21).all()) and bool(((ent.double() - most.log()).abs() <= 2.0 ** -21).all())
    assert ids.tolist() == [[7, 0], [100, 101], [0, 100]] and top_lp[0].tolist() == [0.0, -math.inf]
    # g / T within fp32 (about 1e33); with no gradient for the entropy: its factor log p is that of the shares alone
    g = torch.tensor([1.0, 0.0, 1.0], device="cuda") * 1e33 * torch.tensor(temperature, dtype=torch.float64).item()
    got = fp8rl.logprobs_backward(x, t, stats, ent, g, g, temperature=temperature).double()
    p = (x == x.amax(1, keepdim=True)).double() / most[:, None]
    pick = torch.zeros_like(p).scatter_(1, t.long()[:, None], 1.0)
    want = g.double()[:, None] * (pick - p) / torch.tensor(temperature, dtype=torch.float32).double().item()
    # the entropy's own gradient is 0 in exact arithmetic: -p (log p + H) with equal shares
    size = g.double()[:, None] / torch.tensor(temperature, dtype=torch.float32).double().item()
    out = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -20
    assert bool(((got - want).abs() <= want.abs() * out + size * p * 2.0 ** -17 + size * pick * 2.0 ** -17).all())
