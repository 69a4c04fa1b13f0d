"""The helpers under torch's autograd: log probabilities and entropy carry their
gradient, what has no backward pass says so, and calls without gradients are as
they are."""
import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8rl.load_library(build_if_missing=True)


def make(rows=37, vocab=2001, dtype=torch.float32):
    g = torch.Generator("cuda").manual_seed(rows)
    x = torch.randn(rows, vocab, generator=g, device="cuda").to(dtype).requires_grad_()
    t = torch.randint(-1, vocab, (rows,), generator=g, device="cuda").int()
    return x, t, torch.randn(rows, generator=g, device="cuda"), torch.randn(rows, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("use", ["both", "lp", "entropy", "sum"])
@pytest.mark.parametrize("with_out", [False, True])
def test_logprobs_gradient(use, dtype, with_out):
    x, t, g, gh = make(dtype=dtype)
    rows = len(t)
    out = (torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")) if with_out else None
    lp, entropy, stats, ids, top_lp = fp8rl.logprobs(x, t, temperature=0.7, out=out)
    with torch.no_grad():
        want = fp8rl.logprobs(x, t, temperature=0.7)
    assert not any(w.requires_grad for w in want if w is not None)
    assert all(torch.equal(a, b) for a, b in zip((lp, entropy, stats), want[:3])) and ids is None and top_lp is None
    one = torch.ones_like(g)
    loss, a, b = {"both": ((g * lp + gh * entropy).sum(), g, gh), "lp": ((g * lp).sum(), g, None),
                  "entropy": ((gh * entropy).sum(), torch.zeros_like(g), gh), "sum": (lp.sum() + entropy.sum(), one, one)}[use]
    loss.backward()
    assert torch.equal(x.grad, fp8rl.logprobs_backward(x.detach(), t, want[2], want[1], a, b, temperature=0.7))
    # and the formula's, in fp64 (the terms of a gradient are within about 2^-16 of themselves)
    z = x.detach().double().requires_grad_()
    lsm = torch.log_softmax(z / 0.7, 1)
    on = t >= 0
    ref = torch.where(on, a.double() * lsm.gather(1, t.clamp(min=0).long()[:, None])[:, 0], 0)
    if b is not None:
        ref = ref - torch.where(on, b.double() * (lsm.exp() * lsm).sum(1), 0)
    ref.sum().backward()
    size = (a.abs() + (0 if b is None else 20 * b.abs()))[:, None] / 0.7
    p = lsm.detach().exp() + torch.zeros_like(z).scatter_(1, t.clamp(min=0).long()[:, None], 1.0)
    out_eps = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -22
    assert bool(((x.grad.double() - z.grad).abs() <= z.grad.abs() * out_eps + size * p * 2.0 ** -15).all())
    assert fp8rl.fp8rl_sync_status() == 0


def test_logprobs_of_a_product():
    """Through torch's own operators in front of it, and from alternatives without one."""
    g = torch.Generator("cuda").manual_seed(1)
    h, w = (torch.randn(n, 64, generator=g, device="cuda").requires_grad_() for n in (20, 500))
    t = torch.randint(0, 500, (20,), generator=g, device="cuda").int()
    lp, entropy, stats, ids, top_lp = fp8rl.logprobs(h @ w.T, t, topk=3)
    assert lp.requires_grad and entropy.requires_grad and not ids.requires_grad
    (lp.mean() + 0.1 * entropy.mean()).backward()
    ref = torch.autograd.grad((lambda l: l.gather(1, t.long()[:, None]).mean() - 0.1 * (l.exp() * l).sum(1).mean())
                              (torch.log_softmax(h.double() @ w.double().T, 1)), (h, w))
    for a, b in zip((h.grad, w.grad), ref):
        assert float((a - b).norm() / b.norm()) < 2.0 ** -10
    for i in (2, 4):
        with pytest.raises(RuntimeError, match="not from stats or top_lp"):
            fp8rl.logprobs(h @ w.T, t, topk=3)[i].sum().backward()


def test_no_backward_pass_is_an_error():
    q = torch.randn(30, 4, 64, device="cuda").bfloat16().requires_grad_()
    k, v = (torch.randn(30, 2, 64, device="cuda").bfloat16().requires_grad_() for _ in range(2))
    plan = fp8rl.attn_prefill_plan(torch.tensor([0, 30], dtype=torch.int32, device="cuda"), 30, 4, 2)
    cache = torch.zeros(32, 128, dtype=torch.uint8, device="cuda")
    table = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    ln, sc = torch.tensor([30], dtype=torch.int32, device="cuda"), torch.ones(2, device="cuda")
    x, r = (torch.randn(5, 256, device="cuda").bfloat16().requires_grad_() for _ in range(2))
    w = torch.ones(256, device="cuda").bfloat16()
    for call in (lambda: fp8rl.attn_prefill(q, k, v, plan), lambda: fp8rl.attn_prefill(q.detach(), k.detach(), v, plan),
                 lambda: fp8rl.attn_decode(q[:1], cache, cache, table, ln, sc, 16), lambda: fp8rl.rmsnorm_quant(x, w, r.detach())[2:],
                 lambda: fp8rl.rmsnorm_quant(x.detach(), w, r)[2:]):
        got = call()
        with torch.no_grad():
            want = call()
        for a, b in zip(got, want):
            assert torch.equal(a.detach(), b) and not b.requires_grad
            with pytest.raises(RuntimeError, match="has no backward pass"):
                a.float().sum().backward(retain_graph=True)
    out, lse = fp8rl.attn_prefill(q.detach(), k.detach(), v.detach(), plan)
    assert not out.requires_grad and not lse.requires_grad
    assert fp8rl.fp8rl_sync_status() == 0
