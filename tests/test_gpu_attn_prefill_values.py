"""Non-finite values in packed causal attention: a NaN or an infinity in v_j
reaches its own column of the rows that see position j and nothing else.  The
rest has the very bits of the same call with a zero in its place (the products
that it takes part in are the same), whatever the prompt's length."""
import math

import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8rl.load_library(build_if_missing=True)


def make(lens, hq, hkv, d, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    total = sum(lens)
    x = torch.randn(total, (hq + 2 * hkv) * d, generator=g, device="cuda").bfloat16()
    cu = torch.tensor([0] + [sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32, device="cuda")
    plan = fp8rl.attn_prefill_plan(cu, total, hq, hkv)
    return x[:, :hq * d].view(total, hq, d), x[:, hq * d:(hq + hkv) * d].view(total, hkv, d), x[:, (hq + hkv) * d:].view(total, hkv, d), plan


def check(lens, hq, hkv, d, at, seed=0):
    """at: (sequence, position, KV head, column, value) of each value put in."""
    q, k, v, plan = make(lens, hq, hkv, d, seed)
    v = v.contiguous()
    clean, bad = v.clone(), v.clone()
    group = hq // hkv
    want_special = torch.zeros(v.shape[0], hq, d, device="cuda")  # the terms that each output gets: 0, an infinity or NaN
    for b, pos, head, col, value in at:
        start = sum(lens[:b])
        clean[start + pos, head, col], bad[start + pos, head, col] = 0.0, value
        want_special[start + pos:start + lens[b], head * group:(head + 1) * group, col] += value
    want, want_lse = fp8rl.attn_prefill(q, k, clean, plan)
    assert fp8rl.fp8rl_sync_status() == 0
    for _ in range(3):
        out, lse = fp8rl.attn_prefill(q, k, bad, plan)
        assert fp8rl.fp8rl_sync_status() == 0
        ref = want.float() + want_special
        nan = ref.isnan()
        assert torch.equal(out.isnan(), nan)
        assert torch.equal(out.float()[~nan], ref[~nan])
        assert torch.equal(lse, want_lse)


HEADS = [(1, 1, 128), (3, 3, 64), (8, 2, 128), (16, 2, 64), (64, 1, 128), (256, 1, 64)]


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_values_in_every_kind_of_place(hq, hkv, d):
    """First and last positions of tiles and items; both infinities in one column
    (their sum is NaN from the second on); in several columns of one row."""
    inf, nan = math.inf, math.nan
    lens = [300, 1, 513, 77]
    last = hkv - 1
    check(lens, hq, hkv, d, [(0, 127, 0, 3, nan), (0, 130, 0, 5, inf), (0, 131, 0, 5, -inf), (0, 299, 0, d - 1, -inf), (1, 0, last, 0, inf),
                             (2, 255, last, 8, nan), (2, 256, last, 9, inf), (2, 512, last, 0, nan), (3, 0, 0, 1, -inf), (3, 76, 0, 1, inf)],
          seed=hq)


@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_second_tile_alone(hq, hkv, d):
    """In positions that only the second query tile of an item sees, many items."""
    span = 256 // next(p for p in (128, 64, 32, 16, 8, 4, 2, 1) if hq // hkv % p == 0)
    n = 1024 + span
    check([n], hq, hkv, d, [(0, p + span // 2 + p // span % (span - span // 2), p // span % hkv, p // span % d, math.nan)
                            for p in range(0, n, span)], seed=hq)


@pytest.mark.parametrize("hq,hkv,d,n", [(1, 1, 128, 70000), (2, 1, 64, 120001)])
def test_late_in_a_long_prompt(hq, hkv, d, n):
    """The waits of the kernel do not depend on how far back the prompt goes, and
    the other sequences of the call are whole."""
    check([200, n, 131, 513], hq, hkv, d, [(1, n - 1, 0, 3, math.nan), (1, n - 40, 0, 7, math.inf), (1, n - 300, 0, 9, -math.inf)], seed=n)


@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 128), (8, 2, 128), (4, 2, 64)])
def test_all_values_of_the_last_positions(hq, hkv, d):
    n, bad = 5000, 400
    q, k, v, plan = make([n], hq, hkv, d, seed=1)
    v = v.contiguous()
    v[n - bad:] = math.nan
    out, lse = fp8rl.attn_prefill(q, k, v, plan)
    assert fp8rl.fp8rl_sync_status() == 0
    v[n - bad:] = 0
    want, want_lse = fp8rl.attn_prefill(q, k, v, plan)
    assert torch.equal(out[:n - bad], want[:n - bad]) and torch.equal(lse, want_lse)
    assert bool(out[n - bad:].isnan().all())


@pytest.mark.parametrize("hq,hkv,d", HEADS)
@pytest.mark.parametrize("masked", [1, 127, 128, 129, 300])
def test_scores_of_minus_infinity(hq, hkv, d, masked):
    """Keys whose scores are -inf for every query have probability 0, whole key
    tiles of them at a prompt's start too; a row of them alone is NaN, as the
    formula's 0 / 0."""
    n = 500
    q, k, v, plan = make([n], hq, hkv, d, seed=masked)
    q, k = q.contiguous(), k.contiguous()
    q[:, :, 0] = q[:, :, 0].abs().clamp(min=0.25)
    k[:masked, :, 0] = -math.inf
    out, lse = fp8rl.attn_prefill(q, k, v, plan)
    assert fp8rl.fp8rl_sync_status() == 0
    assert bool(out[:masked].isnan().all())
    later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
    for h in range(0, hq, max(1, hq // 3)):
        kh = h // (hq // hkv)
        s = (q[:, h].double() @ k[:, kh].double().T * d ** -0.5).masked_fill(later, -math.inf)[masked:]
        assert bool((s[:, :masked] == -math.inf).all())
        z = torch.logsumexp(s, 1)
        p = torch.exp(s - z[:, None])
        ref = p @ v[:, kh].double()
        size = (q[masked:, h].double().abs() @ k[masked:, kh].double().abs().T * d ** -0.5).masked_fill(later[masked:, masked:], 0)
        eps = size.amax(1) * (2.0 ** -19 + 2.0 ** -21 + 2.0 ** -22)
        tol = (2.0 ** -8 + 2.0 ** -10 + 4 * eps)[:, None] * (p @ v[:, kh].double().abs()) + ref.abs() * 2.0 ** -8
        assert bool(((out[masked:, h].double() - ref).abs() <= tol).all())
        assert bool(((lse[masked:, h].double() - z).abs() <= 4 * eps + 2.0 ** -19 + z.abs() * 2.0 ** -22).all())
