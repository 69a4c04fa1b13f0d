"""GPU parity of the packed causal attention against the formula in fp64.

Bounds, from the arithmetic: a score is d bf16 products added in fp32 on the
tensor cores (each addition within 2^-22 of the magnitudes in it):
eps = (2^-19 + 2^-21) sum|q k| scale, plus |s| 2^-22 for the exponent.  A
probability is rounded to bf16 (2^-8), so an output is within
(2^-8 + 2^-10 + 4 eps) sum p|v| of its value, plus bf16's own 2^-8; lse is
within 2 eps + 2^-19 + |lse| 2^-22 (the row's reference times the scale is
rounded, and added back, as one number)."""
import math

import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8rl.load_library(build_if_missing=True)


def make(lens, hq, hkv, d, seed=0, q_scale=1.5, tail=0):
    """Packed q, k, v as column ranges of one projection output; `tail` more
    tokens of no sequence behind them, NaN."""
    g = torch.Generator("cuda").manual_seed(seed)
    total = sum(lens) + tail
    x = torch.randn(total, (hq + 2 * hkv) * d, generator=g, device="cuda").bfloat16()
    x[:, :hq * d] *= q_scale
    if tail:
        x[sum(lens):] = math.nan
    q = x[:, :hq * d].view(total, hq, d)
    k = x[:, hq * d:(hq + hkv) * d].view(total, hkv, d)
    v = x[:, (hq + hkv) * d:].view(total, hkv, d)
    cu = torch.tensor([0] + [sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32, device="cuda")
    return q, k, v, cu


def compare(out, lse, q, k, v, start, n, scale=None):
    hq, d = q.shape[1:]
    group = hq // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
    for h in range(hq):
        qq, kk, vv = q[start:start + n, h].double(), k[start:start + n, h // group].double(), v[start:start + n, h // group].double()
        s = (qq @ kk.T * scale).masked_fill(later, -math.inf)
        size = (qq.abs() @ kk.abs().T * scale).masked_fill(later, 0.0)
        z = torch.logsumexp(s, 1)
        p = torch.exp(s - z[:, None])
        ref = p @ vv
        eps = (size * (2.0 ** -19 + 2.0 ** -21) + s.masked_fill(later, 0.0).abs() * 2.0 ** -22).amax(1)
        tol = (2.0 ** -8 + 2.0 ** -10 + 4 * eps)[:, None] * (p @ vv.abs()) + ref.abs() * 2.0 ** -8
        got = out[start:start + n, h].double()
        assert bool(((got - ref).abs() <= tol).all()), (h, ((got - ref).abs() / tol).max().item())
        lt = 2 * eps + 2.0 ** -19 + z.abs() * 2.0 ** -22 + s.masked_fill(later, 0.0).abs().amax(1) * 2.0 ** -22
        assert bool(((lse[start:start + n, h].double() - z).abs() <= lt).all())


def check(lens, hq, hkv, d, seed=0, scale=None, **more):
    q, k, v, cu = make(lens, hq, hkv, d, seed, **more)
    plan = fp8rl.attn_prefill_plan(cu, q.shape[0], hq, hkv)
    out, lse = fp8rl.attn_prefill(q, k, v, plan, softmax_scale=scale)
    assert fp8rl.fp8rl_sync_status() == 0
    start = 0
    for n in lens:
        if n:
            compare(out, lse, q, k, v, start, n, scale)
        start += n
    return q, k, v, plan, out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (8, 2), (32, 4), (6, 2), (12, 2), (5, 1), (36, 4), (16, 1), (64, 1), (256, 1)])
def test_heads(hq, hkv, d):
    check([300, 77, 1], hq, hkv, d, seed=hq + d)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 384, 385, 640, 1000])
def test_lengths(n):
    check([n], 8, 2, 128, seed=n)
    check([n], 2, 2, 128, seed=n)  # one head a tile: 128 positions
    check([n], 2, 2, 64, seed=n)


def test_packed():
    check([5, 0, 300, 1, 0, 128, 129, 64, 700, 31], 8, 2, 128, seed=1)
    check([0, 0], 8, 2, 128, seed=1, tail=1)
    check([3] * 500, 4, 1, 128, seed=2)
    check([200] * 40 + [1500], 16, 2, 64, seed=3)


@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (1, 1, 64), (8, 1, 128), (32, 8, 64)])
def test_many_short_prompts(hq, hkv, d):
    """Thousands of items of one or two key tiles: every ring of the kernel
    turns over many times with nothing to wait for in between.  Checked against
    the same prompts alone."""
    g = torch.Generator().manual_seed(hq)
    kinds = [int(x) for x in torch.randint(1, 200, (12,), generator=g)] + [1, 128, 129]
    order = [kinds[int(x)] for x in torch.randint(0, len(kinds), (3000,), generator=g)]
    q, k, v, cu = make(order, hq, hkv, d, seed=hq)
    plan = fp8rl.attn_prefill_plan(cu, q.shape[0], hq, hkv)
    outs = [fp8rl.attn_prefill(q, k, v, plan) for _ in range(5)]
    assert fp8rl.fp8rl_sync_status() == 0
    for o, z in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(z, outs[0][1])
    starts = cu.tolist()
    for b in range(0, 3000, 211):
        compare(*outs[0], q, k, v, starts[b], order[b])


def test_long_prompt():
    check([5001], 4, 1, 128, seed=4)
    check([4100], 2, 2, 64, seed=5)


def test_other_sequences_do_not_leak():
    """NaN and infinities in the neighbouring sequences and behind the last one."""
    lens = [100, 57, 131, 300]
    q, k, v, cu = make(lens, 8, 2, 128, seed=6, tail=50)
    for t in (q, k, v):
        t[100:157] = math.nan
        t[288:588:2] = math.inf
    plan = fp8rl.attn_prefill_plan(cu, q.shape[0], 8, 2)
    out, lse = fp8rl.attn_prefill(q, k, v, plan)
    assert fp8rl.fp8rl_sync_status() == 0
    compare(out, lse, q, k, v, 0, 100)
    compare(out, lse, q, k, v, 157, 131)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (2, 2, 128), (16, 2, 64), (2, 2, 64)])
@pytest.mark.parametrize("bad", [0, 1, 63, 64, 100, 127, 128, 200, 299])
def test_later_positions_do_not_leak(hq, hkv, d, bad):
    """A NaN or an infinity in v_j or k_j reaches no position before j; from j
    on the formula's own NaN or infinity appears."""
    n = 300
    q, k, v, cu = make([n], hq, hkv, d, seed=bad + 1)
    plan = fp8rl.attn_prefill_plan(cu, n, hq, hkv)
    for value in (math.nan, math.inf, -math.inf):
        vv = v.clone()
        vv[bad, 0, 3] = value
        out, lse = fp8rl.attn_prefill(q, k, vv, plan)
        assert fp8rl.fp8rl_sync_status() == 0
        clean = torch.where(torch.isfinite(vv), vv, 0.0)
        if bad:
            compare(out, lse, q, k, vv, 0, bad)
        group = hq // hkv
        hit = out[bad:, :group, 3].float()
        assert bool(torch.isnan(hit).all()) if math.isnan(value) else bool((~torch.isfinite(hit)).all())
        # every other column and the other KV heads are as without it
        want, want_lse = fp8rl.attn_prefill(q, k, clean, plan)
        keep = torch.ones(hq, d, dtype=torch.bool, device="cuda")
        keep[:group, 3] = False
        diff = (out.float() - want.float()).abs()[:, keep]
        assert bool((diff <= 2.0 ** -6 * want.float().abs()[:, keep] + 2.0 ** -6).all())
        assert torch.equal(lse, want_lse)
    kk = k.clone()
    kk[bad, hkv - 1, 5] = math.nan
    out, lse = fp8rl.attn_prefill(q, kk, v, plan)
    if bad:
        compare(out, lse, q, kk, v, 0, bad)
    assert bool(torch.isnan(out[bad:, hq - 1].float()).all()) and bool(torch.isnan(lse[bad:, hq - 1]).all())


def test_tokens_of_no_sequence_are_not_written():
    q, k, v, cu = make([100, 60], 8, 2, 128, seed=7, tail=33)
    plan = fp8rl.attn_prefill_plan(cu, q.shape[0], 8, 2)
    out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 3.0, device="cuda")
    fp8rl.attn_prefill(q, k, v, plan, out=(out, lse))
    assert fp8rl.fp8rl_sync_status() == 0
    assert bool((out[160:] == 3).all()) and bool((lse[160:] == 3).all())


def test_scores_that_grow_and_peak():
    """Keys in ascending and descending score order (the reference maximum
    moves, or never does), scores in the hundreds, and q = 0."""
    n, d = 900, 128
    q, k, v, cu = make([n], 2, 1, d, seed=8)
    q = torch.ones_like(q)
    ramp = torch.linspace(-3, 3, n, device="cuda").bfloat16()
    plan = fp8rl.attn_prefill_plan(cu, n, 2, 1)
    for r in (ramp, ramp.flip(0)):
        kk = r[:, None, None].expand(n, 1, d).contiguous()
        out, lse = fp8rl.attn_prefill(q, kk, v.contiguous(), plan)
        assert fp8rl.fp8rl_sync_status() == 0
        compare(out, lse, q, kk, v, 0, n)
    check([700], 4, 2, 128, seed=9, q_scale=40.0)
    check([700], 4, 2, 64, seed=9, q_scale=0.0)
    check([300], 4, 2, 128, seed=10, scale=1.0)


def test_clamped_ends_and_wrong_plan():
    q, k, v, cu = make([100, 60], 8, 2, 128, seed=11)
    want = fp8rl.attn_prefill(q, k, v, fp8rl.attn_prefill_plan(cu, 160, 8, 2))
    wild = torch.tensor([-5, 100, 1 << 30, 7], dtype=torch.int32, device="cuda")  # the last sequence ends before it starts
    got = fp8rl.attn_prefill(q, k, v, fp8rl.attn_prefill_plan(wild, 160, 8, 2))
    assert fp8rl.fp8rl_sync_status() == 0
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    with pytest.raises(ValueError, match="other sizes"):
        fp8rl.attn_prefill(q, k, v, fp8rl.attn_prefill_plan(cu, 160, 8, 4))
    # the same through the C entry point: nothing written, reported by the status
    plan = fp8rl.attn_prefill_plan(cu, 160, 8, 8)
    out = torch.zeros_like(want[0])
    big = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    big[:plan.data.numel()] = plan.data
    fp8rl.fp8rl_attn_prefill(q, q.stride(0), k, k.stride(0), v, v.stride(0), big, big.numel(), 2, 160, 8, 2, 128, 0.1, out, 1024, None)
    assert fp8rl.fp8rl_sync_status() == 7
    assert bool((out == 0).all())
    got = fp8rl.attn_prefill(q, k, v, fp8rl.attn_prefill_plan(cu, 160, 8, 2))
    assert fp8rl.fp8rl_sync_status() == 0 and torch.equal(want[0], got[0])


def test_offsets_past_32_bits():
    """Rows 2^22 elements apart: the last token starts past 2^31 elements."""
    n, ld = 530, 1 << 22
    q, k, v, cu = make([n], 8, 2, 128, seed=12)
    big = torch.empty(n * ld, dtype=torch.bfloat16, device="cuda")
    wide = big.as_strided((n, 12 * 128), (ld, 1))
    wide.copy_(torch.cat([t.reshape(n, -1) for t in (q, k, v)], 1))
    plan = fp8rl.attn_prefill_plan(cu, n, 8, 2)
    want = fp8rl.attn_prefill(q, k, v, plan)
    got = fp8rl.attn_prefill(wide[:, :1024].view(n, 8, 128), wide[:, 1024:1280].view(n, 2, 128), wide[:, 1280:].view(n, 2, 128), plan)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_same_bits_streams_and_graph():
    q, k, v, plan, out, lse = check([700, 20, 333], 32, 8, 128, seed=13)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        again = fp8rl.attn_prefill(q, k, v, plan)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    buf = (torch.empty_like(out), torch.empty_like(lse))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fp8rl.attn_prefill(q, k, v, plan, out=buf)
    for _ in range(3):
        buf[0].zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, buf[0]) and torch.equal(lse, buf[1])
    assert fp8rl.fp8rl_sync_status() == 0
