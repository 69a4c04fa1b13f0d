"""GPU parity of the RMS norm with the residual's addition and the E4M3
output, against the same formula in fp64.

Bounds, from the arithmetic: a row's sum of squares is a sum of positive fp32
terms, at most 32 of them in sequence per thread and 15 levels of tree above
(relative error below 50 * 2^-24, halved by the square root); h = x + residual
rounds once (2^-24), rsqrtf is within 2 ulp (2^-22) and two products round
(2^-23): y is within DELTA = 2^-18 of its exact value with a factor of two to
spare.  Scales are amax / 448 of such y (one more rounding): within DELTA.  A
code is E4M3 of y / scale, so its value lies between the roundings of
v (1 - 2 DELTA) and v (1 + 2 DELTA), v the exact quotient.  A UE8M0 scale may
be the next power of two only where amax is within DELTA of the boundary."""
import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu
DELTA = 2.0 ** -18
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8rl.load_library(build_if_missing=True)


def rounded(v):
    """The E4M3 value nearest to v (fp64), saturating."""
    return v.clamp(-448, 448).float().to(E4M3).double()


def check(x, w, res, q, s, h, fmt, eps=1e-6):
    m, k = x.shape
    groups = -(-k // 128)
    hh = x.double() + (0 if res is None else res.double())
    y = hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + eps) * w.double()
    amax = torch.zeros(groups, m, dtype=torch.float64, device=x.device)
    for g in range(groups):
        amax[g] = y[:, 128 * g:128 * g + 128].abs().amax(1)
    if fmt == fp8rl.SCALE_FP32:
        sv = s.double()
        ref = torch.where(amax == 0, 1.0, amax / 448)
        assert bool(((sv - ref).abs() <= DELTA * ref).all())
    else:
        sv = torch.pow(2.0, s.double() - 127)
        for f, up in ((1 - DELTA, False), (1 + DELTA, True)):
            e = torch.where(amax == 0, 0.0, torch.ceil(torch.log2(amax * f / 448)).clamp(-127, 127))
            b = torch.pow(2.0, e)
            assert bool(((sv <= b) if up else (sv >= b)).all())
    per = sv.t().repeat_interleave(128, 1)[:, :k]
    v = y / per
    got = q.view(E4M3).double()
    lo, hi = rounded(v * (1 - 2 * DELTA)), rounded(v * (1 + 2 * DELTA))
    assert bool(((got >= torch.minimum(lo, hi)) & (got <= torch.maximum(lo, hi))).all())
    if res is not None:
        assert torch.equal(h, (x.float() + res.float()).bfloat16())


def inputs(m, k, seed=0, scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    channel = torch.exp(torch.randn(k, generator=g, device="cuda"))
    x = (torch.randn(m, k, generator=g, device="cuda") * channel * scale).bfloat16()
    res = (torch.randn(m, k, generator=g, device="cuda") * 3 * scale).bfloat16()
    w = (1 + 0.2 * torch.randn(k, generator=g, device="cuda")).bfloat16()
    return x, res, w


@pytest.mark.parametrize("fmt", [fp8rl.SCALE_FP32, fp8rl.SCALE_UE8M0])
@pytest.mark.parametrize("m,k", [(1, 1), (3, 5), (5, 127), (4, 128), (4, 129), (2, 1000), (1, 1024), (9, 1032), (6, 2048), (1, 4096),
                                 (17, 4096), (700, 4096), (7, 4100), (7, 5120), (3, 8192), (3, 8200), (2, 12288), (2, 16384),
                                 (2, 20001), (1, 32768)])
def test_norm_matches_fp64(m, k, fmt):
    x, res, w = inputs(m, k, seed=m + k)
    for r in (res, None):
        q, s, h = fp8rl.rmsnorm_quant(x, w, r, fmt=fmt)
        assert fp8rl.fp8rl_sync_status() == 0
        assert (h is None) == (r is None)
        check(x, w, r, q, s, h, fmt)


@pytest.mark.parametrize("off,pad", [(0, 8), (1, 8), (8, 3), (3, 5)])
def test_norm_strides_and_alignment(off, pad):
    """Column ranges of wider tensors: aligned and unaligned starts and strides."""
    m, k = 5, 1000
    x, res, w = inputs(m, k, seed=3)

    def place(t):
        big = torch.full((m, k + off + pad), 7.0, dtype=t.dtype, device="cuda")
        big[:, off:off + k] = t
        return big, big[:, off:off + k]

    _, xs = place(x)
    _, rs = place(res)
    hb, hs = place(torch.zeros_like(x))
    qb = torch.full((m, k + 16), 0x55, dtype=torch.uint8, device="cuda")
    qs = qb[:, :k]
    s = torch.empty(8, m, device="cuda")
    fp8rl.rmsnorm_quant(xs, w, rs, out=(qs, s, hs))
    assert fp8rl.fp8rl_sync_status() == 0
    check(x, w, res, qs, s, hs, fp8rl.SCALE_FP32)
    assert bool((qb[:, k:] == 0x55).all())
    assert bool((hb[:, :off] == 7).all()) and bool((hb[:, off + k:] == 7).all())


def test_norm_h_in_place_and_without_residual():
    x, res, w = inputs(33, 4096, seed=9)
    want = fp8rl.rmsnorm_quant(x, w, res)
    r2 = res.clone()
    got = fp8rl.rmsnorm_quant(x, w, r2, out=(torch.empty_like(want[0]), torch.empty_like(want[1]), r2))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    h = torch.zeros_like(x)  # h without a residual is x itself
    fp8rl.rmsnorm_quant(x, w, None, out=(torch.empty_like(want[0]), torch.empty_like(want[1]), h))
    assert torch.equal(h, x)


def test_norm_extreme_magnitudes():
    """Rows of zeros (scale 1, codes 0), tiny rows under eps, and rows near the
    top of bf16 whose squares still fit fp32."""
    for fmt in (fp8rl.SCALE_FP32, fp8rl.SCALE_UE8M0):
        for scale in (1e-18, 1e-6, 1e15):
            x, res, w = inputs(4, 512, seed=1, scale=scale)
            x[1] = 0
            res[1] = 0
            q, s, h = fp8rl.rmsnorm_quant(x, w, res, fmt=fmt)
            check(x, w, res, q, s, h, fmt)
            assert bool((q[1] == 0).all())


def test_norm_offsets_past_32_bits():
    """Rows 2^23 elements apart: the last one's offset is past 2^31 elements."""
    ld, m, k = 1 << 23, 300, 2048
    x0, res, w = inputs(m, k, seed=5)
    big = torch.empty(m * ld, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((m, k), (ld, 1))
    x.copy_(x0)
    q, s, h = fp8rl.rmsnorm_quant(x, w, res)
    check(x0, w, res, q, s, h, fp8rl.SCALE_FP32)


def test_norm_empty_and_another_stream():
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    q, s, h = fp8rl.rmsnorm_quant(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), w)
    assert q.shape == (0, 256) and s.shape == (2, 0)
    x, res, w = inputs(64, 4096, seed=2)
    want = fp8rl.rmsnorm_quant(x, w, res)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = fp8rl.rmsnorm_quant(x, w, res)
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_norm_chains_into_the_gemm():
    """Norm, then the W8A8 linear on its codes, captured in a graph: the
    result is the GEMM of exactly those codes, replay after replay."""
    x, res, w = inputs(16, 4096, seed=11)
    wq, sw = fp8rl.quant_weight(torch.randn(512, 4096, device="cuda").bfloat16())
    q, s, h = fp8rl.rmsnorm_quant(x, w, res)
    want = fp8rl.gemm(q, s, wq, sw)
    out = (torch.empty_like(q), torch.empty_like(s), torch.empty_like(h))
    y = torch.empty_like(want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        fp8rl.rmsnorm_quant(x, w, res, out=out)
        fp8rl.gemm(out[0], out[1], wq, sw, out=y)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fp8rl.rmsnorm_quant(x, w, res, out=out)
        fp8rl.gemm(out[0], out[1], wq, sw, out=y)
    for _ in range(3):
        y.zero_()
        out[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(out[0], q)
