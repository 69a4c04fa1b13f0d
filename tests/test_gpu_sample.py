"""Drawing tokens: against the definition in 64 bits, row by row.

Tokens and the numbers of kept ones have to be equal: weights and sums are known to
about 2^-43 of the sum, so that a draw among 10^5 borders falls between the two
calculations once in 10^7 rows.

lp is fp32 from x - m (one rounding), its quotient by T, ln of a sum of at least 1
(2 ulp) and their difference, of one sign: 2^-21 relative, and 2^-40 for the sums'
own error where S is near 1.  S itself may come from fp32 exponentials and sums of 32
of them, four roundings deep: 4 x 2^-24 of S, 2^-22 in ln S.  Each weight but the
largest (exactly 1) is off by at most 2^-22 (the exponential) + 2^-22 (the moves to a
larger maximum, which meet shrinking shares of S) + 2^-22 t (its exponent t in base
2: x - m, log2(e) / T and their product are rounded, 2^-24 each, and ln 2 of that is
2.1 x 2^-24 t), so ln S by at most 2^-21 (1 - 1 / S) + 2^-22 E[t].  The kept
mass of a row where something is cut off is exact to 2^-40."""
import math

import numpy as np
import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu

LAST_U = 1 - 2.0 ** -53


def ref_row(x, u, t, k, p, q):
    """(token, lp, lp_kept, kept, how far ln S may be off) of one row (fp64 tensor on the host)."""
    if not 0 <= u < 1 or not 0 <= t < math.inf or math.isnan(p) or math.isnan(q):
        return -1, 0.0, 0.0, 0, 0.0
    if torch.isnan(x).any() or (x == math.inf).any():
        return -1, math.nan, math.nan, 0, 0.0
    finite = int((x > -math.inf).sum())
    if finite == 0:
        return -1, -math.inf, -math.inf, 0, 0.0
    if t == 0:
        t, k = 1.0, 1
    if p <= 0:
        k = 1
    x = x + 0.0
    m = x.max()
    y = (x - m) / t
    w = torch.where(y > -100 * math.log(2), torch.exp(y), 0.0)
    order = torch.sort(x, descending=True, stable=True).indices[:finite]
    n = min(k, finite) if k > 0 else finite
    if 0 < p < 1:
        mass = torch.cumsum(w[order[:n]], 0)
        n = min(n, int((mass < p * mass[-1]).sum()) + 1)
    if q > 0:
        n = min(n, int((x[order] >= m + t * math.log(min(q, 1.0))).sum()))
    ids = torch.sort(order[:n]).values
    c = torch.cumsum(w[ids], 0)
    at = int((c <= u * c[-1]).sum())
    at = min(at, int((w[ids] > 0).nonzero().max()))
    j = ids[at]
    off = 2.0 ** -22 + 2.0 ** -21 * (1 - 1 / float(w.sum())) + 2.0 ** -22 * float((w * torch.where(w > 0, -y, 0)).sum() / w.sum()) / math.log(2)
    return int(j), float(y[j] - torch.log(w.sum())), float(y[j] - torch.log(c[-1])), n, off


def f32(v):
    return torch.tensor(v, dtype=torch.float32).item()


def check(logits, u, t=1.0, k=0, p=1.0, q=0.0, **more):
    rows = logits.shape[0]
    got = fp8rl.sample(logits, u, t, k, p, q, **more)
    token, lp, lp_kept, kept = (v.cpu() for v in got)
    cols = [v.tolist() if isinstance(v, torch.Tensor) else [v if n == 1 else f32(v)] * rows for n, v in enumerate((t, k, p, q))]
    x, us = logits.double().cpu(), u.tolist()
    for r in range(rows):
        want = ref_row(x[r], us[r], *(c[r] for c in cols))
        assert (int(token[r]), int(kept[r])) == (want[0], want[3]), (r, us[r], want, int(token[r]), int(kept[r]))
        off = want[4] if want[3] == int((x[r] > -math.inf).sum()) else 0.0
        for have, w, off in ((float(lp[r]), want[1], want[4]), (float(lp_kept[r]), want[2], off)):
            if math.isnan(w):
                assert math.isnan(have), r
            elif math.isinf(w):
                assert have == w, r
            else:
                assert abs(have - w) <= 2.0 ** -21 * abs(w) + 2.0 ** -40 + off, (r, have, w)
    return got


def make(rows, vocab, dtype, seed, pad=0, spread=2.5):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, vocab + pad, generator=g, device="cuda") * spread
    best = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    x[torch.arange(rows, device="cuda"), best] += 12 * torch.rand(rows, generator=g, device="cuda")
    return x.to(dtype)[:, :vocab], torch.rand(rows, generator=g, device="cuda", dtype=torch.float64)


DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 31, 33, 100, 255, 257, 1000, 4099, 32001])
@pytest.mark.parametrize("pad", [0, 3])
def test_nothing_cut_off(dtype, vocab, pad):
    check(*make(23, vocab, dtype, vocab + pad, pad))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k,p,q", [(1, 1.0, 0.0), (20, 1.0, 0.0), (300, 1.0, 0.0), (5000, 1.0, 0.0), (0, 0.95, 0.0), (0, 0.5, 0.0),
                                   (0, 0.9999, 0.0), (0, f32(1 - 2.0 ** -24), 0.0), (0, 1e-6, 0.0), (0, 1.0, 0.05), (0, 1.0, 1.0), (50, 0.9, 0.02),
                                   (2000, 0.99, 0.0), (40000, 0.3, 1e-4)])
@pytest.mark.parametrize("vocab", [3, 777, 32001])
def test_cuts(dtype, k, p, q, vocab):
    check(*make(9, vocab, dtype, vocab + k, 1), 0.8, k, p, q)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 16, 700])
def test_sizes_of_a_rollout(dtype, rows):
    # flat and sure rows; with 700 a CTA has a row to itself
    vocab = 151936 if rows < 100 else 4001
    x, u = make(rows, vocab, dtype, rows, spread=1.5)
    check(x, u, 1.0)
    check(x, u, 0.7, 50, 0.95, 0.01)
    check(x, u, 1.3, 0, 0.9, 0.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_parameters_of_each_row(dtype):
    rows = 64
    x, u = make(rows, 5003, dtype, 5)
    g = torch.Generator("cuda").manual_seed(6)
    t = torch.rand(rows, generator=g, device="cuda") * 1.5
    k = torch.randint(-1, 100, (rows,), generator=g, device="cuda", dtype=torch.int32)
    p = torch.rand(rows, generator=g, device="cuda") * 1.2
    q = torch.rand(rows, generator=g, device="cuda") * 0.2
    t[:8] = torch.tensor([0.0, 1e-6, 100.0, -1.0, math.nan, math.inf, 0.0, 1.0])
    k[8:12] = torch.tensor([0, -5, 1, 2 ** 31 - 1])
    p[12:18] = torch.tensor([0.0, -1.0, math.nan, 1.0, 7.0, 1e-30])
    q[18:23] = torch.tensor([0.0, -1.0, math.nan, 1.0, 7.0])
    u[23:28] = torch.tensor([0.0, LAST_U, -1.0, 1.0, math.nan], dtype=torch.float64)
    check(x, u, t, k, p, q)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_grid_of_numbers_meets_every_token_by_its_share(dtype):
    # one row of logits, drawn with u = (i + 1/2) / n: the tokens ascend, each as often as its probability says
    n, vocab = 2000, 50
    x, _ = make(1, vocab, dtype, 1)
    u = (torch.arange(n, device="cuda", dtype=torch.float64) + 0.5) / n
    x = x.repeat(n, 1)
    token, lp, _, kept = fp8rl.sample(x, u)
    token = token.long()
    assert (token[1:] >= token[:-1]).all() and (kept == vocab).all()
    share = torch.bincount(token, minlength=vocab).double() / n
    assert (share - torch.softmax(x[0].double(), 0)).abs().max() <= 1.0 / n
    lps, _, _, _, _ = fp8rl.logprobs(x, token.int())
    assert (lp - lps).abs().max() <= 2e-6


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [5, 1000, 20011])
def test_equal_logits_go_by_the_lower_index(dtype, vocab):
    rows = 12
    u = torch.rand(rows, device="cuda", dtype=torch.float64, generator=torch.Generator("cuda").manual_seed(vocab))
    x = torch.full((rows, vocab), 3.25, device="cuda", dtype=dtype)
    check(x, u)
    check(x, u, 1.0, max(1, vocab // 3))
    check(x, u, 1.0, 0, 0.5)
    check(x, u, 1.0, vocab // 2 + 1, 0.25, 1.0)
    # three values, zeros of both signs among them
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.tensor([-1.0, -0.0, 0.0, 2.0], device="cuda")[torch.randint(0, 3 if vocab < 1000 else 4, (rows, vocab), generator=g, device="cuda")].to(dtype)
    for k, p in ((0, 1.0), (vocab // 2, 1.0), (0, 0.4), (vocab // 2 + 1, 0.8), (2, 0.99)):
        check(x, u, 0.9, k, p)


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_logits(dtype):
    rows, vocab = 14, 3001
    x, u = make(rows, vocab, dtype, 3)
    u[0], u[1] = 0.0, LAST_U
    x = x.clone()
    x[:, :40] = -math.inf
    x[:, -40:] = -math.inf
    x[2] = -math.inf
    x[3] = -math.inf
    x[3, 77] = 1.0
    x[4, 50] = math.nan
    x[5, 60] = math.inf
    x[6] = torch.finfo(dtype).min
    x[7, ::2] = torch.finfo(dtype).min
    x[8] = math.inf
    x[9, 100:] = torch.finfo(dtype).min
    x[10, :] = torch.finfo(dtype).max
    x[10, 5:9] = torch.finfo(dtype).min
    x[11, 9] = 3e38
    x[12] = -3e38
    x[13] = 0.0
    for t, k, p, q in ((1.0, 0, 1.0, 0.0), (0.7, 30, 1.0, 0.0), (1.0, 2990, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 2000, 0.999, 1e-3),
                       (1e-30, 0, 1.0, 0.0), (1e30, 0, 0.5, 0.0)):
        check(x, u, t, k, p, q)


def test_values_that_differ_in_their_last_bits():
    # the histograms have to look closer, several times; subnormal logits too
    rows, vocab = 6, 9001
    g = torch.Generator("cuda").manual_seed(9)
    i = torch.randint(0, 4000, (rows, vocab), generator=g, device="cuda", dtype=torch.int32)
    x = (torch.tensor(17.0, device="cuda").view(torch.int32) + i).view(torch.float32)
    x[1] = i[1].view(torch.float32)             # subnormal
    x[2, ::2] = -x[2, ::2]
    x[3, ::3] = -40.0
    x[4] = x[4] * 1e30
    x[5] = i[5].float() * 1e-38
    u = torch.rand(rows, generator=g, device="cuda", dtype=torch.float64)
    for t, k, p in ((1.0, 0, 0.5), (1.0, 4000, 1.0), (1e-4, 0, 0.5), (1.0, 700, 0.9), (100.0, 8000, 0.999)):
        check(x, u, t, k, p)


def test_rows_of_other_strides_streams_and_outputs():
    x, u = make(5, 1000, torch.bfloat16, 8)
    wide = torch.zeros(5, 1311, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:1003] = x
    want = check(x, u, 0.9, 0, 0.9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = tuple(torch.empty_like(t) for t in want)
    got = fp8rl.sample(wide[:, 3:1003], u, 0.9, 0, 0.9, out=out, stream=side)
    side.synchronize()
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, out))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert fp8rl.sample(x[:0], u[:0])[0].shape == (0,)


def test_same_bits_captured_and_replayed():
    x, u = make(16, 32001, torch.bfloat16, 12)
    want = fp8rl.sample(x, u, 1.0, 50, 0.9, 0.01)
    out = tuple(torch.empty_like(t) for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8rl.sample(x, u, 1.0, 50, 0.9, 0.01, out=out)
    for _ in range(3):
        for t in out:
            t.fill_(-7)
        graph.replay()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_a_draw_has_no_gradient():
    x, u = make(4, 100, torch.float32, 2)
    x.requires_grad_()
    token, lp, lp_kept, kept = fp8rl.sample(x, u)
    assert not token.requires_grad and lp.requires_grad
    with pytest.raises(RuntimeError, match="no backward pass"):
        lp.sum().backward()


def test_a_row_far_into_memory():
    # element offsets past 2^31
    vocab, ld = 1000, 1 << 30
    x = torch.empty(3 * ld, dtype=torch.bfloat16, device="cuda")
    rows = x.as_strided((3, vocab), (ld, 1))
    src, u = make(3, vocab, torch.bfloat16, 4)
    rows.copy_(src)
    check(rows, u, 0.9, 0, 0.9)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_vocabulary_of_a_million(dtype):
    x, u = make(3, 1200007, dtype, 21, spread=1.5)
    for k, p in ((0, 1.0), (40, 1.0), (0, 0.9)):
        check(x, u, 1.0, k, p)


def test_more_rows_than_a_grid_has():
    rows, vocab = 70001, 8  # (rows of whole 16-byte pieces: the same bits wherever they lie)
    x, u = make(rows, vocab, torch.float32, 22)
    u[69000:69010] = -1
    token, lp, lp_kept, kept = fp8rl.sample(x, u, 1.0, 3)
    some = [0, 1, 65534, 65535, 65536, 68999, 69000, 69009, 69010, 70000]
    at = torch.tensor(some, device="cuda")
    want = fp8rl.sample(x[at].contiguous(), u[at], 1.0, 3)
    for a, b in zip((token, lp, lp_kept, kept), want):
        assert torch.equal(a[at], b)
    on = u >= 0
    assert ((token >= 0) == on).all() and (kept[on] == 3).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_tokens_alone(dtype):
    # the C call without its optional outputs
    x, u = make(40, 9001, dtype, 23, spread=1.0)
    for k, p in ((0, 1.0), (30, 0.9), (0, 0.9)):
        want = fp8rl.sample(x, u, 1.0, k, p)
        token = torch.full((40,), -9, dtype=torch.int32, device="cuda")
        fp8rl.fp8rl_sample(x, int(dtype == torch.float32), 40, 9001, x.stride(0), u, 1.0, k, p, 0.0, None, None, None, None, token, None,
                           None, None)
        assert torch.equal(token, want[0])


def test_two_streams_at_once():
    x, u = make(64, 32001, torch.bfloat16, 24)
    y, v = make(64, 32001, torch.float32, 25)
    want = fp8rl.sample(x, u, 1.0, 0, 0.9), fp8rl.sample(y, v)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        pair = []
        for s, (a, b, p) in zip(streams, ((x, u, 0.9), (y, v, 1.0))):
            with torch.cuda.stream(s):
                pair.append(fp8rl.sample(a, b, 1.0, 0, p))
        got.append(pair)
    torch.cuda.synchronize()
    for pair in got:
        for a, b in zip(pair, want):
            assert all(torch.equal(c, d) for c, d in zip(a, b))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,rows", [(151936, 24), (151936, 320), (151936, 1300), (4001, 320), (1500, 320)])
@pytest.mark.parametrize("t,k,p", [(1.0, 0, 1.0), (0.6, 0, 1.0), (1.0, 300, 0.9), (1.0, 0, 0.9)])
@pytest.mark.parametrize("spread", [1.0, 4.0])
def test_draws_next_to_a_border(dtype, vocab, rows, t, k, p, spread):
    """u beside borders between tokens, 2^-34 to 2^-19 to both sides: what fp32 sums cannot tell apart, can just tell,
    and can.  The borders are known to 2^-45 (extended sums of 64-bit weights).  The draws' weights are off by up to
    2^-41.6 each; a lane's sum of n pairs by n roundings, 2^-25 each, of a low part that n roundings have made
    (n 2^-50 of the sum as they come, n <= 150: 2^-42.8); u is held to 2^-48.  So a token may be the
    neighbour of the one it should be where u W lies within 2^-40 W of a border (of any: light tokens have many)."""
    x, _ = make(1, vocab, dtype, vocab + rows, spread=spread)
    rng = np.random.default_rng(vocab + rows)
    y = x[0].double().cpu().numpy()
    w = np.exp((y - y.max()) / f32(t)).astype(np.longdouble)
    order = np.argsort(-y, kind="stable")
    order = order[:k] if k else order
    mass = np.cumsum(w[order])
    order = order[:int(np.searchsorted(mass, f32(p) * mass[-1])) + 1] if p < 1 else order
    kept = np.zeros(vocab, dtype=bool)
    kept[order] = True
    upto = np.cumsum(np.where(kept, w, 0))
    # borders of any token, and of tokens as they are drawn
    at = np.concatenate([rng.choice(order, rows // 2), np.searchsorted(upto, rng.random(rows - rows // 2) * upto[-1], side="right")])
    off = np.array([s * 2.0 ** -e for e in (34, 30, 27, 25, 23, 22, 21, 20, 19) for s in (-1, 1)])
    u = np.clip((upto[at] / upto[-1]).astype(np.float64) + off[np.arange(rows) % len(off)], 0.0, LAST_U)
    want = np.searchsorted(upto, u.astype(np.longdouble) * upto[-1], side="right")
    token, _, _, n = fp8rl.sample(x.repeat(rows, 1), torch.tensor(u, device="cuda"), t, k, p)
    assert (n == len(order)).all()
    token, goal, near = token.cpu().numpy(), u.astype(np.longdouble) * upto[-1], np.longdouble(2.0) ** -40 * upto[-1]
    ahead = np.concatenate([np.zeros(1, dtype=upto.dtype), upto])[token]
    assert kept[token].all() and (ahead <= goal + near).all() and (goal - near <= upto[token]).all()
    assert (token == want).mean() >= 0.99
