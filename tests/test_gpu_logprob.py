"""GPU parity of the log probabilities, entropy, top alternatives and their
gradient against the formulas in fp64.

Bounds, from the arithmetic (fp32 throughout).  An exponent (x - m) log2e / T
carries three roundings, so e_j is within |y_j| 2^-22 + 2^-21 (the exponential)
of its value; a thread adds about vocab / 256 terms in sequence, the tree above
about 20: S is within tol_s = (vocab / 256 + 60) 2^-24 + 2^-21 + E|y| 2^-22.
lp adds |y_t| 2^-22 and its own rounding; the entropy's second sum doubles the
terms weighted by |y|.  A gradient is p (..) with p within tol_s + |y| 2^-21,
rounded once to the logits' type."""
import math

import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8rl.load_library(build_if_missing=True)


def make(rows, vocab, dtype, seed=0, spread=3.0, ld=None, offset=0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * spread).to(dtype)
    if ld or offset:
        ld = ld or vocab
        buf = torch.full((rows * ld + offset,), 50.0, dtype=dtype, device="cuda")  # a wrong read would dominate
        view = buf[offset:].as_strided((rows, vocab), (ld, 1), storage_offset=offset)
        view.copy_(x)
        x = view
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda").to(torch.int32)
    return x, t


def forward64(x, t, temperature):
    x = x.double()
    m = x.amax(1, keepdim=True)
    y = (x - m) / temperature
    e = torch.exp(y)
    s = e.sum(1, keepdim=True)
    lp = y - torch.log(s)
    p = e / s
    yy = torch.where(p > 0, y, 0.0)
    ent = -(p * torch.where(p > 0, lp, 0.0)).sum(1)
    return lp, p, ent, (p * yy.abs()).sum(1), torch.log(s[:, 0]), m[:, 0], y


def tol_s(vocab, ey):
    return (vocab / 256 + 60) * 2.0 ** -24 + 2.0 ** -21 + ey * 2.0 ** -22


def check(x, t, temperature=1.0, topk=0):
    lp, ent, stats, ids, top_lp = fp8rl.logprobs(x, t, temperature=temperature, topk=topk)
    assert fp8rl.fp8rl_sync_status() == 0
    rlp, p, rent, ey, ln_s, m, y = forward64(x, t, temperature)
    ts = tol_s(x.shape[1], ey)
    at = t.long()[:, None]
    yt = y.gather(1, at)[:, 0].abs()
    ref = rlp.gather(1, at)[:, 0]
    assert bool(((lp - ref).abs() <= ts + yt * 2.0 ** -22 + ref.abs() * 2.0 ** -23).all())
    assert bool(((ent - rent).abs() <= 2 * ts * (1 + ey) + rent * 2.0 ** -22).all())
    assert bool((stats[:, 0] == m).all())
    assert bool(((stats[:, 1] - ln_s).abs() <= ts + ln_s.abs() * 2.0 ** -23).all())
    if topk:
        order = torch.sort(x.double() + 0.0, dim=1, descending=True, stable=True).indices[:, :topk]
        assert torch.equal(ids.long(), order)
        r = rlp.gather(1, order)
        assert bool(((top_lp - r).abs() <= ts[:, None] + y.gather(1, order).abs() * 2.0 ** -22 + r.abs() * 2.0 ** -23).all())
    return lp, ent, stats


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,topk", [(1, 1, 1), (2, 7, 7), (3, 31, 5), (1, 255, 32), (5, 1000, 20), (3, 2049, 1), (700, 513, 3),
                                             (2, 32001, 20), (40, 50257, 5), (1, 151936, 32), (400, 32000, 20)])
def test_logprob_matches_fp64(rows, vocab, topk, dtype):
    x, t = make(rows, vocab, dtype, seed=vocab)
    check(x, t, topk=topk)
    check(x, t, topk=0)
    check(x, t, temperature=0.6, topk=topk)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset,pad", [(1, 0), (3, 1), (8, 5), (0, 9)])
def test_logprob_unaligned_rows(offset, pad, dtype):
    x, t = make(6, 4001, dtype, seed=offset, ld=4001 + pad, offset=offset)
    check(x, t, topk=17)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,pieces", [(400, 255), (400, 256), (400, 257), (400, 2048), (400, 2049), (30, 256), (30, 2047), (303, 1000), (608, 2100)])
def test_row_lengths_where_the_split_changes(rows, pieces, dtype):
    """Rows of so many 16-byte pieces, give or take an element."""
    n = 8 if dtype == torch.bfloat16 else 4
    for vocab in (pieces * n - 1, pieces * n, pieces * n + 1):
        x, t = make(rows, vocab, dtype, seed=vocab, ld=vocab + 3)
        check(x, t, topk=20)
        check(x, t)


@pytest.mark.parametrize("rows,vocab", [(3, 131), (400, 900), (400, 5000), (20, 40000)])
def test_top_of_values_that_differ_in_their_low_bits(rows, vocab):
    """fp32 logits that share their upper 16 bits: as many at the bound as elements;
    then a few dozen above the rest."""
    g = torch.Generator("cuda").manual_seed(vocab)
    x = 1.0 + torch.rand(rows, vocab, generator=g, device="cuda") * 2.0 ** -9
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda").int()
    check(x, t, topk=32)
    for extra in (30, 33, 63, 64, 65, 100):
        y = x.clone()
        at = torch.rand(rows, vocab, generator=g, device="cuda").argsort(1)[:, :extra]
        y.scatter_(1, at, 2.0 + torch.rand(rows, extra, generator=g, device="cuda") * 2.0 ** -9)
        check(y, t, topk=32)
        check(y.bfloat16(), t, topk=25)


@pytest.mark.parametrize("rows", [1, 30, 700])
def test_top_ties_go_to_the_lower_id(rows):
    """Few distinct values, constant rows, ascending and descending rows, and
    -0 beside 0: every thread's maximum ties."""
    vocab = 5000
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randint(-2, 3, (rows, vocab), generator=g, device="cuda").bfloat16()
    x[::3] = 1.5
    x[1::5] = torch.arange(vocab, device="cuda").bfloat16()
    x[2::7] = -torch.arange(vocab, device="cuda").bfloat16()
    x[:, ::2] = torch.where(x[:, ::2] == 0, -0.0, x[:, ::2])
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda").to(torch.int32)
    check(x, t, topk=32)
    check(x.float(), t, topk=32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_logits_and_rows(dtype):
    """-inf logits have probability 0; a row of them alone, rows of the type's
    lowest value, rows without a token, a single finite logit, and NaN or +inf
    in one row only."""
    vocab, rows = 3001, 9
    x, t = make(rows, vocab, dtype, seed=8)
    x[:, 1000:] = -math.inf
    t.clamp_(max=999)
    x[1] = -math.inf                                      # nothing left
    x[2] = torch.finfo(dtype).min                         # the lowest value everywhere: uniform
    t[3], t[4] = -1, vocab                                # padding
    x[5] = -math.inf
    x[5, 77], t[5] = 3.0, 77                              # one survivor
    x[6, 5] = math.nan
    x[7, 5] = math.inf
    t[0] = 2500                                           # a token that the mask excludes
    top = 8
    lp, ent, stats, ids, top_lp = fp8rl.logprobs(x, t, topk=top)
    gl, ge = torch.ones(rows, device="cuda"), torch.ones(rows, device="cuda")
    grad = fp8rl.logprobs_backward(x, t, stats, ent, gl, ge).double()
    assert fp8rl.fp8rl_sync_status() == 0
    assert lp[0] == -math.inf and math.isfinite(ent[0])
    assert lp[1] == -math.inf and ent[1] == 0 and bool((top_lp[1] == -math.inf).all())
    assert ids[1].tolist() == list(range(top)) and bool((grad[1] == 0).all())
    tol = tol_s(vocab, 0.0) + math.log(vocab) * 2.0 ** -22
    assert abs(lp[2].item() + math.log(vocab)) <= tol and abs(ent[2].item() - math.log(vocab)) <= 2 * tol
    assert ids[2].tolist() == list(range(top))
    for r in (3, 4):
        assert lp[r] == 0 and ent[r] == 0 and bool((stats[r] == 0).all()) and bool((grad[r] == 0).all())
        assert bool((ids[r] == -1).all()) and bool((top_lp[r] == 0).all())
    assert lp[5] == 0 and ent[5] == 0 and ids[5, 0] == 77 and ids[5, 1] == 0 and top_lp[5, 1] == -math.inf
    assert bool((grad[5] == 0).all())
    for r in (6, 7):
        assert math.isnan(lp[r]) and math.isnan(ent[r]) and bool(torch.isnan(grad[r]).all())
    # the neighbours are untouched by them
    ok = [8]
    check(x[8:9].clone(), t[8:9].clone(), topk=top)
    assert bool(torch.isfinite(grad[ok]).all()) and bool((grad[8, 1000:] == 0).all())


def grad64(x, t, g, gh, temperature):
    lp, p, ent, ey, _, _, y = forward64(x, t, temperature)
    pick = torch.zeros_like(p).scatter_(1, t.long()[:, None], 1.0)
    lpz = torch.where(p > 0, lp, 0.0)
    inner = g.double()[:, None] + gh.double()[:, None] * (lpz + ent[:, None])
    d = (g.double()[:, None] * pick - p * inner) / temperature
    size = p * (g.abs().double()[:, None] + gh.abs().double()[:, None] * (lpz.abs() + ent[:, None] + 1)) / temperature
    tol_p = 4 * tol_s(x.shape[1], ey)[:, None] + torch.where(p > 0, y, 0.0).abs() * 2.0 ** -20
    out = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -22
    tol = d.abs() * out + size * tol_p + pick * g.abs().double()[:, None] * 2.0 ** -21 / temperature + 1e-38
    return d, tol


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,temperature", [(1, 1, 1.0), (3, 37, 1.0), (5, 1000, 0.7), (2, 32001, 1.3), (300, 4096, 1.0),
                                                    (2, 151936, 1.0)])
def test_gradient_matches_formula(rows, vocab, temperature, dtype):
    x, t = make(rows, vocab, dtype, seed=rows)
    gen = torch.Generator("cuda").manual_seed(1)
    g, gh = torch.randn(rows, generator=gen, device="cuda"), torch.randn(rows, generator=gen, device="cuda")
    _, ent, stats, _, _ = fp8rl.logprobs(x, t, temperature=temperature)
    got = fp8rl.logprobs_backward(x, t, stats, ent, g, gh, temperature=temperature)
    d, tol = grad64(x, t, g, gh, temperature)
    assert bool(((got.double() - d).abs() <= tol).all())
    plain = fp8rl.logprobs_backward(x, t, stats, None, g, temperature=temperature)
    d, tol = grad64(x, t, g, torch.zeros_like(g), temperature)
    assert bool(((plain.double() - d).abs() <= tol).all())
    # in place, and into rows that start at another place of a 16-byte piece
    buf = torch.zeros(rows * (vocab + 3) + 1, dtype=dtype, device="cuda")
    other = buf[1:].as_strided((rows, vocab), (vocab + 3, 1), storage_offset=1)
    fp8rl.logprobs_backward(x, t, stats, ent, g, gh, temperature=temperature, out=other)
    assert torch.equal(other, got)
    y = x.clone()
    fp8rl.logprobs_backward(y, t, stats, ent, g, gh, temperature=temperature, out=y)
    assert torch.equal(y, got)
    assert fp8rl.fp8rl_sync_status() == 0


def test_gradient_matches_differences():
    """Central differences of the kernel's own forward pass, step 2^-6: the
    truncation error is h^2 / 6 times a third derivative below 1 (4e-5), the
    forward's rounding 2 * 2^-19 / 2^-5 (1.2e-4)."""
    rows, vocab, temperature, step = 2, 23, 1.0, 2.0 ** -6
    x, t = make(rows, vocab, torch.float32, seed=5, spread=1.0)
    g, gh = torch.tensor([0.7, -1.1], device="cuda"), torch.tensor([0.5, 0.3], device="cuda")

    def loss(z):
        lp, ent, _, _, _ = fp8rl.logprobs(z, t, temperature=temperature)
        return (g * lp + gh * ent).double()

    _, ent, stats, _, _ = fp8rl.logprobs(x, t, temperature=temperature)
    got = fp8rl.logprobs_backward(x, t, stats, ent, g, gh, temperature=temperature).double()
    for j in range(vocab):
        up, down = x.clone(), x.clone()
        up[:, j] += step
        down[:, j] -= step
        width = (up[:, j].double() - down[:, j].double())
        diff = (loss(up) - loss(down)) / width
        assert bool(((diff - got[:, j]).abs() <= 4e-4).all())


def test_offsets_past_32_bits_and_rows_past_one_grid():
    vocab, ld, rows = 1001, 1 << 21, 1100  # the last row starts past 2^31 elements
    x0, t = make(rows, vocab, torch.bfloat16, seed=2)
    big = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((rows, vocab), (ld, 1))
    x.copy_(x0)
    # (the rows start at other places of a 16-byte piece than x0's, so sums are in another order: bounds, not bits)
    _, ent, stats = check(x, t, topk=4)
    g = torch.ones(rows, device="cuda")
    d, tol = grad64(x0, t, g, g, 1.0)
    assert bool(((fp8rl.logprobs_backward(x, t, stats, ent, g, g).double() - d).abs() <= tol).all())
    x, t = make(70000, 33, torch.bfloat16, seed=3)
    check(x, t, topk=2)
    g = torch.ones(70000, device="cuda")
    _, ent, stats, _, _ = fp8rl.logprobs(x, t)
    d, tol = grad64(x, t, g, g, 1.0)
    assert bool(((fp8rl.logprobs_backward(x, t, stats, ent, g, g).double() - d).abs() <= tol).all())


def test_same_bits_on_every_run_and_stream():
    x, t = make(37, 50257, torch.bfloat16, seed=6)
    want = fp8rl.logprobs(x, t, topk=9)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = fp8rl.logprobs(x, t, topk=9)
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_empty_and_into_tis_weights():
    lp, ent, stats, ids, top_lp = fp8rl.logprobs(torch.empty(0, 100, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), topk=3)
    assert lp.shape == (0,) and ids.shape == (0, 3)
    x, t = make(64, 1000, torch.bfloat16, seed=1)
    lp, _, _, _, _ = fp8rl.logprobs(x, t)
    noisy, _, _, _, _ = fp8rl.logprobs((x.float() + 0.05).bfloat16(), t)
    w, kl = fp8rl.tis_weights(lp, noisy)
    assert bool(((w.double() - torch.exp((lp - noisy).double()).clamp(max=2.0)).abs() <= 1e-5).all())
