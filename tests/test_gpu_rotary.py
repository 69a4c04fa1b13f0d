"""Rotary positions against the formula in 64 bits.

The angle's sine and cosine are fp32 numbers off by at most 2^-22 (2^-25 of a half
turn from its conversion, times pi, and 2 ulp of sincospi); the rotation adds two
roundings of 2^-24 (|a| + |b|).  So before its rounding an output is within
2^-20 (|a| + |b|) of the formula's; bf16 adds 2^-8 of the value (half a step), an
E4M3 code 2^-4 of it, or half the smallest step, 2^-10 of the scale."""
import math

import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def ref(x, positions, inv, axis, interleaved, inverse=False):
    """(turned fp64, |a| + |b| per element)."""
    pos = positions.double().reshape(-1, positions.shape[-1])
    angle = pos[torch.tensor(axis, device=x.device, dtype=torch.long)].t() * torch.tensor(inv, dtype=torch.float64, device=x.device)
    if inverse:
        angle = -angle
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    n = len(inv)
    y, size = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    at = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., at[0]].double(), x[..., at[1]].double()
    y[..., at[0]], y[..., at[1]] = a * c - b * s, a * s + b * c
    size[..., at[0]] = size[..., at[1]] = a.abs() + b.abs()
    return y, size


def near(got, want, size):
    err = (got.double() - want).abs()
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -20 * size + 1e-39
    assert (err <= tol).all(), float((err - tol).max())


def qkv(tokens, hq, hkv, d, seed, pad=0):
    g = torch.Generator("cuda").manual_seed(seed)
    t = torch.randn(tokens, (hq + 2 * hkv) * d + pad, generator=g, device="cuda").bfloat16()
    q, k, v = t[:, :hq * d], t[:, hq * d:(hq + hkv) * d], t[:, (hq + hkv) * d:(hq + 2 * hkv) * d]
    return tuple(x.unflatten(1, (-1, d)) for x in (q, k, v))


def plan(d, part, axes, theta=10000.0):
    pairs = int(d * part) // 2
    inv = [theta ** (-i / max(1, pairs)) for i in range(pairs)]
    sections = [pairs - 2 * (pairs // 3), pairs // 3, pairs // 3] if axes == 3 else [pairs]
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    return fp8rl.rotary_freqs(2 * pairs, theta, sections), inv, axis


def positions_of(tokens, axes, far, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(0, far + 1, (axes, tokens), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("tokens,hq,hkv,d", [(1, 32, 8, 128), (2, 1, 1, 64), (37, 12, 2, 128), (1300, 16, 16, 64), (5000, 8, 2, 128),
                                             (9, 40, 4, 128), (3, 5, 3, 80), (7, 3, 1, 48), (5, 2, 1, 6), (4, 3, 2, 2), (6, 2, 1, 200),
                                             (4000, 3, 1, 96), (3, 2, 1, 1024)])
@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_against_the_formula(tokens, hq, hkv, d, axes, interleaved, inverse):
    q, k, _ = qkv(tokens, hq, hkv, d, tokens + d)
    freqs, inv, axis = plan(d, 1.0, axes)
    pos = positions_of(tokens, axes, 5000)
    got = fp8rl.rotary(q, k, pos, freqs, interleaved=interleaved, inverse=inverse)
    for x, y in zip((q, k), got):
        near(y, *ref(x, pos, inv, axis, interleaved, inverse))


@pytest.mark.parametrize("d,part", [(128, 0.5), (128, 0.25), (64, 0.5), (128, 0.125), (96, 0.5), (128, 0.0), (10, 0.8)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_part_of_the_head(d, part, interleaved):
    q, k, _ = qkv(19, 4, 2, d, 3)
    freqs, inv, axis = plan(d, part, 1)
    pos = positions_of(19, 1, 300)
    for x, y in zip((q, k), fp8rl.rotary(q, k, pos[0], freqs, interleaved=interleaved)):
        near(y, *ref(x, pos, inv, axis, interleaved))
        assert torch.equal(y[..., freqs.rotary_dim:], x[..., freqs.rotary_dim:])


@pytest.mark.parametrize("theta", [10000.0, 1e6])
def test_far_positions(theta):
    # angles of 10^9: fp32 would know nothing of them; negative positions turn the other way
    q, k, _ = qkv(64, 2, 1, 128, 4)
    freqs, inv, axis = plan(128, 1.0, 1, theta)
    pos = torch.cat([2 ** 31 - 1 - torch.arange(32, device="cuda"), -(2 ** 31) + torch.arange(16, device="cuda"), torch.arange(-8, 8, device="cuda")])
    pos = pos.to(torch.int32)[None]
    got = fp8rl.rotary(q, k, pos, freqs)
    # fp64 itself knows an angle of 2 * 10^9 to 2^-22
    for x, y in zip((q, k), got):
        want, size = ref(x, pos, inv, axis, False)
        near(y, want, 2 * size)


def test_given_frequencies_and_axes():
    q, k, _ = qkv(11, 2, 2, 16, 5)
    inv = [0.5, -0.25, 1e-3, 7.5, 0.0, 3.0, 100.0, 1e-9]
    axis = [0, 1, 2, 0, 1, 2, 0, 1]
    freqs = fp8rl.rotary_freqs(16, inv_freq=inv, axis=axis)
    assert freqs.axes == 3
    pos = positions_of(11, 3, 1000)
    for x, y in zip((q, k), fp8rl.rotary(q, k, pos, freqs)):
        near(y, *ref(x, pos, inv, axis, False))


@pytest.mark.parametrize("pad", [0, 8, 1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_strides(pad, interleaved):
    q, k, _ = qkv(33, 4, 2, 128, 6, pad)
    freqs, inv, axis = plan(128, 1.0, 1)
    pos = positions_of(33, 1, 40)
    want = fp8rl.rotary(q.contiguous(), k.contiguous(), pos, freqs, interleaved=interleaved)
    got = fp8rl.rotary(q, k, pos, freqs, interleaved=interleaved)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = fp8rl.rotary(q, k, pos, freqs, interleaved=interleaved, out=(q, k))
    assert got[0].data_ptr() == q.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip((q, k), want))
    wide = torch.empty(33, 1, 129, dtype=torch.bfloat16, device="cuda")[..., 1:]  # rows of odd alignment
    one = fp8rl.rotary(want[0][:, :1], None, pos, freqs, interleaved=interleaved, out=(wide, None))
    assert one[1] is None and torch.equal(wide, fp8rl.rotary(want[0][:, :1].contiguous(), None, pos, freqs, interleaved=interleaved)[0])


def test_no_tokens():
    q, k, v = qkv(0, 4, 2, 128, 1)
    freqs, _, _ = plan(128, 1.0, 1)
    pos = torch.empty(0, dtype=torch.int32, device="cuda")
    assert fp8rl.rotary(q, k, pos, freqs)[0].shape == (0, 4, 128)
    cache = torch.zeros(4, 256, dtype=torch.uint8, device="cuda")
    assert fp8rl.rotary_kv_append(q, k, v, pos, freqs, pos, cache, cache.clone(), torch.ones(2, device="cuda"))[0].shape == (0, 4, 128)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
def test_gradient(interleaved, axes):
    tokens, hq, hkv, d = 21, 3, 2, 32
    q, k, _ = qkv(tokens, hq, hkv, d, 7)
    freqs, inv, axis = plan(d, 0.75, axes)
    pos = positions_of(tokens, axes, 100)
    q, k = (x.detach().clone().requires_grad_() for x in (q, k))
    yq, yk = fp8rl.rotary(q, k, pos, freqs, interleaved=interleaved)
    g = torch.Generator("cuda").manual_seed(8)
    gq, gk = (torch.randn(y.shape, generator=g, device="cuda").bfloat16() for y in (yq, yk))
    torch.autograd.backward((yq, yk), (gq, gk))
    for x, gx in ((q, gq), (k, gk)):
        near(x.grad, *ref(gx, pos, inv, axis, interleaved, True))  # the formula's
        # differences of sum(g * turned x) in 64 bits (linear: exact but for fp64's rounding)
        x64 = x.detach().double()
        for _ in range(20):
            i = tuple(int(torch.randint(0, n, (1,), generator=torch.Generator().manual_seed(_ * 7 + n))) for n in x.shape)
            step = torch.zeros_like(x64)
            step[i] = 0.5
            up, dn = (float((gx.double() * ref(x64 + sign * step, pos, inv, axis, interleaved)[0]).sum()) for sign in (1, -1))
            _, size = ref(gx, pos, inv, axis, interleaved, True)
            assert abs(float(x.grad[i]) - (up - dn)) <= 2.0 ** -8 * abs(up - dn) + 2.0 ** -20 * float(size[i]) + 1e-9
    # one output alone, an expanded gradient
    q2 = q.detach().clone().requires_grad_()
    k2 = k.detach().clone().requires_grad_()
    _, yk = fp8rl.rotary(q2, k2, pos, freqs, interleaved=interleaved)
    yk.sum().backward()
    assert q2.grad is None or not q2.grad.any()
    near(k2.grad, *ref(torch.ones_like(k2), pos, inv, axis, interleaved, True))


def codes_near(cache, rows, want, size, scale):
    """E4M3 codes of `want` (fp64 [n, width]) in cache rows `rows`."""
    got = cache.view(E4M3)[rows].double() * scale
    exact = want.clamp(-448 * scale, 448 * scale)
    err = (got - exact).abs()
    tol = 2.0 ** -4 * exact.abs() + 2.0 ** -10 * scale + 2.0 ** -20 * size
    assert (err <= tol).all(), float((err - tol).max())


@pytest.mark.parametrize("tokens,hq,hkv,d", [(1, 32, 8, 128), (16, 32, 4, 128), (700, 12, 2, 64), (5000, 4, 2, 128), (9, 3, 1, 48), (7, 5, 3, 6)])
@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("keys", [False, True])
def test_append(tokens, hq, hkv, d, axes, interleaved, keys):
    q, k, v = qkv(tokens, hq, hkv, d, tokens + 1)
    freqs, inv, axis = plan(d, 1.0, axes)
    pos = positions_of(tokens, axes, 9000)
    slots = 2 * tokens + 5
    g = torch.Generator("cuda").manual_seed(tokens)
    at = torch.randperm(slots, generator=g, device="cuda")[:tokens].to(torch.int32)
    if tokens > 4:
        at[1], at[3] = -1, slots  # padding, and behind the cache
    caches = [torch.randint(0, 255, (slots, hkv * d), generator=g, device="cuda", dtype=torch.int64).to(torch.uint8) for _ in range(2)]
    before = [c.clone() for c in caches]
    scales = torch.tensor([5.3 / 448, 2.5 / 448], device="cuda")  # the values' saturates some
    yq, yk = fp8rl.rotary_kv_append(q, k, v, pos, freqs, at, *caches, scales, interleaved=interleaved, keys=keys)
    assert (yk is not None) == keys
    near(yq, *ref(q, pos, inv, axis, interleaved))
    want, size = ref(k, pos, inv, axis, interleaved)
    if keys:
        near(yk, want, size)
    on = (at >= 0) & (at < slots)
    rows = at[on].long()
    codes_near(caches[0], rows, want[on].flatten(1), size[on].flatten(1), float(scales[0]))
    # the values' codes are kv_append's
    k_ref, v_ref = (c.clone() for c in before)
    fp8rl.kv_append(k.flatten(1), v.flatten(1), at, k_ref, v_ref, scales)
    assert torch.equal(caches[1], v_ref)
    rest = torch.ones(slots, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert all(torch.equal(c[rest], b[rest]) for c, b in zip(caches, before))


def test_append_saturates_and_keeps_tiny_scales():
    q, k, v = qkv(4, 2, 2, 128, 2)
    freqs, inv, axis = plan(128, 1.0, 1)
    pos = positions_of(4, 1, 50)
    at = torch.arange(4, device="cuda", dtype=torch.int32)
    for scale in (1e-30, 1e-19, 1.0, 1e30):
        for size in (1.0, 1e30, 1e-30):
            caches = [torch.zeros(4, 256, dtype=torch.uint8, device="cuda") for _ in range(2)]
            scales = torch.full((2,), scale, device="cuda")
            x = (k.float() * size).bfloat16()
            fp8rl.rotary_kv_append(q, x, v, pos, freqs, at, *caches, scales)
            want, mag = ref(x, pos, inv, axis, False)
            codes_near(caches[0], at.long(), want.flatten(1), mag.flatten(1), float(scales[0]))


def test_append_has_no_backward_pass():
    q, k, v = qkv(4, 2, 1, 64, 2)
    freqs, _, _ = plan(64, 1.0, 1)
    pos = positions_of(4, 1, 50)
    caches = [torch.zeros(4, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    q = q.detach().clone().requires_grad_()
    y, _ = fp8rl.rotary_kv_append(q, k, v, pos, freqs, torch.arange(4, device="cuda", dtype=torch.int32), *caches, torch.ones(2, device="cuda"))
    with pytest.raises(RuntimeError, match="no backward pass"):
        y.sum().backward()


def test_streams_and_graphs():
    q, k, v = qkv(65, 8, 2, 128, 9)
    freqs, _, _ = plan(128, 1.0, 1)
    pos = positions_of(65, 1, 500)
    want = fp8rl.rotary(q, k, pos, freqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = fp8rl.rotary(q, k, pos, freqs, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = tuple(torch.zeros_like(t) for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fp8rl.rotary(q, k, pos, freqs, out=out)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_rows_far_into_memory():
    # element offsets past 2^31
    tokens, ld = 3, 1 << 30
    base = torch.empty(3 * ld, dtype=torch.bfloat16, device="cuda")
    q = base.as_strided((tokens, 2, 128), (ld, 128, 1))
    src, _, _ = qkv(tokens, 2, 1, 128, 1)
    q.copy_(src)
    freqs, inv, axis = plan(128, 1.0, 1)
    pos = positions_of(tokens, 1, 100)
    near(fp8rl.rotary(q, None, pos, freqs)[0], *ref(src, pos, inv, axis, False))


def test_gradient_of_strided_and_shared_inputs():
    # q and k are views of one projection: its gradient gathers both; a backward pass of a sum (an expanded gradient)
    tokens, d = 9, 64
    x = torch.randn(tokens, 5 * d, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16().requires_grad_()
    freqs, inv, axis = plan(d, 1.0, 1)
    pos = positions_of(tokens, 1, 100)
    h = x.view(tokens, 5, d)
    q, k = fp8rl.rotary(h[:, :3], h[:, 3:], pos, freqs)
    (q.sum() + 2 * k.sum()).backward()
    g = torch.ones(tokens, 5, d, dtype=torch.bfloat16, device="cuda")
    g[:, 3:] = 2
    near(x.grad.view(tokens, 5, d), *ref(g, pos, inv, axis, False, True))
    # back and forth: the rotation undoes itself but for two roundings to bf16
    back = fp8rl.rotary(q.detach(), None, pos, freqs, inverse=True)[0]
    assert ((back - h[:, :3]).abs().max() <= 2.0 ** -6 * h.abs().max()).item()


@pytest.mark.parametrize("d", [128, 6])  # the vector path, any layout
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_keeps_nan(d, interleaved):
    # a NaN in a pair makes both its elements NaN, in bf16 and as a code; what is infinite saturates
    q, k, v = (x.contiguous() for x in qkv(5, 2, 2, d, 3))
    freqs, inv, axis = plan(d, 1.0, 1)
    pos = positions_of(5, 1, 50) + 1
    k[1, 0, 0] = v[2, 1, 1] = float("nan")
    k[3, 1, 1], v[4, 0, 0] = float("inf"), -float("inf")
    at = torch.arange(5, device="cuda", dtype=torch.int32)
    caches = [torch.zeros(5, 2 * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    _, yk = fp8rl.rotary_kv_append(q, k, v, pos, freqs, at, *caches, torch.full((2,), 0.01, device="cuda"), interleaved=interleaved, keys=True)
    codes = caches[0].view(5, 2, d)
    want, _ = ref(k, pos, inv, axis, interleaved)
    assert torch.equal(yk.isnan(), want.isnan()) and int(want.isnan().sum()) == 2
    assert torch.equal((codes & 0x7F) == 0x7F, want.isnan())
    far = want.abs() == float("inf")
    assert int(far.sum()) == 2 and torch.equal(codes[far], torch.where(want[far] > 0, 0x7E, 0xFE).to(torch.uint8))
    k_ref, v_ref = (torch.zeros_like(c) for c in caches)
    fp8rl.kv_append(k.flatten(1), v.flatten(1), at, k_ref, v_ref, torch.full((2,), 0.01, device="cuda"))
    assert torch.equal(caches[1], v_ref)


def test_captured_backward_pass():
    tokens, hq, hkv, d = 40, 4, 2, 128
    freqs, _, _ = plan(d, 1.0, 1)
    pos = positions_of(tokens, 1, 500)
    q0, k0, _ = (x.contiguous() for x in qkv(tokens, hq, hkv, d, 1))
    gq, gk = (torch.randn_like(x) for x in (q0, k0))
    q, k = (torch.zeros_like(x).requires_grad_() for x in (q0, k0))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yq, yk = fp8rl.rotary(q, k, pos, freqs)
        grads = torch.autograd.grad((yq, yk), (q, k), (gq, gk))
    with torch.no_grad():
        q.copy_(q0), k.copy_(k0)
    for _ in range(2):
        graph.replay()
        want = fp8rl.rotary(q0, k0, pos, freqs)
        back = fp8rl.rotary(gq, gk, pos, freqs, inverse=True)
        assert all(torch.equal(x, y) for x, y in zip((yq, yk, *grads), (*want, *back)))
        gq.neg_()
