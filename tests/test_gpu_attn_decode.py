"""GPU parity of the attention over the paged E4M3 cache against the formula
in fp64 on the dequantised cache.

Bounds, from the arithmetic: codes enter exactly, q loses nothing above 2^-14
of its largest element and 2^-25 of it below; the d products of a score are
added in fp32 on the tensor cores (each addition within 2^-22 of the
magnitudes in it): eps = (2^-19 + 2^-21) sum|q k| scale, plus |s| 2^-22 for the exponent.
p is rounded to f16 (2^-11, or 2^-24 of the row's reference below its normal
range, which lags the maximum by at most 2^8): an output is within
(2^-10 + 4 eps) sum p|v| of its value, plus n 2^-24 max|v| for the tiny p and
bf16's 2^-8."""
import math

import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8rl.load_library(build_if_missing=True)


def make(lens, hq, hkv, d, page, seed=0, spare=3, ld_pad=0, q_scale=1.5, width=None):
    g = torch.Generator("cuda").manual_seed(seed)
    batch = len(lens)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    width = width or max(1, max(need, default=1))
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    caches = []
    for _ in range(2):
        wide = torch.full((pages * page, hkv * d + ld_pad), 0x7F, dtype=torch.uint8, device="cuda")  # NaN codes around
        x = (torch.randn(pages * page, hkv * d, generator=g, device="cuda") * 80).clamp(-448, 448)
        wide[:, :hkv * d] = x.to(E4M3).view(torch.uint8)
        caches.append(wide[:, :hkv * d])
    # cache rows that no sequence holds are NaN: nothing may read them into a sum
    held = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        if n:
            rows = (table[b, :need[b]].long()[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]
            held[rows] = True
    for c in caches:
        c[~held] = 0x7F
    q = (torch.randn(batch, hq, d, generator=g, device="cuda") * q_scale).bfloat16()
    scales = torch.tensor([0.0121, 0.0117], device="cuda")
    return q, caches[0], caches[1], table, torch.tensor(lens, dtype=torch.int32, device="cuda"), scales


def reference(q, kc, vc, table, lens, scales, page, scale=None, skip=None):
    batch, hq, d = q.shape
    hkv = kc.shape[1] // d
    scale = d ** -0.5 if scale is None else scale
    out = torch.zeros(batch, hq, d, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    lse = torch.full((batch, hq), -math.inf, dtype=torch.float64, device="cuda")
    lse_tol = torch.zeros_like(lse)
    for b in range(batch):
        n = int(lens[b])
        pages = table[b, :-(-n // page)].long()
        rows = (pages[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]
        rows = rows[(rows >= 0) & (rows < kc.shape[0])]
        if rows.numel() == 0:
            continue
        n = rows.numel()
        k = kc[rows].view(E4M3).double().view(n, hkv, d) * scales[0].double()
        v = vc[rows].view(E4M3).double().view(n, hkv, d) * scales[1].double()
        qq = q[b].double().view(hkv, hq // hkv, d)
        s = torch.einsum("hgd,nhd->hgn", qq, k) * scale
        size = torch.einsum("hgd,nhd->hgn", qq.abs(), k.abs()) * scale
        z = torch.logsumexp(s, 2)
        p = torch.exp(s - z[..., None])
        o = torch.einsum("hgn,nhd->hgd", p, v)
        eps = (size * (2.0 ** -19 + 2.0 ** -21) + s.abs() * 2.0 ** -22).amax(2)
        spread = torch.einsum("hgn,nhd->hgd", p, v.abs())
        out[b] = o.reshape(hq, d)
        tol[b] = ((2.0 ** -10 + 4 * eps)[..., None] * spread + n * 2.0 ** -24 * v.abs().max() + o.abs() * 2.0 ** -8).reshape(hq, d)
        lse[b] = z.reshape(hq)
        lse_tol[b] = (2 * eps + 2.0 ** -19 + z.abs() * 2.0 ** -22 + n * 2.0 ** -24 / 16).reshape(hq)
    return out, tol, lse, lse_tol


def check(lens, hq, hkv, d, page, seed=0, **more):
    scale = more.pop("scale", None)
    q, kc, vc, table, ln, scales = make(lens, hq, hkv, d, page, seed, **more)
    out, lse = fp8rl.attn_decode(q, kc, vc, table, ln, scales, page, softmax_scale=scale)
    assert fp8rl.fp8rl_sync_status() == 0
    ref, tol, rl, rl_tol = reference(q, kc, vc, table, ln, scales, page, scale)
    assert bool(((out.double() - ref).abs() <= tol).all()), ((out.double() - ref).abs() / tol.clamp(min=1e-30)).max().item()
    none = rl == -math.inf
    assert bool((lse[none] == -math.inf).all()) and bool((out[none] == 0).all())
    assert bool(((lse.double() - rl).abs()[~none] <= rl_tol[~none]).all())
    return q, kc, vc, table, ln, scales, out, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (32, 8), (32, 4), (6, 2), (9, 1), (40, 4), (16, 1), (40, 1)])
def test_heads(hq, hkv, d):
    check([1, 17, 300, 64], hq, hkv, d, 16, seed=hq)


@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 256])
def test_pages(page):
    check([0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 511, 1000], 8, 2, 128, page, seed=page)


@pytest.mark.parametrize("lens", [[1], [63], [64], [65], [5000], [20000, 3], [0], [0, 0, 7, 0], [100] * 300, [2000, 1] * 40])
def test_lengths(lens):
    check(lens, 32, 8, 128, 16, seed=len(lens))


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (6, 2), (8, 2), (10, 2), (14, 2), (16, 2), (18, 2), (12, 3), (12, 4), (20, 4)])
@pytest.mark.parametrize("ld_pad", [0, 16])
def test_heads_of_64(hq, hkv, ld_pad):
    check([0, 1, 31, 32, 33, 127, 128, 129, 900, 4000], hq, hkv, 64, 16, seed=hq + hkv, ld_pad=ld_pad)


@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (8, 2, 64), (12, 2, 64), (16, 4, 64), (18, 2, 64), (6, 3, 64), (8, 2, 128), (16, 2, 128)])
def test_nan_codes_stay_in_their_head(hq, hkv, d):
    """NaN codes in a head's keys or values reach its own query heads alone."""
    q, kc, vc, table, ln, scales = make([150, 40, 700], hq, hkv, d, 16, seed=11)
    want, wl = fp8rl.attn_decode(q, kc, vc, table, ln, scales, 16)
    group = hq // hkv
    for head in range(hkv):
        mine = torch.zeros(hq, dtype=torch.bool, device="cuda")
        mine[head * group:(head + 1) * group] = True
        for which in range(2):
            caches = [kc.clone(), vc.clone()]
            caches[which][:, head * d:(head + 1) * d] = 0x7F
            out, lse = fp8rl.attn_decode(q, caches[0], caches[1], table, ln, scales, 16)
            assert torch.equal(out[:, ~mine], want[:, ~mine]) and torch.equal(lse[:, ~mine], wl[:, ~mine])
            assert bool(out[:, mine].isnan().all())


@pytest.mark.parametrize("batch,hq,hkv,d", [(470, 8, 4, 128), (920, 16, 2, 128), (920, 24, 2, 128), (920, 4, 4, 64), (920, 16, 4, 64),
                                            (920, 32, 4, 64), (920, 3, 3, 64), (470, 36, 4, 128)])
def test_many_caches(batch, hq, hkv, d):
    """Enough sequences for items of two heads, of ragged lengths, some of them shared by CTAs."""
    g = torch.Generator().manual_seed(batch + hq)
    lens = torch.randint(0, 300, (batch,), generator=g).tolist()
    lens[3], lens[batch // 2], lens[-1] = 5000, 0, 2500
    q, kc, vc, table, ln, scales, out, lse = check(lens, hq, hkv, d, 16, seed=hq)
    group = hq // hkv
    mine = torch.zeros(hq, dtype=torch.bool, device="cuda")
    mine[group:2 * group] = True
    vc = vc.clone()
    vc[:, d:2 * d] = 0x7F  # NaN codes of one KV head stay in its query heads
    got, got_lse = fp8rl.attn_decode(q, kc, vc, table, ln, scales, 16)
    assert torch.equal(got[:, ~mine], out[:, ~mine]) and torch.equal(got_lse, lse)
    assert bool(got[ln > 0][:, mine].isnan().all())


def test_one_long_sequence_of_one_head():
    check([70001], 4, 1, 128, 64, seed=1)


def test_lengths_past_the_table_and_negative_are_clamped():
    q, kc, vc, table, ln, scales = make([64, 40, 30], 8, 2, 128, 16, seed=2)
    want = fp8rl.attn_decode(q, kc, vc, table, torch.tensor([64, 40, 0], dtype=torch.int32, device="cuda"), scales, 16)
    got = fp8rl.attn_decode(q, kc, vc, table, torch.tensor([1 << 30, 40, -5], dtype=torch.int32, device="cuda"), scales, 16)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_pages_outside_the_cache_are_left_out():
    q, kc, vc, table, ln, scales = make([200, 200, 60], 8, 2, 128, 16, seed=3)
    table[0, 3] = -1
    table[0, 7] = kc.shape[0]  # far past the last page
    table[2, :] = -7           # nothing left
    out, lse = fp8rl.attn_decode(q, kc, vc, table, ln, scales, 16)
    ref, tol, rl, rl_tol = reference(q, kc, vc, table, ln, scales, 16)
    assert bool(((out.double() - ref).abs() <= tol).all())
    assert bool((out[2] == 0).all()) and bool((lse[2] == -math.inf).all())


def test_strides_scale_and_peaked_scores():
    check([500, 77], 8, 2, 128, 16, seed=4, ld_pad=64)
    check([500, 77], 8, 2, 128, 16, seed=5, scale=0.5)
    check([900, 77], 8, 2, 128, 16, seed=6, q_scale=40.0)    # scores in the hundreds: one key takes all
    check([900, 77], 8, 2, 128, 16, seed=7, q_scale=1e-30)   # q far below f16's range
    check([900, 77], 8, 2, 64, 16, seed=8, q_scale=0.0)


def test_growing_scores_rescale():
    """Keys in ascending score order: the running maximum keeps moving."""
    d, n = 128, 3000
    q = torch.ones(1, 4, d, dtype=torch.bfloat16, device="cuda")
    codes = (torch.linspace(0, 400, n, device="cuda")[:, None].expand(n, d)).contiguous().to(E4M3).view(torch.uint8)
    v = torch.randn(n, d, device="cuda").clamp(-4, 4).to(E4M3).view(torch.uint8)
    table = torch.arange(-(-n // 16), device="cuda").int()[None]
    kc = torch.zeros(table.shape[1] * 16, d, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    kc[:n], vc[:n] = codes, v
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    scales = torch.tensor([0.05, 1.0], device="cuda")
    for order in (slice(None), None):
        if order is None:
            kc[:n] = kc[:n].flip(0)
        out, lse = fp8rl.attn_decode(q, kc, vc, table, ln, scales, 16)
        ref, tol, rl, rl_tol = reference(q, kc, vc, table, ln, scales, 16)
        assert bool(((out.double() - ref).abs() <= tol).all())
        assert bool(((lse.double() - rl).abs() <= rl_tol).all())


def test_offsets_past_32_bits():
    """A cache of 5 GB: its last pages are past 2^32 bytes."""
    hkv, d, page = 8, 128, 16
    slots = 5 * (1 << 20)
    kc = torch.zeros(slots, hkv * d, dtype=torch.uint8, device="cuda")
    vc = torch.zeros(slots, hkv * d, dtype=torch.uint8, device="cuda")
    q, k0, v0, t0, ln, scales = make([333, 64], 32, hkv, d, page, seed=10, spare=0)
    base = slots // page - k0.shape[0] // page
    kc[base * page:], vc[base * page:] = k0, v0
    want = fp8rl.attn_decode(q, k0, v0, t0, ln, scales, page)
    got = fp8rl.attn_decode(q, kc, vc, torch.where(t0 >= 0, t0 + base, -1).int(), ln, scales, page)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_one_workspace_across_calls_and_same_bits():
    ws = fp8rl.attn_decode_workspace(32, 8, 128)
    first = {}
    for lens in ([5000, 1, 700], [64] * 50, [9], [5000, 1, 700], [64] * 50):
        q, kc, vc, table, ln, scales = make(lens, 32, 8, 128, 16, seed=len(lens))
        got = fp8rl.attn_decode(q, kc, vc, table, ln, scales, 16, workspace=ws)
        key = tuple(lens)
        if key in first:
            assert torch.equal(first[key][0], got[0]) and torch.equal(first[key][1], got[1])
        first[key] = got
    # a graph of it, on another stream's pool
    graph = torch.cuda.CUDAGraph()
    out = (torch.empty_like(got[0]), torch.empty_like(got[1]))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fp8rl.attn_decode(q, kc, vc, table, ln, scales, 16, workspace=ws, out=out)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], got[0])


@pytest.mark.parametrize("lens,hq,hkv,d", [([9000], 40, 4, 128), ([50000], 32, 4, 64), ([30000, 5, 20000], 12, 2, 64), ([60000], 16, 1, 128),
                                           ([40000], 3, 3, 64), ([7000], 8, 1, 128), ([100000, 200], 8, 1, 64)])
def test_partials_merged_in_two_steps(lens, hq, hkv, d):
    """Few long sequences, each over hundreds of CTAs: right, the same bits again on the
    same workspace, and the workspace's counters left at zero."""
    q, kc, vc, table, ln, scales, out, lse = check(lens, hq, hkv, d, 16, seed=hq)
    ws = fp8rl.attn_decode_workspace(hq, hkv, d)
    for _ in range(3):
        got = fp8rl.attn_decode(q, kc, vc, table, ln, scales, 16, workspace=ws)
        assert torch.equal(got[0], out) and torch.equal(got[1], lse)
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert not bool(ws[:sms * 4 * 3 * 4].any())


def test_one_workspace_across_shapes():
    """Shapes that need it in different sizes, on one workspace: the counters of
    one are never another's partials."""
    shapes = [(32, 8, 128), (40, 4, 128), (16, 16, 64), (9, 1, 64), (32, 4, 64), (12, 3, 64)]
    ws = max((fp8rl.attn_decode_workspace(*x) for x in shapes), key=torch.Tensor.numel)
    for turn in range(2):
        for hq, hkv, d in shapes:
            q, kc, vc, table, ln, scales = make([6000, 3000, 7, 9000] * 4, hq, hkv, d, 16, seed=hq)
            want = fp8rl.attn_decode(q, kc, vc, table, ln, scales, 16, workspace=fp8rl.attn_decode_workspace(hq, hkv, d))
            got = fp8rl.attn_decode(q, kc, vc, table, ln, scales, 16, workspace=ws,
                                    out=(torch.full_like(want[0], 7), torch.full_like(want[1], 7)))
            assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_reads_what_the_append_wrote():
    """kv_calibrate, kv_append, then attention: against fp64 attention on the
    cache's own dequantised rows."""
    d, hkv, hq, page, n = 128, 8, 32, 16, 300
    g = torch.Generator("cuda").manual_seed(1)
    k = torch.randn(n, hkv * d, generator=g, device="cuda").bfloat16()
    v = torch.randn(n, hkv * d, generator=g, device="cuda").bfloat16()
    scales = fp8rl.kv_calibrate(k, v)
    pages = torch.randperm(64, generator=g, device="cuda").int()[:-(-n // page)]
    pos = torch.arange(n, device="cuda")
    slots = (pages[pos // page] * page + pos % page).int()
    kc = torch.zeros(64 * page, hkv * d, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    fp8rl.kv_append(k, v, slots, kc, vc, scales)
    q = torch.randn(1, hq, d, generator=g, device="cuda").bfloat16()
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    out, lse = fp8rl.attn_decode(q, kc, vc, pages[None].contiguous(), ln, scales, page)
    ref, tol, _, _ = reference(q, kc, vc, pages[None], ln, scales, page)
    assert bool(((out.double() - ref).abs() <= tol).all())
