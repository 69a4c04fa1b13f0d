"""The attention over the paged E4M3 cache, held to what its arithmetic allows.

The products as in test_gpu_attn_decode.py: scores within eps = (2^-19 + 2^-21)
sum|q k| scale + |s| 2^-22, a probability within 2^-11 of itself in f16's normal
range.  Below that range f16 has steps of 2^-24; the kernel's reference lies at
least 2^11 below the largest key's p, so such a p is within 2^-25 / 2^11 of the
largest key's: an output is within (2^-10 + 4 eps) sum p|v| + 2^-36
exp(s_max - lse) sum|v| of its value, plus bf16's 2^-8."""
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


def codes(x):
    return x.clamp(-448, 448).to(E4M3)


def check(q, kv, scales, lens, scale, page=16, seed=0, shared=False):
    """q [batch, hq, d]; kv: per sequence (k, v) E4M3 [n, hkv, d], put on scattered
    pages; `shared`: all sequences (and queries) are the first one."""
    batch, hq, d = q.shape
    hkv = kv[0][0].shape[1]
    need = [-(-n // page) for n in (lens[:1] if shared else lens)]
    g = torch.Generator("cuda").manual_seed(seed)
    perm = torch.randperm(sum(need) + 2, generator=g, device="cuda").int()
    table = torch.full((batch, max(need)), -1, dtype=torch.int32, device="cuda")
    caches = [torch.full(((sum(need) + 2) * page, hkv * d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]  # NaN codes
    at = 0
    for b, n in enumerate(lens[:1] if shared else lens):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        rows = (table[b, :need[b]].long()[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]
        for c, x in zip(caches, kv[b]):
            c[rows] = x.reshape(n, hkv * d).view(torch.uint8)
    if shared:
        table[1:] = table[:1]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = fp8rl.attn_decode(q, *caches, table, ln, scales, page, softmax_scale=scale)
    assert fp8rl.fp8rl_sync_status() == 0
    for b in range(1 if shared else batch):
        k, v = (x.double() * s.double() for x, s in zip(kv[b], scales))
        qq = q[b].double().view(hkv, hq // hkv, d)
        s = torch.einsum("hgd,nhd->hgn", qq, k) * scale
        size = torch.einsum("hgd,nhd->hgn", qq.abs(), k.abs()) * scale
        z = torch.logsumexp(s, 2)
        p = torch.exp(s - z[..., None])
        eps = (size * (2.0 ** -19 + 2.0 ** -21) + s.abs() * 2.0 ** -22).amax(2)
        ref = torch.einsum("hgn,nhd->hgd", p, v)
        tol = (2.0 ** -10 + 4 * eps)[..., None] * torch.einsum("hgn,nhd->hgd", p, v.abs()) + ref.abs() * 2.0 ** -8 + \
            2.0 ** -36 * torch.exp(s.amax(2) - z)[..., None] * v.abs().sum(0)[:, None]
        rows = slice(None) if shared else slice(b, b + 1)
        err = (out[rows].double().view(-1, *ref.shape) - ref).abs()
        assert bool((err <= tol).all()), (b, (err / tol).max().item())
        assert bool(((lse[rows].double().view(-1, *z.shape) - z).abs() <= 2 * eps + 2.0 ** -19 + z.abs() * 2.0 ** -22).all())


@pytest.mark.parametrize("gap", [10.0, 14.0, 17.0, 17.5, 19.0, 21.0])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
def test_many_small_beside_one_large(gap, at):
    """One key without a value takes nearly all the probability; what the output
    is made of lies `gap` e-folds below it, 131 072 times."""
    n, d, hq = 131073, 128, 4
    g = torch.Generator("cuda").manual_seed(int(gap * 10))
    k = torch.tensor([3.75, 4.0, 4.5], device="cuda")[torch.randint(0, 3, (n, 1, d), generator=g, device="cuda")]
    v = codes(1 + 0.5 * torch.randn(n, 1, d, generator=g, device="cuda"))
    sink = {"first": 0, "middle": 70001, "last": n - 1}[at]
    k[sink], v[sink] = 8.0, torch.zeros(d, device="cuda").to(E4M3)
    q = torch.ones(1, hq, d, device="cuda").bfloat16()
    # the others' mean is 49/12, the sink's distance from it 47/12, times 128 columns
    check(q, [(codes(k), v)], torch.tensor([1.0, 1.0], device="cuda"), [n], gap / (128 * 47 / 12))


@pytest.mark.parametrize("gap", [10.0, 14.0, 17.0, 17.5, 19.0, 21.0])
@pytest.mark.parametrize("at", [0, 4096, 8064])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (2, 2, 64), (8, 2, 128), (16, 1, 128)])
def test_many_small_beside_a_large_one_of_each_warp(gap, at, hq, hkv, d):
    """The same where a CTA has whole sequences (hundreds of them, on the same
    pages) and each of its four warps, which take 32 keys each in turn, has a large
    key of its own."""
    n, batch = 8192, 600
    g = torch.Generator("cuda").manual_seed(int(gap * 10))
    k = torch.tensor([3.75, 4.0, 4.5], device="cuda")[torch.randint(0, 3, (n, hkv, d), generator=g, device="cuda")]
    v = 1 + 0.5 * torch.randn(n, hkv, d, generator=g, device="cuda")
    sinks = at + 32 * torch.arange(4, device="cuda")
    k[sinks], v[sinks] = 8.0, 0.0
    q = torch.ones(batch, hq, d, device="cuda").bfloat16()
    check(q, [(codes(k), codes(v))] * batch, torch.tensor([1.0, 1.0], device="cuda"), [n] * batch, gap / (d * 47 / 12), shared=True)


@pytest.mark.parametrize("lens,hq,hkv,d", [([100000, 200], 8, 1, 64), ([70001], 4, 1, 128), ([50000], 32, 4, 64), ([9000], 40, 4, 128),
                                           ([30000, 5, 20000], 12, 2, 64), ([60000], 16, 1, 128), ([40000], 3, 3, 64), ([7000], 8, 1, 128),
                                           ([2500, 800, 1300] * 60, 32, 8, 128), ([3000] * 310, 8, 4, 128)])
def test_every_part_of_a_cache_counts_once(lens, hq, hkv, d):
    """Column d of the values is 1 in a range of the keys of its own and 0 outside,
    so the output is the ranges' shares of the probability: a partial that is left
    out, counted twice or scaled wrongly changes a column by far more than its bound."""
    g = torch.Generator("cuda").manual_seed(sum(lens) + hq)
    kv = []
    for n in lens:
        k = codes(torch.randn(n, hkv, d, generator=g, device="cuda") * 80)
        v = torch.nn.functional.one_hot(torch.arange(n, device="cuda") * d // n, d).float()
        kv.append((k, (v[:, None] * torch.arange(1, hkv + 1, device="cuda")[:, None]).to(E4M3)))
    q = (torch.randn(len(lens), hq, d, generator=g, device="cuda") * 0.5).bfloat16()
    check(q, kv, torch.tensor([0.0121, 1.0], device="cuda"), lens, d ** -0.5, seed=hq)
