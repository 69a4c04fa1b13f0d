"""Rotary positions at the ends of their ranges: positions that several axes share,
as many tokens as a call takes, keys past the cache's scale."""
import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("tokens", [1, 2, 37])
@pytest.mark.parametrize("d", [128, 6])  # the vector path, any layout
def test_positions_that_all_axes_share(tokens, d):
    # text among images: one row of positions, expanded over the axes
    g = torch.Generator("cuda").manual_seed(tokens)
    q, k, v = (torch.randn(tokens, h, d, generator=g, device="cuda").bfloat16() for h in (4, 2, 2))
    freqs = fp8rl.rotary_freqs(d, sections=(d // 2 - 2, 1, 1))
    pos = torch.randint(0, 5000, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    shared, apart = pos.expand(3, -1), pos.repeat(3, 1)
    want = fp8rl.rotary(q, k, apart, freqs)
    assert all(torch.equal(a, b) for a, b in zip(fp8rl.rotary(q, k, shared, freqs), want))
    caches = [[torch.zeros(tokens, 2 * d, dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(2)]
    at = torch.arange(tokens, device="cuda", dtype=torch.int32)
    got = [fp8rl.rotary_kv_append(q, k, v, p, freqs, at, *c, torch.ones(2, device="cuda"))[0] for p, c in zip((shared, apart), caches)]
    assert torch.equal(*got) and all(torch.equal(a, b) for a, b in zip(*caches))
    x, y = (q.clone().requires_grad_() for _ in range(2))
    fp8rl.rotary(x, None, shared, freqs)[0].sum().backward()
    fp8rl.rotary(y, None, apart, freqs)[0].sum().backward()
    assert torch.equal(x.grad, y.grad)


def test_as_many_tokens_as_a_call_takes():
    tokens, d = 2 ** 31 - 1, 16
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB")
    q = torch.zeros(tokens, 1, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    freqs = fp8rl.rotary_freqs(d)
    ends = (slice(0, 33), slice(tokens // 2, tokens // 2 + 33), slice(tokens - 33, tokens))
    want = []
    for s in ends:
        q[s] = torch.randn(33, 1, d, generator=g, device="cuda").bfloat16()
        pos[s] = torch.randint(0, 1000, (33,), generator=g, device="cuda", dtype=torch.int32)
        want.append(fp8rl.rotary(q[s].clone(), None, pos[s].clone(), freqs)[0])
    fp8rl.rotary(q, None, pos, freqs, out=(q, None))
    assert all(torch.equal(q[s], w) for s, w in zip(ends, want))
    del q, pos
    torch.cuda.empty_cache()


@pytest.mark.parametrize("d", [128, 6])  # the vector path, any layout
@pytest.mark.parametrize("scale", [5e35, 7.5e35, 0.01])
def test_keys_that_are_infinite_saturate_at_every_scale(d, scale):
    # 1024 scales are past fp32's range from 3.3e35 on (the largest bf16 calibrates to 7.6e35)
    k = torch.zeros(4, 1, d, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 0], k[1, 0, 1], k[2, 0, 0], k[2, 0, d // 2], k[3, 0, 0] = INF, -INF, 3e38, -3e38, 208 * scale
    pos = torch.tensor([0, 0, 1, 0], dtype=torch.int32, device="cuda")
    freqs = fp8rl.rotary_freqs(d, inv_freq=[0.7853981633974483] * (d // 2))  # (an eighth of a turn: sums of both halves)
    caches = [torch.zeros(4, d, dtype=torch.uint8, device="cuda") for _ in range(2)]
    # a turn by 0 would meet 0 x infinity in the pair's other element
    fp8rl.rotary_kv_append(k, k, k, pos, freqs, torch.arange(4, device="cuda", dtype=torch.int32), *caches,
                           torch.tensor([scale, 1.0], device="cuda"))
    codes = caches[0].cpu()
    assert int(codes[0, 0]) == 0x7E and int(codes[1, 1]) == 0xFE
    assert int(codes[3, 0]) == int(torch.tensor(208.0).to(torch.float8_e4m3fn).view(torch.uint8))
    # (3e38 + 3e38) / sqrt(2) is infinite in fp32
    assert int(codes[2, 0]) == 0x7E
