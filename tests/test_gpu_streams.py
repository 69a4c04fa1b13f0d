"""The helpers with an explicit ``stream`` other than torch's current one: what
a helper makes and clears for one call belongs to that stream.  The current
stream is kept busy, so that anything left on it would come too late, and memory
of the same size is filled right after the call, so that scratch given back to
the current stream too early would be overwritten."""
import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8rl.load_library(build_if_missing=True)


def aside(call, nbytes):
    """call(stream handle) on a stream of its own while the current stream is busy;
    freed memory of `nbytes` on either stream holds ones."""
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            for _ in range(3):
                torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about a tenth of a second
    got = call(side.cuda_stream)
    trample = [torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    del trample
    assert fp8rl.fp8rl_sync_status() == 0
    return got


def same(want, got):
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("lens,hq,hkv,d", [([9000], 32, 8, 128), ([70, 4000, 0, 1], 8, 2, 64)])
def test_attn_decode_without_a_workspace(lens, hq, hkv, d):
    g = torch.Generator("cuda").manual_seed(1)
    blocks = -(-max(lens) // 16)
    kc, vc = (torch.randint(0, 0x78, (len(lens) * blocks * 16, hkv * d), generator=g, device="cuda").to(torch.uint8) for _ in range(2))
    table = torch.arange(len(lens) * blocks, device="cuda").int().view(len(lens), blocks)
    q = torch.randn(len(lens), hq, d, generator=g, device="cuda").bfloat16()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scales = torch.tensor([0.001, 0.01], device="cuda")
    ws = fp8rl.attn_decode_workspace(hq, hkv, d)
    want = fp8rl.attn_decode(q, kc, vc, table, ln, scales, 16, workspace=ws)
    same(want, aside(lambda s: fp8rl.attn_decode(q, kc, vc, table, ln, scales, 16, stream=s), ws.numel()))
    # the legacy default stream by its null handle
    same(want, fp8rl.attn_decode(q, kc, vc, table, ln, scales, 16, stream=0))


@pytest.mark.parametrize("n", [1, 100_000, 3_000_001])
def test_tis_weights_without_a_workspace(n):
    g = torch.Generator("cuda").manual_seed(2)
    lt, lr = (-torch.rand(n, generator=g, device="cuda") for _ in range(2))
    mask = (torch.rand(n, generator=g, device="cuda") < 0.7).to(torch.uint8)
    need = max(fp8rl.fp8rl_tis_workspace_size(n), 32)
    want = fp8rl.tis_weights(lt, lr, mask, workspace=torch.zeros(need, dtype=torch.uint8, device="cuda"))
    same(want, aside(lambda s: fp8rl.tis_weights(lt, lr, mask, stream=s), need))


def test_moe_plan_without_a_workspace():
    g = torch.Generator("cuda").manual_seed(3)
    topk = torch.rand(5000, 64, generator=g, device="cuda").argsort(1)[:, :8].int().contiguous()
    need = max(fp8rl.fp8rl_moe_plan_workspace_size(5000, 8, 64), 256)
    want = fp8rl.moe_plan(topk, 64, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    same(want, aside(lambda s: fp8rl.moe_plan(topk, 64, stream=s), need))


@pytest.mark.parametrize("with_q", [False, True])
def test_kv_calibrate(with_q):
    g = torch.Generator("cuda").manual_seed(4)
    k, v, q = (torch.randn(3000, 256, generator=g, device="cuda").bfloat16() for _ in range(3))
    q = q if with_q else None
    want = fp8rl.kv_calibrate(k, v, q)
    assert bool((want[:2] > 0).all()) and bool(want[2] > 0) == with_q
    same([want], aside(lambda s: [fp8rl.kv_calibrate(k, v, q, stream=s)], 512))


def test_guarded_outputs(monkeypatch):
    """The guards' fill does not land on what the other stream's kernel wrote."""
    monkeypatch.setenv("FP8RL_CANARY", "1")
    x = torch.randn(300, 512, device="cuda").bfloat16()
    want = fp8rl.quant_act(x)
    same(want, aside(lambda s: fp8rl.quant_act(x, stream=s), 1 << 18))
