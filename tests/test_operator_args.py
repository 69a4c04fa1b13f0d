"""The norm, attention and log-probability entry points refuse bad arguments on
the host before touching the GPU.  CPU only: no call here reaches a launch."""
import math

import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl
from fp8_w8a8_rollout_gb300 import _build

P = 1 << 20  # an aligned fake address, never dereferenced: validation fails first, or there is no work


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fp8rl.load_library()


def call(lib, name, defaults, **changes):
    assert set(changes) <= set(defaults), changes
    return getattr(lib, name)(*{**defaults, **changes}.values())


NORM = dict(x=P, ldx=256, res=P, ldr=256, w=P, eps=1e-6, m=4, k=256, h=P, ldh=256, q=P, ldq=256, s=P, fmt=0, stream=None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(x=None)), (1, dict(w=None)), (1, dict(q=None)), (1, dict(s=None)), (1, dict(m=-1)), (1, dict(k=-1)),
    (1, dict(ldx=255)), (1, dict(ldr=255)), (1, dict(ldh=255)), (1, dict(ldq=255)), (1, dict(eps=-1.0)),
    (1, dict(eps=math.nan)), (1, dict(fmt=2)), (2, dict(k=40000, ldx=40000, ldr=40000, ldh=40000, ldq=40000)),
    (2, dict(m=1 << 31)), (3, dict(x=P + 1)), (3, dict(res=P + 1)), (3, dict(w=P + 1)), (3, dict(h=P + 1)), (3, dict(s=P + 2)),
    (0, dict(m=0)), (0, dict(k=0)),
])
def test_norm(lib, status, changes):
    assert call(lib, "fp8rl_rmsnorm_quant", NORM, **changes) == status


DECODE = dict(q=P, ldq=4096, batch=2, hq=32, hkv=8, d=128, kc=P, vc=P, ldc=1024, slots=64, table=P, ldt=4, blocks=4, page=16,
              lens=P, scales=P, scale=0.1, out=P, ldo=4096, lse=P, ws=P, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(q=None)), (1, dict(kc=None)), (1, dict(vc=None)), (1, dict(table=None)), (1, dict(lens=None)), (1, dict(scales=None)),
    (1, dict(out=None)), (1, dict(ws=None)), (1, dict(batch=-1)), (1, dict(hq=30)), (1, dict(hkv=0)), (1, dict(hq=0)),
    (1, dict(ldq=4095)), (1, dict(ldo=4095)), (1, dict(ldc=1023)), (1, dict(ldt=3)), (1, dict(page=0)), (1, dict(slots=-1)),
    (1, dict(blocks=-1)), (1, dict(scale=0.0)), (1, dict(scale=math.inf)), (1, dict(scale=math.nan)), (1, dict(ws_bytes=1000)),
    (2, dict(d=96)), (2, dict(batch=8193)), (2, dict(blocks=1 << 27, ldt=1 << 27)), (2, dict(page=1 << 31)), (2, dict(slots=1 << 27)),
    (3, dict(q=P + 2)), (3, dict(ldq=4097)), (3, dict(kc=P + 8)), (3, dict(vc=P + 8)), (3, dict(ldc=1032)), (3, dict(out=P + 1)),
    (3, dict(table=P + 2)), (3, dict(lens=P + 2)), (3, dict(scales=P + 2)), (3, dict(lse=P + 2)), (3, dict(ws=P + 8)),
    (0, dict(batch=0)),
])
def test_decode(lib, status, changes):
    assert call(lib, "fp8rl_attn_decode", DECODE, **changes) == status


def test_decode_workspace_size(lib):
    f = lib.fp8rl_attn_decode_workspace_size
    assert f(32, 8, 128) > 0 and f(40, 4, 64) > 0
    assert f(32, 5, 128) == 0 and f(32, 8, 96) == 0 and f(0, 1, 128) == 0 and f(8, 0, 128) == 0


PREFILL = dict(q=P, ldq=6144, k=P, ldk=6144, v=P, ldv=6144, plan=P, plan_bytes=1 << 30, batch=2, total=100, hq=32, hkv=8, d=128,
               scale=0.1, out=P, ldo=4096, lse=P, stream=None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(q=None)), (1, dict(k=None)), (1, dict(v=None)), (1, dict(plan=None)), (1, dict(out=None)), (1, dict(batch=-1)),
    (1, dict(total=-1)), (1, dict(hq=30)), (1, dict(hkv=0)), (1, dict(ldq=4088)), (1, dict(ldk=1016)), (1, dict(ldv=1016)),
    (1, dict(ldo=4088)), (1, dict(scale=0.0)), (1, dict(scale=math.nan)), (1, dict(plan_bytes=16)), (2, dict(d=96)),
    (2, dict(total=(1 << 26) + 1)), (2, dict(batch=(1 << 20) + 1)), (3, dict(q=P + 8)), (3, dict(k=P + 8)), (3, dict(v=P + 8)),
    (3, dict(out=P + 8)), (3, dict(ldq=6145)), (3, dict(ldk=6148)), (3, dict(ldv=6148)), (3, dict(ldo=4100)), (3, dict(plan=P + 8)),
    (3, dict(lse=P + 2)), (0, dict(batch=0)), (0, dict(total=0)),
])
def test_prefill(lib, status, changes):
    assert call(lib, "fp8rl_attn_prefill", PREFILL, **changes) == status


PLAN = dict(cu=P, batch=2, total=100, hq=32, hkv=8, plan=P, plan_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(cu=None)), (1, dict(plan=None)), (1, dict(batch=-1)), (1, dict(total=-1)), (1, dict(hq=30)), (1, dict(plan_bytes=16)),
    (2, dict(total=(1 << 26) + 1)), (2, dict(batch=(1 << 20) + 1)), (3, dict(cu=P + 2)), (3, dict(plan=P + 8)),
])
def test_prefill_plan(lib, status, changes):
    assert call(lib, "fp8rl_attn_prefill_plan", PLAN, **changes) == status


def test_prefill_plan_size(lib):
    f = lib.fp8rl_attn_prefill_plan_size
    assert f(1000, 3, 32, 8) >= 16 * (1 + 1000 // 64 + 3) and f(0, 0, 1, 1) == 16
    assert f(-1, 1, 8, 8) == 0 and f(1, -1, 8, 8) == 0 and f(1, 1, 8, 3) == 0 and f((1 << 26) + 1, 1, 8, 8) == 0 and f(1 << 26, 1, 8, 8) > 0


LP = dict(x=P, fp32=0, rows=4, vocab=100, ld=100, T=1.0, tokens=P, lp=P, ent=P, stats=P, topk=4, ids=P, top=P, stream=None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(x=None)), (1, dict(tokens=None)), (1, dict(lp=None)), (1, dict(ent=None)), (1, dict(stats=None)), (1, dict(ids=None)),
    (1, dict(top=None)), (1, dict(fp32=2)), (1, dict(rows=-1)), (1, dict(vocab=0)), (1, dict(ld=99)), (1, dict(T=0.0)),
    (1, dict(T=-1.0)), (1, dict(T=math.inf)), (1, dict(T=math.nan)), (1, dict(topk=-1)), (2, dict(topk=33)),
    (2, dict(vocab=3, topk=4)), (2, dict(vocab=1 << 31, ld=1 << 31)), (3, dict(x=P + 1)), (3, dict(fp32=1, x=P + 2)),
    (3, dict(tokens=P + 1)), (3, dict(stats=P + 4)), (3, dict(ids=P + 2)), (0, dict(rows=0)),
])
def test_logprob(lib, status, changes):
    assert call(lib, "fp8rl_logprob", LP, **changes) == status


GRAD = dict(x=P, fp32=0, rows=4, vocab=100, ld=100, T=1.0, tokens=P, stats=P, ent=P, g=P, gh=P, dx=2 * P, ldd=100, stream=None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(x=None)), (1, dict(tokens=None)), (1, dict(stats=None)), (1, dict(ent=None)), (1, dict(g=None)), (1, dict(dx=None)),
    (1, dict(fp32=-1)), (1, dict(rows=-1)), (1, dict(vocab=0)), (1, dict(ld=99)), (1, dict(ldd=99)), (1, dict(T=0.0)),
    (1, dict(dx=P, ldd=128)), (2, dict(vocab=1 << 31, ld=1 << 31, ldd=1 << 31)), (3, dict(x=P + 1)), (3, dict(dx=P + 1)),
    (3, dict(stats=P + 4)), (3, dict(g=P + 2)), (3, dict(gh=P + 2)), (0, dict(rows=0)),
])
def test_logprob_backward(lib, status, changes):
    assert call(lib, "fp8rl_logprob_backward", GRAD, **changes) == status


def test_helpers_reject_host_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(4)
    u8 = torch.zeros(64, 128, dtype=torch.uint8)
    for one in (lambda: fp8rl.rmsnorm_quant(x, x[0]),
                lambda: fp8rl.attn_decode(x.view(4, 2, 128), u8, u8, t.view(4, 1), t, f, 16),
                lambda: fp8rl.attn_prefill_plan(t, 4, 2, 1),
                lambda: fp8rl.attn_prefill(x.view(4, 2, 128), x.view(4, 2, 128), x.view(4, 2, 128), fp8rl.AttnPlan(t, 1, 4, 2, 2)),
                lambda: fp8rl.logprobs(x, t),
                lambda: fp8rl.logprobs_backward(x, t, f.view(2, 2), f, f)):
        with pytest.raises(ValueError, match="CUDA tensors"):
            one()
