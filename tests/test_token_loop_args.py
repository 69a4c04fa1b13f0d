"""The sampling, rotary and page entry points refuse bad arguments on the host
before touching the GPU.  CPU only: no call here reaches a launch."""
import ctypes
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


SAMPLE = dict(x=P, fp32=0, rows=4, vocab=100, ld=100, u=P, T=1.0, k=0, p=1.0, q=0.0, dT=None, dk=None, dp=None, dq=None, token=P, lp=P,
              lpk=P, kept=P, stream=None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(x=None)), (1, dict(u=None)), (1, dict(token=None)), (1, dict(fp32=2)), (1, dict(rows=-1)), (1, dict(vocab=0)), (1, dict(ld=99)),
    (1, dict(T=-1.0)), (1, dict(T=math.inf)), (1, dict(T=math.nan)), (1, dict(k=-1)), (1, dict(p=0.0)), (1, dict(p=-0.5)),
    (1, dict(p=math.nan)), (1, dict(q=-0.1)), (1, dict(q=1.5)), (1, dict(q=math.nan)), (2, dict(vocab=1 << 31, ld=1 << 31)),
    (3, dict(x=P + 1)), (3, dict(fp32=1, x=P + 2)), (3, dict(u=P + 4)), (3, dict(token=P + 2)), (3, dict(lp=P + 1)), (3, dict(lpk=P + 2)),
    (3, dict(kept=P + 2)), (3, dict(dT=P + 2)), (3, dict(dk=P + 2)), (3, dict(dp=P + 2)), (3, dict(dq=P + 2)), (0, dict(rows=0)),
    (0, dict(rows=0, T=math.nan, dT=P)),
])
def test_sample(lib, status, changes):
    assert call(lib, "fp8rl_sample", SAMPLE, **changes) == status


ROTARY = dict(q=P, ldq=4096, hq=32, k=P, ldk=1024, hkv=8, tokens=4, d=128, freqs=P, pairs=64, pos=P, ldp=4, axes=1, inter=0, inv=0,
              qo=2 * P, ldqo=4096, ko=2 * P, ldko=1024, stream=None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(q=None)), (1, dict(k=None)), (1, dict(qo=None)), (1, dict(ko=None)), (1, dict(freqs=None)), (1, dict(pos=None)),
    (1, dict(ldq=4095)), (1, dict(ldk=1023)), (1, dict(ldqo=4095)), (1, dict(ldko=1023)), (1, dict(ldp=3)), (1, dict(tokens=-1)),
    (1, dict(hq=-1)), (1, dict(hkv=-1)), (1, dict(hq=0, hkv=0)), (1, dict(d=0)), (1, dict(pairs=65)), (1, dict(pairs=-1)), (1, dict(axes=0)),
    (1, dict(inter=2)), (1, dict(inv=-1)), (1, dict(qo=P, ldqo=4104)), (1, dict(ko=P, ldko=2048)), (2, dict(d=1025, hq=1, hkv=1, ldk=2048, ldko=2048)),
    (2, dict(hq=9000, ldq=1 << 24, ldqo=1 << 24)), (2, dict(tokens=1 << 31, ldp=1 << 31)), (2, dict(axes=65)), (3, dict(q=P + 1)),
    (3, dict(k=P + 1)), (3, dict(qo=P + 1)), (3, dict(ko=P + 1)), (3, dict(pos=P + 2)), (3, dict(freqs=P + 4)), (0, dict(tokens=0)),
])
def test_rotary(lib, status, changes):
    assert call(lib, "fp8rl_rotary", ROTARY, **changes) == status


APPEND = dict(q=P, ldq=4096, hq=32, k=P, ldk=1024, v=P, ldv=1024, hkv=8, tokens=4, d=128, freqs=P, pairs=64, pos=P, ldp=4, axes=1, inter=0,
              qo=2 * P, ldqo=4096, ko=None, ldko=0, slots=P, kc=P, vc=P, ldc=1024, num=64, scales=P, stream=None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(q=None)), (1, dict(k=None)), (1, dict(v=None)), (1, dict(qo=None)), (1, dict(slots=None)), (1, dict(kc=None)),
    (1, dict(vc=None)), (1, dict(scales=None)), (1, dict(ldv=1023)), (1, dict(ldc=1023)), (1, dict(num=-1)), (1, dict(hkv=0)),
    (1, dict(ko=2 * P, ldko=1023)), (1, dict(inter=-1)), (2, dict(d=1026, hq=1, hkv=1, ldv=2048, ldc=2048)), (3, dict(v=P + 1)),
    (3, dict(slots=P + 2)), (3, dict(scales=P + 2)), (0, dict(tokens=0)),
])
def test_rotary_kv_append(lib, status, changes):
    assert call(lib, "fp8rl_rotary_kv_append", APPEND, **changes) == status


CACHES = (ctypes.c_void_p * 2)(P, P)
HOLES = (ctypes.c_void_p * 2)(P, None)
RESERVE = dict(table=P, ldt=8, rows=4, cols=8, page=16, lens=P, refs=P, pages=64, cu=None, count=None, total=4, slots=P, info=P, caches=CACHES,
               n=2, width=1024, ld=1024, ws=P, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(table=None)), (1, dict(lens=None)), (1, dict(refs=None)), (1, dict(slots=None)), (1, dict(ws=None)), (1, dict(ws_bytes=64)),
    (1, dict(rows=-1)), (1, dict(cols=-1)), (1, dict(ldt=7)), (1, dict(page=0)), (1, dict(pages=-1)), (1, dict(total=-1)),
    (1, dict(total=6)), (1, dict(n=-1)), (1, dict(caches=None)), (1, dict(caches=HOLES)), (1, dict(width=0)), (1, dict(ld=1000)),
    (2, dict(rows=8193, total=8193)), (2, dict(pages=1 << 28)), (2, dict(cols=1 << 28, ldt=1 << 28)), (2, dict(total=1 << 31, cu=P)),
    (2, dict(width=1 << 28, ld=1 << 28)), (3, dict(table=P + 2)), (3, dict(lens=P + 2)), (3, dict(refs=P + 2)), (3, dict(cu=P + 1)),
    (3, dict(count=P + 1)), (3, dict(slots=P + 2)), (3, dict(info=P + 2)), (3, dict(ws=P + 8)), (0, dict(rows=0, total=0)),
])
def test_kv_reserve(lib, status, changes):
    assert call(lib, "fp8rl_kv_reserve", RESERVE, **changes) == status


FORK = dict(table=P, ldt=8, rows=4, cols=8, page=16, lens=P, parent=P, new=4, to=2 * P, ld=8, to_lens=2 * P, refs=P, pages=64, stream=None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(table=None)), (1, dict(lens=None)), (1, dict(parent=None)), (1, dict(to=None)), (1, dict(to_lens=None)), (1, dict(refs=None)),
    (1, dict(new=-1)), (1, dict(ld=7)), (1, dict(rows=-1)), (1, dict(to=P)), (1, dict(to_lens=P)), (1, dict(to=P, to_lens=P, new=5)),
    (1, dict(to=P, to_lens=P, ld=9)), (2, dict(new=8193)), (2, dict(rows=8193)), (3, dict(parent=P + 2)), (3, dict(to=2 * P + 2)),
    (3, dict(to_lens=2 * P + 1)), (0, dict(rows=0, new=0)),
])
def test_kv_fork(lib, status, changes):
    assert call(lib, "fp8rl_kv_fork", FORK, **changes) == status


COMPACT = dict(table=P, ldt=8, rows=4, cols=8, page=16, lens=P, refs=P, pages=64, used=P, caches=CACHES, n=2, width=1024, ld=1024, ws=P,
               ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("status,changes", [
    (1, dict(table=None)), (1, dict(lens=None)), (1, dict(refs=None)), (1, dict(used=None)), (1, dict(ws=None)), (1, dict(ws_bytes=64)),
    (1, dict(caches=HOLES)), (1, dict(ld=1)), (1, dict(page=-1)), (2, dict(pages=1 << 28)), (3, dict(used=P + 2)), (3, dict(ws=P + 4)),
    (3, dict(refs=P + 1)),
])
def test_kv_compact(lib, status, changes):
    assert call(lib, "fp8rl_kv_compact", COMPACT, **changes) == status


def test_workspace_sizes(lib):
    f, g = lib.fp8rl_kv_reserve_workspace_size, lib.fp8rl_kv_compact_workspace_size
    assert f(0, 0, 16) > 0 and f(256, 256, 16) >= 256 * 32 + 4 * (16 + 512)
    assert f(-1, 0, 16) == 0 and f(8193, 0, 16) == 0 and f(1, -1, 16) == 0 and f(1, 1, 0) == 0
    assert g(0) > 0 and g(1000) >= 16 * 501 + 4000 and g(-1) == 0


def test_frequencies():
    f = fp8rl.rotary_freqs(8, 10000.0, (1, 2, 1), device="cpu")
    assert f.axes == 3 and f.rotary_dim == 8 and f.data[1].tolist() == [0, 1, 1, 2]
    for i, word in enumerate(f.data[0].tolist()):
        turn = 10000.0 ** (-i / 4) / (2 * math.pi)
        assert abs((word % (1 << 64)) / 2.0 ** 64 - turn) < 1e-16
    g = fp8rl.rotary_freqs(4, inv_freq=[-1.0, 7.0], device="cpu")
    assert [w % (1 << 64) / 2.0 ** 64 for w in g.data[0].tolist()] == pytest.approx([1 - 1 / (2 * math.pi), 7 / (2 * math.pi) - 1])
    for bad in (dict(rotary_dim=7), dict(rotary_dim=8, sections=(1, 2)), dict(rotary_dim=4, inv_freq=[1.0]), dict(rotary_dim=4, theta=0.0),
                dict(rotary_dim=4, inv_freq=[1.0, math.inf]), dict(rotary_dim=4, sections=(1, 1), axis=(0, 1)), dict(rotary_dim=4, axis=(0, -1))):
        with pytest.raises(ValueError):
            fp8rl.rotary_freqs(**bad, device="cpu")


def test_helpers_reject_host_tensors_and_wrong_types():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    u = torch.zeros(4, dtype=torch.float64)
    t = torch.zeros(4, dtype=torch.int32)
    u8 = torch.zeros(64, 256, dtype=torch.uint8)
    table = torch.zeros(4, 4, dtype=torch.int32)
    f = fp8rl.rotary_freqs(128, device="cpu")
    h = x.view(4, 2, 128)
    for one in (lambda: fp8rl.sample(x, u), lambda: fp8rl.rotary(h, h, t, f),
                lambda: fp8rl.rotary_kv_append(h, h, h, t, f, t, u8, u8, torch.ones(2)),
                lambda: fp8rl.kv_reserve(table, t, t, 16, [u8]), lambda: fp8rl.kv_fork(table, t, t, t, 16),
                lambda: fp8rl.kv_compact(table, t, t, 16, [u8])):
        with pytest.raises(ValueError, match="CUDA tensors"):
            one()
    with pytest.raises(ValueError, match="temperature"):
        fp8rl.sample(x, u, temperature=u)
    with pytest.raises(ValueError, match="top_k"):
        fp8rl.sample(x, u, top_k=u)
    with pytest.raises(ValueError, match="logits"):
        fp8rl.sample(x.double(), u)
    with pytest.raises(ValueError, match="one shape"):
        fp8rl.KvCaches([u8, u8[:, :128]])
    with pytest.raises(ValueError, match="uint8"):
        fp8rl.KvCaches([table])
