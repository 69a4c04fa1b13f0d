"""The norm, attention and log-probability kernels launch before the kernel in
front of them has finished and wait for it: a chain of them, each reading what
the one before wrote, from buffers poisoned before every pass, gives the same
bits with the overlap, without it (test hook 13), and replayed from a graph."""
import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    fp8rl.load_library(build_if_missing=True)


@pytest.mark.parametrize("tokens", [7, 200, 1500])
def test_chain(tokens):
    hq, hkv, d, hidden, vocab = 8, 2, 128, 1024, 4096
    g = torch.Generator("cuda").manual_seed(tokens)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").bfloat16()

    x, res, w = normal(tokens, hidden), normal(tokens, hidden), normal(hidden)
    wqkv, wo, head = (fp8rl.quant_weight(normal(n, k) * k ** -0.5) for n, k in
                      (((hq + 2 * hkv) * d, hidden), (hidden, hq * d), (vocab, hidden)))
    ends = torch.tensor([0, tokens // 3, tokens], dtype=torch.int32, device="cuda")
    plan = fp8rl.attn_prefill_plan(ends, tokens, hq, hkv)
    pages = -(-tokens // 16)
    table = torch.randperm(pages, generator=g, device="cuda").int()[None]
    pos = torch.arange(tokens, device="cuda")
    slots = (table[0, pos // 16] * 16 + pos % 16).int()
    kc, vc = (torch.empty(pages * 16, hkv * d, dtype=torch.uint8, device="cuda") for _ in range(2))
    scales = torch.tensor([0.02, 0.02], device="cuda")
    length = torch.tensor([tokens], dtype=torch.int32, device="cuda")
    ws = fp8rl.attn_decode_workspace(hq, hkv, d)
    target = torch.randint(0, vocab, (tokens,), generator=g, device="cuda").int()
    gl, ge = torch.randn(tokens, generator=g, device="cuda"), torch.randn(tokens, generator=g, device="cuda")

    def out(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    f32, u8 = torch.float32, torch.uint8
    n1 = (out(tokens, hidden, dtype=u8), out(hidden // 128, tokens, dtype=f32), out(tokens, hidden))
    qkv = out(tokens, (hq + 2 * hkv) * d)
    att = (out(tokens, hq, d), out(tokens, hq, dtype=f32))
    one = (out(1, hq, d), out(1, hq, dtype=f32))
    o = out(tokens, hidden)
    n2 = (out(tokens, hidden, dtype=u8), out(hidden // 128, tokens, dtype=f32), out(tokens, hidden))
    logits = out(tokens, vocab)
    lp = (out(tokens, dtype=f32), out(tokens, dtype=f32), out(tokens, 2, dtype=f32), out(tokens, 4, dtype=torch.int32), out(tokens, 4, dtype=f32))
    grad = out(tokens, vocab)
    buffers = [*n1, qkv, *att, *one, o, *n2, logits, *lp, grad, kc, vc]

    def chain():
        fp8rl.rmsnorm_quant(x, w, res, out=n1)
        fp8rl.gemm(n1[0], n1[1], *wqkv, out=qkv)
        h = qkv.view(tokens, hq + 2 * hkv, d)
        q, k, v = h[:, :hq], h[:, hq:hq + hkv], h[:, hq + hkv:]
        fp8rl.kv_append(qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:], slots, kc, vc, scales)
        fp8rl.attn_decode(q[-1:], kc, vc, table, length, scales, 16, workspace=ws, out=one)
        fp8rl.attn_prefill(q, k, v, plan, out=att)
        fp8rl.gemm_act_quant(att[0].view(tokens, hq * d), *wo, out=o)
        fp8rl.rmsnorm_quant(o, w, n1[2], out=n2)
        fp8rl.gemm(n2[0], n2[1], *head, out=logits)
        fp8rl.logprobs(logits, target, topk=4, out=lp)
        fp8rl.logprobs_backward(logits, target, lp[2], lp[1], gl, ge, out=grad)

    def poisoned(run):
        for b in buffers:
            b.view(torch.uint8).fill_(0x5A)
        torch.cuda.synchronize()
        run()
        assert fp8rl.fp8rl_sync_status() == 0
        return [b.clone() for b in buffers]

    want = poisoned(chain)
    try:
        fp8rl.fp8rl_debug_set(fp8rl.DEBUG_PDL, 1)
        serial = poisoned(chain)
    finally:
        fp8rl.fp8rl_debug_set(fp8rl.DEBUG_RESET, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    runs = [serial, poisoned(graph.replay), poisoned(graph.replay), poisoned(chain)]
    for got in runs:
        for a, b in zip(want, got):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
