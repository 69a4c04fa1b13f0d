"""The token loop as a whole: prompts into reserved pages, forked for several
answers, tokens drawn, rotated, appended and attended, answers that end freed, the
rest compacted (the example rollout step, and the calls captured in one graph)."""
import importlib.util
import os
import sys

import pytest
import torch

import fp8_w8a8_rollout_gb300 as fp8rl

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("rollout_step_loop", os.path.join(ROOT, "examples", "rollout_step.py"))
    m = importlib.util.module_from_spec(spec)
    sys.modules["rollout_step_loop"] = m
    spec.loader.exec_module(m)
    return m


def test_answers_share_their_prompt(example):
    prompts, answers, new = 3, 4, 10
    r = example.run(example.Config(layers=2), prompts=prompts, new_tokens=new, seed=5, answers=answers)
    assert r["answer"].shape == (prompts * answers, new) and (r["answer"] >= 0).all()
    assert int(r["scored"].sum()) == prompts * answers * new
    assert torch.isfinite(r["lp_rollout"]).all() and (r["lp_rollout"] <= 0).all()
    # answers to one prompt differ, and their first tokens come from one row of logits
    assert len({tuple(a) for a in r["answer"].tolist()}) > prompts
    # the rollout's and the trainer's probabilities of the drawn tokens agree to well within a nat on average
    assert abs(r["kl"][0].item()) < 0.5
    c = r["cache"]
    held = torch.zeros_like(c.refs)
    for row, n in zip(c.table.tolist(), c.lens.tolist()):
        for p in row[:-(-n // c.page)]:
            held[p] += 1
    assert torch.equal(held, c.refs)
    # whole pages of a prompt stay shared by its answers
    for i in range(prompts):
        mine, whole = c.table[i * answers:(i + 1) * answers], (int(c.lens[i * answers]) - new) // c.page
        assert (mine[:, :whole] == mine[:1, :whole]).all() and (c.refs[mine[0, :whole].long()] == answers).all()
    used = c.compact()
    assert used == int((held > 0).sum()) and not c.refs[used:].any()


def test_answers_that_end_give_their_pages_back(example):
    cfg = example.Config(layers=2, vocab=128)  # (small, so that the last token comes up)
    r = example.run(cfg, prompts=4, new_tokens=24, seed=9, answers=4, eos=7, temperature=2.0)
    ended = r["going"] == 0
    assert ended.any()
    hit = r["answer"] == 7
    for row, end, h in zip(r["answer"].tolist(), ended.tolist(), hit.tolist()):
        if end:
            at = h.index(True)
            assert all(t == -1 for t in row[at + 1:])
        assert all(t >= 0 for t in row[:row.index(7) if 7 in row else len(row)])
    assert (r["lp_rollout"][r["answer"] < 0] == 0).all()
    assert int(r["scored"].sum()) == int((r["answer"] >= 0).sum())
    c = r["cache"]
    assert (c.lens[ended] == 0).all() and (c.lens[~ended] > 0).all()
    used = c.compact()
    assert used == int((c.refs > 0).sum())
    c.select(torch.full_like(c.lens, -1))
    assert not c.refs.any() and c.compact() == 0


def test_a_decode_step_in_a_graph_gives_the_eager_steps():
    """reserve, rotary_kv_append, attn_decode, sample: captured once and replayed, against the same calls made one by one."""
    rows, hq, hkv, d, page, blocks, pages, vocab = 6, 8, 2, 128, 16, 8, 64, 3001
    g = torch.Generator("cuda").manual_seed(3)
    qkv = torch.randn(rows, (hq + 2 * hkv) * d, generator=g, device="cuda").bfloat16()
    head = (torch.randn(vocab, hq * d, generator=g, device="cuda") * 0.1).bfloat16()
    freqs = fp8rl.rotary_freqs(d)
    scales = torch.full((2,), 0.01, device="cuda")
    uniforms = torch.rand(12, rows, generator=g, device="cuda", dtype=torch.float64)

    class State:
        def __init__(self):
            self.caches = [torch.zeros(pages * page, hkv * d, dtype=torch.uint8, device="cuda") for _ in range(2)]
            self.handle = fp8rl.KvCaches(self.caches)
            self.table = torch.full((rows, blocks), -1, dtype=torch.int32, device="cuda")
            self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
            self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
            cu = torch.tensor([0, 20, 20, 20, 20, 20, 20], dtype=torch.int32, device="cuda")
            slots, _ = fp8rl.kv_reserve(self.table, self.lens, self.refs, page, self.handle, cu_seqlens=cu, total_tokens=20)
            k = torch.randn(20, hkv * d, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
            fp8rl.kv_append(k, k, slots, *self.caches, scales)
            fp8rl.kv_fork(self.table, self.lens, self.refs, torch.tensor([0, 0, 0, -1, 0, 0], dtype=torch.int32, device="cuda"), page,
                          out=(self.table, self.lens))
            self.uniform = uniforms[0].clone()
            self.workspace = fp8rl.attn_decode_workspace(hq, hkv, d)

        def step(self):
            before = self.lens.clone()
            slots, info = fp8rl.kv_reserve(self.table, self.lens, self.refs, page, self.handle)
            h = qkv.view(rows, -1, d)
            q, _ = fp8rl.rotary_kv_append(h[:, :hq], h[:, hq:hq + hkv], h[:, hq + hkv:], before, freqs, slots, *self.caches, scales)
            out, _ = fp8rl.attn_decode(q, *self.caches, self.table, self.lens, scales, page, workspace=self.workspace)
            logits = out.view(rows, -1) @ head.T
            return (*fp8rl.sample(logits, self.uniform, 0.8, 20, 0.9), slots, info)

    eager, captured = State(), State()
    warm = State()
    warm.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = captured.step()
    for u in uniforms:
        eager.uniform.copy_(u)
        captured.uniform.copy_(u)
        want = eager.step()
        graph.replay()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for name in ("table", "lens", "refs"):
            assert torch.equal(getattr(eager, name), getattr(captured, name))
        assert all(torch.equal(a, b) for a, b in zip(eager.caches, captured.caches))
    assert fp8rl.fp8rl_sync_status() == 0
    assert int(eager.lens[0]) == 32 and int(eager.lens[3]) == 12
