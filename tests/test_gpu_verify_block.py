"""The append, attention and verify calls of a sampled verify step together, as examples/verify_block.py makes them."""
import os
import sys

import numpy as np
import pytest

from oracle import paged

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import verify_block
    verify_block.lb.lowbit_device_error()
    yield verify_block
    assert verify_block.lb.lowbit_device_error() == 0


def test_it_runs(example):
    answers, lens = example.main(batch=3, prompt=48, steps=5, drafts=3)
    for row, n in zip(answers, lens):
        assert 5 <= len(row) <= 20 and n == 48 + len(row)
        assert all(0 <= t < example.VOCAB for t in row)


def start(example, seed=0):
    a = example.Answers(4, 80, 160, 3, seed)
    a.read_prompt(torch.randint(0, example.VOCAB, (a.prompt,), dtype=torch.int32, device="cuda", generator=a.gen))
    return a


def test_replayed_steps_are_the_plain_ones(example):
    a, b = start(example), start(example)
    for x in (a, b):
        x.numbers.fill_(0.4)
        x.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for u in (0.1, 0.73, 0.99):
        for x in (a, b):
            x.numbers.copy_(((torch.arange(x.numbers.numel(), device="cuda") * 0.377 + u) % 1).view_as(x.numbers))
        a.step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.ids, b.ids) and torch.equal(a.kv_lens, b.kv_lens) and torch.equal(a.last, b.last)
        assert torch.equal(a.logits.view(torch.int16), b.logits.view(torch.int16))


def test_every_part_against_its_oracle(example):
    from test_gpu_append_norm import within
    from test_gpu_verify_drafts import Case, plain
    a = start(example)
    for s in range(2):
        a.numbers.uniform_(generator=a.gen)
        before = a.kv_lens.clone()
        raw = []
        project = a.project

        def watched(x, T):
            project(x, T)
            raw.append([t.clone() for t in (a.q, a.k)])

        a.project = watched
        a.step()
        a.project = project
        torch.cuda.synchronize()
        lens = (before + 4).tolist()
        pos = np.concatenate([np.arange(n - 4, n) for n in lens])
        rows = a.rope.cpu().numpy()[pos]
        for x, weight, got in ((raw[0][0], a.q_weight, a.q), (raw[0][1], a.k_weight, None)):
            y = paged.normalise(x.double().cpu().numpy(), weight.cpu().numpy(), 1e-6)
            y, size = paged.rotate64(y, rows, False)
            if got is None:
                table = a.block_table.cpu().numpy()
                got = torch.stack([a.cache.k[table[t // 4][p // 16], p % 16] for t, p in enumerate(pos)])
            within(got, y, size)
        for b in range(4):
            k, v = (paged.gather(c.double().cpu().numpy(), a.block_table[b].cpu().numpy(), lens[b], 16) for c in (a.cache.k, a.cache.v))
            want, _, spread = paged.attention(a.q[4 * b:4 * b + 4].double().cpu().numpy(), k, v, paged.visible(4, lens[b], True, 0),
                                              128 ** -0.5)
            got = a.out[4 * b:4 * b + 4].double().cpu().numpy()
            # as in test_gpu_paged.py: weights and outputs rounded to bf16 once, fp32 scores
            assert (np.abs(got - want) <= 1.05 * (2.0 ** -8 * (spread + np.abs(want)) + 1e-4 * spread) + 1e-30).all()
        c = Case.__new__(Case)
        c.cu, c.z, c.y, c.index = np.arange(5) * 3, a.logits, a.draft_logits.view(-1, example.VOCAB), None
        f = np.float32
        c.settings = [(float(f(0.8)), 0, float(f(0.95)), 0.0)] * 4
        c.draft_settings = [(float(f(0.8)), 0, 1.0, 0.0)] * 4
        c.drafts, c.u, c.v = a.tokens[:, 1:].reshape(-1), a.numbers[3:6].t().reshape(-1).cpu().numpy(), a.numbers[6].cpu().numpy()
        for b in range(4):
            n, tokens, _ = plain(c, b)
            assert (int(a.n_accept[b]), a.ids[4 * b:4 * b + 4].tolist()) == (n, tokens)
            assert int(a.kv_lens[b]) == int(before[b]) + n + 1 and int(a.last[b]) == tokens[n]
