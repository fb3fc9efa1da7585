"""A sampled verify step: several answers to one prompt, each moving on by a block of drafted tokens.

The requests share the prompt's pages.  In a step every request has its last token and a few drafts after it:

  draft      lowbit_sample               tokens drawn from a cheap drafter's rows (here the vocabulary head
                                         on the token's embedding), which are kept
  q, k, v    lowbit_gemm_int4_grouped    one launch on the same activations
  append     lowbit_kv_append_norm       a norm of each head of q and k, rotary positions; keys and values into
                                         the paged cache
  attention  lowbit_prefix_attention     the prompt's pages read once for all requests
  o, head    lowbit_gemm_int4            all rows of the block, all vocabulary rows
  verify     lowbit_verify_drafts        accepted drafts and the token that follows them, distributed as drawn
                                         from the target alone

A request's length then grows by what was accepted and one; the positions of rejected drafts are written over by
the next step.  Everything stays on the stream and has one shape, so the step is captured in a graph.

  python examples/verify_block.py            # four answers of 8 steps with up to 4 tokens each
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from decode_block import DIM, HEADS, HIDDEN, KV_HEADS, PAGE, VOCAB, int4_matrix, lb  # noqa: E402


class Answers:
    """`batch` requests behind one prompt of whole pages; blocks of `drafts` tokens and the one before them."""

    def __init__(self, batch, prompt, longest, drafts=3, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        q, kv = HEADS * DIM, KV_HEADS * DIM
        self.wq, self.wk, self.wv = (int4_matrix(n, HIDDEN, gen) for n in (q, kv, kv))
        self.wo, self.head = int4_matrix(HIDDEN, q, gen), int4_matrix(VOCAB, HIDDEN, gen)
        self.embed = torch.randn((VOCAB, HIDDEN), device="cuda", generator=gen).to(torch.bfloat16)
        self.q_weight, self.k_weight = (1 + 0.1 * torch.randn(DIM, device="cuda", generator=gen) for _ in "qk")
        rate = 1.0 / 10000.0 ** (torch.arange(0, DIM, 2, device="cuda") / DIM)
        angle = torch.arange(longest, device="cuda")[:, None] * rate
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float()
        whole, per = prompt // PAGE, -(-longest // PAGE)
        k, v = (torch.zeros((whole + batch * (per - whole), PAGE, KV_HEADS, DIM), dtype=torch.bfloat16, device="cuda")
                for _ in "kv")
        self.cache = lb.lowbit_paged_cache(k, v)
        i32 = dict(dtype=torch.int32, device="cuda")
        own = whole + torch.arange(batch * (per - whole), **i32).view(batch, per - whole)
        room = torch.zeros((batch, 4096 // PAGE), **i32)  # columns for longer answers, as a server's table has
        self.block_table = torch.cat([torch.arange(whole, **i32).expand(batch, whole), own, room], 1).contiguous()
        self.prompt, self.batch, self.drafts, self.gen = whole * PAGE, batch, drafts, gen
        self.kv_lens = torch.full((batch,), self.prompt, **i32)
        self.last = torch.zeros(batch, **i32)
        n = drafts + 1
        T, f = batch * n, dict(dtype=torch.bfloat16, device="cuda")
        self.cu_q, self.cu_drafts = torch.arange(0, T + 1, n, **i32), torch.arange(0, batch * drafts + 1, drafts, **i32)
        self.cu_groups = torch.tensor([0, batch], **i32)
        self.prefix_lens = torch.tensor([self.prompt], **i32)
        self.tokens = torch.zeros((batch, n), **i32)
        self.x, self.q = torch.empty((T, HIDDEN), **f), torch.empty((T, HEADS, DIM), **f)
        self.k, self.v = (torch.empty((T, KV_HEADS, DIM), **f) for _ in "kv")
        self.out, self.y, self.logits = torch.empty((T, HEADS, DIM), **f), torch.empty((T, HIDDEN), **f), torch.empty((T, VOCAB), **f)
        self.one, self.row = torch.empty((batch, HIDDEN), **f), torch.empty((batch, VOCAB), **f)
        self.draft_logits = torch.empty((batch, drafts, VOCAB), **f)
        self.ids, self.n_accept = torch.empty(T, **i32), torch.empty(batch, **i32)
        self.workspace = torch.empty(lb.lowbit_prefix_attention_workspace_bytes(T, batch, HEADS, KV_HEADS, DIM),
                                     dtype=torch.uint8, device="cuda")
        self.verify_workspace = torch.empty(lb.lowbit_verify_drafts_workspace_bytes(T, batch * drafts), dtype=torch.uint8,
                                            device="cuda")
        self.temperature = torch.full((batch,), 0.8, device="cuda")
        self.top_p = torch.full((batch,), 0.95, device="cuda")
        self.numbers = torch.zeros((2 * drafts + 1, batch), device="cuda")   # a step's uniform numbers

    def project(self, x, T):
        q, kv = HEADS * DIM, KV_HEADS * DIM
        lb.lowbit_gemm_int4_grouped([(x, self.wq, q, HIDDEN, self.q), (x, self.wk, kv, HIDDEN, self.k),
                                     (x, self.wv, kv, HIDDEN, self.v)], T)

    def read_prompt(self, tokens):
        """The prompt's keys and values into the shared pages, as many tokens at a time as a block has."""
        i32 = dict(dtype=torch.int32, device="cuda")
        for at in range(0, self.prompt, self.tokens.numel()):
            n = min(self.tokens.numel(), self.prompt - at)
            self.project(self.embed[tokens[at:at + n].long()].contiguous(), n)
            lb.lowbit_kv_append_norm(None, self.k[:n], self.v[:n], None, self.k_weight, 1e-6, self.rope,
                                     torch.tensor([0, n], **i32), torch.tensor([at + n], **i32), self.block_table[:1],
                                     self.cache, None)
        self.last.copy_(tokens[-1].expand(self.batch))

    def step(self):
        """Draft, verify, move on; ids and n_accept hold what became of the block."""
        d, T = self.drafts, self.batch * (self.drafts + 1)
        self.tokens[:, 0] = self.last
        for i in range(d):
            torch.index_select(self.embed, 0, self.tokens[:, i].contiguous(), out=self.one)
            lb.lowbit_gemm_int4(self.one, self.head, self.batch, VOCAB, HIDDEN, self.row)
            self.draft_logits[:, i] = self.row
            drawn = torch.empty(self.batch, dtype=torch.int32, device="cuda")
            lb.lowbit_sample(self.row, self.numbers[i], drawn, self.temperature)
            self.tokens[:, i + 1] = drawn
        self.kv_lens += d + 1
        torch.index_select(self.embed, 0, self.tokens.view(-1), out=self.x)
        self.project(self.x, T)
        lb.lowbit_kv_append_norm(self.q, self.k, self.v, self.q_weight, self.k_weight, 1e-6, self.rope, self.cu_q,
                                 self.kv_lens, self.block_table, self.cache, self.q)
        lb.lowbit_prefix_attention(self.q, self.cache, self.cu_q, self.kv_lens, self.block_table, self.cu_groups,
                                   self.prefix_lens, self.out, self.workspace)
        lb.lowbit_gemm_int4(self.out, self.wo, T, HIDDEN, HEADS * DIM, self.y)
        self.y += self.x
        lb.lowbit_gemm_int4(self.y, self.head, T, VOCAB, HIDDEN, self.logits)
        lb.lowbit_verify_drafts(self.logits, self.cu_drafts, self.tokens[:, 1:].reshape(-1),
                                self.numbers[d:2 * d].t().reshape(-1), self.numbers[2 * d], self.n_accept, self.ids,
                                self.verify_workspace, draft_logits=self.draft_logits.view(-1, VOCAB),
                                temperature=self.temperature, top_p=self.top_p, draft_temperature=self.temperature)
        self.kv_lens += self.n_accept - d
        at = self.cu_q[:-1] + self.n_accept
        self.last.copy_(self.ids[at.long()])


def main(batch=4, prompt=64, steps=8, drafts=3):
    a = Answers(batch, prompt, prompt + steps * (drafts + 1) + PAGE, drafts)
    a.read_prompt(torch.randint(0, VOCAB, (a.prompt,), dtype=torch.int32, device="cuda", generator=a.gen))
    answers = [[] for _ in range(batch)]

    def keep():
        for b, row in enumerate(a.ids.view(batch, -1).tolist()):
            answers[b] += [t for t in row if t >= 0]

    a.numbers.uniform_(generator=a.gen)
    a.step()                                             # a plain step, also the graph's warm-up
    keep()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step()
    for _ in range(steps - 1):
        a.numbers.uniform_(generator=a.gen)
        graph.replay()
        keep()
    if lb.lowbit_device_error():
        raise RuntimeError("a kernel recorded an error")
    return answers, a.kv_lens.tolist()


if __name__ == "__main__":
    for b, (row, n) in enumerate(zip(*main())):
        print(f"answer {b}: {n} tokens cached, drew {row}")
