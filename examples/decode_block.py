"""One decoder layer's attention and a sampled vocabulary head, as a serving step runs them.

A batch of requests of different lengths, each with a block of new tokens (one when it decodes, a
prompt's or draft's piece otherwise), goes through

  q, k, v    lowbit_gemm_int4_grouped    one launch on the same activations
  append     lowbit_kv_append            rotary positions; keys and values into the paged cache
  attention  lowbit_paged_attention      the new tokens over everything cached
  o          lowbit_gemm_int4
  head       lowbit_gemm_int4            the last token of each request, all vocabulary rows
  sample     lowbit_sample               temperature, top-k, top-p, min-p from given numbers

Weights are random: what is shown is how the calls fit together.  The batch's description (cu_q,
kv_lens, block_table) lives on the device and every buffer is the caller's, so a step whose block
sizes repeat is captured once in a CUDA graph and replayed while the lengths grow.

  python examples/decode_block.py            # a prompt of 40 tokens per request, then 8 decoded
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_weight_gemv_gb300 as lb  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, VOCAB, PAGE = 2560, 32, 8, 128, 32768, 16


def int4_matrix(rows, inputs, gen):
    """A random INT4 matrix, packed."""
    codes = torch.randint(-8, 8, (rows, inputs), dtype=torch.int8, device="cuda", generator=gen)
    scales = torch.full((rows, inputs // 128), 0.006, dtype=torch.float16, device="cuda")
    packed = torch.empty(lb.lowbit_int4_packed_bytes(rows, inputs), dtype=torch.uint8, device="cuda")
    lb.lowbit_pack_int4(codes, scales, rows, inputs, packed)
    return packed


class Decoder:
    """Weights, cache and buffers for `batch` requests of up to `longest` tokens."""

    def __init__(self, batch, longest, seed=0, fp8_cache=False):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        q, kv = HEADS * DIM, KV_HEADS * DIM
        self.wq, self.wk, self.wv = (int4_matrix(n, HIDDEN, gen) for n in (q, kv, kv))
        self.wo, self.head = int4_matrix(HIDDEN, q, gen), int4_matrix(VOCAB, HIDDEN, gen)
        self.embed = torch.randn((VOCAB, HIDDEN), device="cuda", generator=gen).to(torch.bfloat16)
        rate = 1.0 / 10000.0 ** (torch.arange(0, DIM, 2, device="cuda") / DIM)
        angle = torch.arange(longest, device="cuda")[:, None] * rate
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float()
        per = -(-longest // PAGE)
        dtype = torch.float8_e4m3fn if fp8_cache else torch.bfloat16
        k, v = (torch.zeros((batch * per, KV_HEADS, PAGE, DIM), device="cuda").to(dtype).transpose(1, 2)
                for _ in range(2))
        scale = torch.full((KV_HEADS,), 1 / 32, device="cuda") if fp8_cache else None
        self.cache = lb.lowbit_paged_cache(k, v, scale, scale)
        order = torch.randperm(batch * per, device="cuda", generator=gen).to(torch.int32)
        self.block_table = order.view(batch, per)
        self.kv_lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.batch, self.gen = batch, gen

    def buffers(self, new):
        """The arrays of a step with `new` tokens per request (at most 32 in all)."""
        T, f = self.batch * new, dict(dtype=torch.bfloat16, device="cuda")
        need = lb.lowbit_paged_attention_workspace_bytes(T, self.batch, HEADS, KV_HEADS, DIM)
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(T=T, cu_q=torch.arange(0, T + 1, new, **i32), new=new,
                    tokens=torch.zeros(T, **i32), u=torch.zeros(self.batch, device="cuda"),
                    x=torch.empty((T, HIDDEN), **f), q=torch.empty((T, HEADS, DIM), **f),
                    k=torch.empty((T, KV_HEADS, DIM), **f), v=torch.empty((T, KV_HEADS, DIM), **f),
                    out=torch.empty((T, HEADS, DIM), **f), y=torch.empty((T, HIDDEN), **f),
                    last=torch.empty((self.batch, HIDDEN), **f), logits=torch.empty((self.batch, VOCAB), **f),
                    ids=torch.empty(self.batch, **i32), logprob=torch.empty(self.batch, device="cuda"),
                    workspace=torch.empty(need, dtype=torch.uint8, device="cuda"),
                    temperature=torch.full((self.batch,), 0.8, device="cuda"),
                    top_k=torch.full((self.batch,), 50, **i32),
                    top_p=torch.full((self.batch,), 0.95, device="cuda"),
                    min_p=torch.full((self.batch,), 0.02, device="cuda"))

    def step(self, s):
        """tokens -> ids: the next token of every request.  Everything stays on the stream."""
        T, q, kv = s["T"], HEADS * DIM, KV_HEADS * DIM
        self.kv_lens += s["new"]
        torch.index_select(self.embed, 0, s["tokens"], out=s["x"])
        lb.lowbit_gemm_int4_grouped([(s["x"], self.wq, q, HIDDEN, s["q"]),
                                     (s["x"], self.wk, kv, HIDDEN, s["k"]),
                                     (s["x"], self.wv, kv, HIDDEN, s["v"])], T)
        lb.lowbit_kv_append(s["q"], s["k"], s["v"], self.rope, s["cu_q"], self.kv_lens,
                            self.block_table, self.cache, s["q"])
        lb.lowbit_paged_attention(s["q"], self.cache, s["cu_q"], self.kv_lens, self.block_table,
                                  s["out"], s["workspace"])
        lb.lowbit_gemm_int4(s["out"], self.wo, T, HIDDEN, q, s["y"])
        s["last"].copy_(s["y"].view(self.batch, s["new"], HIDDEN)[:, -1])
        lb.lowbit_gemm_int4(s["last"], self.head, self.batch, VOCAB, HIDDEN, s["logits"])
        lb.lowbit_sample(s["logits"], s["u"], s["ids"], s["temperature"], s["top_k"], s["top_p"],
                         s["min_p"], logprob=s["logprob"])
        return s["ids"]


def main(batch=4, prompt=40, decode=8):
    d = Decoder(batch, prompt + decode + PAGE)
    piece = d.buffers(32 // batch)                       # the prompt, in pieces of 32 tokens in all
    tokens = torch.randint(0, VOCAB, (batch, prompt), dtype=torch.int32, device="cuda", generator=d.gen)
    for i in range(0, prompt, piece["new"]):
        piece["tokens"].copy_(tokens[:, i:i + piece["new"]].reshape(-1))
        ids = d.step(piece)
    one = d.buffers(1)
    one["tokens"].copy_(ids)
    one["u"].uniform_(generator=d.gen)
    one["tokens"].copy_(d.step(one))                     # a plain step, also the graph's warm-up
    drawn = [one["ids"].tolist()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.step(one)
    for _ in range(decode - 1):
        one["u"].uniform_(generator=d.gen)
        graph.replay()
        one["tokens"].copy_(one["ids"])
        drawn.append(one["ids"].tolist())
    if lb.lowbit_device_error():
        raise RuntimeError("a kernel recorded an error")
    return torch.tensor(drawn).T.tolist(), d.kv_lens.tolist()


if __name__ == "__main__":
    rows, lens = main()
    for b, (row, n) in enumerate(zip(rows, lens)):
        print(f"request {b}: {n} tokens cached, drew {row}")
