"""Operators of a sampled verify step over a shared context, as cases to be timed and compared.

Three operators next to the paged append, attention and sampling calls, in the order of a step that
verifies drafted tokens of many requests at a temperature:

  append     queries and keys normalised head by head (root mean square, a weight per element), rotary
             positions on both, and keys and values written into a paged cache
             (lowbit_kv_append_norm);
  attention  the new tokens of requests whose first pages are the same ones: the shared pages are read
             once for all of them (lowbit_prefix_attention);
  verify     drafted tokens accepted or rejected against the target's probabilities from given uniform
             numbers, and the token that follows them (lowbit_verify_drafts).

`own` chooses between the plain form of each (elementary torch operations in 32 bits) and the
library's calls.  Heads of 128 with 32 query and 8 key/value heads are the 4B-class decoder
layer's q, k and v widths (4096 and 1024); 248,320 and 32,768 rows are the full and trimmed
vocabularies; 16 rows are one draft block: 15 drafted tokens and the one before them.
"""
import math
import random

import numpy as np
import torch

own = False

FIXED = 2.0 ** 40      # a probability or a sampling weight of 1 in whole numbers


def listed():
    return [
        # One token of one request: the append between two small launches of a decode step.
        dict(name="norm_append_one", op="append", batch=1, new=1, max_kv=4000, heads=32, kv_heads=8,
             dim=128, page=64, order="head", cache="bf16", rot=128, pairs="half", ragged=0),
        # 32 requests verifying a draft block each, cache in 8 bits with a scale per head.
        dict(name="norm_append_verify_fp8", op="append", batch=32, new=16, max_kv=4100, heads=32,
             kv_heads=8, dim=128, page=16, order="head", cache="fp8", rot=128, pairs="half",
             ragged=1),
        # Two prompts' chunks with wide heads, rotary on the first quarter of each, adjacent pairs.
        dict(name="norm_append_wide", op="append", batch=2, new=1111, max_kv=5001, heads=16,
             kv_heads=4, dim=256, page=64, order="token", cache="bf16", rot=64, pairs="adjacent",
             ragged=1),
        # Four prompts' chunks at once: bound by memory.
        dict(name="norm_append_prompt", op="append", batch=4, new=4099, max_kv=9001, heads=32,
             kv_heads=8, dim=128, page=64, order="token", cache="bf16", rot=128, pairs="half",
             ragged=0),
        # Eight answers sampled from one prompt, one token each: latency.
        dict(name="prefix_samples", op="attention", batch=8, groups=1, new=1, prefix=4001, own=300,
             heads=32, kv_heads=8, dim=128, page=64, order="head", cache="bf16", causal=True,
             ragged=0),
        # A decode batch behind one long system prompt, cache in 8 bits, own contexts of all lengths.
        dict(name="prefix_decode_fp8", op="attention", batch=64, groups=1, new=1, prefix=16384,
             own=2000, heads=32, kv_heads=8, dim=128, page=16, order="head", cache="fp8",
             causal=True, ragged=1),
        # Draft blocks of four system prompts' requests being verified, some slots idle.
        dict(name="prefix_verify", op="attention", batch=48, groups=4, new=16, prefix=20000,
             own=1500, heads=32, kv_heads=8, dim=128, page=64, order="token", cache="bf16",
             causal=True, ragged=1),
        # Questions of several hundred tokens about one long document: bound by arithmetic.
        dict(name="prefix_chunks", op="attention", batch=6, groups=1, new=701, prefix=12345, own=64,
             heads=32, kv_heads=8, dim=128, page=64, order="head", cache="bf16", causal=True,
             ragged=1),
        # One request's block from a drafter that proposes its likeliest tokens; usual truncation.
        dict(name="verify_one", op="verify", batch=1, drafts=15, vocab=248320, draft_vocab=0,
             type="fp32", mix=0, ragged=0),
        # Four requests, the drafter's own distribution over the full vocabulary, temperature alone.
        dict(name="verify_full_bf16", op="verify", batch=4, drafts=7, vocab=248320,
             draft_vocab=248320, type="bf16", mix=2, ragged=0),
        # Nine requests with a trimmed draft head, some with few drafts or none, settings of all kinds.
        dict(name="verify_trimmed", op="verify", batch=9, drafts=15, vocab=248320,
             draft_vocab=32768, type="bf16", mix=1, ragged=1),
        # A large batch with the trimmed head.
        dict(name="verify_batch", op="verify", batch=32, drafts=15, vocab=248320, draft_vocab=32768,
             type="fp32", mix=1, ragged=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "attention", "attention", "verify"))
    if op == "verify":
        batch = _log(rng, 1, 24)
        vocab = _log(rng, 1000, 248320)
        return dict(op=op, batch=batch, drafts=rng.randint(0, 15), vocab=vocab,
                    draft_vocab=rng.choice((0, vocab, _log(rng, 500, vocab))),
                    type=rng.choice(("fp32", "bf16")), mix=rng.choice((0, 1, 1, 2)),
                    ragged=rng.choice((0, 1)))
    kv_heads = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 4, 4, 5, 8) if kv_heads < 8 else (1, 2, 4, 4))
    case = dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, page=rng.choice((16, 32, 64, 128)),
                order=rng.choice(("head", "token")), cache=rng.choice(("bf16", "bf16", "fp8")),
                ragged=rng.choice((0, 1, 1)))
    if op == "append":
        batch = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 12000 // batch))
        dim = rng.choice((64, 128, 128, 256))
        case |= dict(batch=batch, new=new, max_kv=new + _log(rng, 1, 4000), dim=dim,
                     rot=rng.choice((dim, dim, dim // 2)), pairs=rng.choice(("half", "half", "adjacent")))
        return case
    batch = _log(rng, 2, 48)
    case |= dict(batch=batch, groups=rng.choice((1, 1, 2, max(1, batch // 4))),
                 dim=rng.choice((64, 128, 128)), causal=rng.choice((True, True, True, False)),
                 prefix=_log(rng, 100, 20000))
    if rng.random() < 0.25:       # prompts' chunks
        case |= dict(new=_log(rng, 40, max(41, 2400 // batch)), own=_log(rng, 1, 500))
    else:                         # decoding and draft blocks
        case |= dict(new=rng.choice((1, 1, 4, 8, 16, 16, 31)), own=_log(rng, 1, 2500))
    case["groups"] = min(case["groups"], batch)
    return case


def _lengths(case):
    """New tokens and whole length of every request, groups' bounds and their shared lengths: plain
    lists, the same for every seed."""
    B, new = case["batch"], case["new"]
    shared = case["op"] == "attention"
    r = random.Random(B * 1000003 + new * 1009 + (case["prefix"] if shared else case["max_kv"]))
    news, kvs, bounds, prefix = [], [], [0, B], [0]
    if shared:
        g = case["groups"]
        bounds = [0] + sorted(r.sample(range(1, B), g - 1)) + [B]
        prefix = [case["prefix"] if i == 0 or not case["ragged"]
                  else r.randint(max(1, case["prefix"] // 4), case["prefix"]) for i in range(g)]
    for b in range(B):
        n = new if new <= 31 or not case["ragged"] else r.randint(max(1, new // 4), new)
        if case["ragged"] and B > 4 and b % 7 == 5:
            n = 0                 # an idle slot of the batch
        if shared:
            of = sum(b >= x for x in bounds[1:])
            mine = case["own"] if not case["ragged"] else int(math.exp(r.uniform(0.0, math.log(case["own"] + 1))))
            kvs.append(prefix[of] + n + mine)
        else:
            top = case["max_kv"]
            kv = top if b == 0 or not case["ragged"] else min(top, n + int(math.exp(r.uniform(0.0, math.log(top + 1)))))
            kvs.append(max(kv, n, 1))
        news.append(n)
    return news, kvs, bounds, prefix


def _rows(case):
    """Drafted tokens of every request."""
    r = random.Random(case["batch"] * 7919 + case["drafts"])
    return [r.randint(0, case["drafts"]) if case["ragged"] else case["drafts"] for _ in range(case["batch"])]


def _cache(case, gen, pages):
    """Key and value pages [pages][page][kv_heads][dim] in the case's order and type."""
    H, D, ps = case["kv_heads"], case["dim"], case["page"]
    shape = (pages, ps, H, D) if case["order"] == "token" else (pages, H, ps, D)
    out = []
    for _ in range(2):
        t = torch.randn(shape, device="cuda", generator=gen)
        if case["cache"] == "fp8":
            t = (t * 32).clamp(-448, 448).to(torch.float8_e4m3fn)
        else:
            t = t.to(torch.bfloat16)
        out.append(t if case["order"] == "token" else t.transpose(1, 2))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 40) + 29)
    if case["op"] == "verify":
        return _prepare_verify(case, seed, gen)
    news, kvs, bounds, prefix = _lengths(case)
    B, Hq, Hk, D, ps = case["batch"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    T = sum(news)
    need = [-(-kv // ps) for kv in kvs]
    shared = [p // ps for p in prefix]           # whole pages only are shared
    group = [sum(b >= x for x in bounds[1:-1]) for b in range(B)]
    width = max(need) + 1
    pages = sum(n - shared[g] for n, g in zip(need, group)) + sum(shared) + 3
    order = np.random.RandomState(int(seed) % (1 << 31)).permutation(pages)
    table = np.zeros((B, width), dtype=np.int32)
    at = 0
    common = []
    for n in shared:
        common.append(order[at:at + n])
        at += n
    for b in range(B):
        n = need[b] - shared[group[b]]
        table[b, :need[b]] = np.concatenate([common[group[b]], order[at:at + n]])
        at += n
    k, v = _cache(case, gen, pages)
    dev = dict(device="cuda", dtype=torch.int32)
    s = dict(op=case["op"], case=case, T=T, k_cache=k, v_cache=v, news=news, kvs=kvs, bounds=bounds,
             shared=shared, block_table=torch.from_numpy(table).cuda(),
             cu_q=torch.tensor(np.concatenate([[0], np.cumsum(news)]), **dev),
             kv_lens=torch.tensor(kvs, **dev), k_scale=None, v_scale=None)
    if case["cache"] == "fp8":
        s["k_scale"] = torch.linspace(0.9, 1.3, Hk, device="cuda") / 32
        s["v_scale"] = torch.linspace(1.2, 0.8, Hk, device="cuda") / 32
    if case["op"] == "append":
        # q, k and v as the three products leave them side by side: rows of one buffer.
        qkv = 3.0 * torch.randn((T, (Hq + 2 * Hk) * D), device="cuda", generator=gen)
        qkv[:, :: 131] *= 20.0    # channels that stick out
        qkv = qkv.to(torch.bfloat16)
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["v"] = qkv[:, (Hq + Hk) * D:].view(T, Hk, D)
        s["q_weight"], s["k_weight"] = (
            (1.0 + 0.3 * torch.randn((D,), device="cuda", generator=gen)).to(torch.bfloat16).float()
            for _ in range(2))
        s["eps"] = 1e-6
        R = case["rot"]
        rate = 1.0 / (1000000.0 ** (torch.arange(0, R, 2, dtype=torch.float64) / R))
        angle = torch.arange(max(kvs) + 1, dtype=torch.float64)[:, None] * rate[None, :]
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        s["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    else:
        for c in (k, v):          # what a page holds past its request's end was never written
            flat = c if c.dtype == torch.bfloat16 else c.view(torch.uint8)
            for b in range(B):
                tail = need[b] * ps - kvs[b]
                if tail and need[b] > shared[group[b]]:
                    flat[int(table[b, need[b] - 1]), ps - tail:] = (
                        float("nan") if c.dtype == torch.bfloat16 else 0x7F)
        # scores of standard deviation 1.5: some rows attend to few positions, some to many
        s["q"] = (1.5 * torch.randn((T, Hq, D), device="cuda", generator=gen)).to(torch.bfloat16)
        s["out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device="cuda")
        s["scale"] = D ** -0.5
        s["cu_groups"] = torch.tensor(bounds, **dev)
        s["prefix_lens"] = torch.tensor(prefix, **dev)
    if own:
        import bit_weight_gemv_gb300 as lb
        s["cache"] = lb.lowbit_paged_cache(k, v, s["k_scale"], s["v_scale"])
        if case["op"] == "attention":
            need_bytes = lb.lowbit_prefix_attention_workspace_bytes(T, B, Hq, Hk, D)
            s["workspace"] = torch.zeros(need_bytes, dtype=torch.uint8, device="cuda")
    return s


def _prepare_verify(case, seed, gen):
    B, V, Vd = case["batch"], case["vocab"], case["draft_vocab"]
    n = _rows(case)
    N, M = sum(n), sum(n) + B
    # a broad body of unlikely tokens and a few likely ones, as a language model's rows have
    z = 2.2 * torch.randn((M, V), device="cuda", generator=gen)
    some = torch.randperm(V, device="cuda", generator=gen)[:Vd or V]      # the trimmed vocabulary
    hot = some[torch.randint(0, some.numel(), (M, 24), device="cuda", generator=gen)]
    hot[:, 20:] = torch.randint(0, V, (M, 4), device="cuda", generator=gen)
    lift = 12.0 + 2.0 * torch.randn((M, 24), device="cuda", generator=gen)
    z.scatter_(1, hot, lift)
    r = random.Random(int(seed) * 7919 + M * 31 + V)
    temp, top_k, top_p, min_p = [], [], [], []
    for b in range(B):
        if case["mix"] != 1:
            temp.append(0.7 if case["mix"] == 0 else r.uniform(0.6, 1.1))
            top_k.append(20 if case["mix"] == 0 else 0)
            top_p.append(0.95 if case["mix"] == 0 else 1.0)
            min_p.append(0.0)
            continue
        kind = (b + int(seed)) % 6
        temp.append(0.0 if kind == 4 else r.uniform(0.3, 1.3))
        top_k.append(0 if kind in (1, 3) else int(math.exp(r.uniform(0, math.log(2000)))))
        top_p.append(1.0 if kind in (2, 3) else r.uniform(0.5, 0.99))
        min_p.append(r.uniform(0.005, 0.1) if kind in (0, 3) else 0.0)
    f, i = dict(device="cuda", dtype=torch.float32), dict(device="cuda", dtype=torch.int32)
    cu = np.concatenate([[0], np.cumsum(n)])
    # target rows that judge a draft: every row of a request but its last
    judge = torch.tensor([int(cu[b]) + b + j for b in range(B) for j in range(n[b])], device="cuda",
                         dtype=torch.int64)
    s = dict(op="verify", case=case, logits=z.to(torch.bfloat16) if case["type"] == "bf16" else z,
             cu_drafts=torch.tensor(cu, **i), u=torch.rand((N,), device="cuda", generator=gen),
             v=torch.rand((B,), device="cuda", generator=gen), temperature=torch.tensor(temp, **f),
             top_k=torch.tensor(top_k, **i), top_p=torch.tensor(top_p, **f),
             min_p=torch.tensor(min_p, **f), draft_logits=None, draft_index=None,
             draft_temperature=None, n_accept=torch.empty((B,), **i), ids=torch.empty((M,), **i),
             accept=torch.empty((N,), **f))
    # the drafter's logits: the target's with noise, over the trimmed vocabulary where there is one
    near = (z[judge][:, some] if Vd and Vd < V else z[judge]) if N else z[:0]
    near = 0.9 * near + 0.8 * torch.randn(near.shape, device="cuda", generator=gen)
    if not Vd:                    # it proposes its likeliest token, and gives no distribution
        s["drafts"] = near.argmax(1).to(torch.int32)
    else:
        near = near.to(torch.bfloat16) if case["type"] == "bf16" else near
        of = [b for b in range(B) for _ in range(n[b])]
        td = torch.tensor([max(temp[b], 0.3) for b in range(B)], **f)
        p = torch.softmax(near.float() / td[of][:, None], 1)
        col = torch.multinomial(p, 1, generator=gen)[:, 0] if N else torch.zeros((0,), device="cuda", dtype=torch.int64)
        s["draft_logits"], s["draft_temperature"] = near, td
        s["drafts"] = col.to(torch.int32)
        if Vd < V:
            s["drafts"] = some[col].to(torch.int32)
            s["draft_index"] = torch.full((V,), -1, **i)
            s["draft_index"][some] = torch.arange(Vd, **i)
    if own:
        import bit_weight_gemv_gb300 as lb
        s["workspace"] = torch.zeros(lb.lowbit_verify_drafts_workspace_bytes(M, N), dtype=torch.uint8,
                                     device="cuda")
    return s


# --------------------------------------------------------------------------------------------
# One pass


def run(s):
    if s["op"] == "append":
        return _run_append(s)
    if s["op"] == "attention":
        return _run_attention(s)
    return _run_verify(s)


def _run_append(s):
    if own:
        import bit_weight_gemv_gb300 as lb
        lb.lowbit_kv_append_norm(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["eps"],
                                 s["rope"], s["cu_q"], s["kv_lens"], s["block_table"], s["cache"],
                                 s["q_out"], interleaved=s["case"]["pairs"] == "adjacent")
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    case, T, ps = s["case"], s["T"], s["case"]["page"]
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = kv[b] - cu[b + 1] + t
    page = s["block_table"][b, pos // ps].long()

    def normed(x, weight):
        x = x.float()
        return x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"])) * weight

    q = _rotate(normed(s["q"], s["q_weight"]), s["rope"][pos], case)
    k = _rotate(normed(s["k"], s["k_weight"]), s["rope"][pos], case)
    v = s["v"].float()
    s["q_out"].copy_(q)
    for x, scale, cache in ((k, s["k_scale"], s["k_cache"]), (v, s["v_scale"], s["v_cache"])):
        if scale is None:
            cache[page, pos % ps] = x.to(cache.dtype)
        else:
            x = (x / scale[None, :, None]).clamp(-448, 448).to(cache.dtype)
            cache.view(torch.uint8)[page, pos % ps] = x.view(torch.uint8)
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _rotate(x, row, case):
    R = case["rot"]
    c, sn = row[:, None, :R // 2], row[:, None, R // 2:]
    if case["pairs"] == "half":
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    else:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    return torch.cat([y, x[..., R:]], -1)


def _run_attention(s):
    case = s["case"]
    if own:
        import bit_weight_gemv_gb300 as lb
        lb.lowbit_prefix_attention(s["q"], s["cache"], s["cu_q"], s["kv_lens"], s["block_table"],
                                   s["cu_groups"], s["prefix_lens"], s["out"], s["workspace"],
                                   scale=s["scale"], causal=case["causal"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    Hq, Hk, D, ps = case["heads"], case["kv_heads"], case["dim"], case["page"]
    G = Hq // Hk

    def read(c, scale, pages):
        """Keys or values [..., Hk, keys, D] of pages [..., n], in 32 bits."""
        if c.dtype == torch.bfloat16:
            x = c[pages].float()
        else:
            x = c.view(torch.uint8)[pages].view(c.dtype).float() * scale[:, None]
        return x.flatten(-4, -3).transpose(-3, -2)

    # group by group: the shared keys once for all rows, and every request's own keys, padded
    news, kvs, bounds, table = s["news"], s["kvs"], s["bounds"], s["block_table"].long()
    cu = np.concatenate([[0], np.cumsum(news)]).tolist()
    for g, P in enumerate(s["shared"]):
        b0, b1 = bounds[g], bounds[g + 1]
        t0, t1 = cu[b0], cu[b1]
        if t1 == t0:
            continue
        B, n, skip = b1 - b0, max(news[b0:b1]), P * ps
        L = -(-(max(kvs[b0:b1]) - skip) // ps) * ps
        first, kv, new = (torch.tensor(x, device="cuda") for x in (cu[b0:b1], kvs[b0:b1], news[b0:b1]))
        i, j = torch.arange(n, device="cuda"), torch.arange(L, device="cuda") + skip
        pos = (kv - new)[:, None] + i[None, :]                              # [B][n]
        see = (j[None, None, :] < kv[:, None, None]) & (i[None, :] < new[:, None])[:, :, None]
        if case["causal"]:
            see = see & (j[None, None, :] <= pos[:, :, None])
        # own part: [B][Hk][n G][...]
        at = (first[:, None] + i[None, :]).clamp(max=t1 - 1)
        q = s["q"][at].float().view(B, n, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, D)
        mine = table[b0:b1, P:P + L // ps]
        x = torch.matmul(q, read(s["k_cache"], s["k_scale"], mine).transpose(2, 3)) * s["scale"]
        x = x.view(B, Hk, n, G, L).masked_fill_(~see[:, None, :, None, :], float("-inf"))
        top = x.amax(-1, keepdim=True)
        # shared part: the group's rows side by side, [Hk][Tg G][...]
        if P:
            qs = s["q"][t0:t1].float().view(t1 - t0, Hk, G, D).transpose(0, 1).reshape(Hk, -1, D)
            xs = torch.matmul(qs, read(s["k_cache"], s["k_scale"], table[b0, :P]).transpose(1, 2)) * s["scale"]
            tops = xs.amax(-1, keepdim=True)
            ps_ = xs.sub_(tops).exp_()
            sums = ps_.sum(-1, keepdim=True)
            ys = torch.matmul(ps_, read(s["v_cache"], s["v_scale"], table[b0, :P]))
        top = torch.where(torch.isfinite(top), top, -3e38)
        p = x.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        vals = read(s["v_cache"], s["v_scale"], mine)
        vals = torch.where(see.any(1)[:, None, :, None], vals, 0.0)
        y = torch.matmul(p.view(B, Hk, n * G, L), vals).view(B, Hk, n, G, D)
        # both together, row by row: [Tg][Hk][G][...]
        t = torch.arange(t0, t1, device="cuda")
        of = torch.searchsorted(first, t, right=True) - 1
        pick = lambda a: a.permute(0, 2, 1, 3, 4)[of, t - first[of]]
        top, total, y = pick(top), pick(total), pick(y)
        if P:
            turn = lambda a: a.view(Hk, t1 - t0, G, -1).transpose(0, 1)
            tops, sums, ys = turn(tops), turn(sums), turn(ys)
            both = torch.maximum(top, tops)
            a, b = (top - both).exp(), (tops - both).exp()
            top, total, y = both, total * a + sums * b, y * a + ys * b
        y = y / torch.where(total > 0, total, 1.0)
        s["out"][t0:t1] = y.reshape(t1 - t0, Hq, D).to(torch.bfloat16)
        s["lse"][t0:t1] = (top + total.log()).reshape(t1 - t0, Hq)
    return {"out": s["out"], "lse": s["lse"]}


def _kept(z, temp, top_k=None, top_p=None, min_p=None):
    """Weights in 32 bits relative to the row's largest, and of those that the settings leave the masses
    in whole numbers, with their sums: the definition of lowbit_sample."""
    V = z.shape[1]
    z = torch.where(torch.isnan(z), float("-inf"), z.float()).clamp(max=torch.finfo(torch.float32).max)
    top = z.amax(1, keepdim=True)
    temp = temp[:, None]
    greedy = ~(temp >= 1e-6)
    rate = 1.0 / torch.where(greedy, 1.0, temp.clamp(max=1e6))
    w = torch.where(z == float("-inf"), 0.0, torch.exp((z - top) * rate))
    mass = (w * FIXED).round().to(torch.int64)
    if top_k is None and top_p is None and min_p is None:
        return w, mass, mass.sum(1)
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    m = mass.gather(1, order)
    rank = torch.arange(V, device="cuda")[None, :]
    k = top_k.long()[:, None]
    k = torch.where((k <= 0) | (k > V), V, k)
    k = torch.where(greedy, 1, k)
    m = torch.where(rank < k, m, 0)
    total = m.sum(1, keepdim=True)
    p = top_p[:, None]
    limit = (p.double() * total.double()).ceil().to(torch.int64).clamp(min=1)
    limit = torch.where(p >= 1.0, total, limit)
    m = torch.where(m.cumsum(1) - m < limit, m, 0)
    keep = torch.zeros_like(mass).scatter(1, order, m)
    keep = torch.where(w >= min_p[:, None], keep, 0)
    return torch.where(keep > 0, w, 0.0), keep, keep.sum(1)


def _run_verify(s):
    if own:
        import bit_weight_gemv_gb300 as lb
        lb.lowbit_verify_drafts(s["logits"], s["cu_drafts"], s["drafts"], s["u"], s["v"], s["n_accept"],
                                s["ids"], s["workspace"], draft_logits=s["draft_logits"],
                                draft_index=s["draft_index"], temperature=s["temperature"],
                                top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                                draft_temperature=s["draft_temperature"], accept=s["accept"])
        return {"n_accept": s["n_accept"], "ids": s["ids"], "accept": s["accept"]}
    M, V = s["logits"].shape
    B, N = s["v"].numel(), s["u"].numel()
    cu = s["cu_drafts"].long()
    n = cu[1:] - cu[:-1]
    req = torch.arange(B, device="cuda")
    # the request of a draft and of a target row; request b has rows cu[b] + b to cu[b + 1] + b
    of = torch.searchsorted(cu[1:].contiguous(), torch.arange(N, device="cuda"), right=True)
    row_of = torch.searchsorted(cu[1:] + req, torch.arange(M, device="cuda"))
    trunc = [s[x][row_of] for x in ("top_k", "top_p", "min_p")] if s["case"]["mix"] != 2 else [None] * 3
    w, mass, total = _kept(s["logits"], s["temperature"][row_of], *trunc)
    row = torch.arange(N, device="cuda") + of                     # the row that judges a draft
    d = s["drafts"].long()
    share = mass[row, d].double() / total[row].clamp(min=1).double()
    index = s["draft_index"]
    if s["draft_logits"] is not None:
        wq, mq, sq = _kept(s["draft_logits"], s["draft_temperature"][of])
        col = d if index is None else index[d].long()
        given = torch.where(col >= 0, mq.gather(1, col.clamp(min=0)[:, None])[:, 0], 0)
        given = given.double() / sq.clamp(min=1).double()
    else:
        given = torch.ones((N,), device="cuda", dtype=torch.float64)
    u = torch.nan_to_num(s["u"], nan=0.0).clamp(0.0, 1.0).double()
    good = u * given < share
    s["accept"].copy_(torch.where(given > 0, (share / given).clamp(max=1.0), (share > 0).double()))
    # the accepted drafts of a request: those before its first rejected one
    bad = torch.where(good, M, torch.arange(N, device="cuda") - cu[of])
    count = n.scatter_reduce(0, of, bad, "amin")
    at = cu[:-1] + req + count                                    # the row that the next token comes from
    final = mass[at]
    # after a rejection: what the target has above the draft
    rejected = count < n
    w_at = w[at] * (FIXED / total[at].clamp(min=1).double()).float()[:, None]
    if s["draft_logits"] is not None:
        which = (cu[:-1] + count).clamp(max=max(N - 1, 0))
        wq_at = wq[which] * (FIXED / sq[which].clamp(min=1).double()).float()[:, None] if N else w_at
        if index is not None and N:
            wq_at = torch.where(index[None, :] >= 0, wq_at[:, index.long().clamp(min=0)], 0.0)
        rest = w_at - wq_at
    else:
        rest = w_at
        if N:
            which = d[(cu[:-1] + count).clamp(max=N - 1)]
            rest = w_at.scatter(1, which[:, None], w_at.gather(1, which[:, None]) - 1.0)
    rest = (rest.clamp(min=0.0) * FIXED).round().to(torch.int64)
    final = torch.where((rejected & (rest.sum(1) > 0))[:, None], rest, final)
    whole = final.sum(1)
    v = torch.nan_to_num(s["v"], nan=0.0).clamp(0.0, 1.0).double()
    aim = torch.minimum((v * whole.double()).floor().to(torch.int64), whole - 1)
    token = (final.cumsum(1) <= aim[:, None]).sum(1).clamp(max=V - 1)
    token = torch.where(whole > 0, token, -1)
    s["n_accept"].copy_(count)
    # a row's token: the accepted draft, the next token, or none
    place = torch.arange(M, device="cuda") - cu[row_of] - row_of
    draft = torch.cat([d, d.new_zeros(1)])[(cu[row_of] + place).clamp(max=N)]
    ids = torch.where(place < count[row_of], draft, -1)
    s["ids"].copy_(torch.where(place == count[row_of], token[row_of], ids))
    return {"n_accept": s["n_accept"], "ids": s["ids"], "accept": s["accept"]}


# --------------------------------------------------------------------------------------------
# What a pass cannot do without, and its outcome in 64 bits


def work(case):
    if case["op"] == "verify":
        n = _rows(case)
        size = 2 if case["type"] == "bf16" else 4
        target, draft = (sum(n) + case["batch"]) * case["vocab"], sum(n) * case["draft_vocab"]
        index = 4 * case["vocab"] if 0 < case["draft_vocab"] < case["vocab"] else 0
        return {"bytes": (target + draft) * size + index + 16 * sum(n) + 32 * case["batch"],
                "flops": 4 * (target + draft)}
    news, kvs, bounds, prefix = _lengths(case)
    T, Hq, Hk, D, ps = sum(news), case["heads"], case["kv_heads"], case["dim"], case["page"]
    size = 1 if case["cache"] == "fp8" else 2
    if case["op"] == "append":
        each = 2 * Hq * D * 2 + 2 * Hk * D * (2 + size) + case["rot"] * 4 + 4
        return {"bytes": T * each, "flops": T * (Hq + Hk) * (case["rot"] * 3 + 4 * D)}
    pairs = span = 0
    for g, P in enumerate(prefix):
        skip, some = P // ps * ps, False
        for b in range(bounds[g], bounds[g + 1]):
            n, kv = news[b], kvs[b]
            if n:
                some = True
                span += kv - skip
                pairs += sum(kv - n + i + 1 for i in range(n)) if case["causal"] else n * kv
        span += skip if some else 0
    return {"bytes": T * Hq * (4 * D + 4) + 2 * span * Hk * D * size + 4 * span // ps,
            "flops": 4 * Hq * D * pairs}


def exact(case, seed):
    if case["op"] == "verify":
        return _exact_verify(case, seed)
    if case["op"] == "attention" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    news, kvs = s["news"], s["kvs"]
    D, ps, G = case["dim"], case["page"], case["heads"] // case["kv_heads"]
    cu = np.concatenate([[0], np.cumsum(news)])
    f64 = torch.float64
    if case["op"] == "append":
        R = case["rot"]
        half = case["pairs"] == "half"
        first = torch.arange(R // 2) if half else torch.arange(0, R, 2)
        second = first + (R // 2 if half else 1)
        res = {"k_cache": s["k_cache"].to(f64), "v_cache": s["v_cache"].to(f64)}
        q_out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
        for b, (n, kv) in enumerate(zip(news, kvs)):
            at = torch.arange(kv - n, kv, device="cuda")
            slot = s["block_table"][b].long()[at // ps]
            turn = torch.complex(s["rope"][at, :R // 2].to(f64), s["rope"][at, R // 2:].to(f64))
            for what in ("q", "k", "v"):
                x = s[what][cu[b]:cu[b + 1]].to(f64)
                if what != "v":
                    x = x / (x.norm(dim=-1, keepdim=True).square() / D + s["eps"]).sqrt()
                    x = x * s[what + "_weight"].to(f64)
                    z = torch.complex(x[..., first], x[..., second]) * turn[:, None, :]
                    x[..., first], x[..., second] = z.real, z.imag
                if what == "q":
                    q_out[cu[b]:cu[b + 1]] = x
                    continue
                if case["cache"] == "fp8":
                    x = (x / s[what + "_scale"].to(f64)[:, None]).clamp(-448, 448)
                res[what + "_cache"][slot, at % ps] = x
        return {"q": q_out, **res}
    out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    lse = torch.full(s["q"].shape[:2], float("-inf"), dtype=f64, device="cuda")
    for b, (n, kv) in enumerate(zip(news, kvs)):     # every request over its own pages, none shared
        if not n:
            continue
        at = torch.arange(kv, device="cuda")
        slot = s["block_table"][b].long()[at // ps]
        kv_of = []
        for what in ("k", "v"):
            c, scale = s[what + "_cache"], s[what + "_scale"]
            x = c.view(torch.uint8)[slot, at % ps].view(c.dtype) if scale is not None else c[slot, at % ps]
            kv_of.append(x.to(f64) * (scale.to(f64)[:, None] if scale is not None else 1.0))
        last = torch.arange(kv - n, kv, device="cuda") if case["causal"] else torch.full((n,), kv - 1, device="cuda")
        hide = at[None, :] > last[:, None]
        for h in range(case["heads"]):
            x = s["q"][cu[b]:cu[b + 1], h].to(f64) @ kv_of[0][:, h // G].T * s["scale"]
            x[hide] = float("-inf")
            norm = torch.logsumexp(x, 1)
            out[cu[b]:cu[b + 1], h] = torch.exp(x - norm[:, None]) @ kv_of[1][:, h // G]
            lse[cu[b]:cu[b + 1], h] = norm
    return {"out": out, "lse": lse}


def _distribution(z, temp, top_k=0, top_p=1.0, min_p=0.0):
    """Probabilities that the settings leave, in 64 bits."""
    z = z.double().cpu().numpy()
    V = len(z)
    order = np.lexsort((np.arange(V), -z)) if top_k or top_p < 1 or min_p or temp < 1e-6 else np.arange(V)
    if temp < 1e-6:
        order, temp = order[:1], 1.0
    elif 0 < top_k < V:
        order = order[:top_k]
    w = np.exp((z[order] - z[order].max()) / temp)
    if top_p < 1:
        stay = np.cumsum(w) - w < top_p * w.sum()
        stay[0] = True
        order, w = order[stay], w[stay]
    stay = w >= min_p
    p = np.zeros(V)
    p[order[stay]] = w[stay] / w[stay].sum()
    return p


def _exact_verify(case, seed):
    if (sum(_rows(case)) + case["batch"]) * case["vocab"] > 5e7:
        return None
    s = prepare(case, seed)
    B, M = case["batch"], s["logits"].shape[0]
    cu = s["cu_drafts"].tolist()
    drafts, u, v = s["drafts"].tolist(), s["u"].tolist(), s["v"].tolist()
    index = None if s["draft_index"] is None else s["draft_index"].cpu().numpy()
    settings = [s[x].tolist() for x in ("temperature", "top_k", "top_p", "min_p")]
    count, ids, accept = np.zeros(B, dtype=np.int64), np.full(M, -1), np.zeros(len(drafts))
    for b in range(B):
        going = True
        for i in range(cu[b + 1] - cu[b] + 1):
            r, t = cu[b] + i, cu[b] + b + i
            last = r == cu[b + 1]
            if last and not going:
                break
            p = _distribution(s["logits"][t], *(x[b] for x in settings))
            if not last:
                d = drafts[r]
                if s["draft_logits"] is None:
                    q = np.zeros_like(p)
                    q[d] = 1.0
                else:
                    q = _distribution(s["draft_logits"][r], float(s["draft_temperature"][b]))
                    if index is not None:
                        q = np.where(index >= 0, q[np.maximum(index, 0)], 0.0)
                accept[r] = min(1.0, p[d] / q[d]) if q[d] > 0 else float(p[d] > 0)
                if not going:
                    continue
                if u[r] * q[d] < p[d]:
                    ids[t] = d
                    count[b] += 1
                    continue
                going = False
                p = np.maximum(p - q, 0.0)
            cum = np.cumsum(p)
            ids[t] = min(int(np.searchsorted(cum, v[b] * cum[-1], side="right")), len(cum) - 1)
    return {"n_accept": torch.from_numpy(count).to(torch.int32), "ids": torch.from_numpy(ids).to(torch.int32),
            "accept": torch.from_numpy(accept)}
