"""The decode-side operators between the quantised projections, as cases to be timed and compared.

Three operators run between a decoder layer's q, k, v products and its o product, and after the
vocabulary head:

  append     rotary positions on q and k, and k and v written into a paged cache
             (lowbit_kv_append);
  attention  a chunk of new tokens per request (one, a draft block, a prompt's chunk) over that
             cache (lowbit_paged_attention);
  sample     a token per row of logits under temperature, top-k, top-p and min-p, from given
             uniform numbers (lowbit_sample).

`own` chooses between the plain form of each (elementary torch operations in 32 bits) and the
library's calls.  Heads of 128 with 32 query and 8 key/value heads are the 4B-class decoder
layer's q, k and v widths (4096 and 1024); 248,320 and 32,768 rows are the full and trimmed
vocabularies; 16 tokens are one draft block.
"""
import math
import random

import numpy as np
import torch

own = False

FIXED = 2.0 ** 40      # a sampling weight of 1 in whole numbers


def listed():
    return [
        # One token of one request: the append between two small launches of a decode step.
        dict(name="append_one", op="append", batch=1, new=1, max_kv=4000, heads=32, kv_heads=8,
             dim=128, page=64, order="head", cache="bf16", rot=128, pairs="half", ragged=0),
        # 32 requests verifying a draft block each, cache in 8 bits with a scale per head.
        dict(name="append_verify_fp8", op="append", batch=32, new=16, max_kv=3000, heads=32,
             kv_heads=8, dim=128, page=16, order="head", cache="fp8", rot=128, pairs="half",
             ragged=1),
        # Three prompts' chunks at once, rotary on the first half of each head, adjacent pairs.
        dict(name="append_prompt", op="append", batch=3, new=5555, max_kv=9001, heads=32,
             kv_heads=8, dim=128, page=64, order="token", cache="bf16", rot=64,
             pairs="adjacent", ragged=1),
        # Plain decoding of one request with a short context: latency.
        dict(name="attn_one_short", op="attention", batch=1, new=1, max_kv=777, heads=32,
             kv_heads=8, dim=128, page=16, order="head", cache="bf16", causal=True, window=0,
             ragged=0),
        # Verifying one draft block against a long context.
        dict(name="attn_verify_long", op="attention", batch=1, new=16, max_kv=32765, heads=32,
             kv_heads=8, dim=128, page=64, order="head", cache="bf16", causal=True, window=0,
             ragged=0),
        # A decode batch with contexts of many lengths, cache in 8 bits.
        dict(name="attn_decode_fp8", op="attention", batch=64, new=1, max_kv=16384, heads=32,
             kv_heads=8, dim=128, page=16, order="head", cache="fp8", causal=True, window=0,
             ragged=1),
        # A batch of draft blocks being verified, some slots idle, lengths of all kinds.
        dict(name="attn_verify_batch", op="attention", batch=24, new=16, max_kv=20000, heads=32,
             kv_heads=8, dim=128, page=64, order="token", cache="bf16", causal=True, window=0,
             ragged=1),
        # A block drafter: every token of the block sees the whole block, and a window of context.
        dict(name="attn_draft_window", op="attention", batch=9, new=16, max_kv=6000, heads=16,
             kv_heads=4, dim=64, page=32, order="head", cache="bf16", causal=False, window=1024,
             ragged=1),
        # A prompt's chunk on top of a long context: bound by arithmetic.
        dict(name="attn_prompt", op="attention", batch=1, new=4001, max_kv=16331, heads=32,
             kv_heads=8, dim=128, page=64, order="head", cache="bf16", causal=True, window=0,
             ragged=0),
        # One token of a chat: the usual truncation, full vocabulary.
        dict(name="sample_one", op="sample", rows=1, vocab=248320, type="fp32", mix=0, masked=0),
        # A draft block sampled from bf16 logits (many exact ties), a grammar masking many tokens.
        dict(name="sample_block_bf16", op="sample", rows=16, vocab=248320, type="bf16", mix=1,
             masked=1),
        # A large batch, every row with its own settings, some rows greedy or without truncation.
        dict(name="sample_batch", op="sample", rows=192, vocab=248320, type="fp32", mix=1,
             masked=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "attention", "attention", "sample"))
    if op == "sample":
        return dict(op=op, rows=_log(rng, 1, 160), vocab=_log(rng, 1000, 248320),
                    type=rng.choice(("fp32", "bf16")), mix=rng.choice((0, 1, 1)),
                    masked=rng.choice((0, 1)))
    kv_heads = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 4, 4, 5, 8) if kv_heads < 8 else (1, 2, 4, 4))
    case = dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, dim=rng.choice((64, 128, 128)),
                page=rng.choice((16, 32, 64, 128)), order=rng.choice(("head", "token")),
                cache=rng.choice(("bf16", "bf16", "fp8")), ragged=rng.choice((0, 1, 1)))
    if op == "append":
        batch = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 12000 // batch))
        case |= dict(batch=batch, new=new, max_kv=new + _log(rng, 1, 3000),
                     rot=rng.choice((case["dim"], case["dim"], case["dim"] // 2)),
                     pairs=rng.choice(("half", "half", "adjacent")))
        return case
    case |= dict(causal=rng.choice((True, True, True, False)), window=0)
    if rng.random() < 0.25:
        case["window"] = _log(rng, 100, 4000)
    if rng.random() < 0.25:       # a prompt's chunks
        case |= dict(batch=rng.choice((1, 1, 2)), new=_log(rng, 200, 1900))
        case["max_kv"] = case["new"] + _log(rng, 1, 10000)
    else:                         # decoding and draft blocks
        batch = _log(rng, 1, 48)
        case |= dict(batch=batch, new=rng.choice((1, 1, 4, 8, 16, 16, 31)))
        case["max_kv"] = case["new"] + _log(rng, 1, 300000 // batch if batch > 9 else 32000)
    return case


def _lengths(case):
    """New tokens and whole length of every request: plain lists, the same for every seed."""
    B, new, top = case["batch"], case["new"], case["max_kv"]
    if not case["ragged"]:
        return [new] * B, [top] * B
    r = random.Random(B * 1000003 + new * 1009 + top)
    news, kvs = [], []
    for b in range(B):
        n = new if new <= 31 else r.randint(max(1, new // 4), new)
        if B > 4 and b % 7 == 5:
            n = 0                 # an idle slot of the batch
        kv = top if b == 0 else min(top, n + int(math.exp(r.uniform(0.0, math.log(top + 1)))))
        news.append(n)
        kvs.append(max(kv, n, 1))
    return news, kvs


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
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 40) + 17)
    if case["op"] == "sample":
        return _prepare_sample(case, seed, gen)
    news, kvs = _lengths(case)
    B, Hq, Hk, D, ps = case["batch"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    T = sum(news)
    need = [-(-kv // ps) for kv in kvs]
    width = max(need) + 1
    pages = sum(need) + 3
    order = np.random.RandomState(int(seed) % (1 << 31)).permutation(pages)
    table = np.zeros((B, width), dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    k, v = _cache(case, gen, pages)
    dev = dict(device="cuda", dtype=torch.int32)
    s = dict(op=case["op"], case=case, T=T, k_cache=k, v_cache=v, max_new=max(news),
             max_kv=max(kvs), block_table=torch.from_numpy(table).cuda(),
             cu_q=torch.tensor(np.concatenate([[0], np.cumsum(news)]), **dev),
             kv_lens=torch.tensor(kvs, **dev), k_scale=None, v_scale=None)
    if case["cache"] == "fp8":
        s["k_scale"] = torch.linspace(0.9, 1.3, Hk, device="cuda") / 32
        s["v_scale"] = torch.linspace(1.2, 0.8, Hk, device="cuda") / 32
    if case["op"] == "append":
        # q, k and v as the three products leave them side by side: rows of one buffer.
        qkv = torch.randn((T, (Hq + 2 * Hk) * D), device="cuda", generator=gen)
        qkv = qkv.to(torch.bfloat16)
        s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["v"] = qkv[:, (Hq + Hk) * D:].view(T, Hk, D)
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
                if tail:
                    flat[int(table[b, need[b] - 1]), ps - tail:] = (
                        float("nan") if c.dtype == torch.bfloat16 else 0x7F)
        # scores of standard deviation 1.5: some rows attend to few positions, some to many
        s["q"] = (1.5 * torch.randn((T, Hq, D), device="cuda", generator=gen)).to(torch.bfloat16)
        s["out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((T, Hq), dtype=torch.float32, device="cuda")
        s["scale"] = D ** -0.5
    if own:
        import bit_weight_gemv_gb300 as lb
        s["cache"] = lb.lowbit_paged_cache(k, v, s["k_scale"], s["v_scale"])
        if case["op"] == "attention":
            need_bytes = lb.lowbit_paged_attention_workspace_bytes(T, B, Hq, Hk, D)
            s["workspace"] = torch.zeros(need_bytes, dtype=torch.uint8, device="cuda")
    return s


def _prepare_sample(case, seed, gen):
    M, V = case["rows"], case["vocab"]
    # a broad body of unlikely tokens and a few likely ones, as a language model's rows have
    z = 2.2 * torch.randn((M, V), device="cuda", generator=gen)
    hot = torch.randint(0, V, (M, 24), device="cuda", generator=gen)
    lift = 12.0 + 2.0 * torch.randn((M, 24), device="cuda", generator=gen)
    z.scatter_(1, hot, lift)
    if case["masked"]:
        ban = torch.rand((M, V), device="cuda", generator=gen) < 0.6
        ban[0] = True             # one row with a single token allowed
        ban[0, V // 3] = False
        z = z.masked_fill(ban, float("-inf"))
    r = random.Random(int(seed) * 7919 + M * 31 + V)
    temp, top_k, top_p, min_p = [], [], [], []
    for m in range(M):
        if not case["mix"]:
            temp.append(0.7), top_k.append(20), top_p.append(0.95), min_p.append(0.0)
            continue
        kind = (m + int(seed)) % 6
        temp.append(0.0 if kind == 4 else r.uniform(0.3, 1.5))
        top_k.append(0 if kind in (1, 3) else int(math.exp(r.uniform(0, math.log(2000)))))
        top_p.append(1.0 if kind in (2, 3) else r.uniform(0.5, 0.99))
        min_p.append(r.uniform(0.005, 0.1) if kind in (0, 3) else 0.0)
    f = dict(device="cuda", dtype=torch.float32)
    return dict(op="sample", case=case,
                logits=z.to(torch.bfloat16) if case["type"] == "bf16" else z,
                temperature=torch.tensor(temp, **f), top_p=torch.tensor(top_p, **f),
                min_p=torch.tensor(min_p, **f),
                top_k=torch.tensor(top_k, device="cuda", dtype=torch.int32),
                u=torch.rand((M,), device="cuda", generator=gen),
                ids=torch.empty((M,), device="cuda", dtype=torch.int32),
                logprob=torch.empty((M,), **f),
                kept=torch.empty((M,), device="cuda", dtype=torch.int32))


# --------------------------------------------------------------------------------------------
# One pass


def run(s):
    if s["op"] == "append":
        return _run_append(s)
    if s["op"] == "attention":
        return _run_attention(s)
    return _run_sample(s)


def _run_append(s):
    if own:
        import bit_weight_gemv_gb300 as lb
        lb.lowbit_kv_append(s["q"], s["k"], s["v"], s["rope"], s["cu_q"], s["kv_lens"],
                            s["block_table"], s["cache"], s["q_out"],
                            interleaved=s["case"]["pairs"] == "adjacent")
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    case, T, ps = s["case"], s["T"], s["case"]["page"]
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    pos = kv[b] - cu[b + 1] + t
    page = s["block_table"][b, pos // ps].long()
    q = _rotate(s["q"].float(), s["rope"][pos], case)
    k = _rotate(s["k"].float(), s["rope"][pos], case)
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
        lb.lowbit_paged_attention(s["q"], s["cache"], s["cu_q"], s["kv_lens"], s["block_table"],
                                  s["out"], s["workspace"], scale=s["scale"],
                                  causal=case["causal"], window=case["window"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    B, Hq, Hk, D, ps = case["batch"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    G, n, T = Hq // Hk, s["max_new"], s["T"]
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    new = cu[1:] - cu[:-1]
    L = -(-s["max_kv"] // ps) * ps
    pages = s["block_table"][:, :L // ps].long()
    i, j = torch.arange(n, device="cuda"), torch.arange(L, device="cuda")
    pos = (kv - new)[:, None] + i[None, :]                               # [B][n]
    see = (j[None, None, :] < kv[:, None, None]) & (i[None, :] < new[:, None])[:, :, None]
    if case["causal"]:
        see = see & (j[None, None, :] <= pos[:, :, None])
    if case["window"]:
        see = see & (j[None, None, :] > pos[:, :, None] - case["window"])

    def keys(c, scale):
        if c.dtype == torch.bfloat16:
            x = c[pages].float()
        else:
            x = c.view(torch.uint8)[pages].view(c.dtype).float() * scale[:, None]
        return x.reshape(B, L, Hk, D).permute(0, 2, 1, 3)                # [B][Hk][L][D]

    token = (cu[:-1, None] + i[None, :]).clamp(max=max(T - 1, 0))
    q = s["q"][token].float().view(B, n, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, n * G, D)
    x = torch.matmul(q, keys(s["k_cache"], s["k_scale"]).transpose(2, 3)) * s["scale"]
    x = x.view(B, Hk, n, G, L).masked_fill_(~see[:, None, :, None, :], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    vals = keys(s["v_cache"], s["v_scale"])
    vals = torch.where(see.any(1)[:, None, :, None], vals, 0.0)
    y = torch.matmul(p.view(B, Hk, n * G, L), vals).view(B, Hk, n, G, D)
    y = y / torch.where(total > 0, total, 1.0)
    lse = (top + total.log())[..., 0]                                    # [B][Hk][n][G]
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu, t, right=True) - 1
    at = t - cu[b]
    s["out"].copy_(y.permute(0, 2, 1, 3, 4)[b, at].reshape(T, Hq, D))
    s["lse"].copy_(lse.permute(0, 2, 1, 3)[b, at].reshape(T, Hq))
    return {"out": s["out"], "lse": s["lse"]}


def _run_sample(s):
    if own:
        import bit_weight_gemv_gb300 as lb
        lb.lowbit_sample(s["logits"], s["u"], s["ids"], temperature=s["temperature"],
                         top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                         logprob=s["logprob"], kept=s["kept"])
        return {"ids": s["ids"], "logprob": s["logprob"], "kept": s["kept"]}
    z = s["logits"].float()
    M, V = z.shape
    z = torch.where(torch.isnan(z), float("-inf"), z).clamp(max=torch.finfo(torch.float32).max)
    top = z.amax(1, keepdim=True)
    temp = s["temperature"][:, None]
    greedy = ~(temp >= 1e-6)
    rate = 1.0 / torch.where(greedy, 1.0, temp.clamp(max=1e6))
    w = torch.where(z == float("-inf"), 0.0, torch.exp((z - top) * rate))
    mass = (w * FIXED).round().to(torch.int64)
    # the order of truncation: larger logits first, lower tokens first among equal ones
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    m = mass.gather(1, order)
    rank = torch.arange(V, device="cuda")[None, :]
    k = s["top_k"].long()[:, None]
    k = torch.where((k <= 0) | (k > V), V, k)
    k = torch.where(greedy, 1, k)
    m = torch.where(rank < k, m, 0)
    total = m.sum(1, keepdim=True)
    p = s["top_p"][:, None]
    limit = (p.double() * total.double()).ceil().to(torch.int64).clamp(min=1)
    limit = torch.where(p >= 1.0, total, limit)
    before = m.cumsum(1) - m
    m = torch.where(before < limit, m, 0)
    keep = torch.zeros_like(mass).scatter(1, order, m)
    keep = torch.where(w >= s["min_p"][:, None], keep, 0)
    total = keep.sum(1, keepdim=True)
    u = torch.nan_to_num(s["u"], nan=0.0).clamp(0.0, 1.0)[:, None].double()
    aim = torch.minimum((u * total.double()).floor().to(torch.int64), total - 1)
    token = (keep.cumsum(1) <= aim).sum(1).clamp(max=V - 1)
    chosen = keep.gather(1, token[:, None])
    some = total[:, 0] > 0
    s["ids"].copy_(torch.where(some, token, -1))
    share = chosen.double() / total.clamp(min=1).double()
    s["logprob"].copy_(torch.where(some, share.float().log()[:, 0], float("-inf")))
    s["kept"].copy_((keep > 0).sum(1))
    return {"ids": s["ids"], "logprob": s["logprob"], "kept": s["kept"]}


# --------------------------------------------------------------------------------------------
# What a pass cannot do without, and its outcome in 64 bits


def _seen(case, n, kv, i):
    """First and one past the last key that token i of a request sees."""
    pos = kv - n + i
    lo = max(0, pos - case["window"] + 1) if case["window"] else 0
    return lo, max(lo, min(kv, pos + 1) if case["causal"] else kv)


def work(case):
    if case["op"] == "sample":
        M, V = case["rows"], case["vocab"]
        return {"bytes": M * V * (2 if case["type"] == "bf16" else 4) + 32 * M, "flops": 4 * M * V}
    news, kvs = _lengths(case)
    T, Hq, Hk, D = sum(news), case["heads"], case["kv_heads"], case["dim"]
    size = 1 if case["cache"] == "fp8" else 2
    if case["op"] == "append":
        each = 2 * Hq * D * 2 + 2 * Hk * D * (2 + size) + case["rot"] * 4 + 4
        return {"bytes": T * each, "flops": T * (Hq + Hk) * case["rot"] * 3}
    pairs = span = 0
    for n, kv in zip(news, kvs):
        if n:
            lo, hi = _seen(case, n, kv, 0)[0], _seen(case, n, kv, n - 1)[1]
            span += hi - lo
            pairs += sum(b - a for a, b in (_seen(case, n, kv, i) for i in range(n)))
    return {"bytes": T * Hq * (4 * D + 4) + 2 * span * Hk * D * size + 4 * span // case["page"],
            "flops": 4 * Hq * D * pairs}


def exact(case, seed):
    if case["op"] == "sample":
        return _exact_sample(case, seed)
    if case["op"] == "attention" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    news, kvs = _lengths(case)
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
                    z = torch.complex(x[..., first], x[..., second]) * turn[:, None, :]
                    x = x.clone()
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
    for b, (n, kv) in enumerate(zip(news, kvs)):
        if not n:
            continue
        lo, hi = _seen(case, n, kv, 0)[0], _seen(case, n, kv, n - 1)[1]
        at = torch.arange(lo, hi, device="cuda")
        slot = s["block_table"][b].long()[at // ps]
        kv_of = []
        for what in ("k", "v"):
            c, scale = s[what + "_cache"], s[what + "_scale"]
            x = c.view(torch.uint8)[slot, at % ps].view(c.dtype) if scale is not None else c[slot, at % ps]
            kv_of.append(x.to(f64) * (scale.to(f64)[:, None] if scale is not None else 1.0))
        edge = torch.tensor([_seen(case, n, kv, i) for i in range(n)], device="cuda")
        hide = (at[None, :] < edge[:, :1]) | (at[None, :] >= edge[:, 1:])
        for h in range(case["heads"]):
            x = s["q"][cu[b]:cu[b + 1], h].to(f64) @ kv_of[0][:, h // G].T * s["scale"]
            x[hide] = float("-inf")
            norm = torch.logsumexp(x, 1)
            some = torch.isfinite(norm)
            y = torch.exp(x - torch.where(some, norm, 0.0)[:, None]) @ kv_of[1][:, h // G]
            out[cu[b]:cu[b + 1], h] = y
            lse[cu[b]:cu[b + 1], h] = norm
    return {"out": out, "lse": lse}


def _exact_sample(case, seed):
    s = prepare(case, seed)
    M, V = case["rows"], case["vocab"]
    ids, logprob, kept = np.full(M, -1), np.full(M, -np.inf), np.zeros(M, dtype=np.int64)
    for m in range(M):
        z = s["logits"][m].double().cpu().numpy()
        temp, u = float(s["temperature"][m]), float(s["u"][m])
        order = np.lexsort((np.arange(V), -z))
        order = order[np.isfinite(z[order])]
        k = int(s["top_k"][m])
        k = 1 if temp < 1e-6 else k if 0 < k < V else V
        order = order[:k]
        if not len(order):
            continue
        w = np.exp((z[order] - z[order[0]]) / (temp if temp >= 1e-6 else 1.0))
        p = float(s["top_p"][m])
        if p < 1:
            stay = np.cumsum(w) - w < p * w.sum()
            stay[0] = True
            order, w = order[stay], w[stay]
        stay = w >= float(s["min_p"][m])
        order, w = order[stay], w[stay]
        by_id = np.argsort(order)
        cum = np.cumsum(w[by_id])
        at = min(int(np.searchsorted(cum, u * cum[-1], side="right")), len(cum) - 1)
        ids[m], logprob[m] = order[by_id[at]], np.log(w[by_id[at]] / cum[-1])
        kept[m] = int((w >= 0.5 / FIXED).sum())
    return {"ids": torch.from_numpy(ids).to(torch.int32), "logprob": torch.from_numpy(logprob),
            "kept": torch.from_numpy(kept).to(torch.int32)}
