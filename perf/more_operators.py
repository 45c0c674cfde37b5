"""Operators of a serving step as they are measured: attention of chunks of new tokens over a paged cache, sampling.

Every case runs in two forms on the same inputs: the plain form (elementary torch operations
in 32 bits, sums of sampled weights in 64) and, with ``own`` set, the library's entry points through
``bucketized_guidance_step_gb300.decode``.

The definitions that both follow:

* A cache holds K and V as [layers, pages, kv_heads, page, dim]. Sequence s has lens[s] tokens;
  token t lies in page table[s, t // page] at row t % page.
* chunk: rows start[i] .. start[i+1]-1 of the queries are the last tokens of sequence seq[i], whose K
  and V the cache holds already. The row at position t sees the positions j <= t (all of them, or the
  first `sinks` and the last `window`). Returns the output and the log-sum-exp of the scaled scores.
  Rows from start[n] on are padding: their output is left as it was.
* sample: z = logits / temperature (temperature <= 0: greedy, z as it is and no noise). In the order of
  falling z (ties: rising index), with weights e^z: the first top_k tokens stay (0: all), of these the
  shortest beginning whose weights reach top_p of their sum, and of these the tokens with at least
  min_p times the largest weight. The token is the lowest index of the largest z + noise among what
  stays, its log-probability that of what stays.
"""

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
LAYER = 0          # attention reads one layer a call


def _chunk(name, seqs, q_heads, kv_heads, dim, page, new_lo, new_hi, past_lo, past_hi, dtype, window=0, sinks=0, pad=0):
    c = {"op": "chunk", "seqs": seqs, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page,
         "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo, "past_hi": past_hi, "dtype": dtype,
         "window": window, "sinks": sinks, "pad": pad}
    return {"name": name, **c} if name else c


def _sample(name, batch, vocab, dtype, spread, top_k, top_p, min_p, greedy, masked):
    c = {"op": "sample", "batch": batch, "vocab": vocab, "dtype": dtype, "spread": spread, "top_k": top_k,
         "top_p": top_p, "min_p": min_p, "greedy": greedy, "masked": masked}
    return {"name": name, **c} if name else c


def listed():
    return [
        # One guided sample's two branches read a few condition tokens after a short prompt. Latency counts.
        _chunk("chunk_two_short", 2, 16, 16, 64, 16, 3, 7, 1, 250, "fp16"),
        # Fresh prompts of ragged lengths, read whole.
        _chunk("chunk_prompts", 8, 32, 8, 128, 16, 1, 2048, 0, 0, "bf16", pad=5),
        # A long prompt is read in chunks: the last of them.
        _chunk("chunk_long_prompt", 1, 32, 8, 128, 64, 2048, 2048, 14336, 14336, "bf16"),
        # A continuous batch whose sequences check a few drafted tokens each.
        _chunk("chunk_verify_32", 32, 32, 8, 128, 16, 1, 8, 1, 8192, "bf16", pad=11),
        # A short question after one long document: the split over the length carries it.
        _chunk("chunk_few_long", 1, 32, 8, 128, 64, 33, 33, 200001, 200001, "bf16"),
        # Streams kept to a window and a few first tokens, with chunks of their own sizes.
        _chunk("chunk_window", 16, 16, 4, 128, 32, 1, 512, 0, 6001, "fp16", window=1024, sinks=4),
        # A 32-bit model, narrow heads and an odd page size.
        _chunk("chunk_fp32", 8, 8, 4, 96, 24, 1, 129, 0, 1001, "fp32", pad=3),
        # One sample of a small codebook. Latency counts.
        _sample("sample_one", 1, 16384, "bf16", 3.0, 50, 0.9, 0.0, False, False),
        # The logits of a guided batch (32 bits) of a large vocabulary, a grammar's tokens left.
        _sample("sample_64", 64, 131072, "fp32", 3.0, 1000, 0.8, 0.05, True, True),
        # Unfiltered or nearly so: flat distributions, whose nucleus is most of an odd vocabulary.
        _sample("sample_flat", 33, 50021, "bf16", 0.7, 0, 0.5, 0.0, False, False),
        # A wide batch with every row's settings its own.
        _sample("sample_128", 128, 32000, "fp16", 2.0, 200, 0.7, 0.1, True, False),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(2 ** rng.uniform(np.log2(lo), np.log2(hi))))))


def draw(rng):
    dtype = rng.choice(["bf16", "fp16", "bf16", "fp16", "fp32"])
    if rng.random() < 0.6:
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        kv_heads, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 6, 8, 16])
        page = rng.choice([8, 16, 24, 32, 64, 128])
        seqs = _log(rng, 1, 48)
        heads, row = kv_heads * group, kv_heads * dim * 2 * SIZE[dtype]
        most = 1.0e9 * 128 if dtype != "fp32" else 5e9            # pairs of a query and a position, times dim
        new_hi = _log(rng, 1, max(2, min(2048, int((most / (seqs * heads * dim)) ** 0.5))))
        longest = min(200000, int(8e8 / (row * seqs)), int(most / (seqs * heads * dim * new_hi))) - new_hi
        past_hi = _log(rng, 1, max(2, longest)) if rng.random() < 0.8 and longest > 1 else 0
        window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        return _chunk(None, seqs, heads, kv_heads, dim, page, rng.randint(1, new_hi), new_hi, rng.randint(0, past_hi), past_hi,
                      dtype, window, rng.randint(0, 16) if window else 0, rng.choice([0, 0, 1, 7]))
    return _sample(None, _log(rng, 1, 64), _log(rng, 1000, 131072), dtype, rng.choice([0.5, 1.0, 2.0, 3.0, 4.0]),
                   rng.choice([0, _log(rng, 1, 1000)]), rng.choice([1.0, rng.uniform(0.3, 0.99)]), rng.choice([0.0, rng.uniform(0.01, 0.3)]),
                   rng.random() < 0.3, rng.random() < 0.4)


def _spread(lo, hi, n):
    """n whole numbers over [lo, hi], the last of them hi."""
    return [lo + (hi - lo) * (i + 1) // n for i in range(n)]


def _up(a, b):
    return -(-a // b)


def _entries(case):
    """(new, past) tokens of every sequence: long pasts meet short chunks too."""
    n = case["seqs"]
    new, past = _spread(case["new_lo"], case["new_hi"], n), _spread(case["past_lo"], case["past_hi"], n)
    return [(new[i], past[(i * 7 + n // 2) % n] if n % 7 else past[n - 1 - i]) for i in range(n)]


def _normal(shape, dtype, g, sd=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(sd).to(dtype)


def prepare(case, seed):
    s = _prepare_chunk(case, seed) if case["op"] == "chunk" else _prepare_sample(case, seed)
    s.update(case=case, op=case["op"])
    if own:
        _plan(s)
    return s


def _prepare_chunk(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, page, dt = case["seqs"], case["page"], DTYPES[case["dtype"]]
    entries = torch.tensor(_entries(case), dtype=torch.int32, device="cuda")
    entries = entries[torch.randperm(n, generator=g, device="cuda")]           # in another order each time
    new, full = entries[:, 0], entries.sum(1, dtype=torch.int32)
    seq = torch.randperm(n, generator=g, device="cuda").int()
    lens = torch.zeros_like(full)
    lens[seq.long()] = full
    both = _entries(case)
    pages = sum(_up(a + b, page) for a, b in both) + n
    cols = max(_up(a + b, page) for a, b in both)
    held = (lens + page - 1) // page
    at = held.cumsum(0) - held
    col = torch.arange(cols, device="cuda")
    live = col < held[:, None]
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.where(live, perm[(at[:, None] + col).clamp(max=pages - 1)], -1).int()
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs.index_add_(0, table.clamp(min=0).flatten(), live.int().flatten())
    shape = (1, pages, case["kv_heads"], page, case["dim"])
    k, v = (torch.empty(shape, device="cuda", dtype=dt).normal_(generator=g) for _ in range(2))
    start = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), new.cumsum(0).int()])
    tokens = sum(a for a, _ in both) + case["pad"]
    q = _normal((tokens, case["q_heads"], case["dim"]), dt, g, 2.0)
    return {"k": k, "v": v, "table": table, "lens": lens, "refs": refs, "seq": seq, "start": start, "q": q,
            "scale": float(case["dim"]) ** -0.5, "out": torch.zeros_like(q),
            "lse": torch.zeros(q.shape[:2], dtype=torch.float32, device="cuda")}


def _prepare_sample(case, seed):
    B, V = case["batch"], case["vocab"]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def uniform(lo, hi):
        return torch.rand(B, generator=g, device="cuda") * (hi - lo) + lo

    z = torch.randn((B, V), generator=g, device="cuda") * case["spread"]
    if case["masked"]:                                              # a grammar allows few tokens or most
        z[torch.rand((B, V), generator=g, device="cuda") >= uniform(0.01, 1.0)[:, None]] = float("-inf")
    s = {"logits": z.to(DTYPES[case["dtype"]])}
    s["temperature"] = uniform(0.5, 1.5)
    if case["greedy"]:
        s["temperature"] = torch.where(torch.rand(B, generator=g, device="cuda") < 0.25, 0.0, s["temperature"])
    off = torch.rand((3, B), generator=g, device="cuda") < 0.15     # some requests leave a filter out
    k = (uniform(0.0, 1.0) * (case["top_k"] - 1)).round().int() + 1 if case["top_k"] else torch.zeros(B, dtype=torch.int32, device="cuda")
    s["top_k"] = torch.where(off[0], 0, k).int()
    s["top_p"] = torch.where(off[1], 1.0, uniform(case["top_p"], 1.0))
    s["min_p"] = torch.where(off[2], 0.0, uniform(0.0, 2.0) * case["min_p"])
    s["noise"] = -torch.log(-torch.log(torch.rand((B, V), generator=g, device="cuda").clamp(1e-7, 1 - 1e-7)))
    s["token"] = torch.empty(B, dtype=torch.int32, device="cuda")
    s["logprob"] = torch.empty(B, dtype=torch.float32, device="cuda")
    return s


def _plan(s):
    """The handles that a user's program keeps: the cache and the prepared call on its buffers."""
    from bucketized_guidance_step_gb300 import decode
    if s["op"] == "sample":
        s["call"] = decode.prepare_sample(s["logits"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                          min_p=s["min_p"], noise=s["noise"], token=s["token"], logprob=s["logprob"])
        return
    s["cache"] = decode.PagedCache(s["k"], s["v"], s["table"], s["lens"], s["refs"])
    s["call"] = s["cache"].prepare_chunk_attention(s["q"], LAYER, s["seq"], s["start"], scale=s["scale"], window=s["case"]["window"],
                                                   sinks=s["case"]["sinks"], out=s["out"], lse=s["lse"])


def run(s):
    if own:
        s["call"]()
    elif s["op"] == "chunk":
        _chunk_attention(s)
    else:
        _sample_tokens(s)
    if s["op"] == "chunk":
        return {"out": s["out"], "lse": s["lse"]}
    return {"token": s["token"], "logprob": s["logprob"]}


# ---- plain forms ---------------------------------------------------------------------------------
def _chunk_attention(s):
    c, page = s["case"], s["case"]["page"]
    T, Hq, D = s["q"].shape
    n, Hkv = c["seqs"], c["kv_heads"]
    m, L = c["new_hi"], max(a + b for a, b in _entries(c))
    lens = s["lens"][s["seq"].long()].long()
    start = s["start"].long()
    new = start[1:] - start[:-1]
    # padded to the longest chunk and the longest sequence
    i = torch.arange(m, device="cuda")
    j = torch.arange(L, device="cuda")
    row = (start[:-1, None] + i).clamp(max=T - 1)                              # [n, m]
    real = i < new[:, None]
    place = lens[:, None] - new[:, None] + i
    seen = (j <= place[:, :, None]) & real[:, :, None]                         # [n, m, L]
    if c["window"]:
        seen &= (j < c["sinks"]) | (j > place[:, :, None] - c["window"])
    held = j < lens[:, None]
    pages = s["table"][s["seq"].long()][:, j // page].clamp(min=0).long()
    k = s["k"][LAYER][pages, :, j % page].float()                              # [n, L, Hkv, D]
    v = s["v"][LAYER][pages, :, j % page].float().masked_fill(~held[:, :, None, None], 0.0)
    q = s["q"][row].float().view(n, m, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)[:, :, None]) * s["scale"]    # [n, Hkv, G, m, L]
    score = score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.transpose(1, 2)[:, :, None])
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n, m, Hq, D)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(n, m, Hq)
    s["out"][row[real]] = o[real].to(s["out"].dtype)
    s["lse"][row[real]] = lse[real]


def _sample_tokens(s):
    V = s["logits"].shape[1]
    hot = s["temperature"][:, None]
    z = s["logits"].float()
    z = torch.where(hot > 0, z / hot, z)
    low = float("-inf")
    down, order = torch.sort(z, dim=1, descending=True, stable=True)
    w = torch.exp(down.double() - down[:, :1].double())
    rank = torch.arange(V, device="cuda")
    k, p = s["top_k"][:, None], s["top_p"][:, None]
    keep = (rank < k) | (k <= 0)
    w = torch.where(keep, w, 0.0)
    before = w.cumsum(1) - w
    keep &= (before < p.double() * w.sum(1, keepdim=True)) | (p >= 1) | (rank == 0)
    keep &= (w >= s["min_p"][:, None]) & (down > low)
    total = torch.where(keep, w, 0.0).sum(1)
    stays = torch.zeros_like(keep).scatter_(1, order, keep)
    pick = torch.where(stays, torch.where(hot > 0, z + s["noise"], z), low)
    v = torch.arange(V, device="cuda")
    token = torch.where(stays & (pick == pick.amax(1, keepdim=True)), v, V).amin(1)
    none = token == V
    token = torch.where(none, 0, token)
    logprob = (z.gather(1, token[:, None])[:, 0].double() - down[:, 0].double()) - torch.log(total)
    s["token"].copy_(torch.where(none, -1, token))
    s["logprob"].copy_(torch.where(none, low, logprob))


# ---- what a pass cannot do without ----------------------------------------------------------------
def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "sample":
        B, V, k = case["batch"], case["vocab"], case["top_k"]
        # a row that keeps k tokens needs no more than their noise
        return {"bytes": B * (V * e + 4 * (k // 2 if k else V) + 24), "flops": 4.0 * B * V}
    token = case["kv_heads"] * case["dim"] * 2 * e                             # K and V of a token
    w, sinks, tokens, read, pairs = case["window"], case["sinks"], 0, 0, 0
    for new, past in _entries(case):
        t = past + np.arange(new, dtype=np.int64)                              # positions of the rows
        tokens += new
        first = max(0, past + 1 - w) if w else 0
        read += past + new - first + min(sinks, first)
        seen = t + 1 if not w else np.minimum(t + 1, w + np.minimum(sinks, np.maximum(t + 1 - w, 0)))
        pairs += int(seen.sum())
    Hq, D = case["q_heads"], case["dim"]
    return {"bytes": read * token + 2 * tokens * Hq * D * e + 4 * tokens * Hq + 4 * (read // case["page"]),
            "flops": 4.0 * pairs * Hq * D}


# ---- 64 bits ------------------------------------------------------------------------------------
def exact(case, seed):
    """The outputs from their definitions in 64 bits, one sequence or row after the other."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _exact_chunk(s) if case["op"] == "chunk" else _exact_sample(s)


def _exact_chunk(s):
    c, page = s["case"], s["case"]["page"]
    out, lse = s["out"].double(), s["lse"].double()
    start, group = s["start"].tolist(), c["q_heads"] // c["kv_heads"]
    for i, b in enumerate(s["seq"].tolist()):
        n, m = int(s["lens"][b]), start[i + 1] - start[i]
        pages = s["table"][b, :_up(n, page)].long()
        at = torch.arange(n - m, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")
        hidden = j > at
        if c["window"]:
            hidden |= (j <= at - c["window"]) & (j >= c["sinks"])
        for h in range(c["q_heads"]):
            k = s["k"][LAYER][pages, h // group].reshape(-1, c["dim"])[:n].double()
            v = s["v"][LAYER][pages, h // group].reshape(-1, c["dim"])[:n].double()
            score = (s["q"][start[i]:start[i + 1], h].double() @ k.T) * s["scale"]
            score[hidden] = -torch.inf
            lse[start[i]:start[i + 1], h] = torch.logsumexp(score, 1)
            out[start[i]:start[i + 1], h] = torch.softmax(score, 1) @ v
    return {"out": out, "lse": lse}


def _exact_sample(s):
    B, V = s["logits"].shape
    token = torch.empty(B, dtype=torch.int32)
    logprob = torch.empty(B, dtype=torch.float64)
    for b in range(B):
        z, hot = s["logits"][b].float(), float(s["temperature"][b])
        z = (z / s["temperature"][b] if hot > 0 else z).double().cpu().numpy()    # (the quotient in 32 bits: its ties are the definition's)
        order = np.argsort(-z, kind="stable")
        k = int(s["top_k"][b])
        order = order[:k] if k > 0 else order
        order = order[z[order] > -np.inf]
        if not len(order):
            token[b], logprob[b] = -1, -torch.inf
            continue
        w = np.exp(z[order] - z[order[0]])
        p = float(s["top_p"][b])
        if p < 1:
            reached = np.cumsum(w) >= p * w.sum()
            order = order[:int(np.argmax(reached)) + 1]
        order = order[np.exp(z[order] - z[order[0]]) >= float(s["min_p"][b])]
        pick = z[order].astype(np.float32) + s["noise"][b].cpu().numpy()[order] if hot > 0 else z[order]
        token[b] = int(order[pick == pick.max()].min())
        logprob[b] = z[token[b]] - z[order[0]] - np.log(np.exp(z[order] - z[order[0]]).sum())
    return {"token": token, "logprob": logprob}
