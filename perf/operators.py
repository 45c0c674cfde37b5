"""The decode operators as they are measured: attention over a paged cache, the cache's pages, guided logits.

Every case runs in two forms on the same inputs: the plain form (elementary torch operations
in 32 bits) and, with ``own`` set, the library's entry points through
``bucketized_guidance_step_gb300.decode``.

The definitions that both follow:

* A cache holds K and V as [layers, pages, kv_heads, page, dim]. Sequence s has lens[s] tokens;
  token t lies in page table[s, t // page] at row t % page. refs[p] counts the sequences that
  hold page p; a page of count 0 is free. Pages are taken lowest number first, in the order of
  the call's list.
* attention: one query token a sequence, over the visible positions (all, or the first `sinks`
  and the last `window`); with `append` the new token's K and V are first stored at position
  lens - 1. Returns the output and the log-sum-exp of the scaled scores.
* fork: the children release what they hold and share the parents' full pages; a partly filled
  last page is copied (its filled rows) into a page of the child's own.
* compact: with n live pages, the k-th lowest free page below n takes over the k-th highest
  live page.
* admit: finished sequences are freed, the same rows take new prompts (extend), and the
  prompts' K and V are written layer by layer.
* logits: z = uncond + s (cond - uncond), with s from a bucket table; + bias; the penalties for
  the tokens of the history; / temperature (0: greedy, z as it is and no noise); -inf where the
  grammar mask forbids. The token is the lowest index of the largest z (+ noise).
"""

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
LAYER = 0          # attention reads one layer a call
STEPS, BUCKETS = 50, 8


def _attn(name, batch, q_heads, kv_heads, dim, page, lo, hi, dtype, window=0, sinks=0, append=False):
    c = {"op": "attention", "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
         "page": page, "len_lo": lo, "len_hi": hi, "dtype": dtype, "window": window, "sinks": sinks,
         "append": append}
    return {"name": name, **c} if name else c


def _fork(name, pairs, layers, kv_heads, dim, page, lo, hi, dtype):
    c = {"op": "fork", "pairs": pairs, "layers": layers, "kv_heads": kv_heads, "dim": dim,
         "page": page, "len_lo": lo, "len_hi": hi, "dtype": dtype}
    return {"name": name, **c} if name else c


def _compact(name, pages, live, seqs, layers, kv_heads, dim, page, dtype):
    c = {"op": "compact", "pages": pages, "live": live, "seqs": seqs, "layers": layers,
         "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype}
    return {"name": name, **c} if name else c


def _admit(name, seqs, done, layers, kv_heads, dim, page, lo, hi, dtype):
    c = {"op": "admit", "seqs": seqs, "done": done, "layers": layers, "kv_heads": kv_heads,
         "dim": dim, "page": page, "len_lo": lo, "len_hi": hi, "dtype": dtype}
    return {"name": name, **c} if name else c


def _logits(name, batch, vocab, dtype, guided, history, masked, bias, noise):
    c = {"op": "logits", "batch": batch, "vocab": vocab, "dtype": dtype, "guided": guided,
         "history": history, "masked": masked, "bias": bias, "noise": noise}
    return {"name": name, **c} if name else c


def listed():
    return [
        # One sample's two branches at the start of an image: a few hundred tokens. Latency counts.
        _attn("attn_two_short", 2, 16, 16, 64, 16, 1, 250, "fp16", append=True),
        # A continuous batch of 16 guided samples (32 branches) at ragged lengths.
        _attn("attn_ragged_32", 32, 32, 8, 128, 16, 1, 4099, "bf16", append=True),
        # One long context: the split over the length carries it.
        _attn("attn_long", 2, 32, 8, 128, 64, 200001, 262143, "bf16"),
        # A stream kept to a window and a few first tokens, many branches.
        _attn("attn_window", 128, 16, 4, 128, 32, 900, 16384, "fp16", window=1024, sinks=4, append=True),
        # A 32-bit model, narrow heads and an odd page size.
        _attn("attn_fp32", 8, 8, 4, 96, 24, 333, 3001, "fp32"),
        # The uncond branches of 16 prompts fork off; few layers: latency.
        _fork("fork_16", 16, 4, 8, 64, 16, 1, 255, "bf16"),
        # Best-of-n over a deep cache with long pages.
        _fork("fork_deep_64", 64, 32, 8, 128, 64, 17, 2047, "bf16"),
        # A half-empty pool is made dense.
        _compact("compact_half", 4096, 2048, 61, 4, 8, 128, 16, "bf16"),
        # Finished samples leave, new prompts come in.
        _admit("admit_24", 64, 24, 2, 8, 128, 16, 1, 1023, "bf16"),
        # One guided sample of a small codebook. Latency counts.
        _logits("logits_one", 1, 16384, "bf16", True, 200, False, False, True),
        # The guided batch of a large vocabulary, with a grammar.
        _logits("logits_64", 64, 131072, "bf16", True, 2048, True, True, True),
        # Unguided rows of an odd vocabulary in 32 bits, greedy and sampled.
        _logits("logits_odd", 33, 50021, "fp32", False, 1500, True, False, False),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(2 ** rng.uniform(np.log2(lo), np.log2(hi))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "fork", "compact", "admit", "logits", "logits"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    layers, kv_heads, dim = rng.randint(1, 8), rng.randint(1, 8), rng.choice([64, 80, 96, 128, 256])
    if op == "attention":
        kv_heads, group = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([1, 2, 3, 4, 6, 8, 16])
        batch = _log(rng, 1, 128)
        row = kv_heads * dim * 2 * SIZE[dtype]
        hi = _log(rng, 1, max(2, min(262143, int(1.2e9 / (row * batch)))))
        lo = rng.randint(0, hi)
        window = rng.choice([0, 0, _log(rng, 1, 4096)])
        return _attn(None, batch, kv_heads * group, kv_heads, dim, page, lo, hi, dtype, window,
                     rng.randint(0, 16) if window else 0, lo > 0 and rng.random() < 0.5)
    if op == "fork":
        hi = _log(rng, 1, 2048)
        return _fork(None, _log(rng, 1, 64), layers, kv_heads, dim, page, rng.randint(1, hi), hi, dtype)
    if op == "compact":
        per = page * kv_heads * dim * layers * 2 * SIZE[dtype]
        pages = _log(rng, 16, max(17, min(16384, int(1e9 / per))))
        return _compact(None, pages, rng.randint(8, pages), rng.randint(1, 64), layers, kv_heads, dim, page, dtype)
    if op == "admit":
        hi = _log(rng, 1, 1024)
        seqs = _log(rng, 1, 64)
        return _admit(None, seqs, rng.randint(1, seqs), min(layers, 4), kv_heads, dim, page,
                      rng.randint(1, hi), hi, dtype)
    return _logits(None, _log(rng, 1, 64), _log(rng, 1000, 160000), dtype, rng.random() < 0.6,
                   _log(rng, 1, 4096), rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5)


def _spread(lo, hi, n):
    """n lengths over [lo, hi], the last of them hi."""
    return [lo + (hi - lo) * (i + 1) // n for i in range(n)]


def _up(a, b):
    return -(-a // b)


def _normal(shape, dtype, g, sd=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(sd).to(dtype)


def _big(shape, dtype, g):
    """A large cache of normal values: drawn by layer, so that no 32-bit copy of it is held."""
    out = torch.empty(shape, device="cuda", dtype=dtype)
    for layer in out:
        layer.normal_(generator=g)
    return out


def _cache(case, seed, lens, seqs, cols, pages, layers):
    """K, V, a table whose sequences (lens, the first of seqs rows) hold random pages, and the counts."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (layers, pages, case["kv_heads"], case["page"], case["dim"])
    dt = DTYPES[case["dtype"]]
    perm = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int64).int()
    order = torch.randperm(len(lens), generator=g, device="cuda")
    full = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    full[:len(lens)] = torch.tensor(lens, dtype=torch.int32, device="cuda")[order]
    held = (full + case["page"] - 1) // case["page"]
    at = held.cumsum(0) - held
    col = torch.arange(cols, device="cuda")
    live = col < held[:, None]
    table = torch.where(live, perm[(at[:, None] + col).clamp(max=pages - 1)], -1).int()
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs.index_add_(0, table.clamp(min=0).flatten(), live.int().flatten())
    return {"k": _big(shape, dt, g), "v": _big(shape, dt, g), "table": table, "lens": full, "refs": refs, "g": g}


def prepare(case, seed):
    s = {"attention": _prepare_attention, "fork": _prepare_fork, "compact": _prepare_compact,
         "admit": _prepare_admit, "logits": _prepare_logits}[case["op"]](case, seed)
    s.update(case=case, op=case["op"])
    if own:
        _plan(s)
    return s


def _prepare_attention(case, seed):
    B, page = case["batch"], case["page"]
    lens = _spread(case["len_lo"], case["len_hi"], B)
    s = _cache(case, seed, lens, B, max(1, _up(case["len_hi"], page)), sum(_up(n, page) for n in lens) + B, 1)
    dt = DTYPES[case["dtype"]]
    s["q"] = _normal((B, case["q_heads"], case["dim"]), dt, s["g"], 2.0)
    s["scale"] = float(case["dim"]) ** -0.5
    for name in ("k_new", "v_new"):
        s[name] = _normal((B, case["kv_heads"], case["dim"]), dt, s["g"]) if case["append"] else None
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((B, case["q_heads"]), dtype=torch.float32, device="cuda")
    return s


def _prepare_fork(case, seed):
    n, page = case["pairs"], case["page"]
    lens = _spread(case["len_lo"], case["len_hi"], n)
    s = _cache(case, seed, lens, 2 * n, _up(case["len_hi"], page) + 1, sum(_up(x, page) for x in lens) + 2 * n, case["layers"])
    s["src"] = torch.arange(n, dtype=torch.int32, device="cuda")
    s["dst"] = torch.randperm(n, generator=s["g"], device="cuda").int() + n
    return s


def _prepare_compact(case, seed):
    page, live, seqs = case["page"], case["live"], case["seqs"]
    lens = [max(0, ((i + 1) * live // seqs - i * live // seqs) * page - 1) for i in range(seqs)]
    s = _cache(case, seed, lens, seqs, _up(live, seqs) + 1, case["pages"], case["layers"])
    s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
    s["live"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def _prepare_admit(case, seed):
    seqs, done, page = case["seqs"], case["done"], case["page"]
    lens = _spread(case["len_lo"], case["len_hi"], seqs)
    add = _spread(case["len_lo"], case["len_hi"], done)
    cols = _up(case["len_hi"], page)
    s = _cache(case, seed, lens, seqs, cols, seqs * cols + 8, case["layers"])
    s["seq"] = torch.randperm(seqs, generator=s["g"], device="cuda")[:done].int()
    s["add"] = torch.tensor(add, dtype=torch.int32, device="cuda")[torch.randperm(done, generator=s["g"], device="cuda")]
    s["start"] = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), s["add"].cumsum(0).int()])
    shape = (case["layers"], sum(add), case["kv_heads"], case["dim"])
    s["k_new"], s["v_new"] = (_normal(shape, DTYPES[case["dtype"]], s["g"]) for _ in range(2))
    return s


def _prepare_logits(case, seed):
    B, V, T = case["batch"], case["vocab"], case["history"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def uniform(lo, hi):
        return torch.rand(B, generator=g, device="cuda") * (hi - lo) + lo

    cond = torch.randn((B, V), generator=g, device="cuda") * 3.0
    s = {}
    if case["guided"]:
        uncond = cond + torch.randn((B, V), generator=g, device="cuda")
        s["logits"] = torch.cat([uncond, cond]).to(dt)              # [uncond; cond]
    else:
        s["logits"] = cond.to(dt)
    bucket = (torch.arange(STEPS, device="cuda") * BUCKETS) // STEPS
    s["lut"] = (2.0 - 0.8 * (bucket + 0.5) / BUCKETS).float()       # 2.0 -> 1.2 over the steps
    s["step_idx"] = torch.randint(0, STEPS, (B,), generator=g, device="cuda", dtype=torch.int32)
    # tokens of a history repeat: small indices often, the rest of the vocabulary now and then
    u = torch.rand((B, T), generator=g, device="cuda")
    s["tokens"] = (V * u.pow(4)).long().clamp(max=V - 1).int()
    order = torch.randperm(B, generator=g, device="cuda")
    s["tokens_len"] = torch.tensor(_spread(0, T, B), dtype=torch.int32, device="cuda")[order]
    s["prompt_len"] = s["tokens_len"] // 3
    s["repetition"], s["frequency"], s["presence"] = uniform(1.0, 1.3), uniform(0.0, 0.5), uniform(0.0, 0.5)
    s["temperature"] = torch.where(torch.rand(B, generator=g, device="cuda") < 0.25, 0.0, uniform(0.5, 1.5))
    words = _up(V, 32)
    s["mask"] = None
    if case["masked"]:                                              # a grammar allows few tokens or most
        bits = torch.rand((B, words, 32), generator=g, device="cuda") < uniform(0.002, 1.0).pow(2)[:, None, None]
        s["mask"] = (bits.long() << torch.arange(32, device="cuda")).sum(2).to(torch.int64)
        s["mask"] = torch.where(s["mask"] >= 1 << 31, s["mask"] - (1 << 32), s["mask"]).int()
    s["bias"] = torch.randn((1, V), generator=g, device="cuda") if case["bias"] else None
    s["noise"] = -torch.log(-torch.log(torch.rand((B, V), generator=g, device="cuda").clamp(1e-7, 1 - 1e-7))) \
        if case["noise"] else None
    s["z"] = torch.empty((B, V), dtype=torch.float32, device="cuda")
    s["token"] = torch.empty(B, dtype=torch.int32, device="cuda")
    s["logprob"] = torch.empty(B, dtype=torch.float32, device="cuda")
    return s


def _plan(s):
    """The handles that a user's program keeps: the cache and the prepared calls on its buffers."""
    from bucketized_guidance_step_gb300 import decode
    if s["op"] == "logits":
        g = s["case"]["guided"]
        s["calls"] = [decode.prepare_guided_logits(
            s["logits"] if not g else None, stacked=s["logits"] if g else None, step_idx=s["step_idx"] if g else None,
            scale_lut=s["lut"] if g else None, tokens=s["tokens"], tokens_len=s["tokens_len"],
            prompt_len=s["prompt_len"], repetition=s["repetition"], frequency=s["frequency"],
            presence=s["presence"], temperature=s["temperature"], mask=s["mask"], bias=s["bias"],
            noise=s["noise"], out=s["z"], token=s["token"], logprob=s["logprob"])]
        return
    c = s["cache"] = decode.PagedCache(s["k"], s["v"], s["table"], s["lens"], s["refs"])
    if s["op"] == "attention":
        s["calls"] = [c.prepare_attention(s["q"], LAYER, k_new=s["k_new"], v_new=s["v_new"], scale=s["scale"],
                                          window=s["case"]["window"], sinks=s["case"]["sinks"], out=s["out"], lse=s["lse"])]
    elif s["op"] == "fork":
        s["calls"] = [c.prepare_fork(s["src"], s["dst"])]
    elif s["op"] == "compact":
        s["calls"] = [c.prepare_compact(table_out=s["table_out"], refs_out=s["refs_out"], live=s["live"])]
    else:
        s["calls"] = [c.prepare_free(s["seq"]), c.prepare_extend(s["seq"], s["add"])]
        s["calls"] += [c.prepare_write(i, s["k_new"][i], s["v_new"][i], s["seq"], s["start"]) for i in range(s["case"]["layers"])]


def _outputs(s):
    if s["op"] == "attention":
        got = {"out": s["out"], "lse": s["lse"]}
        return {**got, "k": s["k"], "v": s["v"]} if s["case"]["append"] else got
    if s["op"] == "logits":
        return {"logits": s["z"], "token": s["token"], "logprob": s["logprob"]}
    if s["op"] == "compact":
        return {"table": s["table_out"], "refs": s["refs_out"], "live": s["live"], "k": s["k"], "v": s["v"]}
    return {"table": s["table"], "refs": s["refs"], "lens": s["lens"], "k": s["k"], "v": s["v"]}


def run(s):
    if own:
        [call() for call in s["calls"]]
    else:
        {"attention": _attention, "fork": _fork_pages, "compact": _compact_pages, "admit": _admit_prompts,
         "logits": _guided_logits}[s["op"]](s)
    return _outputs(s)


# ---- plain forms ---------------------------------------------------------------------------------
def _attention(s):
    c, page = s["case"], s["case"]["page"]
    B, Hq, D = s["q"].shape
    Hkv = c["kv_heads"]
    lens = s["lens"].long()
    if c["append"]:
        at = lens - 1
        where = s["table"].gather(1, (at // page)[:, None])[:, 0].long()
        s["k"][LAYER][where, :, at % page] = s["k_new"]
        s["v"][LAYER][where, :, at % page] = s["v_new"]
    n = c["sinks"] + c["window"] if c["window"] else c["len_hi"]
    j = torch.arange(min(n, c["len_hi"]), device="cuda")
    first = (lens - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(lens)
    sinks = torch.minimum(first, torch.full_like(first, c["sinks"]))
    pos = torch.where(j < sinks[:, None], j, j + (first - sinks)[:, None])
    seen = pos < lens[:, None]
    pos = torch.where(seen, pos, 0)
    pages = s["table"].gather(1, pos // page).clamp(min=0).long()
    k = s["k"][LAYER][pages, :, pos % page].float()                 # [B, n, Hkv, D]
    v = s["v"][LAYER][pages, :, pos % page].float()
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]     # [B, Hkv, G, n]
    score = score.masked_fill(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(score - top).masked_fill(~seen[:, None, None], 0.0)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.transpose(1, 2).masked_fill(~seen[:, None, :, None], 0.0))
    o = torch.where(total > 0, o / total, 0.0)
    s["out"].copy_(o.view(B, Hq, D))
    s["lse"].copy_((top + torch.log(total)).view(B, Hq))


def _free_pages(refs):
    """The free pages' numbers in rising order (those held come after them)."""
    return torch.sort((refs > 0).int(), stable=True).indices


def _release(s, seq):
    page, table, lens, refs = s["case"]["page"], s["table"], s["lens"], s["refs"]
    held = torch.arange(table.shape[1], device="cuda") < ((lens[seq] + page - 1) // page)[:, None]
    refs.index_add_(0, table[seq].clamp(min=0).flatten(), -held.int().flatten())


def _fork_pages(s):
    page, table, lens, refs = s["case"]["page"], s["table"], s["lens"], s["refs"]
    src, dst = s["src"].long(), s["dst"].long()
    _release(s, dst)
    rows, n = table[src], lens[src]
    col = torch.arange(table.shape[1], device="cuda")
    full = n // page
    shared = col < full[:, None]
    refs.index_add_(0, rows.clamp(min=0).flatten(), shared.int().flatten())
    part = n % page
    need = part > 0
    last = rows.gather(1, ((n - 1) // page).long()[:, None])[:, 0].long()
    taken = _free_pages(refs)[(need.cumsum(0) - need.long()).clamp(min=0)]
    fresh = torch.where(need, taken, last)
    refs.index_add_(0, fresh, need.int())
    table[dst] = torch.where(shared, rows, torch.where((col == full[:, None]) & need[:, None], fresh[:, None].int(), -1))
    lens[dst] = n
    filled = (torch.arange(page, device="cuda") < part[:, None])[None, :, None, :, None]
    s["k"][:, fresh] = torch.where(filled, s["k"][:, last], s["k"][:, fresh])
    s["v"][:, fresh] = torch.where(filled, s["v"][:, last], s["v"][:, fresh])


def _compact_pages(s):
    refs, table = s["refs"], s["table"]
    P = refs.shape[0]
    live = refs > 0
    n = live.sum()
    page = torch.arange(P, device="cuda")
    holes = torch.sort((live | (page >= n)).int(), stable=True).indices          # holes below n, rising
    top = (live & (page >= n)).flip(0)
    movers = P - 1 - torch.sort((~top).int(), stable=True).indices               # live pages from n on, falling
    count = int(top.sum())
    holes, movers = holes[:count], movers[:count]
    to = page.clone()
    to[movers] = holes
    s["table_out"].copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    s["refs_out"].copy_(torch.where(page < n, refs, 0))
    s["refs_out"][holes] = refs[movers]
    s["live"].copy_(n)
    s["k"][:, holes] = s["k"][:, movers]
    s["v"][:, holes] = s["v"][:, movers]


def _admit_prompts(s):
    page, table, lens, refs = s["case"]["page"], s["table"], s["lens"], s["refs"]
    seq, add = s["seq"].long(), s["add"]
    _release(s, seq)
    need = (add + page - 1) // page
    at = need.cumsum(0) - need
    col = torch.arange(table.shape[1], device="cuda")
    mine = col < need[:, None]
    taken = _free_pages(refs)[(at[:, None] + col).clamp(max=refs.shape[0] - 1)]
    refs.index_add_(0, taken.flatten(), mine.int().flatten())
    table[seq] = torch.where(mine, taken.int(), -1)
    lens[seq] = add
    t = torch.arange(s["k_new"].shape[1], device="cuda")
    row = torch.searchsorted(s["start"][1:].contiguous(), t.int(), right=True)
    pos = t - s["start"][row]
    where = table[seq[row], pos // page].long()
    # one assignment: [tokens, layers, kv_heads, dim]
    s["k"].permute(1, 3, 0, 2, 4)[where, pos % page] = s["k_new"].transpose(0, 1)
    s["v"].permute(1, 3, 0, 2, 4)[where, pos % page] = s["v_new"].transpose(0, 1)


def _guided_logits(s):
    c = s["case"]
    B, V = c["batch"], c["vocab"]
    low = float("-inf")
    if c["guided"]:
        scale = s["lut"][s["step_idx"].long()][:, None]
        uncond, cond = s["logits"][:B].float(), s["logits"][B:].float()
        z = uncond + scale * (cond - uncond)
        z = torch.where(cond == low, low, torch.where(uncond == low, cond, z))
    else:
        z = s["logits"].float()
    if s["bias"] is not None:
        z = z + s["bias"]
    t = torch.arange(s["tokens"].shape[1], device="cuda")
    known = t < s["tokens_len"][:, None]
    said = (known & (t >= s["prompt_len"][:, None])).float()
    tokens = s["tokens"].long()
    seen = torch.zeros((B, V), device="cuda").scatter_add_(1, tokens, known.float()) > 0
    count = torch.zeros((B, V), device="cuda").scatter_add_(1, tokens, said)
    r = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
    z = z - (s["frequency"][:, None] * count + s["presence"][:, None] * (count > 0))
    hot = s["temperature"][:, None]
    z = torch.where(hot > 0, z / hot, z)
    if s["mask"] is not None:
        v = torch.arange(V, device="cuda")
        z = torch.where(((s["mask"][:, v // 32] >> (v % 32).int()) & 1) > 0, z, low)
    pick = z if s["noise"] is None else torch.where(hot > 0, z + s["noise"], z)
    best = pick.amax(1, keepdim=True)
    v = torch.arange(V, device="cuda")
    token = torch.where((pick == best) & (pick > low), v, V).amin(1)
    top = z.amax(1, keepdim=True).clamp(min=-3e38)
    lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
    none = token == V
    s["z"].copy_(z)
    s["token"].copy_(torch.where(none, -1, token))
    s["logprob"].copy_(torch.where(none, low, z.gather(1, token.clamp(max=V - 1)[:, None])[:, 0] - lse))


# ---- what a pass cannot do without ----------------------------------------------------------------
def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "logits":
        B, V = case["batch"], case["vocab"]
        words = e * (2 if case["guided"] else 1) + 4 + (4 if case["noise"] else 0)   # in, out, noise
        known = sum(_spread(0, case["history"], B))
        return {"bytes": B * (V * words + (V // 8 if case["masked"] else 0) + 40) + 4 * V * bool(case["bias"]) + 4 * known,
                "flops": B * V * (12 if case["guided"] else 8)}
    page, token = case["page"], case["kv_heads"] * case["dim"] * 2 * e                 # K and V of a token
    if case["op"] == "attention":
        lens = _spread(case["len_lo"], case["len_hi"], case["batch"])
        seen = sum(min(n, case["sinks"] + case["window"]) if case["window"] else n for n in lens)
        B, Hq, D = case["batch"], case["q_heads"], case["dim"]
        return {"bytes": seen * token + (B * token if case["append"] else 0) + 2 * B * Hq * D * e + 4 * B * Hq + 4 * (seen // page),
                "flops": 4.0 * seen * Hq * D}
    if case["op"] == "fork":
        lens = _spread(case["len_lo"], case["len_hi"], case["pairs"])
        pages = sum(_up(n, page) for n in lens)
        return {"bytes": 2 * case["layers"] * token * sum(n % page for n in lens) + 4 * (4 * pages + case["pairs"] * 4), "flops": 0}
    if case["op"] == "compact":
        moved = case["live"] * (case["pages"] - case["live"]) / case["pages"]          # of a random pool
        return {"bytes": 2 * case["layers"] * token * page * moved + 8 * (case["pages"] + case["live"]), "flops": 0}
    add = sum(_spread(case["len_lo"], case["len_hi"], case["done"]))
    return {"bytes": 2 * case["layers"] * token * add + 4 * 6 * (add // page) + 4 * case["seqs"], "flops": 0}


# ---- 64 bits ------------------------------------------------------------------------------------
def exact(case, seed):
    """The computed outputs from their definitions in 64 bits, one row after the other. Pages hold
    copies of their inputs: nothing is computed there."""
    if case["op"] not in ("attention", "logits"):
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _exact_attention(s) if case["op"] == "attention" else _exact_logits(s)


def _exact_attention(s):
    c, page = s["case"], s["case"]["page"]
    B, Hq, D = s["q"].shape
    Hkv = c["kv_heads"]
    out = torch.zeros((B, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        pages = s["table"][b, :_up(n, page)].long()
        for h in range(Hkv):
            k = s["k"][LAYER][pages, h].reshape(-1, D)[:n].double()
            v = s["v"][LAYER][pages, h].reshape(-1, D)[:n].double()
            if c["append"]:
                k[n - 1], v[n - 1] = s["k_new"][b, h].double(), s["v_new"][b, h].double()
            if c["window"] and n > c["window"]:
                first = n - c["window"]
                keep = torch.cat([torch.arange(min(c["sinks"], first)), torch.arange(first, n)]).to(k.device)
                k, v = k[keep], v[keep]
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            score = (s["q"][b, heads].double() @ k.T) * s["scale"]
            lse[b, heads] = torch.logsumexp(score, 1)
            out[b, heads] = torch.softmax(score, 1) @ v
    got = {"out": out, "lse": lse}
    return {**got, "k": None, "v": None} if c["append"] else got


def _exact_logits(s):
    c = s["case"]
    B, V = c["batch"], c["vocab"]
    z = torch.empty((B, V), dtype=torch.float64, device="cuda")
    token = torch.empty(B, dtype=torch.int32)
    logprob = torch.empty(B, dtype=torch.float64)
    for b in range(B):
        if c["guided"]:
            w = s["lut"][int(s["step_idx"][b])].double()
            u, k = s["logits"][b].double(), s["logits"][B + b].double()
            row = (1.0 - w) * u + w * k
            row[u == -torch.inf] = k[u == -torch.inf]
            row[k == -torch.inf] = -torch.inf
        else:
            row = s["logits"][b].double()
        if s["bias"] is not None:
            row = row + s["bias"][0].double()
        n, first = int(s["tokens_len"][b]), int(s["prompt_len"][b])
        seen = torch.unique(s["tokens"][b, :n].long())
        r = float(s["repetition"][b])
        row[seen] = torch.where(row[seen] > 0, row[seen] / r, row[seen] * r)
        said, times = torch.unique(s["tokens"][b, first:n].long(), return_counts=True)
        row[said] -= float(s["frequency"][b]) * times + float(s["presence"][b])
        hot = float(s["temperature"][b])
        if hot > 0:
            row = row / hot
        if s["mask"] is not None:
            bits = np.unpackbits(s["mask"][b].cpu().numpy().view(np.uint8), bitorder="little")[:V]
            row[torch.from_numpy(bits == 0).to(row.device)] = -torch.inf
        pick = row + s["noise"][b].double() if s["noise"] is not None and hot > 0 else row
        z[b] = row
        if bool((row > -torch.inf).any()):
            token[b] = int((pick == pick.max()).nonzero()[0])
            logprob[b] = float(row[token[b]] - torch.logsumexp(row, 0))
        else:
            token[b], logprob[b] = -1, -torch.inf
    return {"logits": z, "token": token, "logprob": logprob}
