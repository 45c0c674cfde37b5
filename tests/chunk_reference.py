"""Chunk attention from its definition in float64, an entry at a time on the GPU: for caches that are too long to be
gone through on the host."""

import torch


def pool(lens, *, heads, dim, page, dtype, seed=0):
    """k, v, table, lens and refs of a cache of one layer, made on the GPU; rows past a sequence's end hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    held = [-(-n // page) for n in lens]
    pages, cols = sum(held) + 2, max(held + [1])
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), cols), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    k, v = (torch.empty((1, pages, heads, page, dim), dtype=dtype, device="cuda").normal_(generator=g) for _ in range(2))
    at = 0
    for s, n in enumerate(lens):
        mine = perm[at:at + held[s]]
        at += held[s]
        table[s, :held[s]] = mine
        refs[mine.long()] = 1
        if n % page:
            for x in (k, v):
                x[0, int(mine[-1]), :, n % page:] = float("nan")
    return k, v, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), refs


def rows_of(cache, q, s, at, m, *, scale=None, window=0, sinks=0, layer=0):
    """Of the rows q[at : at + m], the last m tokens of sequence s: the output [m, heads, dim], the log-sum-exp, the
    largest sum of |q k| * |scale| of a row, the weighted mean of |v|, and how many positions a row sees."""
    n, page = int(cache.lens[s]), cache.k.shape[3]
    heads, dim = cache.k.shape[2], cache.k.shape[4]
    scale = dim ** -0.5 if scale is None else scale
    pages = cache.table[s, :-(-n // page)].long()
    k, v = (x[layer, pages].transpose(0, 1).reshape(heads, -1, dim)[:, :n].double() for x in (cache.k, cache.v))
    rows = q[at:at + m].double().unflatten(1, (heads, -1)).permute(1, 2, 0, 3)          # [heads, group, m, dim]
    pos = torch.arange(n - m, n, device="cuda")[:, None]
    j = torch.arange(n, device="cuda")
    seen = j <= pos
    if window:
        seen &= (j < sinks) | (j > pos - window)
    score = (rows @ k[:, None].transpose(2, 3) * scale).masked_fill(~seen, float("-inf"))
    most = (rows.abs() @ k[:, None].abs().transpose(2, 3) * abs(scale)).masked_fill(~seen, 0.0).amax(-1)
    w = torch.softmax(score, -1)

    def back(x):
        return x.permute(2, 0, 1, *range(3, x.dim())).flatten(1, 2)

    return (back(w @ v[:, None]), back(torch.logsumexp(score, -1)), back(most), back(w @ v[:, None].abs()),
            seen.sum(1))
