"""Sampling (CUDA) against its definition in float64 (GPU).

z = logits / temperature is a quotient in 32 bits (correctly rounded: numpy's is bit for bit the same),
so the order of the tokens and its ties are exact. Where a filter's sum or bound decides, a token whose
sum (or weight) is within 2^-18 of its bound may be kept or not: the expected token and log-probability
are computed both ways and either is taken (weights are good to about 2^-21, their sums to the same).

Tolerance of a log-probability: the weights' relative error 2^-21, the logarithm's 2^-22 |lse|, and the
roundings of z - max and of the difference, 2^-23 (|z - max| + |logprob|).
"""

import numpy as np
import pytest
import torch

from bucketized_guidance_step_gb300 import decode

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SLACK = 2.0 ** -18


def kept(z, k, p, m, way):
    """Indices that stay, in order; way -1, 0, 1: what lies on a bound goes, as computed, stays."""
    order = np.argsort(-z, kind="stable")
    order = order[z[order] > -np.inf]
    if not len(order):
        return order
    if k > 0:
        order = order[:k]
    top = z[order[0]]
    with np.errstate(invalid="ignore"):
        w = np.where(z[order] == top, 1.0, np.exp(z[order] - top))
    if p < 1:
        before = np.cumsum(w) - w
        keep = before < max(p, 0.0) * w.sum() * (1 + way * SLACK) + way * SLACK * 2.0 ** -20
        keep[0] = True
        order, w = order[keep], w[keep]
    return order[(w >= m * (1 - way * SLACK)) | (z[order] == top)]


def expected(z, k, p, m, noise):
    """The (token, logprob) that are right."""
    answers = []
    for way in (0, -1, 1):
        order = kept(z, k, p, m, way)
        if not len(order):
            answers.append((-1, -np.inf, 0.0))
            continue
        pick = z[order].astype(np.float32)
        if noise is not None:
            pick = pick + noise[order]
        best = np.nanmax(pick) if not np.all(np.isnan(pick)) else np.nan
        if np.isnan(best):
            answers.append((-1, -np.inf, 0.0))
            continue
        token = int(order[pick == best].min())
        top = z[order[0]]
        with np.errstate(invalid="ignore"):
            rel = np.where(z[order] == top, 0.0, z[order] - top)
        mine = 0.0 if z[token] == top else z[token] - top
        lp = mine - np.log(np.exp(rel).sum())
        answers.append((token, lp, 2.0 ** -21 + 2.0 ** -22 * abs(lp) + 2.0 ** -23 * (2 * abs(mine) + abs(lp)) + 2.0 ** -22))
    return answers


def check(logits, token, logprob, *, temperature=None, top_k=None, top_p=None, min_p=None, noise=None):
    torch.cuda.synchronize()
    x = logits.float().cpu().numpy()
    B = x.shape[0]

    def row(t, b, default):
        return default if t is None else t[b].item()

    n = None if noise is None else noise.cpu().numpy()
    for b in range(B):
        hot = row(temperature, b, 1.0)
        with np.errstate(over="ignore", invalid="ignore"):
            z = x[b] / np.float32(hot) if hot > 0 else x[b]
        z = np.where(np.isnan(z), -np.inf, z).astype(np.float64)
        got = int(token[b]), float(logprob[b])
        right = expected(z, row(top_k, b, 0), row(top_p, b, 1.0), row(min_p, b, 0.0),
                         n[b if n.shape[0] > 1 else 0] if n is not None and hot > 0 else None)
        assert any(got[0] == t and (got[1] == lp or abs(got[1] - lp) <= tol) for t, lp, tol in right), (b, got, right)


def gumbel(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand(shape, generator=g, device="cuda").clamp(1e-7, 1 - 1e-7)
    return -torch.log(-torch.log(u))


def draw(B, V, dtype, seed, spread=3.0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = (torch.randn(B * (V + offset) + offset, generator=g, device="cuda") * spread).to(dtype)
    return flat[offset:].view(B, V + offset)[:, :V] if offset else flat.view(B, V)


def settings(B, seed, k=50):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = torch.rand((5, B), generator=g, device="cuda")
    return dict(temperature=torch.where(r[0] < 0.2, 0.0, 0.4 + r[0]), top_k=(r[1] * k).int(),
                top_p=torch.where(r[2] < 0.2, 1.0, r[2]), min_p=torch.where(r[3] < 0.3, 0.0, r[3] * 0.3))


def run(logits, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    token, logprob = decode.sample(logits, status=status, **kw)
    return token, logprob, int(status)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("B,V", [(1, 1), (3, 2), (5, 7), (2, 31), (9, 100), (4, 1000), (3, 4095), (2, 4096), (2, 8193),
                                 (1, 16384), (70, 5003), (3, 50021), (2, 131072), (160, 9000), (1, 262147)])
def test_sizes(dtype, B, V):
    x = draw(B, V, dtype, V)
    kw = settings(B, V, min(V + 2, 300))
    kw["noise"] = gumbel((B, V), V)
    token, logprob, word = run(x, **kw)
    check(x, token, logprob, **kw)
    assert word == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [500000, 3000001])
def test_rows_that_no_cluster_holds(dtype, V):
    x = draw(2, V, dtype, 5)
    for kw in (dict(top_k=torch.tensor([1000, 100000]).int().cuda()), dict(top_p=torch.tensor([0.9, 0.3]).cuda()),
               dict(top_p=torch.tensor([0.99, 0.5]).cuda(), top_k=torch.tensor([0, 7000]).int().cuda(),
                    min_p=torch.tensor([0.0, 0.01]).cuda(), temperature=torch.tensor([0.7, 1.3]).cuda())):
        kw["noise"] = gumbel((1, V), 3)
        token, logprob, word = run(x, **kw)
        check(x, token, logprob, **kw)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("offset", [1, 2, 3, 5, 7, 9])
def test_rows_of_any_alignment(dtype, offset):
    x = draw(6, 4100, dtype, offset, offset=offset)
    kw = settings(6, offset)
    kw["noise"] = gumbel((1, 4103), 1)[:, 3:]
    token, logprob, _ = run(x, **kw)
    check(x, token, logprob, **kw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [64, 9001, 70000])
@pytest.mark.parametrize("values", [1, 2, 5])
def test_ties_go_to_the_lowest_index(dtype, V, values):
    """Few values of z: the border lies among many tokens that share one."""
    g = torch.Generator(device="cuda").manual_seed(V + values)
    B = 12
    x = (torch.randint(0, values, (B, V), generator=g, device="cuda").float() * 0.5).to(dtype)
    ks = torch.tensor([1, 2, 3, V // 7, V // 3, V // 2, V - 1, V, 0, 5, 17, V // 5], dtype=torch.int32, device="cuda")
    ps = torch.linspace(0.05, 0.999, B, device="cuda")
    for kw in (dict(top_k=ks), dict(top_p=ps), dict(top_k=ks, top_p=ps)):
        for noise in (None, gumbel((B, V), values)):
            token, logprob, _ = run(x, noise=noise, **kw)
            check(x, token, logprob, noise=noise, **kw)


def test_flat_and_peaked_rows():
    V = 30000
    for spread in (0.0, 0.01, 0.5, 10.0, 100.0, 3e4):
        x = draw(8, V, F32, 3, spread=spread)
        kw = dict(top_p=torch.linspace(0.1, 0.9, 8, device="cuda"), noise=gumbel((8, V), 4))
        token, logprob, _ = run(x, **kw)
        check(x, token, logprob, **kw)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_infinities_and_nan(dtype):
    inf, nan = float("inf"), float("nan")
    V = 5000
    x = draw(9, V, dtype, 8)
    x[0] = -inf
    x[1] = nan
    x[2, ::2] = -inf
    x[3, 100] = inf
    x[4, 100:200] = inf
    x[5, ::3] = nan
    x[6] = -inf
    x[6, 4321] = -5.0
    x[7, 1:] = -inf
    x[8] = torch.finfo(dtype).min
    kw = settings(9, 9, 300)
    for key in (None, "top_k", "top_p", "min_p", "temperature"):
        some = {k: v for k, v in kw.items() if k != key}
        for noise in (None, gumbel((9, V), 2)):
            token, logprob, word = run(x, noise=noise, **some)
            check(x, token, logprob, noise=noise, **some)
            assert word == decode.GS_DEV_EMPTY_ROW
    noise = gumbel((9, V), 2)
    noise[:, ::2] = nan
    noise[:, 1::4] = -inf
    token, logprob, word = run(x, noise=noise)
    check(x, token, logprob, noise=noise)
    noise.fill_(-inf)
    token, logprob, word = run(x, noise=noise)
    check(x, token, logprob, noise=noise)
    noise.fill_(nan)
    token, logprob, word = run(x, noise=noise)
    assert torch.all(token == -1) and torch.all(torch.isneginf(logprob)) and word == decode.GS_DEV_EMPTY_ROW


@pytest.mark.parametrize("V", [1000, 40000, 600000])
def test_endless_temperature(V):
    """z is 0 for finite logits, and NaN, not kept, for infinite ones."""
    inf = float("inf")
    x = draw(4, V, F32, 12)
    x[0, ::3] = inf
    x[1, 1::2] = -inf
    x[2] = inf
    x[2, V - 7] = 2.0
    x[3] = -inf
    kw = dict(temperature=torch.full((4,), inf, device="cuda"))
    for some in ({}, dict(top_k=torch.tensor([3, 50, 2, 1]).int().cuda()), dict(top_p=torch.full((4,), 0.4, device="cuda"))):
        for noise in (None, gumbel((4, V), 3)):
            token, logprob, word = run(x, noise=noise, **kw, **some)
            check(x, token, logprob, noise=noise, **kw, **some)
            assert word == decode.GS_DEV_EMPTY_ROW and int(token[2]) == V - 7 and int(token[3]) == -1


def test_settings_outside_their_ranges():
    """Negative, zero, huge and tiny settings."""
    V = 3000
    x = draw(8, V, F32, 8)
    noise = gumbel((8, V), 1)
    for kw in (dict(top_k=torch.tensor([-1, 0, 1, V, V + 1, 1 << 30, -(1 << 31), 2]).int().cuda()),
               dict(top_p=torch.tensor([-1.0, 0.0, 1e-30, 1.0, 1.5, 0.9999999, 1e30, 0.5]).cuda()),
               dict(min_p=torch.tensor([-1.0, 0.0, 1e-30, 1.0, 0.999, 2.0, 1e-5, 0.5]).cuda()),
               dict(temperature=torch.tensor([-1.0, 0.0, 1e-30, 1e-3, 1e3, 1e30, 1e-45, float("inf")]).cuda())):
        token, logprob, _ = run(x, noise=noise, **kw)
        check(x, token, logprob, noise=noise, **kw)
    minus = torch.tensor([[-0.0, 0.0, -0.0, -1.0]] * 2, device="cuda")           # zeros of both signs tie
    token, _, _ = run(minus, top_k=torch.tensor([1, 2]).int().cuda())
    assert token.tolist() == [0, 0]


def test_draws_follow_the_filtered_distribution():
    """Over many rows of the same logits, tokens come as often as their probabilities say."""
    V, B = 200, 8192
    x = draw(1, V, F32, 12, spread=1.0)
    k, p = 20, 0.8
    token, logprob, _ = run(x.expand(B, V).contiguous(), noise=gumbel((B, V), 77), top_k=torch.full((B,), k).int().cuda(),
                            top_p=torch.full((B,), p).cuda())
    z = x[0].double().cpu().numpy()
    order = kept(z, k, p, 0.0, 0)
    prob = np.exp(z[order] - z[order[0]])
    prob /= prob.sum()
    count = np.bincount(token.cpu().numpy(), minlength=V)
    assert count[order].sum() == B
    # a binomial count is within 6 standard deviations
    assert np.all(np.abs(count[order] - B * prob) <= 6 * np.sqrt(B * prob * (1 - prob)) + 1)
    lp = dict(zip(order.tolist(), np.log(prob)))
    assert max(abs(lp[t] - q) for t, q in zip(token.tolist(), logprob.tolist())) < 1e-5


def test_outputs_apart_and_repeated():
    x = draw(40, 20000, BF16, 1)
    kw = settings(40, 3, 500)
    kw["noise"] = gumbel((40, 20000), 2)
    token, logprob, _ = run(x, **kw)
    one = torch.full((40,), -7, dtype=torch.int32, device="cuda")
    two = torch.full((40,), 7.0, device="cuda")
    decode.prepare_sample(x, token=one, **kw)()
    decode.prepare_sample(x, logprob=two, **kw)()
    assert torch.equal(one, token) and torch.equal(two, logprob)             # bit for bit, whatever the timing
    for _ in range(5):
        again = run(x, **kw)
        assert torch.equal(again[0], token) and torch.equal(again[1], logprob)


def test_replay_and_streams():
    B, V = 16, 30000
    x, noise = draw(B, V, F32, 1), gumbel((B, V), 2)
    kw = settings(B, 3, 500)
    token, logprob = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, device="cuda")
    call = decode.prepare_sample(x, noise=noise, token=token, logprob=logprob, **kw)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (5, 6):
        x.copy_(draw(B, V, F32, seed))
        noise.copy_(gumbel((B, V), seed))
        kw["top_p"].fill_(0.1 * seed)
        g.replay()
        check(x, token, logprob, noise=noise, **kw)
    outs = [torch.zeros_like(token) for _ in range(2)]
    calls = [decode.prepare_sample(x, noise=noise, token=o, **kw) for o in outs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            with torch.cuda.stream(s):
                c()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], token) and torch.equal(outs[1], token)


def test_large_batches_and_offsets():
    """Rows past 2^31 elements."""
    V, B = 300000, 8000
    x = torch.full((B, V), -30.0, dtype=BF16, device="cuda")
    at = torch.randint(0, V, (B, 4), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    x.scatter_(1, at, torch.tensor([1.0, 2.0, 3.0, 4.0], dtype=BF16, device="cuda").expand(B, 4).contiguous())
    token, logprob, _ = run(x, top_k=torch.full((B,), 1).int().cuda())
    assert torch.equal(token.long(), at[:, 3]) and torch.all(logprob == 0)


def test_after_guided_logits():
    """The two together, as a decode step uses them: penalties and the grammar first, then the filters."""
    B, V = 5, 3001
    logits = draw(2 * B, V, BF16, 4)
    tokens = torch.randint(0, V, (B, 30), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").int()
    mask = torch.randint(-(1 << 31), 1 << 31, (1, (V + 31) // 32), device="cuda",
                         generator=torch.Generator(device="cuda").manual_seed(2)).int()
    z, greedy, lp = decode.guided_logits(stacked=logits, cfg=1.5, tokens=tokens, mask=mask,
                                         tokens_len=torch.full((B,), 30).int().cuda(),
                                         repetition=torch.full((B,), 1.2, device="cuda"))
    kw = settings(B, 6)
    kw["noise"] = gumbel((B, V), 3)
    token, logprob, _ = run(z, **kw)
    check(z, token, logprob, **kw)
    # no filter and no noise: the token and log-probability of guided_logits itself
    token, logprob, _ = run(z)
    assert torch.equal(token, greedy) and (logprob - lp).abs().max() < 1e-5


@pytest.mark.parametrize("name,value", [
    ("temperature", torch.ones(3)), ("top_k", torch.ones(4, dtype=torch.int64)), ("top_p", torch.ones(4).double()),
    ("min_p", torch.ones(4, 1)), ("noise", torch.zeros(2, 100)), ("noise", torch.zeros(4, 99)),
    ("token", torch.zeros(4)), ("logprob", torch.zeros(5)),
])
def test_the_binding_refuses(name, value):
    x = torch.zeros(4, 100, device="cuda")
    with pytest.raises(ValueError):
        decode.sample(x, **{name: value.cuda()})
    with pytest.raises(ValueError):
        decode.sample(x, noise=torch.zeros(4, 200, device="cuda")[:, ::2])
    with pytest.raises(ValueError):
        decode.sample(x[:, ::2])
    with pytest.raises(ValueError):
        decode.sample(x[:1].expand(4, 100))
    with pytest.raises(ValueError):
        decode.prepare_sample(x)
