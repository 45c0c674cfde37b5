"""Guided logits (CUDA) against the oracle in float64 (GPU).

Tolerance of z: every step rounds once in fp32, at most eight of them (product, fma, bias,
repetition, penalty and its sum, reciprocal, temperature), each relative to the magnitude
`size` that the oracle carries along: 8 * 2^-24 * size. The log-probability adds the same
for the token and for the sum, 2^-24 (vocab / 8 + 64) for the sum's roundings, and 2^-22 of its
own size. A token may differ from the oracle's only where the two picks lie within twice
the tolerance of each other.
"""

import numpy as np
import pytest
import torch

from bucketized_guidance_step_gb300 import decode, gs
from oracle import decode as O

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 2.0 ** -24


def words(allowed):
    """Bool [B, V] -> int32 bit words [B, ceil(V / 32)]."""
    B, V = allowed.shape
    padded = np.zeros((B, -(-V // 32) * 32), bool)
    padded[:, :V] = allowed
    return torch.from_numpy(np.packbits(padded, axis=1, bitorder="little").view(np.int32).copy()).cuda()


def check(got, rows, noise=None, temperature=None):
    out, token, logprob = (x.double().cpu().numpy() for x in got)
    for b, (z, tok, lp, size, pick) in enumerate(rows):
        V = len(z)
        tol = 8 * EPS * size + 1e-37
        assert np.array_equal(np.isneginf(out[b]), np.isneginf(z)), b
        fin = np.isfinite(z)
        assert np.all(np.abs(out[b][fin] - z[fin]) <= tol[fin]), (b, np.max(np.abs(out[b][fin] - z[fin]) / tol[fin]))
        t = int(token[b])
        if tok < 0:
            assert t == -1 and np.isneginf(logprob[b])
            continue
        slack = 2 * (tol.max() + EPS * np.abs(pick[np.isfinite(pick)]).max())
        assert t == tok or pick[t] >= pick[tok] - slack, (b, t, tok)
        want = z[t] - z[tok] + lp
        bound = 2 * tol[fin].max() + EPS * (V / 8 + 64) + 4 * EPS * abs(want) + 4 * EPS * np.abs(z[fin]).max()
        assert abs(logprob[b] - want) <= bound, (b, logprob[b], want)


def inputs(B, V, T, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    cond = (torch.randn((B, V), generator=g) * 4).to(dtype)
    uncond = (cond.float() + torch.randn((B, V), generator=g)).to(dtype)
    tokens = torch.randint(-1, V + 1, (B, T), generator=g, dtype=torch.int32)     # some outside
    tokens[:, ::2] = tokens[:, ::2] % max(1, V // 50)                             # many repeats
    length = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32)
    length[0] = T
    prompt = (length * torch.rand(B, generator=g)).int()
    vec = lambda lo, hi: torch.rand(B, generator=g) * (hi - lo) + lo               # noqa: E731
    return dict(cond=cond, uncond=uncond, tokens=tokens, tokens_len=length, prompt_len=prompt,
                repetition=vec(0.8, 1.5), frequency=vec(-0.2, 0.6), presence=vec(-0.2, 0.6),
                temperature=torch.where(torch.arange(B) % 4 == 1, 0.0, vec(0.3, 2.0)),
                bias=torch.randn((B, V), generator=g), noise=-torch.log(-torch.log(
                    torch.rand((B, V), generator=g).clamp(1e-6, 1 - 1e-6))),
                allowed=(torch.rand((B, V), generator=g) < 0.3).numpy())


def oracle_rows(x, scale, masked=True, noise=True):
    rows = []
    for b in range(x["cond"].shape[0]):
        n = int(x["tokens_len"][b])
        rows.append(O.guided_logits(
            x["cond"][b].double().numpy(), x["uncond"][b].double().numpy(), float(scale[b]),
            x["bias"][b].double().numpy(), x["tokens"][b, :n].tolist(), int(x["prompt_len"][b]),
            *(float(x[n][b]) for n in ("repetition", "frequency", "presence", "temperature")),
            allowed=x["allowed"][b] if masked else None,
            noise=x["noise"][b].double().numpy() if noise else None))
    return rows


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("B,V,T", [(1, 1, 1), (3, 7, 5), (5, 33, 40), (2, 2048, 300), (4, 4099, 1000),
                                   (3, 20000, 5000), (70, 8200, 64), (700, 513, 9)])
def test_everything_together(dtype, B, V, T):
    x = inputs(B, V, T, dtype, seed=V + B)
    lut = torch.tensor([3.0, 1.0, 0.0, 7.5, -1.25])
    idx = torch.arange(B, dtype=torch.int32) % 5
    dev = {n: v.cuda() for n, v in x.items() if n != "allowed"}
    got = decode.guided_logits(step_idx=idx.cuda(), scale_lut=lut.cuda(), mask=words(x["allowed"]), **dev)
    check(got, oracle_rows(x, lut[idx.long()]))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_alignment(dtype):
    """Rows of wider tensors, off the 16-byte boundary, and one row shared by all."""
    B, V = 5, 1000
    x = inputs(B, V, 50, dtype, seed=3)
    both = torch.zeros((2 * B, V + 13), dtype=dtype).cuda()
    both[:B, 5:5 + V], both[B:, 5:5 + V] = x["uncond"].cuda(), x["cond"].cuda()
    out = torch.full((B, V + 3), 9.0, device="cuda")
    for n in ("bias", "noise"):
        x[n] = x[n][:1].expand(B, V)
    x["allowed"] = np.repeat(x["allowed"][:1], B, 0)
    dev = {n: v.cuda() for n, v in x.items() if n not in ("allowed", "cond", "uncond", "bias", "noise")}
    token, logprob = torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(B, device="cuda")
    decode.guided_logits(stacked=both[:, 5:5 + V], cfg=2.5, bias=x["bias"][:1].cuda(),
                         noise=x["noise"][:1].cuda(), mask=words(x["allowed"][:1]), out=out[:, 1:1 + V],
                         token=token, logprob=logprob, **dev)
    check((out[:, 1:1 + V], token, logprob), oracle_rows(x, [2.5] * B))
    assert (out[:, 0] == 9).all() and (out[:, 1 + V:] == 9).all()


def test_masks_that_leave_a_row_empty_and_absent_masks():
    B, V = 4, 5000
    x = inputs(B, V, 10, F32, seed=1)
    x["allowed"][1] = False
    x["allowed"][2] = False
    x["allowed"][2, 4999] = True                       # one token left: its probability is 1
    status = torch.zeros(1, dtype=torch.int32).cuda()
    present = torch.tensor([1, 1, 1, 0], dtype=torch.uint8).cuda()
    dev = {n: v.cuda() for n, v in x.items() if n != "allowed"}
    got = decode.guided_logits(cfg=1.5, mask=words(x["allowed"]), mask_present=present, status=status, **dev)
    x["allowed"][3] = True
    check(got, oracle_rows(x, [1.5] * B))
    assert got[1].tolist()[1:3] == [-1, 4999] and float(got[2][2]) == 0.0
    assert int(status) == decode.GS_DEV_EMPTY_ROW


def test_infinities_and_nan():
    V = 3000
    g = torch.Generator().manual_seed(0)
    cond, uncond = torch.randn((2, V), generator=g), torch.randn((2, V), generator=g)
    cond[0, 7], uncond[0, 7] = -torch.inf, -torch.inf          # forbidden by both
    cond[0, 8] = -torch.inf                                    # by cond alone
    uncond[0, 9] = -torch.inf                                  # by uncond alone: not guided
    cond[0, 10] = torch.finfo(F32).min
    cond[1, 100] = torch.nan
    allowed = np.ones((2, V), bool)
    allowed[1, 100] = False                                    # NaN in a masked place
    out, token, logprob = decode.guided_logits(cond=cond.cuda(), uncond=uncond.cuda(), cfg=3.0, mask=words(allowed))
    out = out.cpu()
    assert torch.isneginf(out[0, 7]) and torch.isneginf(out[0, 8]) and out[0, 9] == cond[0, 9]
    assert not torch.isnan(out).any() and torch.isneginf(out[1, 100])
    assert torch.isfinite(logprob).all()
    out, token, logprob = decode.guided_logits(cond.cuda())
    assert torch.isnan(out[1, 100]) and int(token[1]) == int(cond[1].nan_to_num(-1e9).argmax())
    assert torch.isnan(logprob[1]) and torch.isfinite(logprob[0])
    out, token, _ = decode.guided_logits(torch.full((1, V), -torch.inf).cuda())
    assert int(token) == -1


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ties_go_to_the_lowest_index(dtype):
    for V, at in ((50, [3, 9]), (9000, [8191, 8192, 8999]), (40000, [39999, 2047, 2048])):
        x = torch.zeros((2, V), dtype=dtype)
        x[0, at] = 5.0
        _, token, logprob = decode.guided_logits(x.cuda())
        assert token.tolist() == [min(at), 0]
        want = 5.0 - np.log(len(at) * np.exp(5.0) + V - len(at))
        assert abs(float(logprob[0]) - want) < 1e-4


def test_scale_one_reads_no_uncond_and_zero_gives_it():
    V = 2500
    g = torch.Generator().manual_seed(5)
    cond, uncond = (torch.randn((3, V), generator=g).to(BF16).cuda() for _ in range(2))
    poison = torch.full_like(uncond, float("nan"))
    lut = torch.tensor([1.0]).cuda()
    out, _, _ = decode.guided_logits(cond=cond, uncond=poison, scale_lut=lut, step=0)
    assert torch.equal(out, cond.float())
    out, _, _ = decode.guided_logits(cond=cond, uncond=uncond, cfg=0.0)
    assert torch.equal(out, uncond.float())


def test_rows_in_error_are_flagged_and_left():
    V = 300
    cond = torch.randn((3, V)).cuda()
    lut = torch.tensor([1.0, 2.0]).cuda()
    status = torch.zeros(1, dtype=torch.int32).cuda()
    out = torch.full((3, V), 7.0).cuda()
    token = torch.full((3,), 5, dtype=torch.int32).cuda()
    decode.guided_logits(cond=cond, scale_lut=lut, step_idx=torch.tensor([0, 2, 1], dtype=torch.int32).cuda(),
                         out=out, token=token, status=status)
    assert int(status) == gs.GS_DEV_STEP_RANGE | gs.GS_DEV_NEED_UNCOND
    assert torch.equal(out[0], cond[0]) and (out[1:] == 7).all() and token.tolist()[1:] == [-1, -1]


def test_outputs_alone_repeats_and_another_stream():
    V, B = 30000, 9
    x = torch.randn((B, V)).to(F16).cuda()
    out, token, logprob = decode.guided_logits(x)
    assert torch.equal(out, x.float())
    for name in ("token", "logprob", "out"):
        t = {"token": torch.empty_like(token), "logprob": torch.empty_like(logprob), "out": torch.empty_like(out)}[name]
        call = decode.prepare_guided_logits(x, **{name: t})
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(4):
                call()
        side.synchronize()
        assert torch.equal(t, {"token": token, "logprob": logprob, "out": out}[name])


def test_refusals_of_the_binding():
    x = torch.zeros((2, 64)).cuda()
    for kw in (dict(cond=x), dict(uncond=x), dict(bias=x[:, :5]), dict(mask=torch.zeros((2, 3), dtype=torch.int32).cuda()),
               dict(tokens=torch.zeros((2, 4), dtype=torch.int32).cuda()), dict(temperature=torch.ones(3).cuda()),
               dict(noise=x.double()), dict(out=torch.zeros((2, 64))), dict(repetition=torch.ones(2))):
        with pytest.raises(ValueError):
            decode.guided_logits(x, **kw)
    with pytest.raises(gs.GSError):
        decode.guided_logits(x, scale_lut=torch.ones(3).cuda(), step=3)
