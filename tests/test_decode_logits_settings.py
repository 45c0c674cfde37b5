"""Guided logits: quotients, settings at the ends of their ranges (GPU).

Without guidance, bias and noise a logit of an fp32 row passes through one operation, so z is the
correctly rounded quotient or product: compared bit for bit with numpy's. A repetition penalty
multiplies by its rounded reciprocal where that is an ordinary number.
"""

import numpy as np
import pytest
import torch

from bucketized_guidance_step_gb300 import decode

pytestmark = pytest.mark.gpu

F32 = np.float32


def rows(B, V, seed=0):
    x = np.random.default_rng(seed).standard_normal((B, V)).astype(F32) * F32(5)
    x[:, :8] = [0.0, -0.0, np.inf, -np.inf, 1e-42, -1e-38, 3e38, -3e38]
    return x


def same(got, want):
    return np.array_equal(got.view(np.int32), want.view(np.int32))


@pytest.mark.parametrize("V", [513, 5000, 40001])
def test_temperature_divides(V):
    hot = np.array([0.7, 1.3, 0.1, 3.0, 1e-6, 1e30, 1.0, 2.0 ** -126, 2.0 ** -130, 1e-45, 3e38, 2.0 ** 127, 1.1754942e-38], F32)
    x = rows(len(hot), V, seed=V)
    out, _, _ = decode.guided_logits(torch.from_numpy(x).cuda(), temperature=torch.from_numpy(hot).cuda())
    with np.errstate(over="ignore"):
        want = x / hot[:, None]
    got = out.cpu().numpy()
    for b in range(len(hot)):
        assert same(got[b], want[b]), (hot[b], np.flatnonzero(got[b] != want[b])[:5])


@pytest.mark.parametrize("V", [513, 40001])
def test_repetition(V):
    rep = np.array([1.1, 0.7, 3.0, 1e-40, 2.0 ** -130, 1e38, 1.5], F32)
    x = rows(len(rep), V, seed=V)
    tokens = torch.arange(V, dtype=torch.int32).repeat(len(rep), 1).cuda()
    n = torch.full((len(rep),), V, dtype=torch.int32).cuda()
    out, _, _ = decode.guided_logits(torch.from_numpy(x).cuda(), tokens=tokens, tokens_len=n, prompt_len=n,
                                     repetition=torch.from_numpy(rep).cuda())
    with np.errstate(over="ignore", invalid="ignore"):
        usual = ((rep >= 2.0 ** -40) & (rep <= 2.0 ** 40))[:, None]
        want = np.where(x > 0, np.where(usual, x * (F32(1) / rep)[:, None], x / rep[:, None]), x * rep[:, None])
    got = out.cpu().numpy()
    for b in range(len(rep)):
        assert same(got[b], want[b]), (rep[b], np.flatnonzero(got[b] != want[b])[:5])


def test_a_very_cold_row_still_chooses():
    """A temperature whose reciprocal is no fp32 number."""
    x = torch.tensor([[-1.0, 0.0, -2.0, -1e-3]], device="cuda")
    _, token, logprob = decode.guided_logits(x, temperature=torch.tensor([1e-40], device="cuda"))
    assert int(token) == 1 and float(logprob) == 0.0
