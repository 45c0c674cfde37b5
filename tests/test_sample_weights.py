"""How exact the weights of sampling are (GPU): a token d below the largest has e^-d of its weight, off by
(2^-22 + 2.3 d 2^-24) of itself at most. min_p tells on which side of a bound a weight lies: with noise that makes the
lower token win wherever it is kept, it is kept where its weight in 64 bits is above min_p by more than that, and not
where it is below by more.
"""

import numpy as np
import pytest
import torch

from bucketized_guidance_step_gb300 import decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [2, 5000, 200000])    # a list; one pass; a row that no cluster holds
@pytest.mark.parametrize("top", [0.0, 1.0, -3.3, 47.11, 1000.5])
def test_weights_are_as_good_as_stated(vocab, top):
    B = 4096 if vocab < 10000 else 1024
    rng = np.random.default_rng(int(abs(top) * 10) + vocab)
    z = np.full((B, vocab), -np.inf, dtype=np.float32)
    z[:, 0] = top
    z[:, vocab - 1] = np.float32(top) - rng.uniform(0.0, 27.0, B).astype(np.float32)
    d = z[:, 0].astype(np.float64) - z[:, vocab - 1].astype(np.float64)
    weight, off = np.exp(-d), 2.0 ** -22 + 2.3 * d * 2.0 ** -24
    min_p = (weight * (1 + rng.uniform(-4, 4, B) * off)).astype(np.float32)
    noise = torch.zeros((1, vocab), device="cuda")
    noise[0, vocab - 1] = 1e6
    token, _ = decode.sample(torch.from_numpy(z).cuda(), min_p=torch.from_numpy(min_p).cuda(), noise=noise,
                             top_k=torch.full((B,), 2, dtype=torch.int32, device="cuda") if vocab == 2 else None)
    kept = token.cpu().numpy() == vocab - 1
    ratio = min_p.astype(np.float64) / weight
    assert kept[ratio < 1 - off].all() and not kept[ratio > 1 + off].any()
    assert (ratio < 1 - off).sum() > B // 8 and (ratio > 1 + off).sum() > B // 8
