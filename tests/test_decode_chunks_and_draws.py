"""Chunks, single tokens and sampling in one decoding run: the example's (GPU).

A prompt read in chunks of any size leaves the same keys and values: layer 1's come after an attention
and products of width 512 in fp32, sums of about 15 in absolute values, so 15 * 512 * 2^-24 = 4.6e-4
each way at worst. A step's token is held to the definition of top_k, top_p and min_p in float64 on the z
of that step, where a token whose sum or weight lies within 2^-18 of its bound may be kept or not.
"""

import numpy as np
import pytest
import torch

from examples import guided_decode as E

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chunk", [7, 16, 200])
def test_the_size_of_chunks_does_not_matter(chunk):
    cfg = E.Config()
    model = E.Model(cfg, torch.float32)
    g = torch.Generator(device="cuda").manual_seed(3)
    tokens = torch.randint(1, cfg.vocab, (3, 139), generator=g, device="cuda", dtype=torch.int32)
    held = []
    for size in (1, chunk):
        d = E.Decoder(model, 2, 8, torch.float32)
        d.read(d.both[:3], tokens, chunk=size)
        assert d.lens.tolist() == [139, 139, 139, 0] and int(d.status) == 0
        rows = d.cache.table[:3, :9].long()
        held.append([x[:, rows].transpose(3, 4).flatten(2, 3).clone() for x in (d.cache.k, d.cache.v)])
    for one, many in zip(*held):
        # [layers, 3, cols * heads, page, dim]: what lies past the last token is as it was made, zero
        assert torch.allclose(one, many, rtol=0, atol=2 * 4.6e-4)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("keep", [dict(top_k=5), dict(top_p=0.6), dict(top_k=40, top_p=0.8, min_p=0.1), dict(top_k=1)])
def test_tokens_come_from_what_is_kept(keep, graph):
    seen = []

    def watch(d):
        seen.append([x.cpu().numpy().copy() for x in (d.z, d.noise, d.token, d.logprob)])

    tokens, logprobs, d = E.run(3, 6, "bf16", graph=graph, watch=watch, keep=keep)
    assert tokens.shape == (3, 6) and len(seen) == 6 and int(d.status) == 0
    for i, (z, noise, token, logprob) in enumerate(seen):
        for b in range(3):
            order = np.argsort(-z[b], kind="stable")
            order = order[z[b][order] > -np.inf]
            right = []
            for slack in (-(2.0 ** -18), 0.0, 2.0 ** -18):
                ids = order[:keep.get("top_k") or None]
                w = np.exp(z[b][ids].astype(np.float64) - z[b][ids[0]])
                before = np.cumsum(w) - w
                stay = (before < keep.get("top_p", 1.0) * w.sum() * (1 + slack)) & (w >= keep.get("min_p", 0.0) * (1 - slack))
                stay[0] = True
                ids, w = ids[stay], w[stay]
                best = int(ids[np.argmax(z[b][ids] + noise[b][ids])])
                right.append((best, float(z[b][best]) - float(z[b][ids[0]]) - np.log(w.sum())))
            assert any(int(token[b]) == t and abs(logprob[b] - lp) < 2.0 ** -18 * (1 + abs(lp)) for t, lp in right), (i, b)
            assert int(tokens[b, i]) == int(token[b])
    if keep.get("top_k") == 1:
        assert torch.equal(tokens[:, 0].cpu(), torch.as_tensor([int(s.argmax()) for s in seen[0][0]], dtype=torch.int32))
        assert (logprobs == 0).all()
