"""The decode operators together: the example's guided decoding against a float64 model that
keeps no cache (GPU).

Every step's logits are recomputed from the whole token sequences in float64 (causal attention
over all positions of both branches) and passed to the oracle's guided logits. The example runs
in fp32; its activations pass through `layers` products and attentions of width 512, so the
logits (of size up to about 20) are held to 2e-3 and the chosen token to the oracle's pick within
that. Also: forked pages are shared, and freeing and compacting leave the other branches whole.
"""

import numpy as np
import pytest
import torch

from examples import guided_decode as E
from oracle import decode as O

pytestmark = pytest.mark.gpu


def plain_logits(model, tokens):
    """Logits of the last position of one sequence, float64, no cache."""
    c = model.cfg
    t = torch.as_tensor(tokens, device="cuda")
    x = (model.embed[t] + model.place[torch.arange(len(t), device="cuda")]).double()
    norm = lambda y: y / torch.sqrt((y * y).mean(-1, keepdim=True) + torch.finfo(torch.float32).eps)  # noqa: E731
    for layer in range(c.layers):
        y = norm(x) @ model.qkv[layer].double()
        a, b = c.q_heads * c.dim, c.kv_heads * c.dim
        q = y[:, :a].view(-1, c.q_heads, c.dim).transpose(0, 1)
        k, v = (z.reshape(-1, c.kv_heads, c.dim).transpose(0, 1).repeat_interleave(c.q_heads // c.kv_heads, 0)
                for z in (y[:, a:a + b], y[:, a + b:]))
        s = q @ k.transpose(1, 2) * c.dim ** -0.5
        s = s.masked_fill(torch.ones_like(s[0]).triu(1).bool(), float("-inf"))
        x = x + (torch.softmax(s, -1) @ v).transpose(0, 1).reshape(len(t), -1) @ model.proj[layer].double()
    return (norm(x[-1]) @ model.head.double()).cpu().numpy()


@pytest.mark.parametrize("graph", [False, True])
def test_guided_decoding_matches_a_model_without_a_cache(graph):
    batch, steps, tf32 = 3, 7, torch.backends.cuda.matmul.allow_tf32
    seen = []

    def watch(d):
        seen.append((d.z.double().cpu().numpy(), d.token.cpu().numpy(), d.noise.double().cpu().numpy()))

    tokens, _, d = E.run(batch, steps, "fp32", prompt=21, condition=5, graph=graph, watch=watch)
    lut = d.lut.double().cpu().numpy()
    prompt, wanted = d.prompt[0].tolist(), d.wanted.tolist()
    allowed = np.arange(d.model.cfg.vocab) != 0
    for b in range(batch):
        said = []
        for i in range(steps):
            last = wanted[b][-1:] + said
            cond = plain_logits(d.model, prompt + wanted[b] + last[:i + 1])
            uncond = plain_logits(d.model, prompt + [0] * len(wanted[b]) + last[:i + 1])
            z, _, _, _, pick = O.guided_logits(cond, uncond, lut[i], tokens=wanted[b] + said, prompt=len(wanted[b]),
                                               repetition=1.1, frequency=0.1, presence=0.1, temperature=1.0,
                                               allowed=allowed, noise=seen[i][2][b])
            got, tok = seen[i][0][b], int(seen[i][1][b])
            assert np.isneginf(got[0]) and np.max(np.abs(got[1:] - z[1:])) < 2e-3, (b, i)
            assert pick[tok] >= pick.max() - 4e-3, (b, i)
            said.append(tok)
        assert said == tokens[b].tolist()
    assert torch.backends.cuda.matmul.allow_tf32 == tf32


def test_branches_share_the_prompt_and_survive_compaction():
    _, _, d = E.run(4, 5, "bf16", prompt=40, condition=3)
    table, refs = d.cache.table.cpu(), d.cache.refs.cpu()
    assert (table[:, :2] == table[0, :2]).all() and (refs[table[0, :2].long()] == 8).all()   # 32 of 40 tokens
    assert len(set(table[:, 2].tolist())) == 8                                              # the partly filled page
    q = torch.randn((8, 8, 64), device="cuda").to(torch.bfloat16)
    before = d.cache.attention(q, 1)
    d.cache.free(torch.tensor([0, 5, 6], dtype=torch.int32, device="cuda"))
    d.cache.compact()
    after = d.cache.attention(q, 1)
    keep = [1, 2, 3, 4, 7]
    assert torch.equal(before[keep], after[keep]) and (after[[0, 5, 6]] == 0).all()
    assert int(d.status) == 0
