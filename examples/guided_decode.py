"""Guided decoding of a small token model with the decode operators, end to end.

A toy transformer (random weights, torch products) writes tokens for a batch of samples under
classifier-free guidance. Every sample has two branches over one shared prompt:

* the prompt's keys and values are stored once (``write``), sequence by sequence;
* the uncond branch forks from it (``fork``: full pages are shared, the last one is copied);
* the cond branch then reads the sample's condition tokens (prompts are read in chunks: ``write``,
  then ``chunk_attention`` over everything stored so far);
* a decode step makes room for one token of every branch (``extend``), attends layer by layer
  while storing the new keys and values (``attention`` with ``k_new`` / ``v_new``), and turns the
  two branches' logits into the next token (``guided_logits``: scale from the bucket plan,
  penalties, temperature, a mask of allowed tokens, Gumbel noise as an input); with ``--top-k``,
  ``--top-p`` or ``--min-p`` the token comes from what these keep of its result (``sample``);
* finished sequences are freed and the pool is made dense (``free``, ``compact``).

The step has no host synchronisation: it is captured in a CUDA graph once and replayed.

    python examples/guided_decode.py [--batch 4] [--steps 32] [--dtype bf16] [--top-k 50] [--top-p 0.9]
"""

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bucketized_guidance_step_gb300 import decode, gs  # noqa: E402

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@dataclass(frozen=True)
class Config:
    layers: int = 2
    q_heads: int = 8
    kv_heads: int = 2
    dim: int = 64
    vocab: int = 1000
    page: int = 16
    length: int = 256             # most tokens of a sequence


class Model:
    """A pre-norm transformer with grouped heads and no feed-forward part."""

    def __init__(self, cfg: Config, dtype, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        width = cfg.q_heads * cfg.dim

        def w(*shape):
            x = torch.randn(shape, generator=g, device="cuda") * shape[0] ** -0.5
            return x.to(dtype)

        self.cfg, self.width = cfg, width
        self.embed = (torch.randn((cfg.vocab, width), generator=g, device="cuda")).to(dtype)
        self.place = (torch.randn((cfg.length, width), generator=g, device="cuda") * 0.1).to(dtype)
        self.qkv = [w(width, (cfg.q_heads + 2 * cfg.kv_heads) * cfg.dim) for _ in range(cfg.layers)]
        self.proj = [w(width, width) for _ in range(cfg.layers)]
        self.head = w(width, cfg.vocab) * 4

    def start(self, tokens, positions):
        return self.embed[tokens.long()] + self.place[positions.long()]

    def split(self, layer, x):
        """q, k, v of rows x ([n, heads, dim] views of one product)."""
        c = self.cfg
        y = torch.nn.functional.rms_norm(x, (self.width,)) @ self.qkv[layer]
        a, b = c.q_heads * c.dim, c.kv_heads * c.dim
        return (y[:, :a].view(-1, c.q_heads, c.dim), y[:, a:a + b].view(-1, c.kv_heads, c.dim),
                y[:, a + b:].view(-1, c.kv_heads, c.dim))

    def join(self, layer, x, attended):
        return x + attended.reshape(len(x), self.width) @ self.proj[layer]

    def logits(self, x):
        return torch.nn.functional.rms_norm(x, (self.width,)) @ self.head


class Decoder:
    """Sequences 0 .. B-1 are the uncond branches, B .. 2B-1 the cond branches."""

    def __init__(self, model: Model, batch: int, steps: int, dtype):
        c, dev = model.cfg, "cuda"
        self.model, self.batch = model, batch
        cols = -(-c.length // c.page)
        pages = 2 * batch * cols
        kv = torch.zeros((2, c.layers, pages, c.kv_heads, c.page, c.dim), dtype=dtype, device=dev)
        i32 = dict(dtype=torch.int32, device=dev)
        self.lens = torch.zeros(2 * batch, **i32)
        self.status = torch.zeros(1, **i32)
        self.cache = decode.PagedCache(kv[0], kv[1], torch.full((2 * batch, cols), -1, **i32), self.lens,
                                       torch.zeros(pages, **i32), status=self.status)
        self.both = torch.arange(2 * batch, **i32)
        self.uncond, self.cond = self.both[:batch], self.both[batch:]
        self.tokens = torch.zeros((batch, c.length), **i32)       # history: condition, then output
        self.tokens_len = torch.zeros(batch, **i32)
        self.prompt_len = torch.zeros(batch, **i32)
        self.token = torch.zeros(batch, **i32)
        self.logprob = torch.zeros(batch, device=dev)
        self.z = torch.zeros((batch, c.vocab), device=dev)
        self.noise = torch.zeros((batch, c.vocab), device=dev)
        _, lut = gs.bucket_plan(steps, min(8, steps), curve="linear", v0=2.0, v1=1.2)
        self.lut = torch.from_numpy(lut).to(dev)
        self.step_idx = torch.zeros(batch, **i32)
        full = torch.ones
        self.settings = dict(repetition=full(batch, device=dev) * 1.1, frequency=full(batch, device=dev) * 0.1,
                             presence=full(batch, device=dev) * 0.1, temperature=full(batch, device=dev))
        words = (c.vocab + 31) // 32
        self.mask = torch.full((1, words), -1, **i32)             # every token allowed
        self.mask[0, 0] = -2                                      # but token 0
        self.kept = None                                          # sample's top_k, top_p and min_p

    def keep(self, top_k=0, top_p=1.0, min_p=0.0):
        """Draw tokens from what top_k, then top_p, then min_p leave of guided_logits' result."""
        full, dev = torch.full, "cuda"
        self.kept = dict(top_k=full((self.batch,), top_k, dtype=torch.int32, device=dev),
                         top_p=full((self.batch,), top_p, device=dev), min_p=full((self.batch,), min_p, device=dev))

    def read(self, seq, tokens, chunk=64):
        """Prompt tokens ([n, t], the same number for every listed sequence) into the cache, up to
        `chunk` of each sequence at a time: their keys and values are stored, and each position
        attends over everything up to itself (in as many bits as the step's attention)."""
        n = len(tokens)
        for part in tokens.split(chunk, 1):
            t = part.shape[1]
            at = self.lens[seq.long()][:, None] + torch.arange(t, device="cuda")
            self.cache.extend(seq, torch.full_like(seq, t))
            start = t * torch.arange(n + 1, dtype=torch.int32, device="cuda")
            x = self.model.start(part.flatten(), at.flatten())
            for layer in range(self.model.cfg.layers):
                q, k, v = self.model.split(layer, x)
                self.cache.write(layer, k, v, seq, start)
                x = self.model.join(layer, x, self.cache.chunk_attention(q, layer, seq, start, split_weights=True))

    def step(self):
        """One token of every sample."""
        m = self.model
        at = self.lens.clone()
        self.cache.extend(self.both)
        x = m.start(self.token.repeat(2), at)
        for layer in range(m.cfg.layers):
            q, k, v = m.split(layer, x)
            x = m.join(layer, x, self.cache.attention(q, layer, k_new=k, v_new=v))
        decode.guided_logits(stacked=m.logits(x), step_idx=self.step_idx, scale_lut=self.lut,
                             tokens=self.tokens, tokens_len=self.tokens_len, prompt_len=self.prompt_len,
                             mask=self.mask, noise=self.noise, out=self.z, token=self.token,
                             logprob=self.logprob, status=self.status, **self.settings)
        if self.kept is not None:                                 # (z has the temperature in it)
            decode.sample(self.z, noise=self.noise, token=self.token, logprob=self.logprob, status=self.status,
                          **self.kept)
        self.tokens.scatter_(1, self.tokens_len.long()[:, None], self.token[:, None])
        self.tokens_len += 1
        self.step_idx += 1


def run(batch=4, steps=32, dtype="bf16", cfg=Config(), prompt=21, condition=5, seed=0, graph=True, watch=None,
        keep=None):
    """Decodes `steps` tokens; returns (tokens [batch, steps], log-probabilities, decoder).
    watch(decoder): called after every step. keep: Decoder.keep's arguments."""
    dt = DTYPES[dtype]
    model = Model(cfg, dt, seed)
    d = Decoder(model, batch, steps, dt)
    if keep is not None:
        d.keep(**keep)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    shared = torch.randint(1, cfg.vocab, (1, prompt), generator=g, device="cuda", dtype=torch.int32)
    wanted = torch.randint(1, cfg.vocab, (batch, condition), generator=g, device="cuda", dtype=torch.int32)
    d.read(d.cond[:1], shared)                                    # the prompt, once
    d.cache.fork(d.cond[:1].expand(2 * batch - 1).contiguous(), torch.cat([d.uncond, d.cond[1:]]))
    d.read(d.cond, wanted)
    d.read(d.uncond, torch.zeros_like(wanted))                    # the null condition
    d.tokens[:, :condition] = wanted
    d.tokens_len += condition
    d.prompt_len += condition
    d.token.copy_(wanted[:, -1])
    d.prompt, d.wanted = shared, wanted
    said, logprobs = [], []
    captured = None
    for i in range(steps):
        u = torch.rand(d.noise.shape, generator=g, device="cuda").clamp(1e-7, 1 - 1e-7)
        d.noise.copy_(-torch.log(-torch.log(u)))
        if graph and i == 1:                                      # (step 0 has warmed everything up)
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                d.step()
        if captured is not None:
            captured.replay()
        else:
            d.step()
        said.append(d.token.clone())
        logprobs.append(d.logprob.clone())
        if watch is not None:
            watch(d)
    status = decode.status_from_word(int(d.status))
    if status != gs.GS_OK:
        raise gs.GSError("guided decode", status)
    return torch.stack(said, 1), torch.stack(logprobs, 1), d


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--dtype", choices=sorted(DTYPES), default="bf16")
    ap.add_argument("--top-k", type=int, default=0, help="0: all")
    ap.add_argument("--top-p", type=float, default=1.0)
    ap.add_argument("--min-p", type=float, default=0.0)
    a = ap.parse_args()
    keep = dict(top_k=a.top_k, top_p=a.top_p, min_p=a.min_p)
    some = a.top_k > 0 or a.top_p < 1 or a.min_p > 0
    tokens, logprobs, d = run(a.batch, a.steps, a.dtype, keep=keep if some else None)
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    for row, lp in zip(tokens.tolist(), logprobs.sum(1).tolist()):
        print(f"log-probability {lp:9.3f}: {row}")
    held = int((d.cache.refs > 0).sum())
    d.cache.free(d.both[::2].contiguous())                        # half the branches leave
    d.cache.compact(live=live)
    print(f"{held} pages held while decoding, {int(live)} after half the branches left, "
          f"dense: {bool((d.cache.refs[:int(live)] > 0).all())}")


if __name__ == "__main__":
    main()
